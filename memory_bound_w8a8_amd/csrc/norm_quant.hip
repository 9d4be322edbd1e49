// Root-mean-square norm with the residual's addition and an 8-bit output, and
// the per-row int8 quantisers, gfx950.
//
// Page 3 (zskr.cn blog), section 3.3, fuses the norm with the quantisation of
// the linear layer's input; section 2.2 stores weights as INT8. Per row:
//   h = bf16(x + r), inv = fp32(1 / sqrt(mean(h^2) + eps)), y = bf16((h inv) w),
// then y is quantised as fp8bq_quant_act does (a scale per 128 columns) or to
// int8 with a scale per row. Rounding y to bf16 is what the separate norm and
// quantiser do (their interface is bf16), so the fused codes equal theirs bit
// for bit; h is rounded because the residual stream is bf16 and the norm has
// to see what the next layer will see. The sum of squares and the root are in
// 64 bits, so that inv does not depend on the order of the sum; the two products
// are rounded to fp32 one after the other, as a norm in fp32 rounds them, which
// puts y on the other side of a bf16 border than products in 64 bits would in
// about 5 values in 10^6.
#include <cfloat>

#include "device_common.h"
#include "step_launch.h"

namespace fp8bq {

namespace {

constexpr float kI8Max = 127.f;

typedef unsigned short v2us __attribute__((ext_vector_type(2)));

// v of the lane ROT further in its DPP row of 16.
template <int ROT>
__device__ __forceinline__ int rotated(int v) {
  return __builtin_amdgcn_update_dpp(0, v, 0x120 + ROT, 0xf, 0xf, true);
}
template <int ROT>
__device__ __forceinline__ double sum_rotated(double v) {
  const v2u w = __builtin_bit_cast(v2u, v);
  const v2u o = {static_cast<unsigned>(rotated<ROT>(static_cast<int>(w[0]))),
                 static_cast<unsigned>(rotated<ROT>(static_cast<int>(w[1])))};
  return v + __builtin_bit_cast(double, o);
}

// Sum over the workgroup (every thread gets it). `slots` holds one value per
// wave; a barrier on both sides lets it be used again.
__device__ __forceinline__ double block_sum(double v, double* slots) {
  v = sum_rotated<1>(sum_rotated<2>(sum_rotated<4>(sum_rotated<8>(v))));
  v += __shfl_xor(v, 16, 64);
  v += __shfl_xor(v, 32, 64);
  const int waves = blockDim.x >> 6;
  if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = v;
  __syncthreads();
  double sum = 0.0;
  for (int i = 0; i < waves; ++i) sum += slots[i];
  __syncthreads();
  return sum;
}

// The larger of two pairs of 16-bit numbers, each for itself. On the
// magnitudes of two bf16 values that is their order, NaN above infinity.
__device__ __forceinline__ unsigned max_pair(unsigned a, unsigned b) {
  return __builtin_bit_cast(unsigned,
                            __builtin_elementwise_max(__builtin_bit_cast(v2us, a), __builtin_bit_cast(v2us, b)));
}
__device__ __forceinline__ unsigned abs_pair(unsigned a) { return a & 0x7fff7fffu; }
// The larger half of a pair, as a number.
__device__ __forceinline__ float top_of(unsigned a) {
  const unsigned hi = a >> 16, lo = a & 0xffffu;
  return __builtin_bit_cast(float, (hi > lo ? hi : lo) << 16);
}

// max_pair over the 16 lanes of a DPP row (rotations by 8, 4, 2 and 1), and
// over the workgroup.
template <int ROT>
__device__ __forceinline__ unsigned max_rotated(unsigned a) {
  return max_pair(a, static_cast<unsigned>(rotated<ROT>(static_cast<int>(a))));
}
__device__ __forceinline__ unsigned row16_max(unsigned a) {
  return max_rotated<1>(max_rotated<2>(max_rotated<4>(max_rotated<8>(a))));
}
__device__ __forceinline__ unsigned block_max(unsigned a, unsigned* slots) {
  a = row16_max(a);
  a = max_pair(a, __shfl_xor(a, 16, 64));
  a = max_pair(a, __shfl_xor(a, 32, 64));
  const int waves = blockDim.x >> 6;
  if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = a;
  __syncthreads();
  unsigned top = 0;
  for (int i = 0; i < waves; ++i) top = max_pair(top, slots[i]);
  __syncthreads();
  return top;
}

// The same for numbers (the quantisers' fp32 rows).
__device__ __forceinline__ float block_max(float v, float* slots) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, 64));
  const int waves = blockDim.x >> 6;
  if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = v;
  __syncthreads();
  float top = 0.f;
  for (int i = 0; i < waves; ++i) top = fmaxf(top, slots[i]);
  __syncthreads();
  return top;
}

// Scale of an int8 row from its amax: 1 where amax / 127 is 0 (a row of
// zeros, or of the smallest subnormal numbers, whose codes are then 0).
__device__ __forceinline__ float row_scale(float amax) {
  const float s = amax / kI8Max;
  return s > 0.f ? s : 1.f;
}

// int8 codes of four quotients, byte i = the i-th. Adding 1.5 * 2^23 rounds to
// a whole number (ties to even) and leaves it in the sum's low bits.
__device__ __forceinline__ unsigned pack4_i8(float q0, float q1, float q2, float q3) {
  const auto code = [](float q) { return __builtin_bit_cast(unsigned, q + 12582912.f); };
  return __builtin_amdgcn_perm(code(q1), code(q0), 0x0c0c0400) | __builtin_amdgcn_perm(code(q3), code(q2), 0x04000c0c);
}
// A quotient held to +-127, which it passes only where the scale is a
// subnormal number.
__device__ __forceinline__ float clamped_i8(float x, float s) { return fminf(fmaxf(x / s, -kI8Max), kI8Max); }

__device__ __forceinline__ void unpack8(const v4u& p, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_lo(p[i]);
    x[2 * i + 1] = bf16_hi(p[i]);
  }
}

// 1 / sqrt(v) rounded to fp32. Held to the largest finite number, which only an
// eps below 2^-256 lets it pass, so that a zero stays a zero. (|h| inv is
// sqrt(K) at most: only the weights can take y out of range.)
__device__ __forceinline__ float inverse_root(double v) { return fminf(static_cast<float>(rsqrt(v)), FLT_MAX); }

// Keeps the compiler from carrying unpacked or 64-bit copies of packed values
// from one use to a later one (four times the registers).
__device__ __forceinline__ void stay_packed(v4u& p) { asm volatile("" : "+v"(p)); }

// The packed y of 8 packed values h and weights w.
__device__ __forceinline__ v4u scaled8(const v4u& h, const v4u& w, float inv) {
  v4u y;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    y[j] = pack_bf16x2((bf16_lo(h[j]) * inv) * bf16_lo(w[j]), (bf16_hi(h[j]) * inv) * bf16_hi(w[j]));
  return y;
}
__device__ __forceinline__ unsigned top8(const v4u& y) {
  return max_pair(max_pair(abs_pair(y[0]), abs_pair(y[1])), max_pair(abs_pair(y[2]), abs_pair(y[3])));
}

// Codes of 8 packed values whose group or row has the scale s; above 2^-96 the
// quotient is the one of the fused product, whose codes are the IEEE
// division's but for the sign of a zero.
__device__ __forceinline__ v2u codes8_e4m3(const v4u& y, float amax, float s) {
  float f[8], q[8];
  unpack8(y, f);
  if (amax >= 0x1p-96f) {
    const RecipPair r = recip_pair(s);
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = copysignf(quotient_e4m3_gemm(f[j], r), f[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = scaled_clamped(f[j], s);
  }
  return v2u{encode4_e4m3(q[0], q[1], q[2], q[3]), encode4_e4m3(q[4], q[5], q[6], q[7])};
}
// The same for int8, up to 2^100: from there on the reciprocal's low part nears
// the subnormal numbers, and above 2^125 it has lost the bits that decide ties (5
// of the 5.2e8 pairs of bf16 numbers). Up to it the code is the IEEE division's
// for every bf16 x and every bf16 row maximum (all pairs checked on the host).
__device__ __forceinline__ v2u codes8_i8(const v4u& y, float amax, float s, const RecipPair& r) {
  float f[8], q[8];
  unpack8(y, f);
  if (amax >= 0x1p-96f && amax < 0x1p100f) {
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = quotient_e4m3_gemm(f[j], r);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = clamped_i8(f[j], s);
  }
  return v2u{pack4_i8(q[0], q[1], q[2], q[3]), pack4_i8(q[4], q[5], q[6], q[7])};
}

// A row per workgroup and trip; thread t holds the 8-value chunks t, t +
// blockDim, ... (CH of them) as packed bf16. All loads of a row, the weight's
// among them, go out before the first is used. x, r and h may be the same
// memory: a thread reads its chunks before it writes them.
//
// Bound by memory for many rows with a residual: 3465 x 5120 to e4m3 moves 125
// MB in 23 .. 27 us (4.7 .. 5.4 TB/s; a copy of 1 GiB reaches 5.2, and some of
// the inputs stay in the memory-side cache at the shorter time). Without a
// residual 2049 x 8704 to int8 takes 14 .. 16.5 us (3.2 .. 3.8 TB/s): fewer
// bytes for the same work a value, and 1.6 rounds of rows that the CUs hold.
template <int CH, bool RES, bool I8>
__global__ __launch_bounds__(1024) void rmsnorm_quant_kernel(int64_t m, int k, double inv_k,
                                                             const unsigned short* x, const unsigned short* r,
                                                             const unsigned short* __restrict__ w, double eps,
                                                             unsigned short* h_out, unsigned char* __restrict__ codes,
                                                             float* __restrict__ scales) {
  __shared__ double sums[16];
  __shared__ unsigned tops[16];
  constexpr bool EARLY = CH <= 4;  // more chunks would not leave the weight registers
  const int chunks = k >> 3;
  const int threads = blockDim.x;
  const int t = threadIdx.x;
  const auto weight = [&](int c) {
    const int i = t + c * threads;
    return *reinterpret_cast<const v4u*>(w + 8 * (i < chunks ? i : 0));
  };
  v4u wv[EARLY ? CH : 1];
  if constexpr (EARLY) {
#pragma unroll
    for (int c = 0; c < CH; ++c) wv[c] = weight(c);
  }
  for (int64_t row = blockIdx.x; row < m; row += gridDim.x) {
    v4u h[CH], rv[RES ? CH : 1];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = t + c * threads;
      h[c] = v4u{0u, 0u, 0u, 0u};
      if (i < chunks) h[c] = *reinterpret_cast<const v4u*>(x + row * k + 8 * i);
      if constexpr (RES) {
        rv[c] = v4u{0u, 0u, 0u, 0u};
        if (i < chunks) rv[c] = *reinterpret_cast<const v4u*>(r + row * k + 8 * i);
      }
    }
    if constexpr (RES) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int i = t + c * threads;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          h[c][j] = pack_bf16x2(bf16_lo(h[c][j]) + bf16_lo(rv[c][j]), bf16_hi(h[c][j]) + bf16_hi(rv[c][j]));
        if (i < chunks) *reinterpret_cast<v4u*>(h_out + row * k + 8 * i) = h[c];
      }
    }
    double sum = 0.0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float f[8];
      unpack8(h[c], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fma(static_cast<double>(f[j]), static_cast<double>(f[j]), sum);
    }
    sum = block_sum(sum, sums);
    const float inv = inverse_root(sum * inv_k + eps);
#pragma unroll
    for (int c = 0; c < CH; ++c) stay_packed(h[c]);
    if constexpr (EARLY) {
#pragma unroll
      for (int c = 0; c < CH; ++c) stay_packed(wv[c]);
    }
    if constexpr (!I8) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int i = t + c * threads;
        const v4u y = scaled8(h[c], EARLY ? wv[EARLY ? c : 0] : weight(c), inv);
        const float amax = top_of(row16_max(top8(y)));
        const float s = group_scale(amax);
        if (i < chunks) {
          *reinterpret_cast<v2u*>(codes + row * k + 8 * i) = codes8_e4m3(y, amax, s);
          if ((i & 15) == 0) scales[row * (k >> 7) + (i >> 4)] = s;
        }
      }
    } else {
      unsigned pair = 0;
      v4u y[CH];
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        y[c] = scaled8(h[c], EARLY ? wv[EARLY ? c : 0] : weight(c), inv);
        pair = max_pair(pair, top8(y[c]));
      }
      const float top = top_of(block_max(pair, tops));
      const float s = row_scale(top);
      const RecipPair recip = recip_pair(s);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        stay_packed(y[c]);
        const int i = t + c * threads;
        if (i < chunks) *reinterpret_cast<v2u*>(codes + row * k + 8 * i) = codes8_i8(y[c], top, s, recip);
      }
      if (t == 0) scales[row] = s;
    }
  }
}

// int8 codes and one scale per row of a bf16 matrix, and of a fp32 one (by the
// IEEE division: its maxima have 24 bits).
template <int CH>
__global__ __launch_bounds__(1024) void quant_rows_i8_kernel(int64_t m, int k, const unsigned short* __restrict__ a,
                                                             unsigned char* __restrict__ codes,
                                                             float* __restrict__ scales) {
  __shared__ unsigned tops[16];
  const int chunks = k >> 3;
  for (int64_t row = blockIdx.x; row < m; row += gridDim.x) {
    v4u x[CH];
    unsigned pair = 0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = threadIdx.x + c * blockDim.x;
      x[c] = v4u{0u, 0u, 0u, 0u};
      if (i < chunks) x[c] = *reinterpret_cast<const v4u*>(a + row * k + 8 * i);
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) pair = max_pair(pair, top8(x[c]));
    const float top = top_of(block_max(pair, tops));
    const float s = row_scale(top);
    const RecipPair recip = recip_pair(s);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = threadIdx.x + c * blockDim.x;
      if (i < chunks) *reinterpret_cast<v2u*>(codes + row * k + 8 * i) = codes8_i8(x[c], top, s, recip);
    }
    if (threadIdx.x == 0) scales[row] = s;
  }
}

template <int CH>
__global__ __launch_bounds__(1024) void quant_rows_i8_kernel(int64_t m, int k, const float* __restrict__ a,
                                                             unsigned char* __restrict__ codes,
                                                             float* __restrict__ scales) {
  __shared__ float tops[16];
  const int chunks = k >> 3;
  for (int64_t row = blockIdx.x; row < m; row += gridDim.x) {
    v4f f[CH][2];
    float top = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = threadIdx.x + c * blockDim.x;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        f[c][j] = v4f{0.f, 0.f, 0.f, 0.f};
        if (i < chunks) f[c][j] = *reinterpret_cast<const v4f*>(a + row * k + 8 * i + 4 * j);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(f[c][j >> 2][j & 3]));
    }
    top = block_max(top, tops);
    const float s = row_scale(top);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = threadIdx.x + c * blockDim.x;
      v2u q;
#pragma unroll
      for (int j = 0; j < 2; ++j)
        q[j] = pack4_i8(clamped_i8(f[c][j][0], s), clamped_i8(f[c][j][1], s), clamped_i8(f[c][j][2], s),
                        clamped_i8(f[c][j][3], s));
      if (i < chunks) *reinterpret_cast<v2u*>(codes + row * k + 8 * i) = q;
    }
    if (threadIdx.x == 0) scales[row] = s;
  }
}

constexpr int64_t kMaxRowsInGrid = 1 << 20;  // workgroups; more rows loop

// Threads of a row's workgroup and chunks of 8 values per thread.
struct RowShape {
  int threads, chunks;
};
RowShape row_shape(int64_t k) {
  const int64_t n = k / 8;
  const int ch = n <= 1024 ? 1 : n <= 2048 ? 2 : n <= 4096 ? 4 : 8;
  const int64_t t = (n + ch - 1) / ch;
  return RowShape{static_cast<int>((t + 63) / 64 * 64), ch};
}

unsigned row_grid(int64_t m) { return static_cast<unsigned>(m < kMaxRowsInGrid ? m : kMaxRowsInGrid); }

template <int CH>
hipError_t run_rmsnorm(int64_t m, int64_t k, const void* x, const void* r, const void* w, double eps, void* h,
                       void* codes, float* scales, bool i8, hipStream_t stream) {
  const int waves = static_cast<int>((k / 8 + 64 * CH - 1) / (64 * CH));
  const auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(row_grid(m)), dim3(64 * waves), 0, stream, m, static_cast<int>(k),
                       1.0 / static_cast<double>(k), static_cast<const unsigned short*>(x),
                       static_cast<const unsigned short*>(r),
                       static_cast<const unsigned short*>(w), eps, static_cast<unsigned short*>(h),
                       static_cast<unsigned char*>(codes), scales);
    return hipGetLastError();
  };
  if (r != nullptr) return i8 ? go(rmsnorm_quant_kernel<CH, true, true>) : go(rmsnorm_quant_kernel<CH, true, false>);
  return i8 ? go(rmsnorm_quant_kernel<CH, false, true>) : go(rmsnorm_quant_kernel<CH, false, false>);
}

template <typename T>
hipError_t run_quant_rows(int64_t m, int64_t k, const void* a, void* codes, float* scales, hipStream_t stream) {
  const RowShape rs = row_shape(k);
  const auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(row_grid(m)), dim3(rs.threads), 0, stream, m, static_cast<int>(k),
                       static_cast<const T*>(a), static_cast<unsigned char*>(codes), scales);
    return hipGetLastError();
  };
  using Kernel = void (*)(int64_t, int, const T*, unsigned char*, float*);
  switch (rs.chunks) {
    case 1: return go(static_cast<Kernel>(quant_rows_i8_kernel<1>));
    case 2: return go(static_cast<Kernel>(quant_rows_i8_kernel<2>));
    case 4: return go(static_cast<Kernel>(quant_rows_i8_kernel<4>));
    default: return go(static_cast<Kernel>(quant_rows_i8_kernel<8>));
  }
}

}  // namespace

hipError_t launch_rmsnorm_quant(int64_t m, int64_t k, const void* x, const void* r, const void* w, double eps,
                                void* h, void* codes, float* scales, bool i8, hipStream_t stream) {
  // Three chunks a lane, or one in the shortest rows: fewer waves share a row's
  // barriers and 64-bit root, and several rows stay in flight on a CU. With
  // inputs from HBM, 3465 x 5120 with residual to e4m3 takes 27.8 / 26.4 / 26.7 /
  // 27.7 / 30.5 us with 1 / 2 / 3 / 4 / 6 chunks, 2049 x 8704 without one to int8
  // 17.2 / 16.5 / 16.7 with 2 / 3 / 4, 3465 x 512 6.2 / 6.7 / 7.4 / 8.0 / 9.4 with
  // 1 / 2 / 3 / 4 / 6. Where the rows do not fill the CUs, a row's own time
  // counts: two chunks (256 x 8704 with residual 7.5 / 8.1 / 8.5 us with 2 / 3 /
  // 4, one row 3.7 / 4.1 / 4.3).
  const int64_t chunks = k / 8;
  if (chunks <= 192) return run_rmsnorm<1>(m, k, x, r, w, eps, h, codes, scales, i8, stream);
  if (chunks <= 2048 && m <= 256) return run_rmsnorm<2>(m, k, x, r, w, eps, h, codes, scales, i8, stream);
  if (chunks <= 3072) return run_rmsnorm<3>(m, k, x, r, w, eps, h, codes, scales, i8, stream);
  if (chunks <= 4096) return run_rmsnorm<4>(m, k, x, r, w, eps, h, codes, scales, i8, stream);
  return run_rmsnorm<8>(m, k, x, r, w, eps, h, codes, scales, i8, stream);
}

hipError_t launch_quant_rows_i8_bf16(int64_t m, int64_t k, const void* a, void* codes, float* scales,
                                     hipStream_t stream) {
  return run_quant_rows<unsigned short>(m, k, a, codes, scales, stream);
}

hipError_t launch_quant_rows_i8_f32(int64_t n, int64_t k, const float* w, void* codes, float* scales,
                                    hipStream_t stream) {
  return run_quant_rows<float>(n, k, w, codes, scales, stream);
}

}  // namespace fp8bq

// Root-mean-square norm with the residual's addition and an 8-bit output, and
// the per-row int8 quantisers, gfx950.
//
// Page 3 (zskr.cn blog), section 3.3, fuses the norm with the quantisation of
// the linear layer's input; section 2.2 stores weights as INT8. Per row:
//   h = bf16(x + r), inv = 1 / sqrt(mean(h^2) + eps), y = bf16((h inv) w),
// the sum of squares, the root and the two products in 64 bits: an fp32
// product rounds a few values in 10^8 to the other side of a bf16 border,
// which moves the scale of their group by 2^-8 where they are its maximum.
// then y is quantised as fp8bq_quant_act does (a scale per 128 columns) or to
// int8 with a scale per row. Rounding y to bf16 is what the separate norm and
// quantiser do (their interface is bf16), so the fused codes equal theirs bit
// for bit; h is rounded because the residual stream is bf16 and the norm has
// to see what the next layer will see.
#include "device_common.h"
#include "step_launch.h"

namespace fp8bq {

namespace {

constexpr float kI8Max = 127.f;

// Sum and maximum over the workgroup (every thread gets it). `slots` holds
// one value per wave; a barrier on both sides lets it be used again.
__device__ __forceinline__ double block_sum(double v, double* slots) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  const int waves = blockDim.x >> 6;
  if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = v;
  __syncthreads();
  double sum = 0.0;
  for (int i = 0; i < waves; ++i) sum += slots[i];
  __syncthreads();
  return sum;
}

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

// Scale of an int8 row from its amax.
__device__ __forceinline__ float row_scale(float amax) { return amax > 0.f ? amax / kI8Max : 1.f; }

// int8 codes of four quotients, byte i = the i-th.
__device__ __forceinline__ unsigned pack4_i8(float q0, float q1, float q2, float q3) {
  const int c0 = static_cast<int>(rintf(q0)), c1 = static_cast<int>(rintf(q1));
  const int c2 = static_cast<int>(rintf(q2)), c3 = static_cast<int>(rintf(q3));
  return (c0 & 0xff) | ((c1 & 0xff) << 8) | ((c2 & 0xff) << 16) | (static_cast<unsigned>(c3) << 24);
}

__device__ __forceinline__ void unpack8(const v4u& p, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_lo(p[i]);
    x[2 * i + 1] = bf16_hi(p[i]);
  }
}

// One row per workgroup and trip; thread t holds the 8-value chunks t,
// t + blockDim, ... (CH of them) as packed bf16.
template <int CH, bool RES, bool I8>
__global__ __launch_bounds__(1024) void rmsnorm_quant_kernel(int64_t m, int k, const unsigned short* __restrict__ x,
                                                             const unsigned short* r,
                                                             const unsigned short* __restrict__ w, double eps,
                                                             unsigned short* h_out, unsigned char* __restrict__ codes,
                                                             float* __restrict__ scales) {
  __shared__ double sums[16];
  __shared__ float tops[16];
  const int chunks = k >> 3;
  for (int64_t row = blockIdx.x; row < m; row += gridDim.x) {
    v4u h[CH];
    double sum = 0.0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = threadIdx.x + c * blockDim.x;
      h[c] = v4u{0u, 0u, 0u, 0u};
      if (i < chunks) {
        const int64_t at = row * k + 8 * i;
        h[c] = *reinterpret_cast<const v4u*>(x + at);
        if constexpr (RES) {
          const v4u rv = *reinterpret_cast<const v4u*>(r + at);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            h[c][j] = pack_bf16x2(bf16_lo(h[c][j]) + bf16_lo(rv[j]), bf16_hi(h[c][j]) + bf16_hi(rv[j]));
          *reinterpret_cast<v4u*>(h_out + at) = h[c];
        }
      }
      float f[8];
      unpack8(h[c], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fma(static_cast<double>(f[j]), static_cast<double>(f[j]), sum);
    }
    sum = block_sum(sum, sums);
    const double inv = 1.0 / sqrt(sum / k + eps);
    float top = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = threadIdx.x + c * blockDim.x;
      v4u wv = v4u{0u, 0u, 0u, 0u};
      if (i < chunks) wv = *reinterpret_cast<const v4u*>(w + 8 * i);
      float f[8], g[8];
      unpack8(h[c], f);
      unpack8(wv, g);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        h[c][j] = pack_bf16x2(static_cast<float>((f[2 * j] * inv) * g[2 * j]),
                              static_cast<float>((f[2 * j + 1] * inv) * g[2 * j + 1]));
      unpack8(h[c], f);
      float amax = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(f[j]));
      if constexpr (I8) {
        top = fmaxf(top, amax);
      } else {
#pragma unroll
        for (int off = 8; off >= 1; off >>= 1) amax = fmaxf(amax, __shfl_xor(amax, off, 16));
        const float s = group_scale(amax);
        float q[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) q[j] = scaled_clamped(f[j], s);
        if (i < chunks) {
          *reinterpret_cast<v2u*>(codes + row * k + 8 * i) =
              v2u{encode4_e4m3(q[0], q[1], q[2], q[3]), encode4_e4m3(q[4], q[5], q[6], q[7])};
          if ((i & 15) == 0) scales[row * (k >> 7) + (i >> 4)] = s;
        }
      }
    }
    if constexpr (I8) {
      top = block_max(top, tops);
      const float s = row_scale(top);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int i = threadIdx.x + c * blockDim.x;
        float f[8];
        unpack8(h[c], f);
        if (i < chunks)
          *reinterpret_cast<v2u*>(codes + row * k + 8 * i) =
              v2u{pack4_i8(f[0] / s, f[1] / s, f[2] / s, f[3] / s), pack4_i8(f[4] / s, f[5] / s, f[6] / s, f[7] / s)};
      }
      if (threadIdx.x == 0) scales[row] = s;
    }
  }
}

// int8 codes and one scale per row of a bf16 or fp32 matrix.
template <int CH, typename T>
__global__ __launch_bounds__(1024) void quant_rows_i8_kernel(int64_t m, int k, const T* __restrict__ a,
                                                             unsigned char* __restrict__ codes,
                                                             float* __restrict__ scales) {
  __shared__ float tops[16];
  const int chunks = k >> 3;
  for (int64_t row = blockIdx.x; row < m; row += gridDim.x) {
    float f[CH][8];
    float top = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = threadIdx.x + c * blockDim.x;
#pragma unroll
      for (int j = 0; j < 8; ++j) f[c][j] = 0.f;
      if (i < chunks) {
        const T* p = a + row * k + 8 * i;
        if constexpr (sizeof(T) == 2) {
          unpack8(*reinterpret_cast<const v4u*>(p), f[c]);
        } else {
          const v4f lo = *reinterpret_cast<const v4f*>(p), hi = *reinterpret_cast<const v4f*>(p + 4);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            f[c][j] = lo[j];
            f[c][4 + j] = hi[j];
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(f[c][j]));
    }
    top = block_max(top, tops);
    const float s = row_scale(top);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = threadIdx.x + c * blockDim.x;
      if (i < chunks)
        *reinterpret_cast<v2u*>(codes + row * k + 8 * i) =
            v2u{pack4_i8(f[c][0] / s, f[c][1] / s, f[c][2] / s, f[c][3] / s),
                pack4_i8(f[c][4] / s, f[c][5] / s, f[c][6] / s, f[c][7] / s)};
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
hipError_t run_rmsnorm(int threads, int64_t m, int64_t k, const void* x, const void* r, const void* w, double eps,
                       void* h, void* codes, float* scales, bool i8, hipStream_t stream) {
  const auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(row_grid(m)), dim3(threads), 0, stream, m, static_cast<int>(k),
                       static_cast<const unsigned short*>(x), static_cast<const unsigned short*>(r),
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
  switch (rs.chunks) {
    case 1: return go(quant_rows_i8_kernel<1, T>);
    case 2: return go(quant_rows_i8_kernel<2, T>);
    case 4: return go(quant_rows_i8_kernel<4, T>);
    default: return go(quant_rows_i8_kernel<8, T>);
  }
}

}  // namespace

hipError_t launch_rmsnorm_quant(int64_t m, int64_t k, const void* x, const void* r, const void* w, double eps,
                                void* h, void* codes, float* scales, bool i8, hipStream_t stream) {
  const RowShape rs = row_shape(k);
  switch (rs.chunks) {
    case 1: return run_rmsnorm<1>(rs.threads, m, k, x, r, w, eps, h, codes, scales, i8, stream);
    case 2: return run_rmsnorm<2>(rs.threads, m, k, x, r, w, eps, h, codes, scales, i8, stream);
    case 4: return run_rmsnorm<4>(rs.threads, m, k, x, r, w, eps, h, codes, scales, i8, stream);
    default: return run_rmsnorm<8>(rs.threads, m, k, x, r, w, eps, h, codes, scales, i8, stream);
  }
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

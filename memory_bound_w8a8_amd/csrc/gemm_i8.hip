// Matrix product in 8-bit integers with a scale per token and per weight row,
// gfx950 (page 3, zskr.cn blog, section 2.2: INT8 weights).
//
// C[m, n] = bf16(fp32(sum_k A[m, k] W[n, k]) * (sa[m] * sw[n])). The sums are
// exact in 32-bit integers (K < 2^17), so the tiles, the order and the split
// of K do not show in the result, and the scales are applied once per output.
#include "device_common.h"
#include "launch.h"
#include "step_launch.h"

namespace fp8bq {

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));

// 16 x 16 outputs, K = 64: lane l supplies 16 bytes of row l % 16 of the
// first operand and of column l % 16 of the second, K-slots 16 (l / 16) ..
// +15; result element i of lane l is row 4 (l / 16) + i, column l % 16.
__device__ __forceinline__ v4i mfma_16x16x64_i8(const v4u& a, const v4u& b, const v4i& c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(v4i, a), __builtin_bit_cast(v4i, b), c, 0, 0, 0);
}

// 64 x 64 tile, 4 waves of 32 x 32, one 128-byte K step at a time through LDS
// (rows of 128 bytes, 16-byte piece c at c ^ (row & 7)).
__global__ __launch_bounds__(256) void gemm_i8_tile_kernel(int64_t m_rows, int64_t n, int64_t k,
                                                           const unsigned char* __restrict__ aq,
                                                           const float* __restrict__ as,
                                                           const unsigned char* __restrict__ wq,
                                                           const float* __restrict__ ws,
                                                           unsigned short* __restrict__ c) {
  __shared__ v4u la[64 * 8], lw[64 * 8];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int lrow = lane & 15, quarter = lane >> 4;
  const int wm = (wave & 1) * 32, wn = (wave >> 1) * 32;
  const int64_t n_tiles = (n + 63) / 64;
  const int64_t m0 = blockIdx.x / n_tiles * 64, n0 = blockIdx.x % n_tiles * 64;
  v4i acc[2][2];
  for (auto& x : acc)
    for (auto& y : x) y = v4i{0, 0, 0, 0};
  for (int64_t g = 0; g < k; g += 128) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = (t >> 3) + 32 * j, piece = t & 7;
      const int64_t ra = m0 + r < m_rows ? m0 + r : m_rows - 1;
      const int64_t rw = n0 + r < n ? n0 + r : n - 1;
      la[8 * r + (piece ^ (r & 7))] = *reinterpret_cast<const v4u*>(aq + ra * k + g + 16 * piece);
      lw[8 * r + (piece ^ (r & 7))] = *reinterpret_cast<const v4u*>(wq + rw * k + g + 16 * piece);
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      v4u af[2], wf[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = 16 * j + lrow;
        af[j] = la[8 * (wm + r) + ((quarter + 4 * h) ^ (r & 7))];
        wf[j] = lw[8 * (wn + r) + ((quarter + 4 * h) ^ (r & 7))];
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = mfma_16x16x64_i8(wf[i], af[j], acc[i][j]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int64_t m = m0 + wm + 16 * j + lrow;
    if (m >= m_rows) continue;
    const float sa = as[m];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t col = n0 + wn + 16 * i + 4 * quarter + e;
        if (col < n)
          c[m * n + col] = static_cast<unsigned short>(
              pack_bf16x2(static_cast<float>(acc[i][j][e]) * (sa * ws[col]), 0.f) & 0xffffu);
      }
  }
}

}  // namespace

int64_t gemm_i8_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_gemm_i8(int64_t m, int64_t n, int64_t k, const void* aq, const float* as, const void* wq,
                          const float* ws, void* c, void*, hipStream_t stream) {
  const int64_t tiles = ((m + 63) / 64) * ((n + 63) / 64);
  if (tiles >= int64_t(1) << 24) return hipErrorInvalidValue;  // 2^32 threads
  hipLaunchKernelGGL(gemm_i8_tile_kernel, dim3(static_cast<unsigned>(tiles)), dim3(256), 0, stream, m, n, k,
                     static_cast<const unsigned char*>(aq), as, static_cast<const unsigned char*>(wq), ws,
                     static_cast<unsigned short*>(c));
  dispatch_log("gemm_i8", m, n, k, "gemm_i8_tile_kernel 64x64");
  return hipGetLastError();
}

}  // namespace fp8bq

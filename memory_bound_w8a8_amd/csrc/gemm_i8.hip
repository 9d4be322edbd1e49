// Matrix product in 8-bit integers with a scale per token and per weight row,
// gfx950 (page 3, zskr.cn blog, section 2.2: INT8 weights).
//
// C[m, n] = bf16(fp32(sum_k A[m, k] W[n, k]) * (sa[m] * sw[n])). The sums are
// exact in 32-bit integers (K < 2^17), so the tiles, the order and the split
// of K do not show in the result, and the scales are applied once per output.
#include "device_common.h"
#include "gemm_i8_tiled.h"
#include "launch.h"
#include "step_launch.h"

namespace fp8bq {

namespace {

template <int BM, int BN, int WM, int WN, int STAGES>
hipError_t tile(int64_t m, int64_t n, int64_t k, const void* aq, const float* as, const void* wq, const float* ws,
                void* c, hipStream_t stream) {
  const int64_t tiles = ((m + BM - 1) / BM) * ((n + BN - 1) / BN);
  if (tiles >= int64_t(1) << 24) return hipErrorInvalidValue;  // 2^32 threads
  hipLaunchKernelGGL((gemm_i8_tiled_kernel<BM, BN, WM, WN, STAGES>), dim3(static_cast<unsigned>(tiles)),
                     dim3(64 * WM * WN), 0, stream, m, n, k, 1, static_cast<const unsigned char*>(aq), as,
                     static_cast<const unsigned char*>(wq), ws, static_cast<unsigned short*>(c), nullptr);
  dispatch_log("gemm_i8", m, n, k, "gemm_i8_tiled_kernel");
  return hipGetLastError();
}

}  // namespace

int64_t gemm_i8_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_gemm_i8(int64_t m, int64_t n, int64_t k, const void* aq, const float* as, const void* wq,
                          const float* ws, void* c, void*, hipStream_t stream) {
  if (m > 512) return tile<256, 256, 2, 2, 2>(m, n, k, aq, as, wq, ws, c, stream);
  if (m > 64) return tile<128, 128, 2, 2, 4>(m, n, k, aq, as, wq, ws, c, stream);
  return launch_gemm_i8_rows(m, n, k, aq, as, wq, ws, c, stream);
}

}  // namespace fp8bq

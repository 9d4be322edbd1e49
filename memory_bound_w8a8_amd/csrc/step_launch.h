// Host-side launchers of the operators of fp8bq_step.h (internal to
// libfp8bq.so). Arguments are validated by step_api.hip first.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8bq {

// norm_quant.hip. r, h: both null or neither. i8: int8 codes with a scale per
// row, else e4m3 codes with a scale per 128 columns.
hipError_t launch_rmsnorm_quant(int64_t m, int64_t k, const void* x, const void* r, const void* w, double eps,
                                void* h, void* codes, float* scales, bool i8, hipStream_t stream);
hipError_t launch_quant_rows_i8_bf16(int64_t m, int64_t k, const void* a, void* codes, float* scales,
                                     hipStream_t stream);
hipError_t launch_quant_rows_i8_f32(int64_t n, int64_t k, const float* w, void* codes, float* scales,
                                    hipStream_t stream);

// gemm_i8.hip. workspace: gemm_i8_workspace_bytes(m, n, k) bytes, or null for
// the plan without one. gemm_i8_fits: whether one grid takes the tiles.
bool gemm_i8_fits(int64_t m, int64_t n);
int64_t gemm_i8_workspace_bytes(int64_t m, int64_t n, int64_t k);
hipError_t launch_gemm_i8(int64_t m, int64_t n, int64_t k, const void* aq, const float* as, const void* wq,
                          const float* ws, void* c, void* workspace, hipStream_t stream);

// gemm_i8_rows.hip: m <= 64
hipError_t launch_gemm_i8_rows(int64_t m, int64_t n, int64_t k, const void* aq, const float* as, const void* wq,
                               const float* ws, void* c, hipStream_t stream);

// verify.hip
int64_t verify_workspace_bytes(int64_t b, int64_t v);
hipError_t launch_verify(int64_t b, int n_drafts, int64_t v, bool bf16, const void* target, const void* draft,
                         const int* drafts, const int* draft_len, const float* u_accept, const float* u_sample,
                         void* workspace, int* tokens, int* accepted, hipStream_t stream);

}  // namespace fp8bq

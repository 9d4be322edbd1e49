// C ABI of the operators of include/fp8bq_step.h: host-side validation and
// dispatch.
#include <cmath>

#include "api_checks.h"
#include "fp8bq_step.h"
#include "launch.h"
#include "step_launch.h"

namespace {

using fp8bq::aligned;
using fp8bq::check_device;
using fp8bq::launch_status;
using fp8bq::product_ok;

constexpr int64_t kMaxIndex = (int64_t(1) << 31) - 1;  // rows form a grid dimension, indices are int32
constexpr int64_t kMaxSequences = 65535;               // sequences form the grid's y dimension

int check_rows(int64_t rows, int64_t k) {
  if (rows < 0 || rows > kMaxIndex || k < 0 || k % 128 != 0 || k > FP8BQ_NORM_MAX_K || !product_ok(rows, k))
    return FP8BQ_ERR_SHAPE;
  return FP8BQ_OK;
}

int rmsnorm_quant(int64_t M, int64_t K, const void* X, const void* R, const void* weight, double eps, void* H,
                  void* codes, float* scales, bool i8, void* stream) {
  int st = check_rows(M, K);
  if (st != FP8BQ_OK) return st;
  if (!(eps > 0.0) || std::isinf(eps)) return FP8BQ_ERR_VALUE;
  if (M == 0 || K == 0) return FP8BQ_OK;
  if (X == nullptr || weight == nullptr || codes == nullptr || scales == nullptr) return FP8BQ_ERR_NULL;
  if (R == nullptr) H = nullptr;
  if (R != nullptr && H == nullptr) return FP8BQ_ERR_NULL;
  if (!aligned(X, 16) || !aligned(R, 16) || !aligned(weight, 16) || !aligned(H, 16) || !aligned(codes, 16) ||
      !aligned(scales, 4))
    return FP8BQ_ERR_ALIGN;
  st = check_device();
  if (st != FP8BQ_OK) return st;
  return launch_status(fp8bq::launch_rmsnorm_quant(M, K, X, R, weight, eps, H, codes, scales, i8,
                                                   static_cast<hipStream_t>(stream)));
}

int check_gemm_i8_sizes(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 0 || K < 0 || K % 128 != 0 || K > FP8BQ_GEMM_I8_MAX_K || M > kMaxIndex || N > kMaxIndex)
    return FP8BQ_ERR_SHAPE;
  if (!product_ok(M, K) || !product_ok(N, K) || !product_ok(M, N) || !fp8bq::gemm_i8_fits(M, N))
    return FP8BQ_ERR_SHAPE;
  return FP8BQ_OK;
}

int check_verify_sizes(int64_t B, int64_t n_drafts, int64_t V) {
  if (B < 0 || B > kMaxSequences || n_drafts < 0 || n_drafts > FP8BQ_MAX_DRAFTS || V < 1 || V > kMaxIndex ||
      !product_ok(B * (n_drafts + 1), V))
    return FP8BQ_ERR_SHAPE;
  return FP8BQ_OK;
}

}  // namespace

extern "C" {

int fp8bq_rmsnorm_quant(int64_t M, int64_t K, const void* X_bf16, const void* R_bf16, const void* weight, double eps,
                        void* H_bf16, void* A_fp8, float* A_scales, void* stream) {
  return rmsnorm_quant(M, K, X_bf16, R_bf16, weight, eps, H_bf16, A_fp8, A_scales, false, stream);
}

int fp8bq_rmsnorm_quant_i8(int64_t M, int64_t K, const void* X_bf16, const void* R_bf16, const void* weight,
                           double eps, void* H_bf16, void* A_i8, float* A_scales, void* stream) {
  return rmsnorm_quant(M, K, X_bf16, R_bf16, weight, eps, H_bf16, A_i8, A_scales, true, stream);
}

int fp8bq_quant_act_i8(int64_t M, int64_t K, const void* A_bf16, void* A_i8, float* A_scales, void* stream) {
  int st = check_rows(M, K);
  if (st != FP8BQ_OK) return st;
  if (M == 0 || K == 0) return FP8BQ_OK;
  if (A_bf16 == nullptr || A_i8 == nullptr || A_scales == nullptr) return FP8BQ_ERR_NULL;
  if (!aligned(A_bf16, 16) || !aligned(A_i8, 16) || !aligned(A_scales, 4)) return FP8BQ_ERR_ALIGN;
  st = check_device();
  if (st != FP8BQ_OK) return st;
  return launch_status(
      fp8bq::launch_quant_rows_i8_bf16(M, K, A_bf16, A_i8, A_scales, static_cast<hipStream_t>(stream)));
}

int fp8bq_quant_weight_i8(int64_t N, int64_t K, const float* W_f32, void* W_i8, float* W_scales, void* stream) {
  int st = check_rows(N, K);
  if (st != FP8BQ_OK) return st;
  if (N == 0 || K == 0) return FP8BQ_OK;
  if (W_f32 == nullptr || W_i8 == nullptr || W_scales == nullptr) return FP8BQ_ERR_NULL;
  if (!aligned(W_f32, 16) || !aligned(W_i8, 16) || !aligned(W_scales, 4)) return FP8BQ_ERR_ALIGN;
  st = check_device();
  if (st != FP8BQ_OK) return st;
  return launch_status(
      fp8bq::launch_quant_rows_i8_f32(N, K, W_f32, W_i8, W_scales, static_cast<hipStream_t>(stream)));
}

int64_t fp8bq_gemm_i8_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  const int st = check_gemm_i8_sizes(M, N, K);
  if (st != FP8BQ_OK) return st;
  if (M == 0 || N == 0 || K == 0) return 0;
  return fp8bq::gemm_i8_workspace_bytes(M, N, K);
}

int fp8bq_gemm_i8(int64_t M, int64_t N, int64_t K, const void* A_i8, const float* A_scales, const void* W_i8,
                  const float* W_scales, void* C_bf16, void* workspace, int64_t workspace_bytes, void* stream) {
  int st = check_gemm_i8_sizes(M, N, K);
  if (st != FP8BQ_OK) return st;
  if (workspace_bytes < 0) return FP8BQ_ERR_SHAPE;
  if (workspace_bytes > 0 && workspace == nullptr) return FP8BQ_ERR_NULL;
  if (!aligned(workspace, 16)) return FP8BQ_ERR_ALIGN;
  if (M == 0 || N == 0) return FP8BQ_OK;
  if (C_bf16 == nullptr) return FP8BQ_ERR_NULL;
  if (!aligned(C_bf16, 16)) return FP8BQ_ERR_ALIGN;
  if (K > 0) {
    if (A_i8 == nullptr || A_scales == nullptr || W_i8 == nullptr || W_scales == nullptr) return FP8BQ_ERR_NULL;
    if (!aligned(A_i8, 16) || !aligned(W_i8, 16) || !aligned(A_scales, 4) || !aligned(W_scales, 4))
      return FP8BQ_ERR_ALIGN;
  }
  st = check_device();
  if (st != FP8BQ_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (K == 0) return launch_status(fp8bq::launch_fill_zero_bf16(M * N, C_bf16, s));
  if (workspace_bytes < fp8bq::gemm_i8_workspace_bytes(M, N, K)) workspace = nullptr;
  return launch_status(fp8bq::launch_gemm_i8(M, N, K, A_i8, A_scales, W_i8, W_scales, C_bf16, workspace, s));
}

int64_t fp8bq_verify_workspace_bytes(int64_t B, int64_t n_drafts, int64_t V) {
  const int st = check_verify_sizes(B, n_drafts, V);
  if (st != FP8BQ_OK) return st;
  return fp8bq::verify_workspace_bytes(B, V);
}

int fp8bq_verify_drafts(int64_t B, int64_t n_drafts, int64_t V, int dtype, const void* target_p, const void* draft_p,
                        const int32_t* drafts, const int32_t* draft_len, const float* u_accept, const float* u_sample,
                        void* workspace, int64_t workspace_bytes, int32_t* tokens, int32_t* accepted, void* stream) {
  int st = check_verify_sizes(B, n_drafts, V);
  if (st != FP8BQ_OK) return st;
  if (dtype != FP8BQ_F32 && dtype != FP8BQ_BF16) return FP8BQ_ERR_VALUE;
  if (B == 0) return FP8BQ_OK;
  if (workspace_bytes < fp8bq::verify_workspace_bytes(B, V)) return FP8BQ_ERR_SHAPE;
  if (target_p == nullptr || u_sample == nullptr || workspace == nullptr || tokens == nullptr || accepted == nullptr)
    return FP8BQ_ERR_NULL;
  if (n_drafts > 0 && (drafts == nullptr || u_accept == nullptr)) return FP8BQ_ERR_NULL;
  const uintptr_t pa = dtype == FP8BQ_F32 ? 4 : 2;
  if (!aligned(target_p, pa) || !aligned(draft_p, pa) || !aligned(workspace, 16) || !aligned(drafts, 4) ||
      !aligned(draft_len, 4) || !aligned(u_accept, 4) || !aligned(u_sample, 4) || !aligned(tokens, 4) ||
      !aligned(accepted, 4))
    return FP8BQ_ERR_ALIGN;
  st = check_device();
  if (st != FP8BQ_OK) return st;
  return launch_status(fp8bq::launch_verify(B, static_cast<int>(n_drafts), V, dtype == FP8BQ_BF16, target_p, draft_p,
                                            drafts, draft_len, u_accept, u_sample, workspace, tokens, accepted,
                                            static_cast<hipStream_t>(stream)));
}

}  // extern "C"

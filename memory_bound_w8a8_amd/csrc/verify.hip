// Verification of drafted tokens against the target's probabilities, gfx950.
//
// Page 1 (SmartX blog), section "single-stream optimisation": a step drafts k
// tokens and verifies them with M = k + 1 rows of the target. Acceptance
// compares u q < p at the drafted tokens; the token after the accepted ones
// is drawn from one row of probabilities (less the drafter's row where a
// draft was rejected), which is all that has to be read whole: the operator
// is bound by that read, 4 or 8 bytes per word and sequence.
//
// The draw works on whole numbers (weights in units of 2^-32, 64-bit sums),
// so splitting a row over workgroups and threads cannot change the token.
//   1. verify_sums_kernel: a row is cut into `splits` pieces, one workgroup
//      each; every workgroup finds its sequence's rejection by itself and
//      writes its piece's sum.
//   2. verify_draw_kernel: one workgroup per sequence finds the piece that
//      holds the drawn point and scans it.
#include "device_common.h"
#include "step_launch.h"

namespace fp8bq {

namespace {

typedef unsigned long long u64;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

struct Verify {
  int n_drafts;
  int64_t v;
  const void* target;
  const void* draft;  // null: drafts are certain
  const int* drafts;
  const int* draft_len;  // null: n_drafts each
  const float* u_accept;
  const float* u_sample;
};

template <bool BF16>
__device__ __forceinline__ float prob(const void* p, int64_t i) {
  if constexpr (BF16) return bf16_lo(static_cast<const unsigned short*>(p)[i]);
  return static_cast<const float*>(p)[i];
}

// Nearest whole number of 2^-32 (ties to even). The hardware conversion
// holds results to 0 .. 2^32 - 1 and gives 0 for NaN.
__device__ __forceinline__ unsigned weight_units(float w) {
  const float x = rintf(w * 0x1p32f);
  unsigned u;
  asm("v_cvt_u32_f32 %0, %1" : "=v"(u) : "v"(x));
  return u;
}

// Drafts of sequence b that are accepted, and whether one was rejected after
// them. Called by whole waves; the result is the same in every lane.
template <bool BF16>
__device__ __forceinline__ int accepted_drafts(const Verify& a, int64_t b, bool* rejected) {
  const int lane = threadIdx.x & 63;
  int len = a.n_drafts;
  if (a.draft_len != nullptr) {
    const int l = a.draft_len[b];
    len = l < 0 ? 0 : (l < len ? l : len);
  }
  bool ok = false;
  if (lane < len) {
    const int64_t i = b * a.n_drafts + lane;
    const int d = a.drafts[i];
    if (d >= 0 && d < a.v) {
      const double p = prob<BF16>(a.target, (b * (a.n_drafts + 1) + lane) * a.v + d);
      const double q = a.draft != nullptr ? static_cast<double>(prob<BF16>(a.draft, i * a.v + d)) : 1.0;
      ok = static_cast<double>(a.u_accept[i]) * q < p;  // 24 x 24 bits: exact
    }
  }
  const u64 no = ~__ballot(ok) & (len == 64 ? ~0ull : (1ull << len) - 1);
  *rejected = no != 0;
  return no != 0 ? __builtin_ctzll(no) : len;
}

// A row of weights: the target's probabilities, less the drafter's.
template <bool BF16>
struct Row {
  const void* p;
  const void* q;      // null: nothing, or 1 at `certain`
  int64_t certain;    // -1: none
  __device__ __forceinline__ Row(const Verify& a, int64_t b, int r, bool less) {
    const int each = BF16 ? 2 : 4;
    p = static_cast<const char*>(a.target) + (b * (a.n_drafts + 1) + r) * a.v * each;
    q = less && a.draft != nullptr ? static_cast<const char*>(a.draft) + (b * a.n_drafts + r) * a.v * each : nullptr;
    certain = less && a.draft == nullptr ? a.drafts[b * a.n_drafts + r] : -1;
  }
  __device__ __forceinline__ unsigned at(int64_t i) const {
    float w = prob<BF16>(p, i);
    if (q != nullptr) w -= prob<BF16>(q, i);
    if (i == certain) w -= 1.f;
    return weight_units(w);
  }
};

__device__ __forceinline__ u64 wave_sum(u64 v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

__device__ __forceinline__ u64 block_sum(u64 v, u64* slots) {
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = v;
  __syncthreads();
  u64 s = 0;
  for (int i = 0; i < kWaves; ++i) s += slots[i];
  __syncthreads();
  return s;
}

template <bool BF16>
__global__ __launch_bounds__(kThreads) void verify_sums_kernel(Verify a, u64* __restrict__ part) {
  __shared__ u64 slots[kWaves];
  const int64_t b = blockIdx.y;
  bool rejected;
  const int r = accepted_drafts<BF16>(a, b, &rejected);
  const Row<BF16> row(a, b, r, rejected);
  const int64_t piece = (a.v + gridDim.x - 1) / gridDim.x;
  const int64_t lo = piece * blockIdx.x;
  const int64_t hi = lo + piece < a.v ? lo + piece : a.v;
  u64 sum = 0;
  for (int64_t i = lo + threadIdx.x; i < hi; i += kThreads) sum += row.at(i);
  sum = block_sum(sum, slots);
  if (threadIdx.x == 0) part[b * gridDim.x + blockIdx.x] = sum;
}

// The lowest index of [lo, hi) whose running sum (starting from `sum`) exceeds
// `goal`, or -1; the same in every thread.
template <bool BF16>
__device__ int64_t scan_row(const Row<BF16>& row, int64_t lo, int64_t hi, u64 sum, u64 goal, u64* slots, int* found) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (threadIdx.x == 0) *found = -1;
  __syncthreads();
  for (int64_t at = lo; at < hi; at += kThreads) {
    const int64_t i = at + threadIdx.x;
    const u64 w = i < hi ? row.at(i) : 0;
    u64 run = w;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const u64 up = __shfl_up(run, off, 64);
      if (lane >= off) run += up;
    }
    if (lane == 63) slots[wave] = run;
    __syncthreads();
    u64 base = sum;
    for (int j = 0; j < kWaves; ++j) {
      if (j < wave) base += slots[j];
      sum += slots[j];
    }
    run += base;
    if (run > goal && run - w <= goal) *found = threadIdx.x;  // one thread at most: sums rise
    __syncthreads();
    if (*found >= 0) return at + *found;
  }
  return -1;
}

template <bool BF16>
__global__ __launch_bounds__(kThreads) void verify_draw_kernel(Verify a, const u64* __restrict__ part, int splits,
                                                               int* __restrict__ tokens, int* __restrict__ accepted) {
  __shared__ u64 slots[kWaves];
  __shared__ int found;
  const int64_t b = blockIdx.x;
  bool rejected;
  const int r = accepted_drafts<BF16>(a, b, &rejected);
  float s = a.u_sample[b] * 0x1p32f;
  unsigned s32;
  asm("v_cvt_u32_f32 %0, %1" : "=v"(s32) : "v"(s));
  const u64 point = static_cast<u64>(s32) << 32;

  u64 total = 0;
  for (int i = 0; i < splits; ++i) total += part[b * splits + i];
  int64_t token = -1;
  if (total > 0) {
    const u64 goal = __umul64hi(total, point);  // floor(total * z / 2^32) < total
    const int64_t piece = (a.v + splits - 1) / splits;
    u64 before = 0;
    int at = 0;
    while (at + 1 < splits && before + part[b * splits + at] <= goal) before += part[b * splits + at++];
    const int64_t lo = piece * at;
    const int64_t hi = lo + piece < a.v ? lo + piece : a.v;
    token = scan_row<BF16>(Row<BF16>(a, b, r, rejected), lo, hi, before, goal, slots, &found);
  } else if (rejected) {  // the drafter's row covers the target's: the target's itself
    const Row<BF16> row(a, b, r, false);
    u64 sum = 0;
    for (int64_t i = threadIdx.x; i < a.v; i += kThreads) sum += row.at(i);
    sum = block_sum(sum, slots);
    if (sum > 0) token = scan_row<BF16>(row, 0, a.v, 0, __umul64hi(sum, point), slots, &found);
  }
  for (int i = threadIdx.x; i <= a.n_drafts; i += kThreads)
    tokens[b * (a.n_drafts + 1) + i] =
        i < r ? a.drafts[b * a.n_drafts + i] : (i == r ? static_cast<int>(token) : -1);
  if (threadIdx.x == 0) accepted[b] = r;
}

int split_count(int64_t b, int64_t v) {
  int64_t s = (1024 + b - 1) / b;
  const int64_t most = (v + 1023) / 1024;  // at least 1024 words per piece
  s = s < most ? s : most;
  return static_cast<int>(s < 256 ? s : 256);
}

}  // namespace

int64_t verify_workspace_bytes(int64_t b, int64_t v) { return b == 0 ? 0 : 8 * b * split_count(b, v); }

hipError_t launch_verify(int64_t b, int n_drafts, int64_t v, bool bf16, const void* target, const void* draft,
                         const int* drafts, const int* draft_len, const float* u_accept, const float* u_sample,
                         void* workspace, int* tokens, int* accepted, hipStream_t stream) {
  const Verify a{n_drafts, v, target, draft, drafts, draft_len, u_accept, u_sample};
  const int splits = split_count(b, v);
  u64* part = static_cast<u64*>(workspace);
  const dim3 grid(static_cast<unsigned>(splits), static_cast<unsigned>(b));
  const dim3 seqs(static_cast<unsigned>(b));
  if (bf16) {
    hipLaunchKernelGGL(verify_sums_kernel<true>, grid, dim3(kThreads), 0, stream, a, part);
    hipLaunchKernelGGL(verify_draw_kernel<true>, seqs, dim3(kThreads), 0, stream, a, part, splits, tokens, accepted);
  } else {
    hipLaunchKernelGGL(verify_sums_kernel<false>, grid, dim3(kThreads), 0, stream, a, part);
    hipLaunchKernelGGL(verify_draw_kernel<false>, seqs, dim3(kThreads), 0, stream, a, part, splits, tokens, accepted);
  }
  return hipGetLastError();
}

}  // namespace fp8bq

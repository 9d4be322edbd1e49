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
// so cutting a row into parts cannot change the token.
//   1. verify_sums_kernel: each wave of a row's workgroups sums one part of
//      it, 16 bytes a lane and load. Every wave finds its sequence's rejection
//      by itself (two dependent loads); the first one writes it down.
//   2. verify_draw_kernel: one workgroup of 8 waves per sequence finds the part
//      that holds the drawn point by a scan over the parts' sums, two a thread,
//      and scans that part the same way, 16 bytes a thread and trip.
#include "device_common.h"
#include "step_launch.h"

namespace fp8bq {

namespace {

typedef unsigned long long u64;

constexpr int kSumThreads = 256;
constexpr int kSumWaves = kSumThreads / 64;
constexpr int kDrawThreads = 512;
constexpr int kDrawWaves = kDrawThreads / 64;
constexpr int kMaxParts = 2 * kDrawThreads;  // the scan over the parts: two a thread

struct Verify {
  int n_drafts;
  int64_t v;
  const void* target;
  const void* draft;  // null: drafts are certain
  const int* drafts;
  const int* draft_len;  // null: n_drafts each
  const float* u_accept;
  const float* u_sample;
  // workspace: a sum of each part of each sequence's row, and what became of
  // the sequence's drafts (accepted ones, + kRejected where one was rejected)
  u64* sums;
  int* state;
  int parts;
  int64_t part_words;
};
constexpr int kRejected = 256;

template <bool BF16>
__device__ __forceinline__ float prob(const void* p, int64_t i) {
  if constexpr (BF16) return bf16_lo(static_cast<const unsigned short*>(p)[i]);
  return static_cast<const float*>(p)[i];
}

// 16 bytes of probabilities from any word: a row of an odd vocabulary starts
// at a multiple of the word's size only.
template <bool BF16>
struct Vec {
  static constexpr int kWords = BF16 ? 8 : 4;
  typedef v4u __attribute__((aligned(2))) at2;
  typedef v4u __attribute__((aligned(4))) at4;
  v4u raw;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    if constexpr (BF16)
      raw = *reinterpret_cast<const at2*>(static_cast<const unsigned short*>(p) + i);
    else
      raw = *reinterpret_cast<const at4*>(static_cast<const float*>(p) + i);
  }
  __device__ __forceinline__ float word(int j) const {
    if constexpr (BF16) return j & 1 ? bf16_hi(raw[j >> 1]) : bf16_lo(raw[j >> 1]);
    return __builtin_bit_cast(float, static_cast<unsigned>(raw[j]));
  }
};

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
  const void* q;    // null: nothing, or 1 at `certain`
  int64_t certain;  // -1: none
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

// This lane's share of the weights of [lo, hi), without the certain draft's 1:
// vectors lane, lane + lanes, ... of the range; LESS: p - q.
template <bool BF16, bool LESS>
__device__ __forceinline__ u64 sum_words(const Row<BF16>& row, int64_t lo, int64_t hi, int lane, int lanes) {
  using V = Vec<BF16>;
  constexpr int W = V::kWords, U = 4;  // U vectors of each tensor in flight
  u64 sum = 0;
  const int64_t step = static_cast<int64_t>(lanes) * W;
  int64_t i = lo + static_cast<int64_t>(lane) * W;
  for (; i + (U - 1) * step + W <= hi; i += U * step) {
    V p[U], q[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      p[u].load(row.p, i + u * step);
      if constexpr (LESS) q[u].load(row.q, i + u * step);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < W; ++j) sum += weight_units(LESS ? p[u].word(j) - q[u].word(j) : p[u].word(j));
  }
  for (; i < hi; i += step) {
    if (i + W <= hi) {
      V p, q;
      p.load(row.p, i);
      if constexpr (LESS) q.load(row.q, i);
#pragma unroll
      for (int j = 0; j < W; ++j) sum += weight_units(LESS ? p.word(j) - q.word(j) : p.word(j));
    } else {
      for (int64_t x = i; x < hi; ++x)
        sum += weight_units(LESS ? prob<BF16>(row.p, x) - prob<BF16>(row.q, x) : prob<BF16>(row.p, x));
    }
  }
  return sum;
}

template <bool BF16>
__global__ __launch_bounds__(kSumThreads) void verify_sums_kernel(Verify a) {
  const int64_t b = blockIdx.y;
  const int lane = threadIdx.x & 63;
  const int part = blockIdx.x * kSumWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  bool rejected;
  const int r = accepted_drafts<BF16>(a, b, &rejected);
  if (part == 0 && lane == 0) a.state[b] = r + (rejected ? kRejected : 0);
  if (part >= a.parts) return;
  const Row<BF16> row(a, b, r, rejected);
  const int64_t lo = a.part_words * part;
  const int64_t hi = lo + a.part_words < a.v ? lo + a.part_words : a.v;
  u64 sum = row.q != nullptr ? sum_words<BF16, true>(row, lo, hi, lane, 64)
                             : sum_words<BF16, false>(row, lo, hi, lane, 64);
  sum = wave_sum(sum);
  if (lane == 0) {
    if (row.certain >= lo && row.certain < hi)
      sum += static_cast<u64>(row.at(row.certain)) - weight_units(prob<BF16>(row.p, row.certain));
    a.sums[b * a.parts + part] = sum;
  }
}

// Inclusive sums over the workgroup's threads in order; *total: all of them.
// A barrier on both sides lets `slots` be used again.
__device__ __forceinline__ u64 block_scan(u64 w, u64* slots, u64* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const u64 up = __shfl_up(w, off, 64);
    if (lane >= off) w += up;
  }
  if (lane == 63) slots[wave] = w;
  __syncthreads();
  u64 base = 0, all = 0;
#pragma unroll
  for (int j = 0; j < kDrawWaves; ++j) {
    const u64 s = slots[j];
    if (j < wave) base += s;
    all += s;
  }
  __syncthreads();
  *total = all;
  return base + w;
}

// The lowest index of [lo, hi) whose running sum (starting from `sum`) exceeds
// `goal`, or -1; the same in every thread.
template <bool BF16>
__device__ int64_t scan_row(const Row<BF16>& row, int64_t lo, int64_t hi, u64 sum, u64 goal, u64* slots, int* found) {
  using V = Vec<BF16>;
  constexpr int W = V::kWords;
  if (threadIdx.x == 0) *found = -1;
  __syncthreads();
  for (int64_t at = lo; at < hi; at += kDrawThreads * W) {
    const int64_t i = at + threadIdx.x * W;
    unsigned w[W];
    if (i + W <= hi) {
      V p, q;
      p.load(row.p, i);
      if (row.q != nullptr) q.load(row.q, i);
#pragma unroll
      for (int j = 0; j < W; ++j) {
        float x = p.word(j);
        if (row.q != nullptr) x -= q.word(j);
        if (i + j == row.certain) x -= 1.f;
        w[j] = weight_units(x);
      }
    } else {
#pragma unroll
      for (int j = 0; j < W; ++j) w[j] = i + j < hi ? row.at(i + j) : 0;
    }
    u64 mine = 0;
#pragma unroll
    for (int j = 0; j < W; ++j) mine += w[j];
    u64 trip;
    u64 run = sum + block_scan(mine, slots, &trip) - mine;
#pragma unroll
    for (int j = 0; j < W; ++j) {
      if (run <= goal && run + w[j] > goal) *found = threadIdx.x * W + j;  // one word at most: sums rise
      run += w[j];
    }
    sum += trip;
    __syncthreads();
    if (*found >= 0) return at + *found;
  }
  return -1;
}

template <bool BF16>
__global__ __launch_bounds__(kDrawThreads) void verify_draw_kernel(Verify a, int* __restrict__ tokens,
                                                                   int* __restrict__ accepted) {
  __shared__ u64 slots[kDrawWaves];
  __shared__ int found;
  __shared__ int at_part;
  __shared__ u64 before_part;
  const int64_t b = blockIdx.x;
  const int t = threadIdx.x;
  const int state = a.state[b];
  const u64* sums = a.sums + b * a.parts;
  const u64 part0 = 2 * t < a.parts ? sums[2 * t] : 0, part1 = 2 * t + 1 < a.parts ? sums[2 * t + 1] : 0;
  const int kept = t < a.n_drafts ? a.drafts[b * a.n_drafts + t] : -1;
  const float s = a.u_sample[b] * 0x1p32f;
  unsigned s32;
  asm("v_cvt_u32_f32 %0, %1" : "=v"(s32) : "v"(s));
  const u64 point = static_cast<u64>(s32) << 32;
  const bool rejected = (state & kRejected) != 0;
  const int r = state & (kRejected - 1);

  u64 total;
  const u64 run1 = block_scan(part0 + part1, slots, &total), run0 = run1 - part1;
  int64_t token = -1;
  if (total > 0) {
    const u64 goal = __umul64hi(total, point);  // floor(total * z / 2^32) < total
    // one part in all: sums rise
    if (run0 > goal && run0 - part0 <= goal) at_part = 2 * t, before_part = run0 - part0;
    if (run1 > goal && run0 <= goal) at_part = 2 * t + 1, before_part = run0;
    __syncthreads();
    const int64_t lo = a.part_words * at_part;
    const int64_t hi = lo + a.part_words < a.v ? lo + a.part_words : a.v;
    token = scan_row<BF16>(Row<BF16>(a, b, r, rejected), lo, hi, before_part, goal, slots, &found);
  } else if (rejected) {  // the drafter's row covers the target's: the target's itself
    const Row<BF16> row(a, b, r, false);
    u64 sum;
    block_scan(sum_words<BF16, false>(row, 0, a.v, t, kDrawThreads), slots, &sum);
    if (sum > 0) token = scan_row<BF16>(row, 0, a.v, 0, __umul64hi(sum, point), slots, &found);
  }
  if (t <= a.n_drafts) tokens[b * (a.n_drafts + 1) + t] = t < r ? kept : (t == r ? static_cast<int>(token) : -1);
  if (t == 0) accepted[b] = r;
}

// Words of a part: all parts are at most 8192 waves (what the CUs hold at
// once) and two a thread of the second kernel; 512 words, or multiples of 1024,
// so that every load of a wave is whole. 33 rows of 151937 bf16 words take 9.2
// us so, and 11.3 in parts of 616 that come to 8316 waves; 64 x 152064 with a
// drafter's rows 12.1 (14.7).
int64_t words_per_part(int64_t b, int64_t v) {
  const int64_t fill = b < 8192 ? 8192 / b : 1, most = fill < kMaxParts ? fill : kMaxParts;
  const int64_t words = (v + most - 1) / most;
  return words <= 512 ? 512 : (words + 1023) / 1024 * 1024;
}
int64_t part_count(int64_t b, int64_t v) {
  const int64_t words = words_per_part(b, v);
  return (v + words - 1) / words;
}

}  // namespace

int64_t verify_workspace_bytes(int64_t b, int64_t v) { return b == 0 ? 0 : b * (8 * part_count(b, v) + 4); }

hipError_t launch_verify(int64_t b, int n_drafts, int64_t v, bool bf16, const void* target, const void* draft,
                         const int* drafts, const int* draft_len, const float* u_accept, const float* u_sample,
                         void* workspace, int* tokens, int* accepted, hipStream_t stream) {
  const int parts = static_cast<int>(part_count(b, v));
  u64* sums = static_cast<u64*>(workspace);
  const Verify a{n_drafts, v,        target,   draft, drafts,
                 draft_len, u_accept, u_sample, sums,  reinterpret_cast<int*>(sums + b * parts),
                 parts,    words_per_part(b, v)};
  const dim3 grid(static_cast<unsigned>((parts + kSumWaves - 1) / kSumWaves), static_cast<unsigned>(b));
  const dim3 seqs(static_cast<unsigned>(b));
  if (bf16) {
    hipLaunchKernelGGL(verify_sums_kernel<true>, grid, dim3(kSumThreads), 0, stream, a);
    hipLaunchKernelGGL(verify_draw_kernel<true>, seqs, dim3(kDrawThreads), 0, stream, a, tokens, accepted);
  } else {
    hipLaunchKernelGGL(verify_sums_kernel<false>, grid, dim3(kSumThreads), 0, stream, a);
    hipLaunchKernelGGL(verify_draw_kernel<false>, seqs, dim3(kDrawThreads), 0, stream, a, tokens, accepted);
  }
  return hipGetLastError();
}

}  // namespace fp8bq

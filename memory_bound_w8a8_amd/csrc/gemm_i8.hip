// Matrix product in 8-bit integers with a scale per token and per weight row,
// gfx950 (page 3, zskr.cn blog, section 2.2: INT8 weights).
//
// C[m, n] = bf16(fp32(sum_k A[m, k] W[n, k]) * (sa[m] * sw[n])). The sums are
// exact in 32-bit integers (K < 2^17), so the tiles, the order and the split
// of K do not show in the result, and the scales are applied once per output.
// Up to 64 tokens gemm_i8_rows.hip streams the weights, but where plan_for finds
// tiles faster; beyond, the tiles below.
#include "device_common.h"
#include "gemm_i8_tiled.h"
#include "launch.h"
#include "step_launch.h"

namespace fp8bq {

namespace {

constexpr int64_t kCUs = 256;
constexpr int64_t kStreamRows = 64;  // tokens of the weight-streaming kernel
constexpr int64_t kSplitRows = 32;   // fewer leave half of a 64-row tile empty
constexpr int64_t kMixedRows = 48;   // from here on a 64-row tile may beat the stream

// Which tile. With c = ceil(tiles / 256) tiles on the busiest CU and s = K /
// 128 steps a call takes, in us,
//   first + s step + (c - 1) (more + s more_step)
// for the numbers of each tile: a least-squares fit over 146 shapes of 65 ..
// 3465 tokens, 512 .. 17408 weight rows and K of 512 .. 17408 drawn evenly over
// their logarithms (mean error 5%). The smallest prediction picks, over the
// same shapes, a tile within 0.3% of the fastest of these and of 256 x 256 with 8
// waves (geometric mean; 16% at worst, where one round of the latter wins).
//
// What the numbers say: a CU gets about 90 bytes a ns out of L2, so a step
// takes (BM + BN) 128 / 90 ns until, at 192 x 256, the MFMAs take as long.
// Small tiles spread few outputs over all CUs, large ones read each operand
// less often: 65 x 5120 x 5120 takes 11.1 us in 64 x 64 tiles and 18 in 128 x
// 128, 1500 x 5120 x 5120 takes 35 in 128 x 256 and 51 in 64 x 128. A CU holds
// two tiles of 64 x 64 at a time, hence their small `more`. The smaller tiles
// are not taken past `rounds`, where the fit ends.
struct Tile {
  int bm, bn;
  double first, step, more, more_step;
  int64_t rounds;
};
constexpr int64_t kAnyRounds = int64_t(1) << 40;
constexpr Tile kTiles[] = {
    {64, 64, 3.3, 0.172, 1.2, 0.171, 6},   {96, 64, 4.0, 0.215, 3.0, 0.241, 6},
    {64, 128, 3.5, 0.274, 1.5, 0.265, 6},  {96, 128, 5.5, 0.300, 3.7, 0.391, 6},
    {128, 128, 4.8, 0.354, 3.3, 0.503, 8}, {192, 128, 5.7, 0.452, 5.0, 0.657, 9},
    {128, 256, 6.4, 0.567, 4.9, 0.865, 9}, {192, 256, 7.1, 0.867, 5.9, 1.314, 9},
    {256, 256, 13.5, 1.035, 8.2, 1.500, kAnyRounds},
};
constexpr int kTileKinds = sizeof(kTiles) / sizeof(kTiles[0]);

// Adding up a split's parts: a launch, and each part's sums written and read.
constexpr double kJoin = 3.5, kJoinPerByte = 4e-7;

// The weight-streaming kernel: a start, the weights from HBM, and each further
// 16 tokens' codes, which every CU reads whole through L2 (63 bytes a ns).
constexpr double kStreamStart = 2.6, kStreamPerByte = 1 / 6.6e6, kStreamPerTokenByte = 1 / 63e3;

struct Plan {
  int kind;   // index of kTiles, or kStream
  int split;  // parts of K
};
constexpr int kStream = -1;

int64_t tile_count(const Tile& t, int64_t m, int64_t n) { return ((m + t.bm - 1) / t.bm) * ((n + t.bn - 1) / t.bn); }

// The K range is split where all tiles of the smallest kind leave most CUs
// idle: over as many workgroups of at least 4 steps as there are CUs, if the
// steps saved outweigh the join (128 x 512 x 8704: 15.9 -> 10.4 us), also up to
// 64 tokens, where the stream's codes weigh most with a deep K (63 x 5120 x
// 8704: 16.6 -> 13.8 us).
Plan plan_for(int64_t m, int64_t n, int64_t k, bool workspace) {
  const double steps = static_cast<double>(k / 128);
  Plan best{kTileKinds - 1, 1};
  double best_us = 1e300;
  if (m <= kStreamRows) {
    best.kind = kStream;
    best_us = kStreamStart + static_cast<double>(n * k) * kStreamPerByte +
              static_cast<double>((m - 1) / 16 * 16 * k) * kStreamPerTokenByte;
    // One round of 64 x 64 tiles has fewer CUs read the codes, but takes the
    // weights at 5.2 TB/s at best: 64 x 12000 x 5120 15.9 -> 12.9 us, 64 x 16384 x
    // 5120 18.7 -> 15.5; 64 x 5120 x 2048 streams in 5.7 and would take 6.4.
    if (m > kMixedRows && tile_count(kTiles[0], m, n) <= kCUs) {
      const double tiles = kTiles[0].first + steps * kTiles[0].step;
      const double read = 1.3 + static_cast<double>(n * k) / 5.2e6;
      const double us = 1.1 * (tiles > read ? tiles : read);
      if (us < best_us) best.kind = 0, best_us = us;
    }
  } else {
    for (int i = 0; i < kTileKinds; ++i) {
      const Tile& t = kTiles[i];
      const int64_t c = (tile_count(t, m, n) + kCUs - 1) / kCUs;
      if (c > t.rounds) continue;
      const double us = t.first + steps * t.step + static_cast<double>(c - 1) * (t.more + steps * t.more_step);
      if (us < best_us) best = Plan{i, 1}, best_us = us;
    }
  }
  if (workspace && m > kSplitRows && best.kind <= 0) {
    const int64_t tiles = tile_count(kTiles[0], m, n), groups = k / 128;
    const int64_t split = kCUs / tiles < groups / 4 ? kCUs / tiles : groups / 4;
    if (split > 1) {
      const double us = kTiles[0].first + static_cast<double>((groups + split - 1) / split) * kTiles[0].step + kJoin +
                        kJoinPerByte * static_cast<double>(8 * split * m * n);
      if (us < best_us) best = Plan{0, static_cast<int>(split)};
    }
  }
  return best;
}

// Workgroups of a launch stay below 2^32 threads of 8 waves. Only 256 x 256 tiles
// are taken that often (the others within `rounds`).
constexpr int64_t kMaxUnits = int64_t(1) << 23;

// Adds the parts of a split: 4 outputs a thread.
__global__ __launch_bounds__(256) void gemm_i8_join_kernel(int64_t m_rows, int64_t n, int split,
                                                           const int* __restrict__ part, const float* __restrict__ as,
                                                           const float* __restrict__ ws,
                                                           unsigned short* __restrict__ c) {
  const int64_t row_threads = (n + 3) / 4;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t m = at / row_threads, col = 4 * (at - m * row_threads);
  if (m >= m_rows) return;
  const int live = n - col < 4 ? static_cast<int>(n - col) : 4;
  v4i sum = {0, 0, 0, 0};
  for (int s = 0; s < split; ++s) {
    const int* p = part + (s * m_rows + m) * n + col;
    if (live == 4) {
      sum += *reinterpret_cast<const v4i_at4*>(p);
    } else {
      for (int e = 0; e < live; ++e) sum[e] += p[e];
    }
  }
  for (int e = 0; e < live; ++e)
    c[m * n + col + e] =
        static_cast<unsigned short>(pack_bf16x2(i8_scaled(sum[e], as[m], ws[col + e]), 0.f) & 0xffffu);
}

template <int BM, int BN, int WM, int WN, int STAGES, bool SPLIT = false, bool FETCH = false>
hipError_t tile(int64_t m, int64_t n, int64_t k, int split, const void* aq, const float* as, const void* wq,
                const float* ws, void* c, void* part, const char* name, hipStream_t stream) {
  const int64_t units = tile_count(Tile{BM, BN, 0, 0, 0, 0, 0}, m, n) * split;
  if (units >= kMaxUnits) return hipErrorInvalidValue;
  hipLaunchKernelGGL((gemm_i8_tiled_kernel<BM, BN, WM, WN, STAGES, SPLIT, FETCH>), dim3(static_cast<unsigned>(units)),
                     dim3(64 * WM * WN), 0, stream, m, n, k, split, static_cast<const unsigned char*>(aq), as,
                     static_cast<const unsigned char*>(wq), ws, static_cast<unsigned short*>(c),
                     static_cast<int*>(part));
  dispatch_log("gemm_i8", m, n, k, name);
  return hipGetLastError();
}

}  // namespace

bool gemm_i8_fits(int64_t m, int64_t n) {
  return m <= kStreamRows || tile_count(kTiles[kTileKinds - 1], m, n) < kMaxUnits;
}

int64_t gemm_i8_workspace_bytes(int64_t m, int64_t n, int64_t k) {
  const Plan p = plan_for(m, n, k, true);
  return p.split > 1 ? 4 * p.split * m * n : 0;
}

hipError_t launch_gemm_i8(int64_t m, int64_t n, int64_t k, const void* aq, const float* as, const void* wq,
                          const float* ws, void* c, void* workspace, hipStream_t stream) {
  const Plan p = plan_for(m, n, k, workspace != nullptr);
  if (p.kind == kStream) return launch_gemm_i8_rows(m, n, k, aq, as, wq, ws, c, stream);
  if (p.split > 1) {
    const hipError_t e = tile<64, 64, 2, 2, 4, true>(
        m, n, k, p.split, aq, as, wq, ws, c, workspace,
        "gemm_i8_tiled_kernel BM=64 BN=64 4 waves 4 stages, K split, + gemm_i8_join_kernel", stream);
    if (e != hipSuccess) return e;
    const int64_t threads = m * ((n + 3) / 4);  // split: below 256 tiles of 64 x 64 outputs
    hipLaunchKernelGGL(gemm_i8_join_kernel, dim3(static_cast<unsigned>((threads + 255) / 256)), dim3(256), 0, stream, m,
                       n, p.split, static_cast<const int*>(workspace), as, ws, static_cast<unsigned short*>(c));
    return hipGetLastError();
  }
  switch (p.kind) {
    case 0:
      return tile<64, 64, 2, 2, 4>(m, n, k, 1, aq, as, wq, ws, c, nullptr,
                                       "gemm_i8_tiled_kernel BM=64 BN=64 4 waves 4 stages", stream);
    case 1:
      return tile<96, 64, 2, 2, 4>(m, n, k, 1, aq, as, wq, ws, c, nullptr,
                                       "gemm_i8_tiled_kernel BM=96 BN=64 4 waves 4 stages", stream);
    case 2:
      return tile<64, 128, 2, 4, 3>(m, n, k, 1, aq, as, wq, ws, c, nullptr,
                                       "gemm_i8_tiled_kernel BM=64 BN=128 8 waves 3 stages", stream);
    case 3:
      return tile<96, 128, 2, 2, 4>(m, n, k, 1, aq, as, wq, ws, c, nullptr,
                                       "gemm_i8_tiled_kernel BM=96 BN=128 4 waves 4 stages", stream);
    case 4:
      return tile<128, 128, 2, 4, 4>(m, n, k, 1, aq, as, wq, ws, c, nullptr,
                                       "gemm_i8_tiled_kernel BM=128 BN=128 8 waves 4 stages", stream);
    case 5:
      return tile<192, 128, 2, 4, 3>(m, n, k, 1, aq, as, wq, ws, c, nullptr,
                                       "gemm_i8_tiled_kernel BM=192 BN=128 8 waves 3 stages", stream);
    case 6:
      return tile<128, 256, 2, 4, 3>(m, n, k, 1, aq, as, wq, ws, c, nullptr,
                                       "gemm_i8_tiled_kernel BM=128 BN=256 8 waves 3 stages", stream);
    case 7:
      return tile<192, 256, 2, 4, 2>(m, n, k, 1, aq, as, wq, ws, c, nullptr,
                                       "gemm_i8_tiled_kernel BM=192 BN=256 8 waves 2 stages", stream);
    default:
      return tile<256, 256, 2, 2, 2, false, true>(m, n, k, 1, aq, as, wq, ws, c, nullptr,
                                       "gemm_i8_tiled_kernel BM=256 BN=256 4 waves 2 stages", stream);
  }
}

}  // namespace fp8bq

// Weight-streaming int8 product for few tokens (M <= 64), gfx950.
//
// Up to some tens of tokens (plan_for in gemm_i8.hip decides) the product reads
// every weight byte once and is bound by HBM, so what matters is that every CU
// streams the same number of bytes and never lets its queue of loads run dry.
//
// One workgroup per CU owns R = N / 256 weight rows (a multiple of 4, at most
// 16 TILES), its 8 waves split K. A wave walks its groups of 128 columns; per
// group first the 16-token blocks of the activation, then the 16-row tiles of
// its weights, each a chunk of 16 rows x 128 bytes. Chunks are copied to the
// wave's own ring of 4 slots in LDS, without registers and without barriers:
// chunk c + 3 goes out before chunk c is used, 48 KB in flight per CU. More
// slots bring nothing while a launch's start grows by 0.1 us for each 16 KB of
// LDS (7168 x 5120 at 1 token: 7.3 / 7.5 / 7.6 / 7.7 / 7.9 us with 3 / 4 / 5 / 6
// / 8 slots; 17408 x 5120 at 64: 20.9 / 20.5 / 20.3 / 20.3 / 20.1), and two
// workgroups per CU of half the rows are slower (16.6 -> 17.4 us at 17408 x
// 5120, 5 tokens: twice the activation). A copy instruction reads 8 whole
// 128-byte lines, the weights' marked as read once (16.9 against 18.1 us
// without the mark); rows past the range lie past the buffer's end and read
// nothing. In a slot, piece c of row r stands at c ^ (r & 7), which spreads the
// fragment reads over the banks.
//
// The sums are 32-bit integers, exact in any order; the 8 waves' sums are
// added through LDS, scaled, rounded to bf16 and stored.
#include "gemm_i8_tiled.h"
#include "launch.h"
#include "step_launch.h"

namespace fp8bq {

namespace {

constexpr int kWaves = 8;
constexpr int kSlots = 4;          // ring slots per wave
constexpr int kSlotBytes = 2048;   // 16 rows x 128 bytes
constexpr int kMaxRowTiles = 5;    // 16-row tiles per workgroup
constexpr int64_t kCUs = 256;

__device__ __forceinline__ v4i mfma_16x16x64_i8(const v4u& a, const v4u& b, const v4i& c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(v4i, a), __builtin_bit_cast(v4i, b), c, 0, 0, 0);
}

// 8 bytes of C at any element.
typedef v2u __attribute__((aligned(2))) v2u_at2;

// MS: 16-token blocks; TILES: 16-row tiles. n: weight rows of this launch; ldc:
// those of C.
template <int MS, int TILES>
__global__ __launch_bounds__(64 * kWaves) void gemm_i8_rows_kernel(int m_rows, int64_t n, int64_t k, int64_t ldc,
                                                                   int rows_per_wg,
                                                                   const unsigned char* __restrict__ aq,
                                                                   const float* __restrict__ as,
                                                                   const unsigned char* __restrict__ wq,
                                                                   const float* __restrict__ ws,
                                                                   unsigned short* __restrict__ c) {
  constexpr int P = MS + TILES;            // chunks per group
  constexpr int AHEAD = kSlots - 1;        // chunks in flight
  constexpr int ITEMS = MS * TILES;        // 16 x 16 outputs per workgroup
  constexpr int ROUND = kSlots * kSlotBytes / 1024;  // of them the ring holds at a time
  __shared__ __attribute__((aligned(16))) unsigned char lds[kWaves * kSlots * kSlotBytes];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lrow = lane & 15, quarter = lane >> 4;
  const int64_t r_begin = static_cast<int64_t>(blockIdx.x) * rows_per_wg;
  const int rows = static_cast<int>(n - r_begin < rows_per_wg ? n - r_begin : rows_per_wg);

  // this wave's groups
  const int groups = static_cast<int>(k >> 7);
  const int g0 = groups * wave / kWaves;
  const int count = groups * (wave + 1) / kWaves - g0;

  // Copies: lane l fetches piece (l % 8) ^ (l / 8) of rows l / 8 and 8 + l / 8
  // of a chunk.
  unsigned off[P][2];
#pragma unroll
  for (int x = 0; x < P; ++x)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int64_t row = 16 * (x < MS ? x : x - MS) + 8 * j + (lane >> 3);
      off[x][j] = static_cast<unsigned>(row * k + 16 * ((lane & 7) ^ (lane >> 3)));
    }
  const v4i a_buf = buffer_words(aq, m_rows * k);
  const v4i w_buf = buffer_words(wq + r_begin * k, rows * k);
  const unsigned ring = lds_addr(lds) + wave * kSlots * kSlotBytes;
  auto copy = [&](int u, int x, int slot) {  // chunk x of the wave's group u; nothing past the last group
    v4i buf = x < MS ? a_buf : w_buf;
    buf[2] = u < count ? buf[2] : 0;
    const unsigned col = u < count ? static_cast<unsigned>(g0 + u) * 128 : 0;
    if (x < MS) {
      buffer_dma16(buf, off[x][0], col, ring + slot * kSlotBytes);
      buffer_dma16(buf, off[x][1], col, ring + slot * kSlotBytes + 1024);
    } else {
      buffer_dma16_once(buf, off[x][0], col, ring + slot * kSlotBytes);
      buffer_dma16_once(buf, off[x][1], col, ring + slot * kSlotBytes + 1024);
    }
  };

  // Scales of the outputs this wave will store (items wave, wave + 8, ...).
  constexpr int MINE = (ITEMS + kWaves - 1) / kWaves;
  float sa[MINE], sw[MINE][4];
#pragma unroll
  for (int y = 0; y < MINE; ++y) {
    const int item = wave + kWaves * y, s = item % MS, t = item / MS;
    const int m = 16 * s + lrow;
    sa[y] = as[m < m_rows ? m : m_rows - 1];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = 16 * t + 4 * quarter + e;
      sw[y][e] = ws[r_begin + (r < rows ? r : rows - 1)];
    }
  }

  v4i acc[TILES][MS];
#pragma unroll
  for (int t = 0; t < TILES; ++t)
#pragma unroll
    for (int s = 0; s < MS; ++s) acc[t][s] = v4i{0, 0, 0, 0};

#pragma unroll
  for (int x = 0; x < AHEAD; ++x) copy(x / P, x % P, x);
  const int frag = wave * kSlots * kSlotBytes + lrow * 128 + 16 * (quarter ^ (lrow & 7));
  int slot = 0;
  v4u a[MS][2];
  for (int u = 0; u < count; ++u) {
#pragma unroll
    for (int x = 0; x < P; ++x) {
      // the slot before this one: its fragments have been read
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      copy(u + (x + AHEAD) / P, (x + AHEAD) % P, (slot + AHEAD) % kSlots);
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * AHEAD) : "memory");
      const unsigned char* at = lds + slot * kSlotBytes;
      const v4u lo = *reinterpret_cast<const v4u*>(at + frag);
      const v4u hi = *reinterpret_cast<const v4u*>(at + (frag ^ 64));
      if (x < MS) {
        a[x][0] = lo;
        a[x][1] = hi;
      } else {
#pragma unroll
        for (int s = 0; s < MS; ++s) acc[x - MS][s] = mfma_16x16x64_i8(lo, a[s][0], acc[x - MS][s]);
#pragma unroll
        for (int s = 0; s < MS; ++s) acc[x - MS][s] = mfma_16x16x64_i8(hi, a[s][1], acc[x - MS][s]);
      }
      slot = (slot + 1) % kSlots;
    }
  }
  // empty copies past the end still write their slots
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");

  v4i* own = reinterpret_cast<v4i*>(lds + wave * kSlots * kSlotBytes);
#pragma unroll
  for (int first = 0; first < ITEMS; first += ROUND) {
#pragma unroll
    for (int t = 0; t < TILES; ++t)
#pragma unroll
      for (int s = 0; s < MS; ++s) {
        const int item = t * MS + s;
        if (item >= first && item < first + ROUND) own[64 * (item - first) + lane] = acc[t][s];
      }
    __syncthreads();
#pragma unroll
    for (int y = 0; y < MINE; ++y) {
      const int item = wave + kWaves * y;
      if (item < first || item >= first + ROUND || item >= ITEMS) continue;
      v4i sum = v4i{0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < kWaves; ++w)
        sum += reinterpret_cast<const v4i*>(lds + w * kSlots * kSlotBytes)[64 * (item - first) + lane];
      const int m = 16 * (item % MS) + lrow;
      const int r = 16 * (item / MS) + 4 * quarter;
      if (m >= m_rows || r >= rows) continue;
      const v2u p = {pack_bf16x2(i8_scaled(sum[0], sa[y], sw[y][0]), i8_scaled(sum[1], sa[y], sw[y][1])),
                     pack_bf16x2(i8_scaled(sum[2], sa[y], sw[y][2]), i8_scaled(sum[3], sa[y], sw[y][3]))};
      unsigned short* dst = c + m * ldc + r_begin + r;
      if (r + 3 < rows) {
        *reinterpret_cast<v2u_at2*>(dst) = p;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (r + e < rows) dst[e] = static_cast<unsigned short>(p[e >> 1] >> (16 * (e & 1)));
      }
    }
    if (first + ROUND < ITEMS) __syncthreads();
  }
}

struct Launch {
  dim3 grid;
  int rows_per_wg;
  int64_t m, n, k, ldc;
  const unsigned char* aq;
  const float* as;
  const unsigned char* wq;
  const float* ws;
  unsigned short* c;
  hipStream_t stream;
};

template <int MS, int TILES>
void run(const Launch& a) {
  hipLaunchKernelGGL((gemm_i8_rows_kernel<MS, TILES>), a.grid, dim3(64 * kWaves), 0, a.stream, static_cast<int>(a.m),
                     a.n, a.k, a.ldc, a.rows_per_wg, a.aq, a.as, a.wq, a.ws, a.c);
}

template <int MS>
void run_tiles(const Launch& a) {
  switch ((a.rows_per_wg + 15) / 16) {
    case 1: return run<MS, 1>(a);
    case 2: return run<MS, 2>(a);
    case 3: return run<MS, 3>(a);
    case 4: return run<MS, 4>(a);
    default: return run<MS, 5>(a);
  }
}

// Workgroups of a launch: fewer than 2^32 threads.
constexpr int64_t kMaxWorkgroups = (int64_t(1) << 23) - 1;

}  // namespace

hipError_t launch_gemm_i8_rows(int64_t m, int64_t n, int64_t k, const void* aq, const float* as, const void* wq,
                               const float* ws, void* c, hipStream_t stream) {
  // rows per workgroup: all rounds of 256 workgroups full, a multiple of 4
  const int64_t rounds = (n + kCUs * 16 * kMaxRowTiles - 1) / (kCUs * 16 * kMaxRowTiles);
  const int64_t even = (n + kCUs * rounds - 1) / (kCUs * rounds);
  const int rows = static_cast<int>((even + 3) / 4 * 4);
  if (m > 64) return hipErrorInvalidValue;
  // One launch, but from about 671 million weight rows on
  const int64_t most = rows * kMaxWorkgroups;
  for (int64_t r0 = 0; r0 < n; r0 += most) {
    const int64_t here = n - r0 < most ? n - r0 : most;
    const Launch a{dim3(static_cast<unsigned>((here + rows - 1) / rows)), rows, m, here, k, n,
                   static_cast<const unsigned char*>(aq), as, static_cast<const unsigned char*>(wq) + r0 * k, ws + r0,
                   static_cast<unsigned short*>(c) + r0, stream};
    if (m <= 16)
      run_tiles<1>(a);
    else if (m <= 32)
      run_tiles<2>(a);
    else if (m <= 48)
      run_tiles<3>(a);
    else
      run_tiles<4>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  dispatch_log("gemm_i8", m, n, k, "gemm_i8_rows_kernel");
  return hipSuccess;
}

}  // namespace fp8bq

// LDS-tiled int8 MFMA kernel for many tokens, gfx950.
//
// C[m, n] = bf16(fp32(sum_k A[m, k] W[n, k]) * (sa[m] * sw[n])). A workgroup
// of WM x WN waves computes BM tokens x BN weight rows, each wave (BM / WM) x
// (BN / WN) of them in 32-bit integer accumulators. There is nothing to do per
// scale group, so the accumulators never leave the matrix core's registers
// and a wave can hold 128 x 128 outputs.
//
// K goes 128 bytes a step through LDS, STAGES steps deep, copied there
// directly (dma16). A tile row is 128 bytes, its 16-byte piece c at c ^ (row
// & 7), so that 8 lanes reading 8 rows hit 8 different bank groups.
//
// In the small tiles of 4 waves (kAhead) all fragments of the next step are
// read while the MFMAs of this one run: one LDS latency and one barrier a step,
// which are longer than their 8 .. 24 MFMAs (64 x 64 tiles, 65 x 512 x 5120: 10.4
// -> 9.4 us; tiles of 8 waves, two on a SIMD, gain nothing).
//
// In the others a step is two halves of K = 64 (one MFMA deep). The fragments of the next
// half are read while the MFMAs of this one run (two register sets). After
// the first half a wave has read all of the step's stage: one wait and barrier
// there says that for every wave, and that the next step's stage has landed;
// the copies of step s + STAGES then go into the stage just read, spread over
// the second half's MFMAs. One barrier a step, and never an idle one between
// a read and its use.
#pragma once

#include "device_common.h"
#include "gemm_tiled.h"

namespace fp8bq {

typedef int v4i __attribute__((ext_vector_type(4)));

// 16 x 16 outputs, K = 64: lane l supplies 16 bytes of row l % 16 of the
// first operand and of column l % 16 of the second, K-slots 16 (l / 16) ..
// +15; result element i of lane l is row 4 (l / 16) + i, column l % 16. The
// sums are in accumulation registers that stay where they are: from the
// builtin the compiler renames the sums of a loop and moves them back (4 moves
// per MFMA in a 128 x 128 wave tile). The compiler sees no MFMA here, so the
// distances it would keep are kept by the callers: mfma_settle() before the
// first (the sums just written) and after the last (before they are read). Two
// on the same sums need none: source and destination are the same registers,
// and the compiler too lets such a pair follow directly. A kernel that keeps
// sums and spilled values in these registers would move them between: every
// instance has exactly its sums there.
__device__ __forceinline__ void mfma_acc_16x16x64_i8(const v4u& a, const v4u& b, v4i& c) {
  asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
}
template <int I, int J>
__device__ __forceinline__ void mfma_settle(v4i (&acc)[I][J]) {
  asm volatile("s_nop 15\n\ts_nop 15");
#pragma unroll
  for (int i = 0; i < I; ++i)
#pragma unroll
    for (int j = 0; j < J; ++j) asm volatile("" : "+a"(acc[i][j]));
  asm volatile("s_nop 15\n\ts_nop 15");
}

// Output of one exact sum: rounded to fp32, times the fp32 product of the
// scales; packed to bf16 by the caller.
__device__ __forceinline__ float i8_scaled(int sum, float sa, float sw) { return static_cast<float>(sum) * (sa * sw); }

// 16 bytes of C at any element (rows of an odd N start at 2-byte addresses),
// and 4 sums at any.
typedef v4u __attribute__((aligned(2))) v4u_at2;
typedef v4i __attribute__((aligned(4))) v4i_at4;

// Workgroup b of `units` -> unit of work: the workgroups of one XCD (b % 8)
// take consecutive units, which share operands through its L2.
__device__ __forceinline__ unsigned xcd_unit(unsigned b, unsigned units) {
  const unsigned x = b & 7, per = units >> 3, rem = units & 7;
  return (x < rem ? x * (per + 1) : rem * (per + 1) + (x - rem) * per) + (b >> 3);
}

// Raw buffer over [base, base + bytes), as its four words, and a direct copy
// from it to LDS (lane i's 16 bytes land at base + 16 i): per-lane offset
// `voff`, checked against the buffer's end, and a uniform `soff`, not checked.
// Written out for the reason given at dma16.
__device__ __forceinline__ v4i buffer_words(const void* base, int64_t bytes) {
  const uint64_t v = reinterpret_cast<uint64_t>(uniform(base));
  return v4i{static_cast<int>(v & 0xffffffffu), static_cast<int>(v >> 32),
             __builtin_amdgcn_readfirstlane(static_cast<int>(bytes)), 0x00020000};
}
__device__ __forceinline__ void buffer_dma16(const v4i& buf, unsigned voff, unsigned soff, unsigned lds_base) {
  asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds" ::"v"(voff), "s"(buf),
               "s"(soff), "s"(__builtin_amdgcn_readfirstlane(static_cast<int>(lds_base)))
               : "memory", "m0");
}

// The same for data that is read once.
__device__ __forceinline__ void buffer_dma16_once(const v4i& buf, unsigned voff, unsigned soff, unsigned lds_base) {
  asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen nt lds" ::"v"(voff), "s"(buf),
               "s"(soff), "s"(__builtin_amdgcn_readfirstlane(static_cast<int>(lds_base)))
               : "memory", "m0");
}

// 4 bytes a lane (lane i's at base + 4 i).
__device__ __forceinline__ void buffer_dma4(const v4i& buf, unsigned voff, unsigned soff, unsigned lds_base) {
  asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dword %0, %1, %2 offen lds" ::"v"(voff), "s"(buf),
               "s"(soff), "s"(__builtin_amdgcn_readfirstlane(static_cast<int>(lds_base)))
               : "memory", "m0");
}

template <int BM, int BN, int WM, int WN, int STAGES>
struct I8Tile {
  static constexpr int kWaves = WM * WN;
  static constexpr int kTM = BM / WM, kTN = BN / WN;
  static constexpr int kJ = kTM / 16, kI = kTN / 16;
  static constexpr int kStageBytes = (BM + BN) * 128;
  static constexpr int kChunks = (BM + BN) / 8 / kWaves;  // copies per wave and step
  // the epilogue's rows in LDS: 32 (16) tokens of kTN bf16, 16 bytes of padding
  static constexpr int kOutRows = kJ % 2 == 0 ? 32 : 16;
  static constexpr int kOutStride = kTN * 2 + 16;
  static constexpr int kOutBytes = kWaves * kOutRows * kOutStride;
  static constexpr int kLdsBytes = STAGES * kStageBytes > kOutBytes ? STAGES * kStageBytes : kOutBytes;
  static constexpr bool kAhead = kWaves == 4 && kI * kJ <= 12;
  static_assert((BM + BN) / 8 % kWaves == 0, "every wave issues the same number of copies");
  static_assert(BM % (16 * WM) == 0 && BN % (16 * WN) == 0 && BM % 8 == 0, "16-row fragments");
  static_assert(kI * kJ >= 4, "other MFMAs while one's sums are under way: for speed, not needed for the result");
  static_assert(STAGES >= 2, "the stage being filled is not the one being read");
};

// SPLIT: the K steps are cut into `split` parts, one workgroup each, whose
// int32 sums go to part [split][m_rows][n] (part s: the steps [G s / split,
// G (s + 1) / split) of G = k / 128); gemm_i8_join_kernel adds them. The host
// keeps tiles x split below 2^23: tiles and steps are counted in 32 bits.
//
// FETCH: with 256 x 256 tiles on all CUs a step's lines come from HBM about as
// late as they may (the copies of a step have half a step to arrive), so each
// wave also asks for 64 of the lines of the step after them, one word of each
// into LDS that nobody reads: they are in L2 when their copies go out. Token
// lines or weight lines by the tile's place, since neighbouring tiles share
// both. 3465 x 17408 x 5120 263 -> 258 us, 3465 x 8192 x 5120 129 -> 124; a step
// or three further ahead brings nothing, nor does it with smaller tiles, whose
// stages are deeper.
template <int BM, int BN, int WM, int WN, int STAGES, bool SPLIT, bool FETCH>
__global__ __launch_bounds__(64 * WM * WN) void gemm_i8_tiled_kernel(int64_t m_rows, int64_t n, int64_t k, int split,
                                                                     const unsigned char* __restrict__ aq,
                                                                     const float* __restrict__ as,
                                                                     const unsigned char* __restrict__ wq,
                                                                     const float* __restrict__ ws,
                                                                     unsigned short* __restrict__ c,
                                                                     int* __restrict__ part) {
  using T = I8Tile<BM, BN, WM, WN, STAGES>;
  constexpr int I = T::kI, J = T::kJ, CH = T::kChunks, WAVES = T::kWaves;
  constexpr bool AHEAD = T::kAhead;
  __shared__ __attribute__((aligned(16))) unsigned char lds[T::kLdsBytes];
  __shared__ float lds_sa[BM], lds_sw[BN];
  __shared__ __attribute__((aligned(16))) unsigned char lds_unread[FETCH ? 256 * WAVES : 1];
  static_assert(!FETCH || (BM == 64 * WAVES && BN == 64 * WAVES), "a line of the tile per thread");
  // the first step's wait allows one fetch besides the copies of the stages after
  // the next: with more stages than two it would allow a copy too many
  static_assert(!FETCH || STAGES == 2, "the wait of a step with fetches is counted for two stages");

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lrow = lane & 15, quarter = lane >> 4;
  const int wave_m = wave % WM, wave_n = wave / WM;

  const unsigned m_tiles = static_cast<unsigned>((m_rows + BM - 1) / BM);
  const unsigned n_tiles = static_cast<unsigned>((n + BN - 1) / BN);
  const unsigned all = static_cast<unsigned>(k >> 7);
  unsigned unit = xcd_unit(blockIdx.x, gridDim.x), ks = 0;
  if constexpr (SPLIT) {
    ks = unit / (m_tiles * n_tiles);
    unit -= ks * (m_tiles * n_tiles);
  }
  // bands of 8 token tiles, in which the token tile runs fastest
  const unsigned band = unit / (8 * n_tiles), at = unit - band * 8 * n_tiles;
  const unsigned width = m_tiles - 8 * band < 8 ? m_tiles - 8 * band : 8;
  const unsigned tn = at / width, tm = 8 * band + (at - tn * width);
  const int64_t m0 = static_cast<int64_t>(tm) * BM, n0 = static_cast<int64_t>(tn) * BN;
  const unsigned g_lo = SPLIT ? all * ks / split : 0;
  const int steps = static_cast<int>(SPLIT ? all * (ks + 1) / split - g_lo : all);

  // Copies: this wave's 8-row chunks (tokens first, then weight rows); lane l
  // fetches piece (l % 8) ^ (row & 7) of row l / 8 of the chunk. The buffers
  // end with the tile's last existing row: rows past it read nothing.
  unsigned off[CH];
#pragma unroll
  for (int q = 0; q < CH; ++q) {
    const int r = 8 * (wave + WAVES * q) + (lane >> 3);
    const int64_t row = 8 * (wave + WAVES * q) < BM ? r : r - BM;
    off[q] = static_cast<unsigned>(row * k + 16 * ((lane & 7) ^ (r & 7)));
  }
  const v4i a_buf = buffer_words(aq + m0 * k, (m_rows - m0 < BM ? m_rows - m0 : BM) * k);
  const v4i w_buf = buffer_words(wq + n0 * k, (n - n0 < BN ? n - n0 : BN) * k);
  // Step s into `stage`; past the last step the buffer is empty, so that every
  // step issues the same number of copies and the wait for them is a constant.
  const unsigned lds_copy = lds_addr(lds) + 1024 * wave;
  auto copy = [&](int s, int stage, int q) {
    // whole rounds of the waves' chunks are tokens or weight rows as a constant
    const bool tok = BM % (8 * WAVES) == 0 ? 8 * WAVES * q < BM : 8 * (wave + WAVES * q) < BM;
    v4i buf = tok ? a_buf : w_buf;
    buf[2] = s < steps ? buf[2] : 0;
    buffer_dma16(buf, off[q], s < steps ? (g_lo + s) * 128 : 0, lds_copy + stage * T::kStageBytes + 1024 * WAVES * q);
  };

  const v4i fetch_buf = (tm & 1) != 0 ? a_buf : w_buf;
  const unsigned fetch_off = static_cast<unsigned>(threadIdx.x * k);
  const unsigned fetch_lds = lds_addr(lds_unread) + 256 * wave;
  auto fetch = [&](int s) {  // one word of each line of step s
    v4i buf = fetch_buf;
    buf[2] = s < steps ? buf[2] : 0;
    buffer_dma4(buf, fetch_off, s < steps ? (g_lo + s) * 128 : 0, fetch_lds);
  };

  // Fragment addresses: row 16 i + lrow of the wave's part, pieces quarter
  // (first half) and quarter + 4 (second).
  const int fa = (T::kTM * wave_m + lrow) * 128 + 16 * (quarter ^ (lrow & 7));
  const int fw = (BM + T::kTN * wave_n + lrow) * 128 + 16 * (quarter ^ (lrow & 7));

  v4i acc[I][J];
#pragma unroll
  for (int i = 0; i < I; ++i)
#pragma unroll
    for (int j = 0; j < J; ++j) acc[i][j] = v4i{0, 0, 0, 0};
  mfma_settle(acc);
  v4u a[AHEAD ? 4 : 2][J], w[AHEAD ? 4 : 2][I];  // register sets: half 0 and 1 of a step, then of the next

  auto read = [&](int set, int stage, int x) {  // x: fragment 0 .. I + J - 1
    const unsigned char* at = lds + stage * T::kStageBytes;
    const int flip = (set & 1) * 64;  // piece 4 further: bit 6 of the swizzled address
    if (x < I)
      w[set][x] = *reinterpret_cast<const v4u*>(at + (fw ^ flip) + 2048 * x);
    else
      a[set][x - I] = *reinterpret_cast<const v4u*>(at + (fa ^ flip) + 2048 * (x - I));
  };
  // The MFMAs of register set `set`; meanwhile the other set is read from
  // `stage`, and (COPY) step s's copies go out into stage `into`. The reads
  // go out within the first three quarters of the MFMAs.
  auto half = [&](auto set_c, auto copy_c, int stage, int s, int into) {
    constexpr int set = decltype(set_c)::value;
    constexpr bool COPY = decltype(copy_c)::value;
    constexpr int MF = I * J, RD = I + J, SPAN = MF * 3 / 4 > 0 ? MF * 3 / 4 : 1;
#pragma unroll
    for (int x = 0; x < MF; ++x) {
      const int i = x / J, j = x % J;
#pragma unroll
      for (int y = RD * x / SPAN; y < (x + 1 >= SPAN ? RD : RD * (x + 1) / SPAN) && x < SPAN; ++y)
        read(1 - set, stage, y);
      mfma_acc_16x16x64_i8(w[set][i], a[set][j], acc[i][j]);
      if constexpr (COPY) {
#pragma unroll
        for (int q = CH * x / MF; q < CH * (x + 1) / MF; ++q) copy(s, into, q);
        if constexpr (FETCH) {
          if (x == MF - 1) fetch(s + 1);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  using Set0 = std::integral_constant<int, 0>;
  using Set1 = std::integral_constant<int, 1>;

#pragma unroll
  for (int s = 0; s < STAGES; ++s)
#pragma unroll
    for (int q = 0; q < CH; ++q) copy(s, s, q);
  if constexpr (FETCH) fetch(STAGES);
  for (int i = threadIdx.x; i < BM; i += 64 * WAVES) lds_sa[i] = as[m0 + i < m_rows ? m0 + i : m_rows - 1];
  for (int i = threadIdx.x; i < BN; i += 64 * WAVES) lds_sw[i] = ws[n0 + i < n ? n0 + i : n - 1];
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((STAGES - 1) * CH + FETCH) : "memory");
#pragma unroll
  for (int x = 0; x < I + J; ++x) read(0, 0, x);

  if constexpr (AHEAD) {
#pragma unroll
    for (int x = 0; x < I + J; ++x) read(1, 0, x);
    // Step s from the sets SET and SET + 1, whose reads are waited for here:
    // then every wave has read stage `stage`, and the next one has landed.
    auto step = [&](auto set_c, int s, int stage, int next) {
      constexpr int set = decltype(set_c)::value, other = 2 - set;
      constexpr int MF = 2 * I * J, RD = 2 * (I + J), SPAN = MF / 2;
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((STAGES - 2) * CH) : "memory");
#pragma unroll
      for (int x = 0; x < MF; ++x) {
        const int h = x / (I * J), i = x % (I * J) / J, j = x % J;
#pragma unroll
        for (int y = RD * x / SPAN; y < RD * (x + 1) / SPAN && y < RD; ++y)
          read(other + y / (I + J), next, y % (I + J));  // past the last step: read, never used
        mfma_acc_16x16x64_i8(w[set + h][i], a[set + h][j], acc[i][j]);
#pragma unroll
        for (int q = CH * x / MF; q < CH * (x + 1) / MF; ++q) copy(s + STAGES, stage, q);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    int stage = 0;
    for (int s = 0; s < steps; s += 2) {
      int next = stage + 1 < STAGES ? stage + 1 : 0;
      step(std::integral_constant<int, 0>{}, s, stage, next);
      if (s + 1 == steps) break;
      stage = next;
      next = stage + 1 < STAGES ? stage + 1 : 0;
      step(std::integral_constant<int, 2>{}, s + 1, stage, next);
      stage = next;
    }
  } else {
    for (int s = 0, stage = 0; s < steps; ++s) {
      const int next = stage + 1 < STAGES ? stage + 1 : 0;
      half(Set0{}, std::false_type{}, stage, 0, 0);
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((STAGES - 2) * (CH + FETCH) + FETCH) : "memory");
      half(Set1{}, std::true_type{}, next, s + STAGES, stage);  // past the last step: read, never used
      stage = next;
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  mfma_settle(acc);

  if constexpr (SPLIT) {
    int* dst = part + ks * m_rows * n;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int64_t m = m0 + T::kTM * wave_m + 16 * j + lrow;
      if (m >= m_rows) continue;
#pragma unroll
      for (int i = 0; i < I; ++i) {
        const int64_t col = n0 + T::kTN * wave_n + 16 * i + 4 * quarter;
        int* at = dst + m * n + col;
        if (col + 3 < n) {
          *reinterpret_cast<v4i_at4*>(at) = acc[i][j];
        } else {
#pragma unroll
          for (int e = 0; e < 3; ++e)
            if (col + e < n) at[e] = acc[i][j][e];
        }
      }
    }
    return;
  }

  // Outputs: a lane holds 4 consecutive columns of a token; through LDS (each
  // wave its own rows) to stores of whole rows, 16 bytes a lane.
  __syncthreads();
  unsigned char* rows = lds + wave * T::kOutRows * T::kOutStride;
  constexpr int JB = T::kOutRows / 16;    // token fragments at a time
  constexpr int LPR = T::kTN / 8;         // lanes per row
  constexpr int RPI = 64 / LPR;           // rows per store
  static_assert(LPR * RPI == 64 && T::kOutRows % RPI == 0, "whole waves store whole rows");
  // Only a tile at an edge of C checks each row and column; its loops are not
  // unrolled, so that the code (which every launch has to fetch) stays small.
  const bool whole = m0 + BM <= m_rows && n0 + BN <= n;
  v4f sw[I];
#pragma unroll
  for (int i = 0; i < I; ++i)
    sw[i] = *reinterpret_cast<const v4f*>(lds_sw + T::kTN * wave_n + 16 * i + 4 * quarter);
#pragma unroll
  for (int j0 = 0; j0 < J; j0 += JB) {
#pragma unroll
    for (int jj = 0; jj < JB; ++jj) {
      const float sa = lds_sa[T::kTM * wave_m + 16 * (j0 + jj) + lrow];
#pragma unroll
      for (int i = 0; i < I; ++i) {
        const v4i v = acc[i][j0 + jj];
        const v2u p = {pack_bf16x2(i8_scaled(v[0], sa, sw[i][0]), i8_scaled(v[1], sa, sw[i][1])),
                       pack_bf16x2(i8_scaled(v[2], sa, sw[i][2]), i8_scaled(v[3], sa, sw[i][3]))};
        *reinterpret_cast<v2u*>(rows + (16 * jj + lrow) * T::kOutStride + (16 * i + 4 * quarter) * 2) = p;
      }
    }
    __builtin_amdgcn_wave_barrier();
    const int lr = lane / LPR, lc = lane % LPR;
    const int64_t col = n0 + T::kTN * wave_n + 8 * lc;
    const int64_t m_first = m0 + T::kTM * wave_m + 16 * j0;
    if (whole) {
      unsigned short* at = c + (m_first + lr) * n + col;
#pragma unroll
      for (int r0 = 0; r0 < T::kOutRows; r0 += RPI, at += RPI * n)
        *reinterpret_cast<v4u_at2*>(at) = *reinterpret_cast<const v4u*>(rows + (r0 + lr) * T::kOutStride + 16 * lc);
    } else {
#pragma unroll 1
      for (int r = lr; r < T::kOutRows; r += RPI) {
        const int64_t m = m_first + r;
        if (m >= m_rows) break;
        unsigned short* at = c + m * n + col;
        if (col + 7 < n) {
          *reinterpret_cast<v4u_at2*>(at) = *reinterpret_cast<const v4u*>(rows + r * T::kOutStride + 16 * lc);
        } else {
#pragma unroll 1
          for (int e = 0; col + e < n; ++e)
            at[e] = *reinterpret_cast<const unsigned short*>(rows + r * T::kOutStride + 16 * lc + 2 * e);
        }
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
}

}  // namespace fp8bq

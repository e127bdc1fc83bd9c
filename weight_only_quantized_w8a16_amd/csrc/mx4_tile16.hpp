// mx4_tile16.hpp -- C = A . value(B)^T on gfx950 for many rows: A in 16 bits,
// B tiled MX4, one BM x BN output tile per workgroup of eight waves.
//
// Per 64-k step the workgroup's BM activation rows (128 bytes each) and the
// codes of its BN channels (32 bytes each) go from global memory straight
// into LDS (buffer_load ... lds, 16 bytes per lane, no VGPRs), NS - 1 steps
// ahead of use.  A wave reads each code once per step -- lane (row, half h)
// the 16 bytes of the 32-value block h of its channel -- and widens it in
// registers right before the matrix instructions, two values an instruction
// with the block scale applied (exact in bf16, one rounding in fp16).  So the
// weights take a quarter of the LDS bytes that 16-bit ones would, and
// nothing is written to LDS by the waves.  Every wave row of the workgroup
// repeats the widening: 16 instructions per 32 channels and step, against
// 16 matrix instructions of 32 cycles each on the 128-row wave tile.
//
// Sub-step ks of a step multiplies k = 32 h + 8 ks + 0 .. 7 (any order of k
// serves as long as both operands use the same): of the codes, word ks of the
// lane's 16 bytes; of the activations, 16-byte chunk 4 h + ks of the row.
//
// Scales: a lane's two scale words per 32 channels hold its blocks of a
// 512-k window (eight steps: word s % 2, byte s / 2 for step s of the
// window); they are loaded into registers one window ahead.
//
// LDS placement: activation chunk c of row r at chunk c ^ ((r / 2) % 8) (16
// lanes reading one chunk of 16 rows touch 16 distinct 16-byte bank groups);
// codes of a 16-channel tile as 512 contiguous bytes, block h first, so 16
// lanes read 256 contiguous bytes.  A direct load cannot be masked: rows past
// the end repeat the last valid row, channel tiles past the end the last
// tile; their outputs are never stored.
#pragma once

#include <type_traits>

#include "mx4_common.hpp"

namespace qg {

template <int BM_, int BN_, int WM_, int WN_, int NS_>
struct Mx4Cfg16 {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NS = NS_;
  static constexpr int NTHR = 64 * WM * WN;
  static constexpr int WTM = BM / WM, WTN = BN / WN;   // wave tile
  static constexpr int TM = WTM / 32, TN = WTN / 32;   // 32x32 accumulators per wave
  static constexpr int A_DMA = BM * 8 / NTHR;          // 16-byte direct loads per thread per step
  static constexpr int B_LOADS = BN * 2 / 64;          // 1 KiB code loads per step and workgroup
  static constexpr int STAGE_A = BM * 128, STAGE_B = BN * 32;
  static_assert(NTHR == 512, "eight waves");
  static_assert(WTM % 32 == 0 && WTN % 32 == 0 && A_DMA >= 1, "tile shape");
  static_assert(B_LOADS <= 8, "at most one code load per wave");
  static_assert((NS == 2 || NS == 4) && NS * (STAGE_A + STAGE_B) <= 160 * 1024, "LDS stages");
};

// One workgroup's tile: rows [row_lo, row_last] of A and C, channels from
// col_lo on, 64-k steps [s0, s1) with s0 a multiple of 8.
struct Mx4Tile {
  int row_lo, row_last, col_lo, s0, s1;
};

struct Mx4Lds {
  char *a[4];
  char *b[4];
};

// s_waitcnt with vmcnt(n), lgkmcnt(0), expcnt untouched.
constexpr int mx4_wait(int n) { return (n & 15) | ((n >> 4) << 14) | (7 << 4); }

// `store(row, col, values)` takes four consecutive columns of one row.
template <class Cfg, int ACT, class Store>
__device__ __forceinline__ void mx4_tile16(const uint16_t *A, int a_rows, const uint8_t *B,
                                           const uint32_t *BS, int N, int K, const Mx4Tile &t,
                                           const Mx4Lds &L, const Store &store) {
  constexpr int TM = Cfg::TM, TN = Cfg::TN, NS = Cfg::NS;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave / Cfg::WN, wn = wave % Cfg::WN;
  const int nb = K >> 7, nw = mx4_scale_windows(K), ntiles = N >> 4;

  constexpr int kRsrcFlags = 0x00020000;
  const uint32_t kb = static_cast<uint32_t>(K) * 2u;   // activation bytes per row
  const auto rA = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint16_t *>(A), 0, static_cast<int>(static_cast<uint32_t>(a_rows) * kb), kRsrcFlags);
  const auto rB = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t *>(B), 0, static_cast<int>(static_cast<uint32_t>(ntiles) * nb * 1024u), kRsrcFlags);

  // A: slot q = (wave * A_DMA + i) * 64 + lane of a stage is row q / 8,
  // placed chunk q % 8, holding the row's chunk (q % 8) ^ ((row / 2) % 8).
  uint32_t a_voff[Cfg::A_DMA];
#pragma unroll
  for (int i = 0; i < Cfg::A_DMA; ++i) {
    const int q = (wave * Cfg::A_DMA + i) * 64 + lane;
    const int r = q >> 3, c = (q & 7) ^ ((r >> 1) & 7);
    a_voff[i] = static_cast<uint32_t>(min(t.row_lo + r, t.row_last)) * kb + c * 16;
  }
  // B: load b brings two 16-channel tiles' 512 bytes of the step, lane l of
  // it tile l / 32, block (l / 16) % 2, channel l % 16.  With fewer loads than
  // waves, the waves past them repeat one (the same bytes to the same place).
  const int bl = wave % Cfg::B_LOADS;
  const uint32_t b_voff =
      static_cast<uint32_t>(min((t.col_lo >> 4) + 2 * bl + (lane >> 5), ntiles - 1)) * static_cast<uint32_t>(nb) * 1024u +
      (lane & 31) * 16;
  // Step `step` into stage ST; past the last step the last one is loaded
  // again (into a stage no later step reads), so every step issues the same
  // number of loads and one wait count fits all.
  auto issue = [&](auto STc, int step) {
    constexpr int ST = decltype(STc)::value;
    const int s = min(step, t.s1 - 1);
    char *da = L.a[ST] + wave * Cfg::A_DMA * 1024;
#pragma unroll
    for (int i = 0; i < Cfg::A_DMA; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rA, (__attribute__((address_space(3))) void *)(da + i * 1024), 16, static_cast<int>(a_voff[i]), s * 128, 0, 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        rB, (__attribute__((address_space(3))) void *)(L.b[ST] + bl * 1024), 16, static_cast<int>(b_voff), s * 512, 0, 0);
  };

  const int h = lane >> 5;
  // Scale words of window w: word (s % 2) of 32-channel block j.
  const uint32_t *sp[TN];
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    const int ch = wn * Cfg::WTN + 32 * j + (lane & 31);
    sp[j] = BS + static_cast<size_t>(min((t.col_lo + ch) >> 4, ntiles - 1)) * nw * 64 + 16 * h + (lane & 15);
  }
  auto load_scales = [&](int w, uint32_t (&sc)[2][TN]) {
    const int ww = min(w, nw - 1);
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int x = 0; x < 2; ++x) sc[x][j] = sp[j][ww * 64 + 32 * x];
  };

  int a_addr[4];
#pragma unroll
  for (int ks = 0; ks < 4; ++ks)
    a_addr[ks] = (wm * Cfg::WTM + (lane & 31)) * 128 + (((4 * h + ks) ^ ((lane >> 1) & 7)) << 4);
  const int b_addr = (wn * Cfg::WTN / 16 + ((lane >> 4) & 1)) * 512 + h * 256 + (lane & 15) * 16;
  auto read_a = [&](const char *As, int ks, u32x4 (&a)[TM]) {
#pragma unroll
    for (int i = 0; i < TM; ++i) a[i] = *reinterpret_cast<const u32x4 *>(As + a_addr[ks] + 4096 * i);
  };

  // acc[i][j] holds C^T, a lane one row of C (32 i + lane % 32) and 16 of its
  // columns, four consecutive ones per group of four values.
  f32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
  auto mma = [&](int ks, const u32x4 (&a)[TM], const u32x4 (&b)[TN], const float (&sc)[TN]) {
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const u32x4 w = mx4_word_to_operand<ACT>(b[j][ks], sc[j]);
#pragma unroll
      for (int i = 0; i < TM; ++i) acc[i][j] = mfma32x32x16<ACT>(w, a[i], acc[i][j]);
    }
  };
  auto barrier = [] {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  // After a step's issue, the loads of the next step are the oldest but
  // those of the NS - 2 steps after it (the scale loads in between only make
  // the wait stricter).
  constexpr int WAIT_NEXT = mx4_wait((NS - 2) * (Cfg::A_DMA + 1));

  uint32_t cur[2][TN], nxt[2][TN];
  // Step s, the I-th of its window, on stage I % NS: issue step s + NS - 1
  // into stage (I - 1) % NS (last read in step s - 1, before the barrier that
  // ended it), run the four sub-steps, wait for this wave's loads of step
  // s + 1, meet the other waves.
  auto body = [&](auto Ic, int step) {
    constexpr int I = decltype(Ic)::value, ST = I % NS;
    issue(std::integral_constant<int, (ST + NS - 1) % NS>{}, step + NS - 1);
    __builtin_amdgcn_sched_barrier(0);
    const char *As = L.a[ST], *Bs = L.b[ST];
    u32x4 a0[TM], a1[TM], b[TN];
    float sc[TN];
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      b[j] = *reinterpret_cast<const u32x4 *>(Bs + b_addr + 1024 * j);
      sc[j] = mx4_scale_operand(cur[I & 1][j], I >> 1);
    }
    read_a(As, 0, a0);
    read_a(As, 1, a1);
    mma(0, a0, b, sc);
    read_a(As, 2, a0);
    mma(1, a1, b, sc);
    read_a(As, 3, a1);
    mma(2, a0, b, sc);
    mma(3, a1, b, sc);
    // Fragment reads one sub-step ahead of the matrix instructions.
    constexpr int NM = TM * TN;
    __builtin_amdgcn_sched_group_barrier(0x100, TN + 2 * TM, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, NM, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, TM, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, NM, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, TM, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, NM, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, NM, 0);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(WAIT_NEXT);
    barrier();
  };
  using std::integral_constant;

  issue(integral_constant<int, 0>{}, t.s0);
  if constexpr (NS > 2) {
    issue(integral_constant<int, 1>{}, t.s0 + 1);
    issue(integral_constant<int, 2>{}, t.s0 + 2);
  }
  load_scales(t.s0 >> 3, cur);
  __builtin_amdgcn_s_waitcnt(mx4_wait(0));
  barrier();
  // Windows of eight steps; the last may have two, four or six (k is a
  // multiple of 128).
  for (int step = t.s0; step < t.s1; step += 8) {
    load_scales((step >> 3) + 1, nxt);
    body(integral_constant<int, 0>{}, step);
    body(integral_constant<int, 1>{}, step + 1);
    if (step + 2 < t.s1) {
      body(integral_constant<int, 2>{}, step + 2);
      body(integral_constant<int, 3>{}, step + 3);
    }
    if (step + 4 < t.s1) {
      body(integral_constant<int, 4>{}, step + 4);
      body(integral_constant<int, 5>{}, step + 5);
    }
    if (step + 6 < t.s1) {
      body(integral_constant<int, 6>{}, step + 6);
      body(integral_constant<int, 7>{}, step + 7);
    }
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      cur[0][j] = nxt[0][j];
      cur[1][j] = nxt[1][j];
    }
  }
  // The re-issued loads of the last steps land before the workgroup (and its
  // LDS) ends.
  __builtin_amdgcn_s_waitcnt(mx4_wait(0));

  // Value v of acc[i][j] is C[row][col], row = wave tile row + 32 i +
  // lane % 32, col = wave tile column + 32 j + 8 (v / 4) + 4 h + v % 4.
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int r = t.row_lo + wm * Cfg::WTM + 32 * i + (lane & 31);
    if (r > t.row_last) continue;
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int col = t.col_lo + wn * Cfg::WTN + 32 * j + 8 * q + 4 * h;
        if (col >= N) continue;
        const float v[4] = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        store(r, col, v);
      }
  }
}

}  // namespace qg

// mx4_tile4.hpp -- C = value(A) . value(B)^T on gfx950 for many rows, both
// operands tiled MX4, one BM x BN output tile per workgroup of eight waves.
//
// The tiled layout is the lane order of the scaled 16 x 16 x 128 matrix
// instruction: a 1 KiB code block (16 rows x 128 k) is one wave's fragment, 16
// bytes -- one 32-value block -- a lane.  Per 128-k step the blocks of the BM
// rows and BN channels go from global memory straight into LDS (buffer_load
// ... lds, one block an instruction, no VGPRs), NS - 1 steps ahead of use, and
// every wave reads the fragments of its wave tile in lane order (no bank
// conflicts, no swizzle).  The block scales are operands of the instruction:
// a lane's scale word holds its blocks of four consecutive steps (a 512-k
// window), byte s % 4 selected by the instruction itself, so a step needs no
// VALU work at all.  Scale words are loaded into registers one window ahead.
//
// A direct load cannot be masked: row tiles past the end repeat the last row
// tile, channel tiles past the end the last channel tile; their outputs are
// never stored.
#pragma once

#include <type_traits>

#include "mx4_common.hpp"
#include "mx4_tile16.hpp"

namespace qg {

template <int BM_, int BN_, int WM_, int WN_, int NS_>
struct Mx4Cfg4 {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NS = NS_;
  static constexpr int NTHR = 64 * WM * WN;
  static constexpr int WTM = BM / WM, WTN = BN / WN;   // wave tile
  static constexpr int TM = WTM / 16, TN = WTN / 16;   // 16x16 accumulators per wave
  static constexpr int A_BLK = BM / 16, B_BLK = BN / 16;   // code blocks per step
  static constexpr int A_DMA = A_BLK / 8 > 0 ? A_BLK / 8 : 1;   // block loads per wave per step
  static constexpr int B_DMA = B_BLK / 8 > 0 ? B_BLK / 8 : 1;
  static constexpr int STAGE_A = BM * 64, STAGE_B = BN * 64;
  static_assert(NTHR == 512, "eight waves");
  static_assert(WTM % 16 == 0 && WTN % 16 == 0, "tile shape");
  static_assert(NS == 4 && NS * (STAGE_A + STAGE_B) <= 160 * 1024, "LDS stages");
};

// 16 x 16 x 128 with byte B of each lane's scale word.
template <int B>
__device__ __forceinline__ f32x4 mx4_mfma_byte(u32x4 a, u32x4 b, f32x4 c, uint32_t sa, uint32_t sb) {
  const i32x4 x = __builtin_bit_cast(i32x4, a), y = __builtin_bit_cast(i32x4, b);
  constexpr int kFP4 = 4;
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
      __builtin_shufflevector(x, x, 0, 1, 2, 3, -1, -1, -1, -1),
      __builtin_shufflevector(y, y, 0, 1, 2, 3, -1, -1, -1, -1), c, kFP4, kFP4, B,
      static_cast<int>(sa), B, static_cast<int>(sb));
}

// Steps [t.s0, t.s1) are of 128 k, s0 a multiple of 4; row_lo a multiple of 16.
template <class Cfg, class Store>
__device__ __forceinline__ void mx4_tile4(const uint8_t *A, const uint32_t *AS, int M, const uint8_t *B,
                                          const uint32_t *BS, int N, int K, const Mx4Tile &t,
                                          const Mx4Lds &L, const Store &store) {
  constexpr int TM = Cfg::TM, TN = Cfg::TN, NS = Cfg::NS;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave / Cfg::WN, wn = wave % Cfg::WN;
  const int nb = K >> 7, nw = mx4_scale_windows(K), ntiles = N >> 4, mtiles = (M + 15) >> 4;
  const int rt0 = t.row_lo >> 4, ct0 = t.col_lo >> 4;

  constexpr int kRsrcFlags = 0x00020000;
  const auto rA = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t *>(A), 0, static_cast<int>(static_cast<uint32_t>(mtiles) * nb * 1024u), kRsrcFlags);
  const auto rB = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t *>(B), 0, static_cast<int>(static_cast<uint32_t>(ntiles) * nb * 1024u), kRsrcFlags);
  // Load i of a wave brings block (wave * DMA + i) of the step; with fewer
  // blocks than waves, waves repeat one (the same bytes to the same place).
  uint32_t a_voff[Cfg::A_DMA], b_voff[Cfg::B_DMA];
#pragma unroll
  for (int i = 0; i < Cfg::A_DMA; ++i)
    a_voff[i] = static_cast<uint32_t>(min(rt0 + (wave * Cfg::A_DMA + i) % Cfg::A_BLK, mtiles - 1)) *
                    static_cast<uint32_t>(nb) * 1024u + lane * 16;
#pragma unroll
  for (int i = 0; i < Cfg::B_DMA; ++i)
    b_voff[i] = static_cast<uint32_t>(min(ct0 + (wave * Cfg::B_DMA + i) % Cfg::B_BLK, ntiles - 1)) *
                    static_cast<uint32_t>(nb) * 1024u + lane * 16;
  // Step `step` into stage ST; past the last step the last one is loaded
  // again (into a stage no later step reads).
  auto issue = [&](auto STc, int step) {
    constexpr int ST = decltype(STc)::value;
    const int so = min(step, t.s1 - 1) * 1024;
#pragma unroll
    for (int i = 0; i < Cfg::A_DMA; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rA, (__attribute__((address_space(3))) void *)(L.a[ST] + (wave * Cfg::A_DMA + i) % Cfg::A_BLK * 1024),
          16, a_voff[i], so, 0, 0);
#pragma unroll
    for (int i = 0; i < Cfg::B_DMA; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rB, (__attribute__((address_space(3))) void *)(L.b[ST] + (wave * Cfg::B_DMA + i) % Cfg::B_BLK * 1024),
          16, b_voff[i], so, 0, 0);
  };

  // Scale words of window w (steps 4 w .. 4 w + 3).
  const uint32_t *ap[TM], *bp[TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
    ap[i] = AS + static_cast<size_t>(min(rt0 + wm * TM + i, mtiles - 1)) * nw * 64 + lane;
#pragma unroll
  for (int j = 0; j < TN; ++j)
    bp[j] = BS + static_cast<size_t>(min(ct0 + wn * TN + j, ntiles - 1)) * nw * 64 + lane;
  struct Scales {
    uint32_t a[TM], b[TN];
  };
  auto load_scales = [&](int w, Scales &s) {
    const int ww = min(w, nw - 1) * 64;
#pragma unroll
    for (int i = 0; i < TM; ++i) s.a[i] = ap[i][ww];
#pragma unroll
    for (int j = 0; j < TN; ++j) s.b[j] = bp[j][ww];
  };

  // acc[i][j]: lane (nl, q) holds row 16 i + nl, columns 16 j + 4 q .. + 3.
  f32x4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  auto barrier = [] {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  constexpr int WAIT_NEXT = mx4_wait((NS - 2) * (Cfg::A_DMA + Cfg::B_DMA));
  Scales cur, nxt;
  // Step s, the I-th of its window, on stage I: issue step s + 3 into the
  // stage read in step s - 1, multiply, wait for this wave's loads of step
  // s + 1, meet the other waves.
  auto body = [&](auto Ic, int step) {
    constexpr int I = decltype(Ic)::value;
    issue(std::integral_constant<int, (I + NS - 1) % NS>{}, step + NS - 1);
    __builtin_amdgcn_sched_barrier(0);
    const char *As = L.a[I] + wm * TM * 1024 + lane * 16, *Bs = L.b[I] + wn * TN * 1024 + lane * 16;
    u32x4 b[TN], a[TM];
#pragma unroll
    for (int j = 0; j < TN; ++j) b[j] = *reinterpret_cast<const u32x4 *>(Bs + j * 1024);
#pragma unroll
    for (int i = 0; i < TM; ++i) a[i] = *reinterpret_cast<const u32x4 *>(As + i * 1024);
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = mx4_mfma_byte<I>(b[j], a[i], acc[i][j], cur.b[j], cur.a[i]);
    // Fragments of one row tile ahead of the matrix instructions.
    __builtin_amdgcn_sched_group_barrier(0x100, TN + (TM > 1 ? 2 : 1), 0);
#pragma unroll
    for (int i = 0; i + 2 < TM; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, TN, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, (TM > 1 ? 2 : 1) * TN, 0);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(WAIT_NEXT);
    barrier();
  };
  using std::integral_constant;
  issue(integral_constant<int, 0>{}, t.s0);
  issue(integral_constant<int, 1>{}, t.s0 + 1);
  issue(integral_constant<int, 2>{}, t.s0 + 2);
  load_scales(t.s0 >> 2, cur);
  __builtin_amdgcn_s_waitcnt(mx4_wait(0));
  barrier();
  for (int step = t.s0; step < t.s1; step += 4) {
    load_scales((step >> 2) + 1, nxt);
    body(integral_constant<int, 0>{}, step);
    if (step + 1 < t.s1) body(integral_constant<int, 1>{}, step + 1);
    if (step + 2 < t.s1) body(integral_constant<int, 2>{}, step + 2);
    if (step + 3 < t.s1) body(integral_constant<int, 3>{}, step + 3);
    cur = nxt;
  }
  // The re-issued loads of the last steps land before the workgroup (and its
  // LDS) ends.
  __builtin_amdgcn_s_waitcnt(mx4_wait(0));

  const int nl = lane & 15, q = lane >> 4;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int r = t.row_lo + wm * Cfg::WTM + 16 * i + nl;
    if (r > t.row_last) continue;
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int col = t.col_lo + wn * Cfg::WTN + 16 * j + 4 * q;
      if (col >= N) continue;
      const float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
      store(r, col, v);
    }
  }
}

}  // namespace qg

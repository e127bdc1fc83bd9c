// mx4_tile.hpp -- tiled products with MX4 weights on gfx950, C = A . value(B)^T
// for many rows.  A fixed set of workgroups walks the output tiles (BM rows x
// BN channels); the k steps of all of a workgroup's tiles form one stream.
//
// Per step the operands' bytes go from global memory straight into one of NS
// LDS stages (buffer_load ... lds, 16 bytes per lane, no VGPRs), almost NS
// steps ahead of use, across tile borders: the first steps of the next tile are on
// their way while the last ones of this tile multiply and while its results
// are stored.  Each wave waits for its own loads of the next step and meets
// the others at one barrier per step.
//
// Two engines fill in what a step is (below): 64 k with 16-bit activations,
// 128 k with MX4 activations.  Block scales are loaded into registers one
// 512-k window (W steps) ahead.  k is a multiple of 128, so a tile's last
// window may be partial: its missing steps load a valid step again and
// multiply nothing, which keeps stages and windows in step with the code.
//
// Results are stored through a buffer resource over the tile's rows: rows past
// its last one fall outside the resource, columns past N get an offset
// outside it, and every wave issues the same number of stores.  So the waits
// after a tile can count them: the next tile's first steps do not wait for
// the stores to land.
#pragma once

#include <type_traits>
#include <utility>

#include "mx4_common.hpp"

namespace qg {

struct Mx4Problem {
  const void *A;
  const uint32_t *AS;
  const uint8_t *B;
  const uint32_t *BS;
  const uint16_t *bias;
  void *C;
  int M, N, K, bias_dt;
  const int32_t *offsets;
  int E;
  float *part;           // K slices: fp32 partial sums [slices, M, N], else null
  int kseg, slices;      // 512-k windows per slice, slices
};

// One tile: rows [row_lo, row_last] of A and C, channels from col_lo on, of
// expert e; steps [s0, s1), s0 at the start of a window.
struct Mx4Item {
  int row_lo, row_last, col_lo, e, slice, s0, s1;
};

// s_waitcnt with vmcnt(n), lgkmcnt(0), expcnt untouched.
constexpr int mx4_wait(int n) {
  return ((n < 63 ? n : 63) & 15) | (((n < 63 ? n : 63) >> 4) << 14) | (7 << 4);
}

constexpr int kRsrcFlags = 0x00020000;
constexpr int kNonTemporal = 2;   // cache policy operand of a buffer store

template <class F, int... I>
__device__ __forceinline__ void mx4_unroll(F &f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}

__device__ __forceinline__ __attribute__((address_space(3))) void *lds_ptr(char *p) {
  return (__attribute__((address_space(3))) void *)p;
}

// A wave's LDS area of ROWS rows of RB bytes on the way to C: written 16 bytes
// of a row at a time, read back so that neighbouring lanes hold neighbouring
// pieces of a row.  A store then covers whole cache lines (64 bytes of a row
// on the narrowest tile), which lets it bypass the caches: with 32-byte
// pieces the cache wrote lines out more than once, and results kept there
// pushed the operands out.  Piece c of row r lies at c ^ f(r), f chosen so
// that neither side has bank conflicts.
template <int RB, int ROWS>
struct Mx4RowBuffer {
  static constexpr int PIECES = RB / 16, PER_STORE = 64 / PIECES > 0 ? 64 / PIECES : 1;   // rows a store covers
  static_assert(RB >= 64 && RB <= 1024 && ROWS % PER_STORE == 0, "row buffer");
  char *base;
  static __device__ __forceinline__ int place(int r, int c) {
    const int f = RB >= 256 ? r & 15 : (r / (256 / RB)) & (PIECES - 1);
    return r * RB + ((c ^ f) << 4);
  }
  __device__ __forceinline__ void write(int r, int c, u32x4 v) const {
    *reinterpret_cast<u32x4 *>(base + place(r, c)) = v;
  }
  template <class Out>
  __device__ __forceinline__ void drain(const Out &out, int r0, int col0, int lane) const {
    const int r = lane / PIECES, c = lane % PIECES;
#pragma unroll
    for (int x = 0; x < ROWS; x += PER_STORE)
      out.put8(r0 + x + r, col0 + 8 * c, *reinterpret_cast<const u32x4 *>(base + place(x + r, c)));
  }
};

// ---------------------------------------------------------------------------
// 16-bit activations, 64 k a step.  LDS stage: BM activation rows of 128
// bytes, 16-byte chunk c of row r at chunk c ^ ((r / 2) % 8) (16 lanes reading
// one chunk of 16 rows touch 16 distinct 16-byte bank groups; the swizzle is
// applied on the source side of the load), then the codes of BN channels, 32
// bytes each: a 16-channel tile is 512 contiguous bytes, 32-value block h of
// the step first, so 16 lanes read 256 contiguous bytes.
//
// A wave reads each code once per step -- lane (row, half h) the 16 bytes of
// block h of its channel -- and widens it in registers right before the
// matrix instructions, two values an instruction with the block scale applied
// (exact in bf16, one rounding in fp16).  So the weights take a quarter of the
// LDS bytes that 16-bit ones would; every wave row repeats the widening: 16
// instructions per 32 channels and step.
//
// Sub-step ks multiplies k = 32 h + 8 ks + 0 .. 7 (any order of k serves as
// long as both operands use the same): of the codes, word ks of the lane's 16
// bytes; of the activations, chunk 4 h + ks of the row.
//
// The buffer resources of the loads span the tile's rows and channels: rows
// and channel tiles past the last one read as zeros, their outputs are not
// stored, and offsets stay small however large the matrices are.
//
// Bound by the matrix cores: the 256 x 256 tile runs at 1.4 to 1.6 PFLOP/s while it
// multiplies, an endless loop of these instructions with nothing else at 1.85
// (the chip lowers its clock under either).
// ---------------------------------------------------------------------------
template <int ACT_, int BM_, int BN_, int WM_, int WN_, int NS_, bool PRE>
struct Mx4Engine16 {
  static constexpr int ACT = ACT_, BM = BM_, BN = BN_, WM = WM_, WN = WN_, NS = NS_;
  static constexpr int NW = WM * WN, NTHR = 64 * NW, W = 8, K_STEP = 64;
  static constexpr int WTM = BM / WM, WTN = BN / WN;   // wave tile
  static constexpr int TM = WTM / 32, TN = WTN / 32;   // 32x32 accumulators per wave
  static constexpr int A_DMA = BM / 8 / NW;            // 1 KiB loads (8 rows) per wave and step
  static constexpr int B_LOADS = BN / 32;              // 1 KiB code loads (32 channels) per step
  static constexpr int B_DMA = (B_LOADS + NW - 1) / NW;
  static constexpr int STAGE_A = BM * 128, STAGE = STAGE_A + BN * 32;
  // Waves a SIMD is bound to hold: a lane's registers (91 to 256 of a SIMD's
  // 512, 32 to 128 of them accumulators) let every tile have two.  A bound of
  // four, which they cannot meet, put accumulators of the smaller tiles into
  // the other half of the register file: 512 x 18944 x 3584 on 128 x 128 82.0
  // us against 81.2, MX4 activations 34.2 against 33.7.
  static constexpr int WAVES = 2;
  static constexpr int LOADS = A_DMA + B_DMA, SCALE_LOADS = 2 * TN;
  static_assert(WTM % 32 == 0 && WTN % 32 == 0 && A_DMA >= 2 && A_DMA % 2 == 0, "tile shape");
  static_assert(B_LOADS % NW == 0 || NW % B_LOADS == 0, "code loads shared out evenly");
  static_assert(NS * STAGE + NW * 32 * WTN * 2 <= 160 * 1024, "LDS");

  struct Scales {
    uint32_t w[2][TN];
  };
  const Mx4Problem &p;
  const int lane, wave, wm, wn, h, nb, nw, ntiles;
  uint32_t a_lane[2], b_lane, s_lane;
  int a_addr[4], b_addr;
  f32x16 acc[TM][TN];

  __device__ __forceinline__ Mx4Engine16(const Mx4Problem &pr, int wave_)
      : p(pr), lane(threadIdx.x & 63), wave(wave_), wm(wave / WN),
        wn(wave % WN), h(lane >> 5), nb(pr.K >> 7), nw(mx4_scale_windows(pr.K)), ntiles(pr.N >> 4) {
    // Load i of a wave brings rows 8 (wave * A_DMA + i) .. + 7, lane l row
    // l / 8, placed chunk l % 8.
#pragma unroll
    for (int x = 0; x < 2; ++x)
      a_lane[x] = static_cast<uint32_t>(lane >> 3) * static_cast<uint32_t>(p.K) * 2u +
                  (((lane & 7) ^ ((4 * x + (lane >> 4)) & 7)) << 4);
    // A code load brings two 16-channel tiles' 512 bytes of the step.
    b_lane = static_cast<uint32_t>(lane >> 5) * static_cast<uint32_t>(nb) * 1024u + (lane & 31) * 16;
    s_lane = static_cast<uint32_t>((lane >> 4) & 1) * static_cast<uint32_t>(nw) * 256u + (16 * h + (lane & 15)) * 4;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks)
      a_addr[ks] = (wm * WTM + (lane & 31)) * 128 + (((4 * h + ks) ^ ((lane >> 1) & 7)) << 4);
    b_addr = STAGE_A + (wn * WTN / 16 + ((lane >> 4) & 1)) * 512 + h * 256 + (lane & 15) * 16;
  }

  __device__ __forceinline__ void issue(char *stage, const Mx4Item &t, int step) const {
    const auto rA = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char *>(static_cast<const char *>(p.A) + static_cast<size_t>(t.row_lo) * p.K * 2), 0,
        static_cast<int>(static_cast<uint32_t>(t.row_last - t.row_lo + 1) * static_cast<uint32_t>(p.K) * 2u), kRsrcFlags);
    const auto rB = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t *>(p.B + (static_cast<size_t>(t.e) * ntiles + (t.col_lo >> 4)) * nb * 1024), 0,
        static_cast<int>(static_cast<uint32_t>(min(BN / 16, ntiles - (t.col_lo >> 4))) * static_cast<uint32_t>(nb) * 1024u),
        kRsrcFlags);
#pragma unroll
    for (int i = 0; i < A_DMA; ++i) {
      const uint32_t row = static_cast<uint32_t>(8 * (wave * A_DMA + i));
      const int off = static_cast<int>(a_lane[i & 1] + row * static_cast<uint32_t>(p.K) * 2u);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rA, lds_ptr(stage + (wave * A_DMA + i) * 1024), 16, off, step * 128, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < B_DMA; ++i) {
      // With fewer code loads than waves, waves repeat one (the same bytes to
      // the same place).
      const int b = (wave * B_DMA + i) % B_LOADS;
      const uint32_t tile = static_cast<uint32_t>(2 * b);
      const int off = static_cast<int>(b_lane + tile * static_cast<uint32_t>(nb) * 1024u);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rB, lds_ptr(stage + STAGE_A + b * 1024), 16, off, step * 512, 0, 0);
    }
  }

  // A lane's two scale words per 32 channels hold its blocks of a window: word
  // s % 2, byte s / 2 for the window's step s.
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t scale_rsrc(const Mx4Item &t) const {
    return __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint32_t *>(p.BS + static_cast<size_t>(t.e) * ntiles * nw * 64), 0,
        static_cast<int>(static_cast<uint32_t>(ntiles) * static_cast<uint32_t>(nw) * 256u), kRsrcFlags);
  }
  __device__ __forceinline__ void load_scales(const Mx4Item &t, int win, Scales &s) const {
    const auto rS = scale_rsrc(t);
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const uint32_t tile = static_cast<uint32_t>((t.col_lo >> 4) + wn * (WTN / 16) + 2 * j);
      const int off = static_cast<int>(s_lane + tile * static_cast<uint32_t>(nw) * 256u);
#pragma unroll
      for (int x = 0; x < 2; ++x)
        s.w[x][j] = __builtin_amdgcn_raw_buffer_load_b32(rS, off, win * 256 + 128 * x, 0);
    }
  }
  __device__ __forceinline__ static void pin(Scales &s) {
#pragma unroll
    for (int j = 0; j < TN; ++j) asm volatile("" : "+v"(s.w[0][j]), "+v"(s.w[1][j]));
  }

  // acc[i][j] holds C^T, a lane one row of C (32 i + lane % 32) and 16 of its
  // columns, four consecutive ones per group of four values.
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
  }
  __device__ __forceinline__ void mma(int ks, const u32x4 (&a)[TM], const u32x4 (&b)[TN], const float (&sc)[TN]) {
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const u32x4 w = mx4_word_to_operand<ACT>(b[j][ks], sc[j]);
#pragma unroll
      for (int i = 0; i < TM; ++i) acc[i][j] = mfma32x32x16<ACT>(w, a[i], acc[i][j]);
    }
  }
  // Fragments of a step.  PRE: the codes and sub-step 0's activations are read
  // during the step before (head), the rest in its first part; the second
  // part, sub-step 3, runs with nothing left to read of its stage.  Without
  // PRE (fewer registers, for two workgroups a CU that hide each other's
  // reads) the first part is the whole step.
  struct Frags {
    u32x4 b[TN], a0[TM], a3[TM];
  };
  __device__ __forceinline__ void read_a(const char *stage, int ks, u32x4 (&a)[TM]) const {
#pragma unroll
    for (int i = 0; i < TM; ++i) a[i] = *reinterpret_cast<const u32x4 *>(stage + a_addr[ks] + 4096 * i);
  }
  __device__ __forceinline__ void read_head(const char *stage, Frags &f) const {
#pragma unroll
    for (int j = 0; j < TN; ++j) f.b[j] = *reinterpret_cast<const u32x4 *>(stage + b_addr + 1024 * j);
    read_a(stage, 0, f.a0);
  }
  __device__ __forceinline__ void head(const char *stage, Frags &f) const {
    if constexpr (PRE) read_head(stage, f);
  }
  template <int I>   // step I of its window
  __device__ __forceinline__ void operands(const Scales &s, float (&sc)[TN]) const {
#pragma unroll
    for (int j = 0; j < TN; ++j) sc[j] = mx4_scale_operand(s.w[I & 1][j], I >> 1);
  }
  template <int I>
  __device__ __forceinline__ void first(const char *stage, Frags &f, const Scales &s) {
    float sc[TN];
    operands<I>(s, sc);
    u32x4 a1[TM], a2[TM];
    if constexpr (!PRE) read_head(stage, f);
    read_a(stage, 1, a1);
    mma(0, f.a0, f.b, sc);
    read_a(stage, 2, a2);
    mma(1, a1, f.b, sc);
    read_a(stage, 3, f.a3);
    mma(2, a2, f.b, sc);
    if constexpr (!PRE) mma(3, f.a3, f.b, sc);
    // Fragment reads one sub-step ahead of the matrix instructions.
    constexpr int NM = TM * TN;
    if constexpr (!PRE) __builtin_amdgcn_sched_group_barrier(0x100, TN + TM, 0);
#pragma unroll
    for (int x = 0; x < 3; ++x) {
      __builtin_amdgcn_sched_group_barrier(0x100, TM, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, NM, 0);
    }
    if constexpr (!PRE) __builtin_amdgcn_sched_group_barrier(0x008, NM, 0);
  }
  template <int I>
  __device__ __forceinline__ void second(const Frags &f, const Scales &s) {
    if constexpr (PRE) {
      float sc[TN];
      operands<I>(s, sc);
      mma(3, f.a3, f.b, sc);
    }
  }

  // One step's scales by themselves, and a whole step on them.
  struct StepScales {
    uint32_t w[TN];
  };
  static constexpr int STEP_SCALE_LOADS = TN;
  __device__ __forceinline__ void load_step_scales(const Mx4Item &t, int step, StepScales &s) const {
    const auto rS = scale_rsrc(t);
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const uint32_t tile = static_cast<uint32_t>((t.col_lo >> 4) + wn * (WTN / 16) + 2 * j);
      s.w[j] = __builtin_amdgcn_raw_buffer_load_b32(rS, static_cast<int>(s_lane + tile * static_cast<uint32_t>(nw) * 256u),
                                                    (step >> 3) * 256 + 128 * (step & 1), 0);
    }
  }
  __device__ __forceinline__ void whole_step(const char *stage, const StepScales &s, int step) {
    Frags f;
    float sc[TN];
#pragma unroll
    for (int j = 0; j < TN; ++j) sc[j] = mx4_scale_operand(s.w[j] >> (8 * ((step >> 1) & 3)), 0);
    u32x4 a1[TM], a2[TM];
    read_head(stage, f);
    read_a(stage, 1, a1);
    read_a(stage, 2, a2);
    read_a(stage, 3, f.a3);
    mma(0, f.a0, f.b, sc);
    mma(1, a1, f.b, sc);
    mma(2, a2, f.b, sc);
    mma(3, f.a3, f.b, sc);
  }
  // Sums of `groups` k groups: all but the first leave theirs in LDS (part:
  // 16 bytes a lane at a time), the first adds them in order.
  static constexpr int PART = TM * TN * 16 * 64 * 4;   // bytes a wave
  __device__ __forceinline__ void put_part(char *part) const {
#pragma unroll
    for (int x = 0; x < TM * TN * 4; ++x) {
      const f32x16 &v = acc[x / (TN * 4)][x / 4 % TN];
      const int q = x % 4;
      *reinterpret_cast<f32x4 *>(part + (x * 64 + lane) * 16) = f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
    }
  }
  __device__ __forceinline__ void add_part(const char *part) {
#pragma unroll
    for (int x = 0; x < TM * TN * 4; ++x) {
      f32x16 &v = acc[x / (TN * 4)][x / 4 % TN];
      const int q = x % 4;
      const f32x4 o = *reinterpret_cast<const f32x4 *>(part + (x * 64 + lane) * 16);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * q + e] += o[e];
    }
  }

  // Value v of acc[i][j] is C[row][col], row = wave tile row + 32 i +
  // lane % 32, col = wave tile column + 32 j + 8 (v / 4) + 4 h + v % 4.
  // 16-bit results: the two halves trade every other group of four, so a lane
  // holds eight consecutive columns (16 bytes) of its row, and 32 rows at a
  // time go through the wave's LDS area to be stored in whole row pieces.
  static constexpr int EP_ROWS = 32, EP = NW * EP_ROWS * WTN * 2;
  template <class Out>
  __device__ __forceinline__ void store(const Mx4Item &t, const Out &out, char *ep) {
    const int col0 = t.col_lo + wn * WTN;
    const Mx4RowBuffer<WTN * 2, EP_ROWS> buf{ep + wave * (EP_ROWS * WTN * 2)};
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int r0 = wm * WTM + 32 * i, r = lane & 31;
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int q = 0; q < 4; q += 2) {
          const int c = 32 * j + 8 * q, col = col0 + c + 4 * h;
          const f32x4 x = out.finish(col - col0, f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]});
          const f32x4 y = out.finish(col - col0 + 8, f32x4{acc[i][j][4 * q + 4], acc[i][j][4 * q + 5], acc[i][j][4 * q + 6], acc[i][j][4 * q + 7]});
          if constexpr (Out::kBytes == 4) {
            out.put4(r0 + r, col, x);
            out.put4(r0 + r, col + 8, y);
          } else {
            const uint32_t x0 = pack2<Out::kType>(x[0], x[1]), x1 = pack2<Out::kType>(x[2], x[3]);
            const uint32_t y0 = pack2<Out::kType>(y[0], y[1]), y1 = pack2<Out::kType>(y[2], y[3]);
            const auto lo = __builtin_amdgcn_permlane32_swap(x0, y0, false, false);
            const auto hi = __builtin_amdgcn_permlane32_swap(x1, y1, false, false);
            buf.write(r, c / 8 + h, u32x4{lo[0], hi[0], lo[1], hi[1]});
          }
        }
      if constexpr (Out::kBytes == 2) buf.drain(out, r0, col0, lane);
      __builtin_amdgcn_sched_barrier(0);   // one row block's values in registers at a time
    }
  }
  template <class Out>
  static constexpr int stores() { return TM * TN * 16 * Out::kBytes / 16; }
};

// ---------------------------------------------------------------------------
// MX4 activations, 128 k a step.  The tiled layout is the lane order of the
// scaled 16 x 16 x 128 matrix instruction: a 1 KiB code block (16 rows x
// 128 k) is one wave's fragment, 16 bytes -- one 32-value block -- a lane.  An
// LDS stage holds the blocks of the BM rows, then of the BN channels, and
// every wave reads the fragments of its wave tile in lane order (no bank
// conflicts, no swizzle).  The block scales are operands of the instruction: a
// lane's scale word holds its blocks of the window's four steps, the byte
// chosen by the instruction, so a step has no VALU work at all.
//
// Bound by the matrix cores and, next to them, the fragment reads (12 KiB a
// wave and step, three quarters of the LDS bandwidth at the instruction rate):
// the 256 x 256 tile runs at 4.3 PFLOP/s while it multiplies, an endless loop
// of the instruction alone at 5.2 to 6.1 (a lowered clock; the 32 x 32 x 64
// form 5.6 to 5.8).  Four waves of 128 x 128, with a third fewer reads, spill:
// 4096 x 18944 x 3584 247 us against 176 on the same chip.
//
// Row tiles past the end repeat the last row tile, channel tiles past the end
// the last channel tile; their outputs are not stored.
// ---------------------------------------------------------------------------
template <int BM_, int BN_, int WM_, int WN_, int NS_>
struct Mx4Engine4 {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NS = NS_;
  static constexpr int NW = WM * WN, NTHR = 64 * NW, W = 4, K_STEP = 128;
  static constexpr int WTM = BM / WM, WTN = BN / WN;   // wave tile
  static constexpr int TM = WTM / 16, TN = WTN / 16;   // 16x16 accumulators per wave
  static constexpr int A_BLK = BM / 16, B_BLK = BN / 16;   // code blocks per step
  static constexpr int A_DMA = (A_BLK + NW - 1) / NW, B_DMA = (B_BLK + NW - 1) / NW;
  static constexpr int STAGE_A = BM * 64, STAGE = STAGE_A + BN * 64;
  static constexpr int WAVES = 2;   // a SIMD, as above
  static constexpr int LOADS = A_DMA + B_DMA, SCALE_LOADS = TM + TN;
  static_assert(WTM % 32 == 0 && WTN % 32 == 0, "tile shape");
  static_assert((A_BLK % NW == 0 || NW % A_BLK == 0) && (B_BLK % NW == 0 || NW % B_BLK == 0),
                "block loads shared out evenly");
  static_assert(NS * STAGE + NW * 16 * WTN * 2 <= 160 * 1024, "LDS");

  struct Scales {
    uint32_t a[TM], b[TN];
  };
  const Mx4Problem &p;
  const int lane, wave, wm, wn, nb, nw, ntiles, mtiles;
  f32x4 acc[TM][TN];

  __device__ __forceinline__ Mx4Engine4(const Mx4Problem &pr, int wave_)
      : p(pr), lane(threadIdx.x & 63), wave(wave_), wm(wave / WN),
        wn(wave % WN), nb(pr.K >> 7), nw(mx4_scale_windows(pr.K)), ntiles(pr.N >> 4), mtiles((pr.M + 15) >> 4) {}

  __device__ __forceinline__ void issue(char *stage, const Mx4Item &t, int step) const {
    const auto rA = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<void *>(p.A), 0, static_cast<int>(static_cast<uint32_t>(mtiles) * static_cast<uint32_t>(nb) * 1024u),
        kRsrcFlags);
    const auto rB = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t *>(p.B), 0, static_cast<int>(static_cast<uint32_t>(ntiles) * static_cast<uint32_t>(nb) * 1024u),
        kRsrcFlags);
    const int off = lane * 16;
    // With fewer blocks than waves, waves repeat one (the same bytes to the
    // same place).
#pragma unroll
    for (int i = 0; i < A_DMA; ++i) {
      const int b = (wave * A_DMA + i) % A_BLK, tile = min((t.row_lo >> 4) + b, mtiles - 1);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rA, lds_ptr(stage + b * 1024), 16, off, (tile * nb + step) * 1024, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < B_DMA; ++i) {
      const int b = (wave * B_DMA + i) % B_BLK, tile = min((t.col_lo >> 4) + b, ntiles - 1);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rB, lds_ptr(stage + STAGE_A + b * 1024), 16, off,
                                               (tile * nb + step) * 1024, 0, 0);
    }
  }
  __device__ __forceinline__ void load_scales(const Mx4Item &t, int win, Scales &s) const {
    const auto rA = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint32_t *>(p.AS), 0, static_cast<int>(static_cast<uint32_t>(mtiles) * static_cast<uint32_t>(nw) * 256u),
        kRsrcFlags);
    const auto rB = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint32_t *>(p.BS), 0, static_cast<int>(static_cast<uint32_t>(ntiles) * static_cast<uint32_t>(nw) * 256u),
        kRsrcFlags);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int tile = min((t.row_lo >> 4) + wm * TM + i, mtiles - 1);
      s.a[i] = __builtin_amdgcn_raw_buffer_load_b32(rA, lane * 4, (tile * nw + win) * 256, 0);
    }
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int tile = min((t.col_lo >> 4) + wn * TN + j, ntiles - 1);
      s.b[j] = __builtin_amdgcn_raw_buffer_load_b32(rB, lane * 4, (tile * nw + win) * 256, 0);
    }
  }
  __device__ __forceinline__ static void pin(Scales &s) {
#pragma unroll
    for (int i = 0; i < TM; ++i) asm volatile("" : "+v"(s.a[i]));
#pragma unroll
    for (int j = 0; j < TN; ++j) asm volatile("" : "+v"(s.b[j]));
  }

  // acc[i][j]: lane (nl, q) holds row 16 i + nl, columns 16 j + 4 q .. + 3.
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  // Fragments of a step: the channels' and the first row tiles' are read
  // during the step before (head), the rest in its first part, which
  // multiplies the first half of the row tiles; the second part runs with
  // nothing left to read of its stage.
  static constexpr int HALF = TM / 2, AHEAD = HALF < 2 ? HALF : 2;
  struct Frags {
    u32x4 b[TN], a[TM];
  };
  __device__ __forceinline__ void head(const char *stage, Frags &f) const {
    const char *As = stage + wm * TM * 1024 + lane * 16, *Bs = stage + STAGE_A + wn * TN * 1024 + lane * 16;
#pragma unroll
    for (int j = 0; j < TN; ++j) f.b[j] = *reinterpret_cast<const u32x4 *>(Bs + j * 1024);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) f.a[i] = *reinterpret_cast<const u32x4 *>(As + i * 1024);
  }
  template <int I>
  __device__ __forceinline__ void first(const char *stage, Frags &f, const Scales &s) {
    const char *As = stage + wm * TM * 1024 + lane * 16;
#pragma unroll
    for (int i = AHEAD; i < TM; ++i) f.a[i] = *reinterpret_cast<const u32x4 *>(As + i * 1024);
#pragma unroll
    for (int i = 0; i < HALF; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = mx4_mfma<I>(f.b[j], f.a[i], acc[i][j], s.b[j], s.a[i]);
    __builtin_amdgcn_sched_group_barrier(0x100, TM - AHEAD, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, HALF * TN, 0);
  }
  template <int I>
  __device__ __forceinline__ void second(const Frags &f, const Scales &s) {
#pragma unroll
    for (int i = HALF; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = mx4_mfma<I>(f.b[j], f.a[i], acc[i][j], s.b[j], s.a[i]);
  }

  // One step's scales by themselves (a window's words), and a whole step on
  // them.
  using StepScales = Scales;
  static constexpr int STEP_SCALE_LOADS = SCALE_LOADS;
  __device__ __forceinline__ void load_step_scales(const Mx4Item &t, int step, StepScales &s) const {
    load_scales(t, step >> 2, s);
  }
  __device__ __forceinline__ void whole_step(const char *stage, const StepScales &s, int step) {
    const char *As = stage + wm * TM * 1024 + lane * 16, *Bs = stage + STAGE_A + wn * TN * 1024 + lane * 16;
    const int sh = 8 * (step & 3);
    u32x4 b[TN], a[TM];
#pragma unroll
    for (int j = 0; j < TN; ++j) b[j] = *reinterpret_cast<const u32x4 *>(Bs + j * 1024);
#pragma unroll
    for (int i = 0; i < TM; ++i) a[i] = *reinterpret_cast<const u32x4 *>(As + i * 1024);
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = mx4_mfma<0>(b[j], a[i], acc[i][j], s.b[j] >> sh, s.a[i] >> sh);
  }
  static constexpr int PART = TM * TN * 64 * 16;
  __device__ __forceinline__ void put_part(char *part) const {
#pragma unroll
    for (int x = 0; x < TM * TN; ++x) *reinterpret_cast<f32x4 *>(part + (x * 64 + lane) * 16) = acc[x / TN][x % TN];
  }
  __device__ __forceinline__ void add_part(const char *part) {
#pragma unroll
    for (int x = 0; x < TM * TN; ++x) acc[x / TN][x % TN] += *reinterpret_cast<const f32x4 *>(part + (x * 64 + lane) * 16);
  }

  // 16-bit results: the lane rows q trade with their neighbours across a pair
  // of column tiles, so a lane holds eight consecutive columns (16 bytes) of
  // its row -- lanes q = 0, 2 those of the first tile, q = 1, 3 of the second
  // -- and 16 rows at a time go through the wave's LDS area to be stored in
  // whole row pieces.
  static constexpr int EP_ROWS = 16, EP = NW * EP_ROWS * WTN * 2;
  template <class Out>
  __device__ __forceinline__ void store(const Mx4Item &t, const Out &out, char *ep) {
    const int nl = lane & 15, q = lane >> 4, col0 = t.col_lo + wn * WTN;
    const Mx4RowBuffer<WTN * 2, EP_ROWS> buf{ep + wave * (EP_ROWS * WTN * 2)};
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int r0 = wm * WTM + 16 * i;
#pragma unroll
      for (int j = 0; j < TN; j += 2) {
        const int col = col0 + 16 * j + 4 * q;
        const f32x4 x = out.finish(col - col0, acc[i][j]), y = out.finish(col - col0 + 16, acc[i][j + 1]);
        if constexpr (Out::kBytes == 4) {
          out.put4(r0 + nl, col, x);
          out.put4(r0 + nl, col + 16, y);
        } else {
          const uint32_t x0 = pack2<Out::kType>(x[0], x[1]), x1 = pack2<Out::kType>(x[2], x[3]);
          const uint32_t y0 = pack2<Out::kType>(y[0], y[1]), y1 = pack2<Out::kType>(y[2], y[3]);
          const auto lo = __builtin_amdgcn_permlane16_swap(x0, y0, false, false);
          const auto hi = __builtin_amdgcn_permlane16_swap(x1, y1, false, false);
          buf.write(nl, 2 * j + 2 * (q & 1) + (q >> 1), u32x4{lo[0], hi[0], lo[1], hi[1]});
        }
      }
      if constexpr (Out::kBytes == 2) buf.drain(out, r0, col0, lane);
      __builtin_amdgcn_sched_barrier(0);   // one row block's values in registers at a time
    }
  }
  template <class Out>
  static constexpr int stores() { return TM * TN * 4 * Out::kBytes / 16; }
};

// Where a tile's sums go: C, with the bias added in fp32 and rounded once to
// the output type, or, unrounded, a K slice's partials.
template <int OUT, bool SPLIT>
struct Mx4Out {
  static constexpr int kType = SPLIT ? QG_FP32 : OUT, kBytes = kType == QG_FP32 ? 4 : 2;
  __amdgpu_buffer_rsrc_t rsrc;   // the tile's rows
  const float *bias;             // LDS: the wave's columns' biases, or null
  int N;

  // The biases of a wave's columns, loaded (a column or two a lane) at the
  // start of its tile so that they are there at the end.
  template <int WTN>
  struct Bias {
    static constexpr int PER = (WTN + 63) / 64;
    uint16_t v[PER];
    __device__ __forceinline__ void load(const Mx4Problem &p, const Mx4Item &t, int col0) {
      if constexpr (!SPLIT) {
        if (!p.bias) return;
#pragma unroll
        for (int x = 0; x < PER; ++x)
          v[x] = p.bias[static_cast<size_t>(t.e) * p.N + min(col0 + 64 * x + static_cast<int>(threadIdx.x & 63), p.N - 1)];
      }
    }
    __device__ __forceinline__ const float *place(const Mx4Problem &p, float *lds) const {
      if constexpr (!SPLIT) {
        if (!p.bias) return nullptr;
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int x = 0; x < PER; ++x)
          if (64 * x + lane < WTN) lds[64 * x + lane] = bits_to_f32_dyn(v[x], p.bias_dt);
        return lds;
      } else {
        return nullptr;
      }
    }
  };

  __device__ __forceinline__ Mx4Out(const Mx4Problem &p, const Mx4Item &t, const float *bias_)
      : bias(bias_), N(p.N) {
    char *base = SPLIT ? reinterpret_cast<char *>(p.part) + static_cast<size_t>(t.slice) * p.M * p.N * 4
                       : static_cast<char *>(p.C);
    base += static_cast<size_t>(t.row_lo) * p.N * kBytes;
    rsrc = __builtin_amdgcn_make_buffer_rsrc(
        base, 0, static_cast<int>(static_cast<uint32_t>(t.row_last - t.row_lo + 1) * static_cast<uint32_t>(p.N) * kBytes),
        kRsrcFlags);
  }
  // c: the column within the wave's.
  __device__ __forceinline__ f32x4 finish(int c, f32x4 v) const {
    if constexpr (!SPLIT) {
      if (bias) v += *reinterpret_cast<const f32x4 *>(bias + c);
    }
    return v;
  }
  __device__ __forceinline__ int offset(int r, int col) const {
    const uint32_t off = (static_cast<uint32_t>(r) * static_cast<uint32_t>(N) + static_cast<uint32_t>(col)) * kBytes;
    return static_cast<int>(col < N ? off : 0xFFFFFFF0u);
  }
  __device__ __forceinline__ void put4(int r, int col, f32x4 v) const {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), rsrc, offset(r, col), 0, 0);
  }
  __device__ __forceinline__ void put8(int r, int col, u32x4 v) const {
    __builtin_amdgcn_raw_buffer_store_b128(v, rsrc, offset(r, col), 0, kNonTemporal);
  }
};

// The stages are separate LDS objects: with one array and a stage index the
// compiler's wait-count pass cannot tell a stage being read from one being
// loaded, and waits for every direct load before each step's first read.
struct Mx4Lds {
  char *s[4];
  char *ep;      // the epilogue's row buffers
  float *bias;   // a wave's columns' biases, [waves][WTN]
};

// `work.get(n, item)`: this workgroup's n-th item, false past the last; its
// fields are uniform over the workgroup.
template <class Eng, class Out, class Work>
__device__ __forceinline__ void mx4_tiles(const Mx4Problem &p, Work &work, const Mx4Lds &L) {
  constexpr int NS = Eng::NS, W = Eng::W;
  static_assert(W % NS == 0 && NS <= 4, "stages and windows in step");
  Mx4Item ci;
  if (!work.get(0, ci)) return;
  Eng eng(p, __builtin_amdgcn_readfirstlane(threadIdx.x >> 6));
  typename Eng::Scales cur, nxt;
  typename Eng::Frags f[2];
  auto barrier = [] {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  auto prologue = [&](auto Ic) {
    constexpr int I = decltype(Ic)::value;
    eng.issue(L.s[I], ci, min(ci.s0 + I, ci.s1 - 1));
  };
  mx4_unroll(prologue, std::make_integer_sequence<int, NS>{});
  eng.load_scales(ci, ci.s0 / W, cur);
  __builtin_amdgcn_s_waitcnt(mx4_wait(0));
  barrier();
  eng.head(L.s[0], f[0]);
  bool stored = false;   // the last tile's stores may still be in flight
  for (int n = 1;; ++n) {
    Mx4Item ni;
    const bool more = work.get(n, ni);
    if (!more) ni = ci;   // its loads land in stages that no step reads
    eng.clear();
    typename Out::template Bias<Eng::WTN> bias;
    bias.load(p, ci, ci.col_lo + eng.wn * Eng::WTN);
    // A wave whose rows all lie past the tile's last multiplies nothing (its
    // loads and barriers are the workgroup's).  Grouped, 2048 rows over 64
    // experts on 128 x 256 tiles: 78 -> 68 us, 12288 rows 160 -> 155.
    const int end = ci.row_lo + eng.wm * Eng::WTM <= ci.row_last ? ci.s1 : ci.s0;
    for (int s = ci.s0; s < ci.s1; s += W) {
      // The window after this one: of this tile, or the next tile's first.
      const bool last = s + W >= ci.s1;
      Mx4Item wi = ci;
      if (last) wi = ni;
      const int ws = last ? ni.s0 : s + W;
      const bool fresh = stored && s == ci.s0;
      eng.load_scales(wi, ws / W, nxt);
      // Step s + I, its stage ST: multiply the first part while the rest of
      // the stage is read; wait for this wave's loads of the next step and
      // meet the others, all of them done with the stage; load the step NS
      // ahead into it and read the next step's first fragments while the
      // second part multiplies.  At the wait the next step's loads are the
      // oldest but those of the NS - 2 steps after it; right after a tile also
      // but its stores and this window's scale loads.
      auto body = [&](auto Ic) {
        constexpr int I = decltype(Ic)::value, ST = I % NS, AHEAD = I + NS;
        const bool live = s + I < end;
        __builtin_amdgcn_sched_barrier(0);
        if (live) eng.template first<I>(L.s[ST], f[I & 1], cur);
        __builtin_amdgcn_sched_barrier(0);
        constexpr int WAIT = (NS - 2) * Eng::LOADS;
        if constexpr (I <= NS - 2) {
          if (fresh) __builtin_amdgcn_s_waitcnt(mx4_wait(WAIT + Eng::template stores<Out>() + Eng::SCALE_LOADS));
          else __builtin_amdgcn_s_waitcnt(mx4_wait(WAIT));
        } else {
          __builtin_amdgcn_s_waitcnt(mx4_wait(WAIT));
        }
        barrier();
        if constexpr (AHEAD < W) eng.issue(L.s[ST], ci, min(s + AHEAD, ci.s1 - 1));
        else if constexpr (AHEAD < 2 * W) eng.issue(L.s[ST], wi, min(ws + AHEAD - W, wi.s1 - 1));
        __builtin_amdgcn_sched_barrier(0);
        eng.head(L.s[(ST + 1) % NS], f[(I + 1) & 1]);
        if (live) {
          eng.template second<I>(f[I & 1], cur);
        }
      };
      mx4_unroll(body, std::make_integer_sequence<int, W>{});
      cur = nxt;
      Eng::pin(cur);   // the scales' own wait here, not after the stores
    }
    eng.store(ci, Out(p, ci, bias.place(p, L.bias + eng.wave * Eng::WTN)), L.ep);
    if (!more) break;
    ci = ni;
    stored = true;
  }
  // The re-issued loads of the last steps land before the workgroup (and its
  // LDS) ends.
  __builtin_amdgcn_s_waitcnt(mx4_wait(0));
}

// One tile (or K slice of one) per workgroup, its k steps dealt out to KW
// groups of waves: for problems with few tiles, where a workgroup's time is
// that of its chain of steps and not of its matrix instructions.  Group g
// takes steps s0 + g, s0 + g + KW, ...; it loads and multiplies its own part
// of a stage, and the groups' sums meet in LDS at the end (in group order).
//
// The loop has no branch around a load: the compiler would have to assume the
// loads after a skipped one missing, and wait for all of them.  So steps past
// the end load the last one again, and only their product is skipped.
template <class Eng, int KW, class Out>
__device__ __forceinline__ void mx4_one_tile(const Mx4Problem &p, const Mx4Item &t, const Mx4Lds &L) {
  constexpr int NS = Eng::NS, LOADS = Eng::LOADS + Eng::STEP_SCALE_LOADS;
  constexpr int PER = KW * Eng::STAGE / Eng::PART;   // waves' sums a stage holds
  static_assert((KW - 1) * Eng::NW <= PER * NS && Eng::EP <= KW * Eng::STAGE, "LDS reuse");
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = wave / Eng::NW;
  Eng eng(p, wave % Eng::NW);
  typename Eng::StepScales sc[NS];
  typename Out::template Bias<Eng::WTN> bias;
  bias.load(p, t, t.col_lo + eng.wn * Eng::WTN);
  auto issue = [&](auto STc, int s) {
    constexpr int ST = decltype(STc)::value;
    const int step = min(t.s0 + s * KW + g, t.s1 - 1);
    eng.issue(L.s[ST] + g * Eng::STAGE, t, step);
    eng.load_step_scales(t, step, sc[ST]);
  };
  auto prologue = [&](auto Ic) { issue(Ic, decltype(Ic)::value); };
  mx4_unroll(prologue, std::make_integer_sequence<int, NS - 1>{});
  eng.clear();
  int s = 0;
  // Step s on stage s % NS: wait for this wave's loads of it (the oldest but
  // those of the NS - 2 steps after it), meet the others, load the step
  // NS - 1 ahead into the stage of the step before, multiply.
  auto body = [&](auto Ic) {
    constexpr int I = decltype(Ic)::value;
    __builtin_amdgcn_s_waitcnt(mx4_wait((NS - 2) * LOADS));
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    issue(std::integral_constant<int, (I + NS - 1) % NS>{}, s + I + NS - 1);
    __builtin_amdgcn_sched_barrier(0);
    const int step = t.s0 + (s + I) * KW + g;
    if (step < t.s1) eng.whole_step(L.s[I] + g * Eng::STAGE, sc[I], step);
    __builtin_amdgcn_sched_barrier(0);
  };
  for (; t.s0 + s * KW < t.s1; s += NS) mx4_unroll(body, std::make_integer_sequence<int, NS>{});
  __builtin_amdgcn_s_waitcnt(mx4_wait(0));
  __syncthreads();   // every group is done with the stages
  if constexpr (KW > 1) {
    // Wave w of group x + 1 at unit x * NW + w of the stages.
    const int w = wave % Eng::NW;
    auto at_unit = [&](int u, auto &&use) {
#pragma unroll
      for (int q = 0; q < NS; ++q)
        if (u / PER == q) use(L.s[q] + u % PER * Eng::PART);
    };
    if (g > 0) at_unit((g - 1) * Eng::NW + w, [&](char *part) { eng.put_part(part); });
    __syncthreads();
    if (g == 0) {
#pragma unroll
      for (int x = 0; x < KW - 1; ++x) at_unit(x * Eng::NW + w, [&](const char *part) { eng.add_part(part); });
    }
    __syncthreads();
    if (g > 0) return;
  }
  eng.store(t, Out(p, t, bias.place(p, L.bias + wave * Eng::WTN)), L.s[0]);
}

}  // namespace qg

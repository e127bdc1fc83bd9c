// f8_tile.hpp -- tiled products of block-scaled 8-bit floats (F8) on gfx950, for
// many rows: a fixed set of workgroups walks the output tiles (BM rows x BN
// channels), 128 k -- one block of scales -- a step, and the steps of all of a
// workgroup's tiles form one stream.
//
// Per step the operands' bytes and scales go from global memory straight into
// one of NS LDS stages (buffer_load ... lds), NS steps ahead of use and across
// tile borders.  Each wave waits for its own loads of the next step and meets
// the others at one barrier a step, in front of the products of its last pair of row
// tiles, when all of the step is in registers.  What is left multiplies while the
// next step's first fragments are read.  Tiles of four such pairs meet once more,
// behind the first: B's fragments are in registers then, and its half of the stage is
// loaded a step's half earlier, so that the loads of a step do not come all at once
// (4096 x 18944 x 3584 275 -> 266 us, 4096 x 3584 x 37888 516 -> 485, 8192^3 477 -> 457,
// gated 4096 x 18944 x 3584 with both sums stored 597 -> 565).
//
// What bounds the large tile: 8192^3 runs at 2.4 PF of the 4.2 that the matrix
// instruction reaches alone (2.07 GHz under this load).  No unit is full by the counters:
// the matrix unit is 53% busy, LDS reads take a quarter of their rate, the L2 is missed
// only by what the tiles' sharing cannot spare, and a step with the scales on the matrix instruction
// (no VALU work) takes as long as one without.  What remains is waiting: two waves a
// SIMD, all that the accumulators leave room for, that meet twice a step.
//
// A stage holds BM rows of A and BN rows of B, 128 bytes each, 16-byte chunk c
// of row r at chunk c ^ ((r / 2) % 8): 16 lanes reading one chunk of 16 rows touch 16
// distinct 16-byte bank groups (the swizzle is applied on the source side of the
// load), then the step's BM + BN scales.  Rows and channels past the last one,
// and chunks past K, read as zeros; their outputs are not stored.
//
// Gated tiles hold BN / 2 gate channels and the BN / 2 up channels beside them: of a
// wave's WTN channels the first half are gate ones, so a lane has both sums of
// each of its outputs.
#pragma once

#include <type_traits>
#include <utility>

#include "f8_common.hpp"
#include "mx4_tile.hpp"
#include "row_groups.hpp"

namespace qg {

enum { kDense, kGrouped, kGated };   // forms of a product
// B's scales: by blocks of 128 x 128, by rows, or by rows and, with A's, normal powers
// of two all of them.
enum { kByBlocks, kByRows, kByPowers };

struct F8Problem {
  const uint8_t *A;
  const float *SA;
  const uint8_t *B;
  const float *SB;
  const uint16_t *bias;
  void *C, *GU;
  int M, N, K, bias_dt;   // N: channels of B, gate and up ones alike
  const int32_t *offsets;
  int E, act;
  float *part;            // K slices: fp32 partial sums [slices, M, N], else null
  int kseg, slices;       // steps per slice, slices
  const uint32_t *powers; // kF8Flags words, 0: all scales are normal powers of two; or null: not known
};

// A lane's part of a wave's loads from A or B.  Load i brings rows 8 i .. 8 i + 7 of the
// wave's, 128 bytes each, lane l row 8 i + l / 8, placed chunk l % 8 (the swizzle above;
// odd loads' rows differ from even ones' by 8).  The whole offset goes into the vector
// register, which a buffer resource checks against its size: the scalar offset may be
// left out of that check, so a resource that ends within the wave's rows would not
// bound loads whose rows are in it.  (Rows as scalar offsets: 4096 x 18944 x 3584 the same
// 266 us, dW by powers of two of that size with its gradient 712 us for 723; rows in the
// resource's base, one for two loads: 268 for 258 and 728 for 723.)
struct F8LaneLoads {
  static constexpr uint32_t kOutside = 0x80000000u;   // past every resource
  uint32_t chunk[2], off[2];
  __host__ __device__ constexpr F8LaneLoads(int lane, uint32_t K) : chunk{}, off{} {
    for (int x = 0; x < 2; ++x) {
      chunk[x] = static_cast<uint32_t>((lane & 7) ^ ((4 * x + (lane >> 4)) & 7)) << 4;
      off[x] = (8u * static_cast<uint32_t>(x) + static_cast<uint32_t>(lane >> 3)) * K + chunk[x];
    }
  }
  // Of loads 0 and 1, with `rem` bytes left of every row; load i is past(i) further.
  __host__ __device__ constexpr uint32_t start(int x, int rem) const {
    return static_cast<int>(chunk[x]) < rem ? off[x] : kOutside;
  }
  static __host__ __device__ constexpr uint32_t past(int i, uint32_t K) { return 16u * static_cast<uint32_t>(i >> 1) * K; }
};

// The first scale of a step among scales that are `per` apart from step to step: 2^30
// rows and more have a step's scales past 2^32 bytes.
__host__ __device__ constexpr size_t f8_scale_offset(int step, uint32_t per) { return static_cast<size_t>(step) * per; }

// A stage: A's rows and the scales, and B's rows.
struct F8Stage {
  char *a, *b;
};

// One tile: rows [row_lo, row_last] of A and C, channels (gated: gate channels)
// from col_lo on, of expert e; steps [s0, s1).
struct F8Item {
  int row_lo, row_last, col_lo, e, slice, s0, s1;
  // Where the wave's loads start, and how far they may reach (F8Engine::prepare).
  const uint8_t *a, *b;
  const float *scales;
  uint32_t a_bytes, b_bytes, scale_bytes;
};

template <int BM_, int BN_, int WM_, int WN_, int NS_, int KIND_, bool GATED_>
struct F8Engine {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NS = NS_;
  static constexpr int KIND = KIND_;
  static constexpr bool BROW = KIND != kByBlocks, GATED = GATED_;
  static constexpr int NW = WM * WN, NTHR = 64 * NW;
  static constexpr int WTM = BM / WM, WTN = BN / WN;   // wave tile
  static constexpr int TM = WTM / 16, TN = WTN / 16;   // 16x16 accumulators per wave
  static constexpr int RP = TM / 2;                    // pairs of row tiles
  static constexpr int COLS = GATED ? BN / 2 : BN;     // columns of C a tile
  static constexpr int A_DMA = BM / 8 / NW, B_DMA = BN / 8 / NW;   // 1 KiB loads (8 rows) a wave and step
  static constexpr int S_LOADS = (BM + BN) / 64;       // 64 scales, a load a wave
  static constexpr int STAGE_S = BM * 128, STAGE_A = STAGE_S + (BM + BN) * 4, STAGE_B = BN * 128, STAGE = STAGE_A + STAGE_B;
  static constexpr int LOADS = A_DMA + B_DMA + 1;
  static constexpr int WAVES = 2;   // a SIMD
  static constexpr int EP_ROWS = 16, EP = NW * EP_ROWS * WTN * 2;
  static_assert(TM % 2 == 0 && TN % 2 == 0 && WTN <= 128 && 128 % (GATED ? WTN / 2 : WTN) == 0, "tile shape");
  static_assert(A_DMA % 2 == 0 && B_DMA % 2 == 0 && (A_DMA * NW * 8 == BM) && (B_DMA * NW * 8 == BN), "row loads");
  static_assert(S_LOADS <= NW && (COLS % 128 == 0 || 128 % COLS == 0), "scale loads");
  static_assert(RP % 2 == 0 || NS % 2 == 0, "fragment buffers in step with the stages");
  static_assert(NS * STAGE + EP <= 160 * 1024, "LDS");

  const F8Problem &p;
  const int lane, wave, wm, wn, nl, q, kb;
  const F8LaneLoads lane_loads;
  int a_addr[2], b_addr[2];
  uint32_t scale_at, scale_step, scale_cut;   // a lane's byte offset; scales from step to step, bytes of them off the end
  f32x4 acc[TM][TN];

  __device__ __forceinline__ F8Engine(const F8Problem &pr, int wave_)
      : p(pr), lane(threadIdx.x & 63), wave(wave_), wm(wave / WN), wn(wave % WN), nl(lane & 15), q(lane >> 4),
        kb(f8_blocks(pr.K)), lane_loads(lane, static_cast<uint32_t>(pr.K)) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      a_addr[x] = (wm * WTM + nl) * 128 + (((4 * x + q) ^ (nl >> 1)) << 4);
      b_addr[x] = (wn * WTN + nl) * 128 + (((4 * x + q) ^ (nl >> 1)) << 4);
    }
    // 64 scales a wave and step: of 64 rows of A or, behind them, channels of B.
    // With fewer such loads than waves, waves repeat one (the same values to the
    // same place).
    const int r = scale_load() * 64 + lane;
    if (r < BM) {
      scale_at = static_cast<uint32_t>(r) * 4u;
      scale_step = static_cast<uint32_t>(p.M);
    } else if (BROW) {
      scale_at = static_cast<uint32_t>(r - BM) * 4u;
      scale_step = static_cast<uint32_t>(p.N);
    } else {
      scale_at = static_cast<uint32_t>(channel(0, r - BM) >> 7) * static_cast<uint32_t>(kb) * 4u;
      scale_step = 1u;
    }
    scale_step = __builtin_amdgcn_readfirstlane(scale_step);
    scale_cut = scale_load() < BM / 64 || BROW ? 0u : 4u;
  }
  __device__ __forceinline__ int scale_load() const { return wave % S_LOADS; }
  // What a tile's loads start from.  A wave's loads bring consecutive rows of A and
  // consecutive channels of B.  (col_lo + r) / 128 = col_lo / 128 + r / 128 for the
  // tile's channels: its columns are a part of 128 or a multiple.
  __device__ __forceinline__ void prepare(F8Item &t) const {
    // Uniform by construction; a division leaves them in vector registers.
    for (int *x : {&t.row_lo, &t.row_last, &t.col_lo, &t.e, &t.slice, &t.s0, &t.s1}) *x = __builtin_amdgcn_readfirstlane(*x);
    const int rows = t.row_last - t.row_lo + 1, row = 8 * A_DMA * wave, chan = 8 * B_DMA * wave;
    const int a_left = rows - row, b_left = GATED ? 8 * B_DMA : p.N - t.col_lo - chan;
    t.a = p.A + static_cast<size_t>(t.row_lo + row) * p.K;
    t.a_bytes = a_left > 0 ? static_cast<uint32_t>(min(a_left, 8 * A_DMA)) * static_cast<uint32_t>(p.K) : 0u;
    t.b = p.B + (static_cast<size_t>(t.e) * p.N + channel(t.col_lo, chan)) * p.K;
    t.b_bytes = b_left > 0 ? static_cast<uint32_t>(min(b_left, 8 * B_DMA)) * static_cast<uint32_t>(p.K) : 0u;
    if (scale_load() < BM / 64) {
      t.scales = p.SA + t.row_lo;
      t.scale_bytes = static_cast<uint32_t>(rows) * 4u;
    } else if (BROW) {
      t.scales = p.SB + t.col_lo;
      t.scale_bytes = static_cast<uint32_t>(p.N - t.col_lo) * 4u;
    } else {
      const uint32_t nb = f8_blocks(p.N), c0 = static_cast<uint32_t>(t.col_lo >> 7);
      t.scales = p.SB + (static_cast<size_t>(t.e) * nb + c0) * kb;
      t.scale_bytes = (nb - c0) * static_cast<uint32_t>(kb) * 4u;
    }
  }

  // Channel of row r of a tile's part of B, the tile's columns from col_lo on.
  __device__ __forceinline__ int channel(int col_lo, int r) const {
    if constexpr (GATED) {
      constexpr int H = WTN / 2;
      const int w = r / WTN, in = r % WTN;
      return col_lo + w * H + in % H + (in >= H ? p.N >> 1 : 0);
    } else {
      return col_lo + r;
    }
  }

  // One step's loads: one resource for the wave's rows and one for its channels.
  struct Loads {
    const void *a, *b, *s;
    uint32_t a_bytes, b_bytes, s_bytes, off[2];
    F8Stage stage;
  };
  // A step past the tile's last loads that one again, its scales as zeros: it adds
  // nothing.
  __device__ __forceinline__ Loads loads(const F8Stage &stage, const F8Item &t, int step_) const {
    const int step = min(step_, t.s1 - 1);
    const uint32_t k0 = static_cast<uint32_t>(step) * 128u;
    const int rem = p.K - step * 128;   // bytes of the rows left
    Loads l;
#pragma unroll
    for (int x = 0; x < 2; ++x) l.off[x] = lane_loads.start(x, rem);
    l.a = t.a + k0;
    l.b = t.b + k0;
    l.s = t.scales + f8_scale_offset(step, scale_step);
    l.a_bytes = t.a_bytes ? t.a_bytes - k0 : 0u;
    l.b_bytes = t.b_bytes ? t.b_bytes - k0 : 0u;
    l.s_bytes = step_ < t.s1 ? t.scale_bytes - static_cast<uint32_t>(step) * scale_cut : 0u;
    l.stage = stage;
    return l;
  }
  static __device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void *base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, static_cast<int>(bytes), kRsrcFlags);
  }
  __device__ __forceinline__ int offset(const Loads &l, int i) const {
    return static_cast<int>(l.off[i & 1] + F8LaneLoads::past(i, static_cast<uint32_t>(p.K)));
  }
  __device__ __forceinline__ void issue_a(const Loads &l, int from, int to) const {
#pragma unroll
    for (int i = from; i < to; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc(l.a, l.a_bytes), lds_ptr(l.stage.a + (wave * A_DMA + i) * 1024), 16,
                                               offset(l, i), 0, 0, 0);
  }
  __device__ __forceinline__ void issue_scales(const Loads &l) const {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc(l.s, l.s_bytes), lds_ptr(l.stage.a + STAGE_S + scale_load() * 256), 4,
                                             static_cast<int>(scale_at), 0, 0, 0);
  }
  __device__ __forceinline__ void issue_b(const Loads &l) const {
#pragma unroll
    for (int i = 0; i < B_DMA; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc(l.b, l.b_bytes), lds_ptr(l.stage.b + (wave * B_DMA + i) * 1024), 16,
                                               offset(l, i), 0, 0, 0);
  }
  __device__ __forceinline__ void issue(const Loads &l) const {
    issue_b(l);
    issue_a(l, 0, A_DMA);
    issue_scales(l);
  }

  // acc[i][j]: lane (nl, q) holds row 16 i + nl, columns 16 j + 4 q .. + 3.
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  // B's scales of a step by blocks: one (gated: two) for the wave.
  struct ScalesB {
    float s[GATED ? 2 : 1];
  };
  struct Frags {
    i32x8 a[2][2], b[BROW ? 2 : TN];
    float sa[2][2];
    ScalesB sb;
  };
  __device__ __forceinline__ i32x8 read(const char *stage, const int (&addr)[2], int i) const {
    return f8_frag(*reinterpret_cast<const u32x4 *>(stage + addr[0] + 2048 * i),
                   *reinterpret_cast<const u32x4 *>(stage + addr[1] + 2048 * i));
  }
  __device__ __forceinline__ void read_a(const F8Stage &stage, int rp, i32x8 (&a)[2], float (&sa)[2]) const {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      a[h] = read(stage.a, a_addr, 2 * rp + h);
      sa[h] = *reinterpret_cast<const float *>(stage.a + STAGE_S + (wm * WTM + 16 * (2 * rp + h) + nl) * 4);
    }
  }
  __device__ __forceinline__ ScalesB read_sb(const F8Stage &stage) const {
    const char *at = stage.a + STAGE_S + (BM + wn * WTN) * 4;
    ScalesB s;
    s.s[0] = *reinterpret_cast<const float *>(at);
    if constexpr (GATED) s.s[1] = *reinterpret_cast<const float *>(at + WTN * 2);
    return s;
  }
  // By rows of B: those of a lane's four columns of column tile j.
  __device__ __forceinline__ f32x4 read_sb(const F8Stage &stage, int j) const {
    return *reinterpret_cast<const f32x4 *>(stage.a + STAGE_S + (BM + wn * WTN + 16 * j + 4 * q) * 4);
  }
  __device__ __forceinline__ void apply(const f32x4 (&t)[2], int rp, int j, const float (&sa)[2], const ScalesB &sb) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      f32x4 &c = acc[2 * rp + h][j];
      const float s = sa[h] * sb.s[GATED && j >= TN / 2 ? 1 : 0];
#pragma unroll
      for (int v = 0; v < 4; ++v) c[v] += t[h][v] * s;
    }
  }
  __device__ __forceinline__ void apply(const f32x4 (&t)[2], int rp, int j, const float (&sa)[2], f32x4 sb) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      f32x4 &c = acc[2 * rp + h][j];
#pragma unroll
      for (int v = 0; v < 4; ++v) c[v] += t[h][v] * (sa[h] * sb[v]);
    }
  }
  // The first fragments of a step.
  __device__ __forceinline__ void head(const F8Stage &stage, Frags &f) const {
    read_a(stage, 0, f.a[0], f.sa[0]);
#pragma unroll
    for (int j = 0; j < (BROW ? 1 : TN); ++j) f.b[j] = read(stage.b, b_addr, j);
    if constexpr (!BROW) f.sb = read_sb(stage);
  }
  // Which half of f.a step I of the stages starts on.
  static constexpr int start(int I) { return RP % 2 ? I & 1 : 0; }
  // A step: two row tiles by one column tile at a time (two matrix instructions), the
  // sums of the two before applied behind them.  The last pair of row tiles has
  // nothing left to read of the stage: behind its first product `meet` waits for the
  // next stage and gives this one up, and its other products run while that stage's
  // first fragments are read and the step's loads are issued -- behind products,
  // since the load path takes eight waves' loads one after the other.
  struct Pending {
    f32x4 t[2][2];
    float s[2][2];   // the scales of t's rows
  };
  __device__ __forceinline__ void product(Pending &d, int g, const i32x8 &b, const i32x8 (&a)[2], const float (&sa)[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      d.t[g & 1][h] = f8_mfma(b, a[h]);
      d.s[g & 1][h] = sa[h];
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  template <class Scales>
  __device__ __forceinline__ void settle(const Pending &d, int g, const Scales &sb) {
    apply(d.t[g & 1], g / TN, g % TN, d.s[g & 1], sb);
    __builtin_amdgcn_sched_barrier(0);
  }
  // The products before the last pair of row tiles.  With four pairs a step's loads
  // are spread: all waves have B's fragments in registers behind the first pair,
  // so there they meet once more, and that part of the stage is loaded early; A's
  // loads come one behind a product.  Steps of fewer products load all at once.
  static constexpr int G0 = (RP - 1) * TN;
  static constexpr bool EARLY = RP >= 4 && KIND != kByRows;
  static constexpr int LATER = EARLY ? B_DMA : 0;   // loads in flight at `meet` that belong to a later step

  // Scales that are powers of two (as the quantizer makes them) ride on the matrix
  // instruction, which adds to the sums itself: no VALU work.
  struct Powers {
    i32x8 a[2][2], b[TN];
    uint32_t ea[2][2], eb[TN];
  };
  __device__ __forceinline__ uint32_t exponent(const F8Stage &stage, int slot) const {
    return *reinterpret_cast<const uint32_t *>(stage.a + STAGE_S + slot * 4) >> 23;
  }
  __device__ __forceinline__ void read_a(const F8Stage &stage, int rp, i32x8 (&a)[2], uint32_t (&ea)[2]) const {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      a[h] = read(stage.a, a_addr, 2 * rp + h);
      ea[h] = exponent(stage, wm * WTM + 16 * (2 * rp + h) + nl);
    }
  }
  __device__ __forceinline__ void read_b(const F8Stage &stage, int j, i32x8 &b, uint32_t &eb) const {
    b = read(stage.b, b_addr, j);
    eb = exponent(stage, BM + wn * WTN + 16 * j + nl);
  }
  __device__ __forceinline__ void head(const F8Stage &stage, Powers &f) const {
    read_a(stage, 0, f.a[0], f.ea[0]);
#pragma unroll
    for (int j = 0; j < TN; ++j) read_b(stage, j, f.b[j], f.eb[j]);
  }
  // The loads of a step (l) around its products: behind product g of it.
  __device__ __forceinline__ void load_behind(const Loads &l, int g) const {
    if (!EARLY) return;
    if (g == TN) issue_b(l);
    if (g == G0 + 1) {
      issue_a(l, 0, A_DMA / 2);
      issue_scales(l);
    }
    if (g == G0 + TN / 2) issue_a(l, A_DMA / 2, A_DMA);
  }
  // `l`: the loads of the step NS ahead; `together`: a barrier; `meet`: the wait for
  // the next stage and a barrier.
  template <class Together, class Meet>
  __device__ __forceinline__ void step(const F8Stage &stage, const F8Stage &next, Powers &f, int x0, const Loads &l,
                                       Together &&together, Meet &&meet) {
#pragma unroll
    for (int g = 0; g < RP * TN; ++g) {
      const int rp = g / TN, j = g % TN, x = (x0 + rp) & 1;
      if (EARLY && g == TN) together();
      if (j == 0 && rp < RP - 1) read_a(stage, rp + 1, f.a[x ^ 1], f.ea[x ^ 1]);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        acc[2 * rp + h][j] = f8_mfma_powers(f.b[j], f.a[x][h], acc[2 * rp + h][j], f.eb[j], f.ea[x][h]);
      __builtin_amdgcn_sched_barrier(0);
      if (g == G0) {
        meet();
        if (!EARLY) issue(l);
        __builtin_amdgcn_sched_barrier(0);
        read_a(next, 0, f.a[x ^ 1], f.ea[x ^ 1]);
      }
      if (rp == RP - 1) read_b(next, j, f.b[j], f.eb[j]);
      load_behind(l, g);
    }
  }
  template <class Together, class Meet>
  __device__ __forceinline__ void step(const F8Stage &stage, const F8Stage &next, Frags &f, int x0, const Loads &l,
                                       Together &&together, Meet &&meet) {
    Pending d;
    if constexpr (BROW) {
      // With scales by rows of B (four a column tile) there are no registers for all
      // of B's fragments: they are read again for each pair of row tiles, their
      // scales with them, and the stage is given up at the step's end.
      f32x4 sb[2];
#pragma unroll
      for (int g = 0; g < RP * TN; ++g) {
        const int rp = g / TN, j = g % TN, x = (x0 + rp) & 1;
        if (j == 0 && rp < RP - 1) read_a(stage, rp + 1, f.a[x ^ 1], f.sa[x ^ 1]);
        if (g + 1 < RP * TN) f.b[(g + 1) & 1] = read(stage.b, b_addr, (g + 1) % TN);
        sb[g & 1] = read_sb(stage, j);
        product(d, g, f.b[g & 1], f.a[x], f.sa[x]);
        if (g) settle(d, g - 1, sb[(g - 1) & 1]);
      }
      meet();
      issue(l);
      read_a(next, 0, f.a[(x0 + RP) & 1], f.sa[(x0 + RP) & 1]);
      f.b[0] = read(next.b, b_addr, 0);
      settle(d, RP * TN - 1, sb[(RP * TN - 1) & 1]);
    } else {
      ScalesB sb;
#pragma unroll
      for (int g = 0; g < RP * TN; ++g) {
        const int rp = g / TN, j = g % TN, x = (x0 + rp) & 1;
        if (EARLY && g == TN) together();
        if (j == 0 && rp < RP - 1) read_a(stage, rp + 1, f.a[x ^ 1], f.sa[x ^ 1]);
        product(d, g, f.b[j], f.a[x], f.sa[x]);
        if (g) settle(d, g - 1, f.sb);
        if (g == G0) {
          meet();
          if (!EARLY) issue(l);
          __builtin_amdgcn_sched_barrier(0);
          read_a(next, 0, f.a[x ^ 1], f.sa[x ^ 1]);
          sb = read_sb(next);
        }
        if (rp == RP - 1) f.b[j] = read(next.b, b_addr, j);
        load_behind(l, g);
      }
      settle(d, RP * TN - 1, f.sb);
      f.sb = sb;
    }
  }

  // 16-bit results: lane rows q trade with their neighbours across a pair of
  // column tiles, so a lane holds eight consecutive columns (16 bytes) of its
  // row -- q = 0, 2 those of the first tile, q = 1, 3 of the second -- and 16 rows
  // at a time go through the wave's LDS area to be stored in whole row pieces.
  // Tiles j0 .. j0 + n - 1 of row tile i, to columns from col0 on.
  template <int N_, class Out, class Value>
  __device__ __forceinline__ void store_row(const Out &out, char *ep, int ln, int i, int col0, Value &&value) const {
    const int r0 = wm * WTM + 16 * i, nl = ln & 15, q = ln >> 4;
    const Mx4RowBuffer<N_ * 32, EP_ROWS> buf{ep + wave * (EP_ROWS * WTN * 2)};
#pragma unroll
    for (int j = 0; j < N_; j += 2) {
      const f32x4 x = value(j), y = value(j + 1);
      if constexpr (Out::kBytes == 4) {
        out.put4(r0 + nl, col0 + 16 * j + 4 * q, x);
        out.put4(r0 + nl, col0 + 16 * j + 16 + 4 * q, y);
      } else {
        const uint32_t x0 = pack2<Out::kType>(x[0], x[1]), x1 = pack2<Out::kType>(x[2], x[3]);
        const uint32_t y0 = pack2<Out::kType>(y[0], y[1]), y1 = pack2<Out::kType>(y[2], y[3]);
        const auto lo = __builtin_amdgcn_permlane16_swap(x0, y0, false, false);
        const auto hi = __builtin_amdgcn_permlane16_swap(x1, y1, false, false);
        buf.write(nl, 2 * j + 2 * (q & 1) + (q >> 1), u32x4{lo[0], hi[0], lo[1], hi[1]});
      }
    }
    if constexpr (Out::kBytes == 2) buf.drain(out, r0, col0, ln);
  }
  // The lane, as a value that is not known before the tile's end: what the results'
  // addresses take from it would else be kept in registers through the steps.
  __device__ __forceinline__ int late_lane() const {
    int l = lane;
    asm volatile("" : "+v"(l));
    return l;
  }
};

// Rows of a result: `cols` columns in a row of N, through a buffer resource over
// the tile's rows, so that rows past its last one are not stored, nor columns
// past `cols`, and every wave issues the same number of stores.
template <int OUT>
struct F8Rows {
  static constexpr int kType = OUT, kBytes = OUT == QG_FP32 ? 4 : 2;
  __amdgpu_buffer_rsrc_t rsrc;
  int stride, cols;
  __device__ __forceinline__ F8Rows(void *base, const F8Item &t, int stride_, int cols_) : stride(stride_), cols(cols_) {
    rsrc = __builtin_amdgcn_make_buffer_rsrc(
        static_cast<char *>(base) + static_cast<size_t>(t.row_lo) * stride * kBytes, 0,
        static_cast<int>(static_cast<uint32_t>(t.row_last - t.row_lo + 1) * static_cast<uint32_t>(stride) * kBytes), kRsrcFlags);
  }
  __device__ __forceinline__ int offset(int r, int col) const {
    const uint32_t off = (static_cast<uint32_t>(r) * static_cast<uint32_t>(stride) + static_cast<uint32_t>(col)) * kBytes;
    return static_cast<int>(col < cols ? off : 0xFFFFFFF0u);
  }
  __device__ __forceinline__ void put4(int r, int col, f32x4 v) const {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), rsrc, offset(r, col), 0, 0);
  }
  __device__ __forceinline__ void put8(int r, int col, u32x4 v) const {
    __builtin_amdgcn_raw_buffer_store_b128(v, rsrc, offset(r, col), 0, 0);
  }
};

// Where a tile's sums go: C with the bias added in fp32, or, unrounded, a K
// slice's partials, or through the gate.  stores(): a wave's stores of a tile.
template <int OUT, bool SPLIT>
struct F8Store {
  static constexpr int kOut = SPLIT ? QG_FP32 : OUT;
  template <class Eng>
  static constexpr int stores() { return Eng::TM * Eng::TN * 4 * F8Rows<kOut>::kBytes / 16; }
  template <class Eng>
  static __device__ __forceinline__ void run(Eng &eng, const F8Problem &p, const F8Item &t, char *ep) {
    const F8Rows<kOut> rows(SPLIT ? p.part + static_cast<size_t>(t.slice) * p.M * p.N : p.C, t, p.N, p.N);
    const int col0 = t.col_lo + eng.wn * Eng::WTN, ln = eng.late_lane();
    f32x4 bias[Eng::TN];
#pragma unroll
    for (int j = 0; j < Eng::TN; ++j) {
      bias[j] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (!SPLIT && p.bias) {
        const int c = min(col0 + 16 * j + 4 * (ln >> 4), p.N - 4);   // columns past N are not stored
        const uint16_t *b = p.bias + static_cast<size_t>(t.e) * p.N + c;
#pragma unroll
        for (int v = 0; v < 4; ++v) bias[j][v] = bits_to_f32_dyn(b[v], p.bias_dt);
      }
    }
#pragma unroll
    for (int i = 0; i < Eng::TM; ++i) {
      eng.template store_row<Eng::TN>(rows, ep, ln, i, col0, [&](int j) {
        f32x4 v = eng.acc[i][j];
        if constexpr (!SPLIT) v += bias[j];
        return v;
      });
      __builtin_amdgcn_sched_barrier(0);   // one row tile's values in registers at a time
    }
  }
};

template <int OUT, bool SAVE>
struct F8StoreGated {
  template <class Eng>
  static constexpr int stores() { return Eng::TM * Eng::TN / 2 * (SAVE ? 3 : 1) * 4 * F8Rows<OUT>::kBytes / 16; }
  template <class Eng>
  static __device__ __forceinline__ void run(Eng &eng, const F8Problem &p, const F8Item &t, char *ep) {
    constexpr int H = Eng::TN / 2;
    const int inter = p.N >> 1, col0 = t.col_lo + eng.wn * (Eng::WTN / 2), ln = eng.late_lane();
    const F8Rows<OUT> rows(p.C, t, inter, inter), gu(SAVE ? p.GU : p.C, t, p.N, p.N);
#pragma unroll
    for (int i = 0; i < Eng::TM; ++i) {
      if constexpr (SAVE) {
        eng.template store_row<H>(gu, ep, ln, i, col0, [&](int j) { return eng.acc[i][j]; });
        eng.template store_row<H>(gu, ep, ln, i, inter + col0, [&](int j) { return eng.acc[i][H + j]; });
      }
      eng.template store_row<H>(rows, ep, ln, i, col0, [&](int j) {
        f32x4 v;
#pragma unroll
        for (int x = 0; x < 4; ++x) v[x] = f8_gate(eng.acc[i][j][x], p.act) * eng.acc[i][H + j][x];
        return v;
      });
      __builtin_amdgcn_sched_barrier(0);
    }
  }
};

// The stages, and their halves, are separate LDS objects: with one array and an index the
// compiler's wait-count pass cannot tell a stage being read from one being
// loaded, and waits for every direct load before each step's first read.
struct F8Lds {
  F8Stage s[2];
  char *ep;      // the epilogue's row buffers
};

// `work.get(n, item)`: this workgroup's n-th item, false past the last; its
// fields are uniform over the workgroup.
template <class Eng, class Store, class Work>
__device__ __forceinline__ void f8_tiles(const F8Problem &p, Work &work, const F8Lds &L) {
  constexpr int NS = Eng::NS;
  static_assert(NS == 2, "stages");
  F8Item ci;
  if (!work.get(0, ci)) return;
  Eng eng(p, __builtin_amdgcn_readfirstlane(threadIdx.x >> 6));
  eng.prepare(ci);
  auto barrier = [] {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  auto prologue = [&](auto Ic) {
    constexpr int I = decltype(Ic)::value;
    eng.issue(eng.loads(L.s[I], ci, ci.s0 + I));
  };
  mx4_unroll(prologue, std::make_integer_sequence<int, NS>{});
  __builtin_amdgcn_s_waitcnt(mx4_wait((NS - 1) * Eng::LOADS));
  barrier();
  F8Item ni;
  bool more;
  auto look_ahead = [&](int n) {
    more = work.get(n, ni);
    if (more) eng.prepare(ni);
    else ni = ci;   // its loads land in stages that no step reads
  };
  // NS steps from s on; those past the tile's last add nothing, which keeps the
  // stages in step with the code.  FRESH: the last tile's stores may still be in
  // flight (a copy of the code of its own, so that the compiler knows how many: else
  // it waits for all of them).  No branch within: one costs a wave its place in the
  // queue of the matrix cores, and around a load all that are in flight.
  auto window = [&](auto Fresh, auto &f, int s) {
    constexpr bool FRESH = decltype(Fresh)::value;
    const bool last = s + NS >= ci.s1;
    F8Item wi = ci;
    if (last) wi = ni;
    const int ws = last ? ni.s0 : s + NS;
    auto body = [&](auto Ic) {
      constexpr int I = decltype(Ic)::value;
      // Wait for this wave's loads of the next step, the oldest but those of
      // the NS - 2 steps after it (right after a tile also but its stores), meet the
      // others, all of them done with the stage, and load the step NS ahead into it.
      auto meet = [&] {
        __builtin_amdgcn_s_waitcnt(
            mx4_wait((NS - 2) * Eng::LOADS + Eng::LATER + (FRESH && I <= NS - 2 ? Store::template stores<Eng>() : 0)));
        barrier();
      };
      eng.step(L.s[I], L.s[(I + 1) % NS], f, Eng::start(I), eng.loads(L.s[I], wi, ws + I), barrier, meet);
      __builtin_amdgcn_sched_barrier(0);
    };
    mx4_unroll(body, std::make_integer_sequence<int, NS>{});
  };
  look_ahead(1);
  auto walk = [&](auto &f) {
    eng.head(L.s[0], f);
    eng.clear();
    window(std::false_type{}, f, ci.s0);
    for (int n = 2;; ++n) {
      for (int s = ci.s0 + NS; s < ci.s1; s += NS) window(std::false_type{}, f, s);
      Store::run(eng, p, ci, L.ep);
      if (!more) break;
      ci = ni;
      look_ahead(n);
      eng.clear();
      window(std::true_type{}, f, ci.s0);
    }
  };
  std::conditional_t<Eng::KIND == kByPowers, typename Eng::Powers, typename Eng::Frags> f;
  walk(f);
  // The re-issued loads of the last steps land before the workgroup (and its
  // LDS) ends.
  __builtin_amdgcn_s_waitcnt(mx4_wait(0));
}

// Dense and gated: bands of four row tiles walked column by column, so one weight
// tile serves the band's row tiles while it is in L2.
template <class Eng>
struct F8DenseWork {
  const F8Problem &p;
  const int tiles_m, tiles_n;
  const WorkShare share;
  __device__ __forceinline__ explicit F8DenseWork(const F8Problem &pr)
      : p(pr), tiles_m((pr.M + Eng::BM - 1) / Eng::BM),
        tiles_n(((Eng::GATED ? pr.N >> 1 : pr.N) + Eng::COLS - 1) / Eng::COLS), share(tiles_m * tiles_n * pr.slices) {}
  __device__ __forceinline__ bool get(int n, F8Item &t) const {
    int id = share.first + n * share.step;
    if (id >= share.end) return false;
    constexpr int G = 4;
    const int per = tiles_m * tiles_n;
    t.slice = id / per;
    id -= t.slice * per;
    const int band = id / (G * tiles_n), first = band * G, gsz = min(G, tiles_m - first);
    const int in = id - band * G * tiles_n, tn = in / gsz;
    t.row_lo = (first + in - tn * gsz) * Eng::BM;
    t.row_last = min(p.M, t.row_lo + Eng::BM) - 1;
    t.col_lo = tn * Eng::COLS;
    t.e = 0;
    t.s0 = t.slice * p.kseg;
    t.s1 = min(f8_blocks(p.K), t.s0 + p.kseg);
    return true;
  }
};

// Grouped: the column tiles of an expert's row tile next to each other.  Items
// come in increasing order, so the wave moves on to the next 64 experts at
// most E / 64 times.
template <class Eng>
struct F8GroupWork {
  const int tiles_n, steps;
  RowGroups groups;
  const WorkShare share;
  static __device__ __forceinline__ int total(const F8Problem &p) {
    RowGroups g(p, Eng::BM);
    while (g.more()) g.next();
    return g.tiles();
  }
  __device__ __forceinline__ explicit F8GroupWork(const F8Problem &p)
      : tiles_n((p.N + Eng::BN - 1) / Eng::BN), steps(f8_blocks(p.K)), groups(p, Eng::BM), share(total(p) * tiles_n) {}
  __device__ __forceinline__ bool get(int n, F8Item &t) {
    const int id = share.first + n * share.step;
    if (id >= share.end) return false;
    const int tm = id / tiles_n;
    int row1;
    if (!groups.find(tm, t.e, t.row_lo, row1)) return false;
    t.row_last = row1 - 1;
    t.col_lo = (id - tm * tiles_n) * Eng::BN;
    t.slice = t.s0 = 0;
    t.s1 = steps;
    return true;
  }
};

template <class Eng, class Store, class Work>
__global__ __launch_bounds__(Eng::NTHR, Eng::WAVES) void k_f8_tiles(F8Problem p) {
  __shared__ __attribute__((aligned(16))) char a0[Eng::STAGE_A], b0[Eng::STAGE_B];
  __shared__ __attribute__((aligned(16))) char a1[Eng::STAGE_A], b1[Eng::STAGE_B];
  __shared__ __attribute__((aligned(16))) char ep[Eng::EP];
  if constexpr (Eng::BROW) {   // where the scales decide, both kinds are launched, and one has the work
    if (p.powers) {
      const bool powers = __ballot(p.powers[threadIdx.x & (kF8Flags - 1)] != 0) == 0;
      if (powers != (Eng::KIND == kByPowers)) return;
    }
  }
  Work work(p);
  f8_tiles<Eng, Store>(p, work, F8Lds{{{a0, b0}, {a1, b1}}, ep});
}

}  // namespace qg

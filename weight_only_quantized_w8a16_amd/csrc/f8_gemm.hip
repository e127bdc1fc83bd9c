// f8_gemm.hip -- products of block-scaled 8-bit floats (F8):
//   C[m, n] = sum_k value(A)[m, k] * value(B)[n, k] (+ bias[n]),
// dense, grouped by expert, or gated (B's rows are gate and up channels, H =
// act(g) * u) (include/qgemm.h).
//
// The scales are any fp32 numbers, so they cannot ride on the matrix
// instruction (whose own are powers of two), but for the weight's gradient, where
// a kernel has looked through them before.  Scales change every 128 k, and
// one 16 x 16 x 128 instruction covers just that: it multiplies on zero, and its
// sum t is added as acc += t * (sa * sb) in fp32, four instructions of a lane
// for every matrix instruction.  The instruction sums eight consecutive k at a
// time and cuts each product at 2^-13 of the eight's largest (measured; all 8-bit
// matrix instructions here do, and 16-bit ones run at half the rate), which on
// normal operands is 3e-5 of a result; everything past the eights is fp32.  The
// product sa * sb is rounded once, and C once.
//
// Weights are the row operand and activations the column operand, so lane
// (nl, q) of a 16 x 16 accumulator holds row m = nl -- one activation scale --
// and the four consecutive columns 4 q .. 4 q + 3.  Any order of k serves as long as
// both operands use the same: lane (nl, q) takes the 16-byte chunks q and q + 4
// of its row's 128 bytes.
#include <algorithm>
#include <cmath>

#include "f8_common.hpp"
#include "f8_tile.hpp"
#include "row_groups.hpp"

namespace qg {

namespace {

template <int OUT>
__device__ __forceinline__ void store4(void *C, size_t off, f32x4 v) {
  if constexpr (OUT == QG_FP32) {
    *reinterpret_cast<f32x4 *>(static_cast<float *>(C) + off) = v;
  } else {
    *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(C) + off) =
        u32x2{pack2<OUT>(v[0], v[1]), pack2<OUT>(v[2], v[3])};
  }
}

typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));

}  // namespace

// ---------------------------------------------------------------------------
// Streaming kernel, for few rows: a workgroup owns 16 rows and NT tiles of 16
// columns (gated: NT / 2 gate tiles and the up tiles beside them), and its waves
// take 128-k blocks in turn.  Nothing is shared between waves until their sums
// meet in LDS.  Bound by HBM: 1 x 131072 x 2048 (268 MB) 43.5 us, 6.2 TB/s, of 6.6 for a plain read.  Loads of
// whole 128-byte pieces of eight rows, and a trade between lanes, against 64 bytes
// of sixteen rows: 50.2 us, and 13 x 18944 x 3584 (68 MB) 16.1 against 19.1 (half
// pieces ask for every line twice).
// ---------------------------------------------------------------------------
template <int NT, bool BROW>
struct F8StreamBlock {
  u32x4 w[NT][2], a[2];
  float sa;
  std::conditional_t<BROW, f32x4, float> sb[NT];
};

template <int OUT, int NT, int FORM, bool BROW>
__global__ __launch_bounds__(512) void k_f8_stream(F8Problem p, int slab0) {
  extern __shared__ __attribute__((aligned(16))) float red[];   // [wave][NT][64][4]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, nwaves = blockDim.x >> 6;
  const int nl = lane & 15, q = lane >> 4;
  const int K = p.K, nb = f8_blocks(K), ntiles = p.N >> 4;
  constexpr int OWN = FORM == kGated ? NT / 2 : NT;   // column tiles of C
  const int half = ntiles >> 1, ctiles = FORM == kGated ? half : ntiles;
  const int nt0 = blockIdx.x * OWN;
  int row0 = (slab0 + static_cast<int>(blockIdx.y)) * 16, row1 = min(p.M, row0 + 16), e = 0;
  if constexpr (FORM == kGrouped) {
    RowGroups groups(p, 16);
    if (!groups.find(slab0 + blockIdx.y, e, row0, row1)) return;
  }
  // Rows and column tiles past the end repeat the last; their sums are not stored.
  const uint8_t *B = p.B + static_cast<size_t>(e) * p.N * K;
  const float *SB = p.SB + static_cast<size_t>(e) * f8_blocks(p.N) * nb;
  const uint8_t *wp[NT];
  const float *sp[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int nt = min(nt0 + i % OWN, ctiles - 1) + (i >= OWN ? half : 0);
    wp[i] = B + static_cast<size_t>(nt * 16 + (nl & 7)) * K;
    sp[i] = BROW ? SB + nt * 16 + 4 * q : SB + static_cast<size_t>(nt >> 3) * nb;
  }
  const int row = min(row0 + nl, row1 - 1);
  const uint8_t *ap = p.A + static_cast<size_t>(row) * K;
  const float *sap = p.SA + row;
  using Block = F8StreamBlock<NT, BROW>;
  auto load = [&](int kb, Block &f) {
    // Chunks past K are read at the row's start and multiplied as zeros.  A load of
    // the weight takes all 128 bytes of eight rows: lane (nl, q) chunk q + 4 (nl / 8)
    // of row nl % 8, then of row nl % 8 + 8.
    const size_t k0 = static_cast<size_t>(kb) * 128 + 16 * q, at0 = k0 < static_cast<size_t>(K) ? k0 : 0,
                 at1 = k0 + 64 < static_cast<size_t>(K) ? k0 + 64 : 0;
    const size_t at = nl < 8 ? at0 : at1;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      f.w[i][0] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(wp[i] + at));
      f.w[i][1] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(wp[i] + at + 8 * static_cast<size_t>(K)));
      if constexpr (BROW) f.sb[i] = *reinterpret_cast<const f32x4u *>(sp[i] + static_cast<size_t>(kb) * p.N);
      else f.sb[i] = sp[i][kb];
    }
    f.a[0] = *reinterpret_cast<const u32x4 *>(ap + at0);
    f.a[1] = *reinterpret_cast<const u32x4 *>(ap + at1);
    f.sa = sap[static_cast<size_t>(kb) * p.M];
  };
  f32x4 acc[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto mma = [&](int kb, Block &f) {
    // Lanes nl and nl + 8 trade halves: chunks q and q + 4 of row nl.
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const uint32_t v0 = f.w[i][0][d], v1 = f.w[i][1][d];
        const uint32_t got = __builtin_amdgcn_mov_dpp(nl < 8 ? v1 : v0, 0x128, 0xF, 0xF, false);   // row_ror:8
        f.w[i][0][d] = nl < 8 ? v0 : got;
        f.w[i][1][d] = nl < 8 ? got : v1;
      }
    if (kb * 128 + 128 > K) {   // a NaN code past K must not count: zeros on both sides
      const u32x4 zero = {0, 0, 0, 0};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool past = kb * 128 + 64 * h + 16 * q >= K;
        f.a[h] = past ? zero : f.a[h];
#pragma unroll
        for (int i = 0; i < NT; ++i) f.w[i][h] = past ? zero : f.w[i][h];
      }
    }
    const i32x8 a = f8_frag(f.a[0], f.a[1]);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const f32x4 t = f8_mfma(f8_frag(f.w[i][0], f.w[i][1]), a);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        if constexpr (BROW) acc[i][v] += t[v] * (f.sa * f.sb[i][v]);
        else acc[i][v] += t[v] * (f.sa * f.sb[i]);
      }
    }
  };
  for (int kb = wave; kb < nb; kb += nwaves) {
    Block f;
    load(kb, f);
    mma(kb, f);
  }
  // The waves' sums meet in LDS and are added in wave order; a thread finishes
  // four consecutive columns, the quads of a tile on neighbouring threads.
#pragma unroll
  for (int i = 0; i < NT; ++i) *reinterpret_cast<f32x4 *>(red + ((wave * NT + i) * 64 + lane) * 4) = acc[i];
  __syncthreads();
  for (int x = threadIdx.x; x < OWN * 64; x += blockDim.x) {
    const int c = x & 3, i = (x >> 2) % OWN, r = x / (4 * OWN);
    if (row0 + r >= row1 || nt0 + i >= ctiles) continue;
    auto total = [&](int tile) {
      f32x4 sum = {0.f, 0.f, 0.f, 0.f};
      for (int w = 0; w < nwaves; ++w)
        sum += *reinterpret_cast<const f32x4 *>(red + ((w * NT + tile) * 64 + 16 * c + r) * 4);
      return sum;
    };
    const int n = (nt0 + i) * 16 + 4 * c;
    const size_t crow = static_cast<size_t>(row0 + r);
    f32x4 v = total(i);
    if constexpr (FORM == kGated) {
      const f32x4 u = total(OWN + i);
      const size_t inter = static_cast<size_t>(p.N >> 1);
      if (p.GU) {
        store4<OUT>(p.GU, crow * p.N + n, v);
        store4<OUT>(p.GU, crow * p.N + inter + n, u);
      }
#pragma unroll
      for (int z = 0; z < 4; ++z) v[z] = f8_gate(v[z], p.act) * u[z];
      store4<OUT>(p.C, crow * inter + n, v);
    } else {
      if (p.bias) {
#pragma unroll
        for (int z = 0; z < 4; ++z) v[z] += bits_to_f32_dyn(p.bias[static_cast<size_t>(e) * p.N + n + z], p.bias_dt);
      }
      store4<OUT>(p.C, crow * p.N + n, v);
    }
  }
}

// K slices: C = RNE_out(the slices' partials summed in slice order + bias).  Bound by
// the partials' way through the 256 MB cache: 6 slices of 333 x 3584 6.6 us.
template <int OUT>
__global__ __launch_bounds__(256) void k_f8_reduce(F8Problem p) {
  const size_t mn = static_cast<size_t>(p.M) * p.N, step = static_cast<size_t>(gridDim.x) * 1024;
  for (size_t i = (static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x) * 4; i < mn; i += step) {
    f32x4 v = *reinterpret_cast<const f32x4 *>(p.part + i);
#pragma unroll 4
    for (int sl = 1; sl < p.slices; ++sl) v += *reinterpret_cast<const f32x4 *>(p.part + sl * mn + i);
    if (p.bias) {
      const int col = static_cast<int>(i % p.N);
#pragma unroll
      for (int x = 0; x < 4; ++x) v[x] += bits_to_f32_dyn(p.bias[col + x], p.bias_dt);
    }
    store4<OUT>(p.C, i, v);
  }
}

namespace {

constexpr int kMaxSlabs = 65535;   // grid.y

template <int OUT, int NT, int FORM, bool BROW>
hipError_t run_stream_as(const F8Problem &p, long slabs, hipStream_t s) {
  const int nb = f8_blocks(p.K), waves = nb < 8 ? nb : 8;
  const size_t lds = static_cast<size_t>(waves) * NT * 256 * sizeof(float);
  const unsigned cols = FORM == kGated ? static_cast<unsigned>(((p.N >> 5) + NT / 2 - 1) / (NT / 2))
                                       : static_cast<unsigned>(((p.N >> 4) + NT - 1) / NT);
  if (static_cast<uint64_t>(cols) * 64 * waves > UINT32_MAX) return hipErrorNotSupported;
  for (long s0 = 0; s0 < slabs; s0 += kMaxSlabs) {
    const unsigned ny = static_cast<unsigned>(std::min<long>(slabs - s0, kMaxSlabs));
    hipLaunchKernelGGL((k_f8_stream<OUT, NT, FORM, BROW>), dim3(cols, ny), dim3(64 * waves), lds, s, p,
                       static_cast<int>(s0));
  }
  return hipGetLastError();
}

// Column tiles a workgroup (NT): a CU reads at most some 24 KB/us whatever its waves
// ask for, so what counts is that every CU has the same share.  As many column tiles as
// let every CU have one workgroup, up to six, then half as many (two rounds of
// workgroups) up to ten, then three.  Measured, NT from 1 on:
//   tiles / CUs 0.5  (N = 2048, K = 2048, M = 1)   4.0  4.6  5.6  6.4  7.5
//               1.0  (N = 4096, K = 4096, M = 4)   6.3  7.4  9.1 10.9 13.7
//               1.25 (N = 5120, K = 5120, M = 8)  11.5  9.4 11.9 14.7 17.5
//               2.5  (N = 10240, K = 2048, M = 1)  6.8  7.7  6.3  6.9  7.9
//               3.25 (N = 13312, K = 2048, M = 12) 9.9  8.5 10.4  8.1  9.6
//               4.6  (N = 18944, K = 3584, M = 13) 19.3 17.9 17.3 19.9 16.1
//               7.0  (N = 28672, K = 4096, M = 1) 25.2 25.1 26.0 24.1 28.2
//               32   (N = 131072, K = 2048, M = 1) 47.2 43.5 43.5 44.6 45.1
// More waves a workgroup (16) and two blocks' loads in flight changed nothing.  Gated
// workgroups (NT / 2 pairs of tiles) two or four: 13312 x 2048 11.8 and 12.1, 16 x
// 18944 x 3584 30.6 and 29.8.  A grouped product's workgroups are bounds, most
// without rows: one, two or four (48 rows over 64 experts of 2816 x 2048 45.6, 35.6
// and 31.9).
template <int OUT, int FORM, bool BROW>
hipError_t run_stream(const F8Problem &p, hipStream_t s) {
  // Row slabs: a grouped product has at most one partial slab per expert
  // with rows.
  const long slabs = FORM == kGrouped ? p.M / 16 + std::min(p.E, p.M) : (static_cast<long>(p.M) + 15) / 16;
  const long cus = device_cus(), tiles = FORM == kGated ? p.N >> 5 : p.N >> 4, rounds = (tiles * slabs + cus - 1) / cus;
  if constexpr (FORM == kGated) {
    if (rounds <= 4) return run_stream_as<OUT, 2, FORM, BROW>(p, slabs, s);
    return run_stream_as<OUT, 4, FORM, BROW>(p, slabs, s);
  } else if constexpr (FORM == kGrouped) {
    if (rounds <= 2) return run_stream_as<OUT, 1, FORM, BROW>(p, slabs, s);
    if (rounds <= 4) return run_stream_as<OUT, 2, FORM, BROW>(p, slabs, s);
    return run_stream_as<OUT, 4, FORM, BROW>(p, slabs, s);
  } else if constexpr (BROW) {
    return run_stream_as<OUT, 2, FORM, BROW>(p, slabs, s);
  } else {
    switch (rounds <= 6 ? rounds : rounds <= 10 ? (rounds + 1) / 2 : 3) {
      case 1: return run_stream_as<OUT, 1, FORM, BROW>(p, slabs, s);
      case 2: return run_stream_as<OUT, 2, FORM, BROW>(p, slabs, s);
      case 3: return run_stream_as<OUT, 3, FORM, BROW>(p, slabs, s);
      case 4: return run_stream_as<OUT, 4, FORM, BROW>(p, slabs, s);
      case 5: return run_stream_as<OUT, 5, FORM, BROW>(p, slabs, s);
      default: return run_stream_as<OUT, 6, FORM, BROW>(p, slabs, s);
    }
  }
}

// The tiles, in the order qg_set_override names them.
template <int TILE, int KIND, bool GATED> struct F8Tiling;
template <int KIND, bool GATED> struct F8Tiling<kF8T256, KIND, GATED> { using Eng = F8Engine<256, 256, 2, 4, 2, KIND, GATED>; };
template <int KIND, bool GATED> struct F8Tiling<kF8T128, KIND, GATED> { using Eng = F8Engine<128, 128, 2, 2, 2, KIND, GATED>; };
template <int KIND, bool GATED> struct F8Tiling<kF8T64, KIND, GATED> { using Eng = F8Engine<64, 128, 2, 2, 2, KIND, GATED>; };

// 32-bit offsets of the tile kernels stay below this.
constexpr uint64_t kF8Span = uint64_t(1) << 31;

struct F8Plan {
  int tile;            // F8Kernel
  int kseg, slices;    // K slices in steps
  size_t bytes;        // partials
};

// What a tile costs, in microseconds: a launch (t0), per step `full` while a CU
// runs as many workgroups as it does at a time (most), lone + shared * q with a
// mean of q < most (lone: a workgroup's chain of steps; shared: what the workgroups
// take from each other), and `again` for every further round.  Fitted to 1200
// timings on MI355X, 16 to 4096 rows and 13 weight shapes of 512 x 8192 to 18944 x
// 3584, dense and gated, each tile and slice count forced, and 90 with B's scales by
// rows (residual 8 and 6 %); the tile so picked is within 0.4 % of the best one on
// average, 20 % at worst (100 x 3584 x 3584 in eight slices instead of three).  The
// steps of the 256 x 256 tile by blocks were 4 % longer then and are scaled by what they
// take since.
struct F8Cost {
  int tile, bm, bn, most;
  float t0, lone, shared, full, again;
};
constexpr F8Cost kCost[] = {{kF8T256, 256, 256, 1, 6.6f, 1.332f, 0.309f, 1.755f, 1.3f},
                            {kF8T128, 128, 128, 2, 3.7f, 0.640f, 0.249f, 1.097f, 0.f},
                            {kF8T64, 64, 128, 2, 2.4f, 0.528f, 0.167f, 0.744f, 0.f}};
constexpr F8Cost kCostRows[] = {{kF8T256, 256, 256, 1, 7.3f, 1.700f, 0.601f, 2.150f, 4.0f},
                                {kF8T128, 128, 128, 2, 4.4f, 0.654f, 0.468f, 1.190f, 2.4f},
                                {kF8T64, 64, 128, 2, 3.7f, 0.510f, 0.120f, 0.682f, 1.6f}};
// K slices: the reduction's launch, one more slice, and a byte of partials; the
// streaming kernel's launch, and a byte that a CU reads (all in the same fit).
constexpr float kSliceLaunch = 2.1f, kSliceEach = 0.24f, kSliceByte = 2.8e-7f;
constexpr float kStreamLaunch = 3.4f, kStreamByte = 4.44e-5f;
// A byte of weights that the tiles read from memory: what bounds them for few rows of
// many channels (1 x 131072 x 2048 50 us on 64 x 128 tiles, 43.5 streamed).
constexpr float kReadByte = 1.8e-7f;

// Time of `tiles` tiles of `steps` steps each.
float tiles_time(const F8Cost &c, float tiles, int steps) {
  const float q = tiles / static_cast<float>(device_cus()), most = static_cast<float>(c.most);
  const float rounds = static_cast<float>(static_cast<int>(q / most)), rest = q - rounds * most;
  steps += steps & 1;   // two stages
  return c.t0 + static_cast<float>(steps) * (rounds * c.full + (rest > 0.f ? c.lone + c.shared * rest : 0.f)) +
         c.again * std::max(0.f, rest > 0.f ? rounds : rounds - 1.f);
}

// The streaming kernel, or the tile and (dense) the K slices, with the least time by
// the measured costs.  A grouped product's row tiles are not known to the host: it
// reckons with half a tile too many for every expert that can have rows, and with a
// row slab of its own for each in the streaming kernel, which so is taken for few rows
// on few experts (8 experts, n = 3584, k = 2560: 4 rows 11.6 us against 15.8, 8 rows
// 17.1 against 16.3; 64 experts, n = 2816, k = 2048: 32 rows 31.4 against 30.8).
// Up to 16 rows, where either kernel reads every weight from memory once, no whole tiles
// are taken: their steps wait for memory longer than the fit, of 16 rows and more, has it
// (us, streamed against 64 x 128: 1 x 26624 x 2048 11.9 and 17.2, 16 x 37888 x 3584 25.6
// and 31.8, 16 x 131072 x 512 14.7 and 16.3, gated 1 x 13312 x 2048 11.8 and 17.4, 16 x
// 17920 x 720 10.8 and 12.8; 17 rows, streamed in two slabs: 37888 x 3584 46.9 and 32.0).
// K slices are (9 x 512 x 18944 16.8 streamed, 14.3 in slices).
F8Plan plan_f8(int M, int N, int K, bool brow, int form, int E) {
  const int steps = f8_blocks(K);
  F8Plan pl{kF8Stream, steps, 1, 0};
  const Override ov = dispatch_override();
  // The tile kernels' offsets span a tile's rows of A, B and C (or partials),
  // and an expert's scales.
  const uint64_t nb = f8_blocks(N);
  if (uint64_t(256) * 4 * N >= kF8Span || uint64_t(256) * K >= kF8Span || nb * steps * 4 >= kF8Span) return pl;
  if (ov.f8_tile >= 0) {
    pl.tile = ov.f8_tile;
  } else {
    const float experts = static_cast<float>(std::min(E, M));
    const float slabs = form == kGrouped ? static_cast<float>(M / 16) + experts : static_cast<float>(M / 16 + (M % 16 != 0));
    const float share = std::ceil(static_cast<float>(N / 16) * slabs / static_cast<float>(device_cus()));
    float best = kStreamLaunch + kStreamByte * share * 16.f * static_cast<float>(K);
    const float read = kReadByte * static_cast<float>(N) * static_cast<float>(K) * (form == kGrouped ? experts : 1.f);
    for (const F8Cost &c : brow ? kCostRows : kCost) {
      const int cols = form == kGated ? c.bn / 2 : c.bn, n = form == kGated ? N / 2 : N;
      const float tiles = static_cast<float>(n / cols + (n % cols != 0)) *
                          (form == kGrouped ? static_cast<float>(M) / static_cast<float>(c.bm) + 0.5f * experts
                                            : static_cast<float>(M / c.bm + (M % c.bm != 0)));
      const int least = M <= 16 && form != kGrouped ? 2 : 1;
      for (int sl = least; sl <= 16 && (sl == 1 || (form == kDense && sl <= steps / 2)); ++sl) {
        const int kseg = (steps + sl - 1) / sl;
        if ((steps + kseg - 1) / kseg != sl) continue;
        float t = std::max(tiles_time(c, tiles * static_cast<float>(sl), kseg), c.t0 + read);
        if (sl > 1)
          t += kSliceLaunch + static_cast<float>(sl) * kSliceEach +
               static_cast<float>(sl + 1) * static_cast<float>(M) * static_cast<float>(N) * 4.f * kSliceByte;
        if (t < best) {
          best = t;
          pl.tile = c.tile;
          pl.slices = sl;
          pl.kseg = kseg;
        }
      }
    }
  }
  if (pl.tile == kF8Stream || form != kDense) {
    pl.slices = 1;
    pl.kseg = steps;
    return pl;
  }
  if (ov.f8_split > 0) {
    const int want = std::min(ov.f8_split, steps);
    pl.kseg = (steps + want - 1) / want;
    pl.slices = (steps + pl.kseg - 1) / pl.kseg;
  }
  if (pl.slices > 1) pl.bytes = static_cast<size_t>(pl.slices) * M * N * sizeof(float);
  return pl;
}

// Workgroups of `Eng` a CU holds: by LDS, and by registers.
template <class Eng>
constexpr int groups_per_cu() {
  const int lds = 160 * 1024 / (Eng::NS * Eng::STAGE + Eng::EP), waves = 4 * Eng::WAVES / Eng::NW;
  return std::max(1, std::min(lds, waves));
}

template <int OUT>
hipError_t reduce_f8(const F8Problem &p, hipStream_t s) {
  const size_t blocks = (static_cast<size_t>(p.M) * p.N / 4 + 255) / 256;
  hipLaunchKernelGGL(k_f8_reduce<OUT>, dim3(static_cast<unsigned>(std::min<size_t>(blocks, 65536))), dim3(256), 0, s, p);
  return hipGetLastError();
}

template <class Eng, class Store, class Work>
hipError_t run_tiles_as(const F8Problem &p, int form, hipStream_t s) {
  const int64_t tn = ((form == kGated ? p.N / 2 : p.N) + Eng::COLS - 1) / Eng::COLS;
  // A grouped product has at most one partial row tile per expert with rows.
  const int64_t tm = form == kGrouped ? p.M / Eng::BM + std::min(p.E, p.M) : (p.M + Eng::BM - 1) / Eng::BM;
  const int64_t items = tm * tn * p.slices;
  if (items > INT32_MAX / 2) return hipErrorNotSupported;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(items, device_cus() * groups_per_cu<Eng>()));
  hipLaunchKernelGGL((k_f8_tiles<Eng, Store, Work>), dim3(grid), dim3(Eng::NTHR), 0, s, p);
  return hipGetLastError();
}

template <int OUT, int FORM, int KIND, int TILE>
hipError_t run_tiles_of(const F8Problem &p, hipStream_t s) {
  using Eng = typename F8Tiling<TILE, KIND, FORM == kGated>::Eng;
  if constexpr (FORM == kGated) {
    return p.GU ? run_tiles_as<Eng, F8StoreGated<OUT, true>, F8DenseWork<Eng>>(p, FORM, s)
                : run_tiles_as<Eng, F8StoreGated<OUT, false>, F8DenseWork<Eng>>(p, FORM, s);
  } else if constexpr (FORM == kGrouped) {
    return run_tiles_as<Eng, F8Store<OUT, false>, F8GroupWork<Eng>>(p, FORM, s);
  } else {
    return p.slices > 1 ? run_tiles_as<Eng, F8Store<OUT, true>, F8DenseWork<Eng>>(p, FORM, s)
                        : run_tiles_as<Eng, F8Store<OUT, false>, F8DenseWork<Eng>>(p, FORM, s);
  }
}

template <int OUT, int FORM, bool BROW, int TILE>
hipError_t run_tiles(const F8Problem &p, hipStream_t s) {
  hipError_t e = hipSuccess;
  if constexpr (BROW) {
    if (p.powers) e = run_tiles_of<OUT, FORM, kByPowers, TILE>(p, s);
  }
  if (e == hipSuccess) e = run_tiles_of<OUT, FORM, BROW ? kByRows : kByBlocks, TILE>(p, s);
  if (e == hipSuccess && p.slices > 1) e = reduce_f8<OUT>(p, s);
  return e;
}

template <int OUT, int FORM, bool BROW>
hipError_t run_form(const F8Problem &p, int tile, hipStream_t s) {
  switch (tile) {
    case kF8T256: return run_tiles<OUT, FORM, BROW, kF8T256>(p, s);
    case kF8T128: return run_tiles<OUT, FORM, BROW, kF8T128>(p, s);
    case kF8T64: return run_tiles<OUT, FORM, BROW, kF8T64>(p, s);
    default: return run_stream<OUT, FORM, BROW>(p, s);
  }
}

template <int OUT>
hipError_t run_f8(const F8Problem &p, int form, bool brow, int tile, hipStream_t s) {
  if (form == kGated) return run_form<OUT, kGated, false>(p, tile, s);
  if (form == kGrouped) return run_form<OUT, kGrouped, false>(p, tile, s);
  return brow ? run_form<OUT, kDense, true>(p, tile, s) : run_form<OUT, kDense, false>(p, tile, s);
}

}  // namespace

size_t f8_workspace_bytes(int m, int n, int k, int b_block) { return plan_f8(m, n, k, b_block == 1, kDense, 0).bytes; }

hipError_t launch_f8_gemm(const F8Args &a, hipStream_t s) {
  const int form = a.gated ? kGated : a.offsets ? kGrouped : kDense;
  const bool brow = a.b_block == 1;
  const F8Plan pl = plan_f8(a.M, a.N, a.K, brow, form, a.E);
  F8Problem p{a.A, a.SA, a.B, a.SB, a.bias, a.C, a.GU, a.M, a.N, a.K, a.bias_dt, a.offsets, a.E, a.act,
              nullptr, f8_blocks(a.K), 1, a.powers};
  if (pl.slices > 1 && a.ws && a.ws_bytes >= pl.bytes) {
    p.part = static_cast<float *>(a.ws);
    p.kseg = pl.kseg;
    p.slices = pl.slices;
  }
  // Two launches, of which the scales let one have the work, pay from some 50 us
  // on (4096 x 18944 x 3584 dB 889 -> 723 us with the gradient's kernel; the idle one
  // takes 4.7).
  if (static_cast<double>(a.M) * a.N * a.K < 4e10) p.powers = nullptr;
  switch (a.out) {
    case QG_FP32: return run_f8<QG_FP32>(p, form, brow, pl.tile, s);
    case QG_FP16: return run_f8<QG_FP16>(p, form, brow, pl.tile, s);
    default: return run_f8<QG_BF16>(p, form, brow, pl.tile, s);
  }
}

}  // namespace qg

// mx4_gemm.hip -- products with MX4 weights:
//   C[m, n] = sum_k A[m, k] * value(B)[n, k] (+ bias[n]),
// A in 16 bits or MX4, dense or grouped by expert (include/qgemm.h).
//
// Every block of 32 weights has a power-of-two scale, so a scaled weight is
// exact in bf16 and the conversion instructions apply the scale while they
// widen the code (two values an instruction): no scale ever reaches the
// accumulators.  MX4 activations go to the scaled matrix instruction as they
// are, 128 k at a time, with each lane's two block scales as operands.
//
// Weights are the row operand and activations the column operand, so lane
// (nl, j) of a 16 x 16 accumulator holds row m = nl and the four consecutive
// columns 4 j .. 4 j + 3.
#include <algorithm>

#include "mx4_common.hpp"
#include "mx4_tile16.hpp"
#include "mx4_tile4.hpp"

namespace qg {

namespace {

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

// Inclusive prefix sum over the wave.
__device__ __forceinline__ int wave_scan(int x, int lane) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int y = __shfl_up(x, off);
    if (lane >= off) x += y;
  }
  return x;
}

// Row tile `id` of a grouped product: expert e and its rows [row0, row1), at
// most BM of them; false past the last tile.  Offsets are clamped to
// [0, M] and a decrease counts as no rows, so no offset leads outside.
__device__ __forceinline__ bool group_tile(const int32_t *offsets, int E, int M, int BM, int id, int &e,
                                           int &row0, int &row1) {
  const int lane = threadIdx.x & 63;
  int before = 0;   // tiles of the experts of earlier rounds
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int x = e0 + lane;
    int lo = 0, hi = 0;
    if (x < E) {
      lo = min(max(offsets[x], 0), M);
      hi = max(min(max(offsets[x + 1], 0), M), lo);
    }
    const int cnt = (hi - lo + BM - 1) / BM;
    const int upto = before + wave_scan(cnt, lane);
    const unsigned long long mine = __ballot(id < upto);
    if (mine) {
      const int l = __builtin_ctzll(mine);
      const int first = __shfl(upto - cnt, l);
      e = e0 + l;
      row0 = __shfl(lo, l) + (id - first) * BM;
      row1 = min(__shfl(hi, l), row0 + BM);
      return true;
    }
    before = __shfl(upto, 63);
  }
  return false;
}

// Row tiles of BM rows of a grouped product.
__device__ __forceinline__ int group_tiles(const int32_t *offsets, int E, int M, int BM) {
  const int lane = threadIdx.x & 63;
  int cnt = 0;
  for (int x = lane; x < E; x += 64) {
    const int lo = min(max(offsets[x], 0), M), hi = max(min(max(offsets[x + 1], 0), M), lo);
    cnt += (hi - lo + BM - 1) / BM;
  }
  return __shfl(wave_scan(cnt, lane), 63);
}

template <int OUT>
__device__ __forceinline__ void store4(void *C, size_t off, const float (&v)[4]) {
  if constexpr (OUT == QG_FP32) {
    *reinterpret_cast<f32x4 *>(static_cast<float *>(C) + off) = f32x4{v[0], v[1], v[2], v[3]};
  } else {
    *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(C) + off) =
        u32x2{pack2<OUT>(v[0], v[1]), pack2<OUT>(v[2], v[3])};
  }
}

}  // namespace

// ---------------------------------------------------------------------------
// Streaming kernel: a workgroup owns 16 rows and NT tiles of 16 columns, its
// waves take 128-k blocks in turn, each lane the 16 bytes of one 32-value
// block.  The waves' sums meet in LDS.
// ---------------------------------------------------------------------------
template <int ACT, int OUT, int NT, bool GROUPED>
__global__ __launch_bounds__(512) void k_mx4_stream(Mx4Problem p, int slab0) {
  extern __shared__ __attribute__((aligned(16))) float red[];   // [wave][NT][64][4]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, nwaves = blockDim.x >> 6;
  const int nl = lane & 15, j = lane >> 4;
  const int K = p.K, nb = K >> 7, nw = mx4_scale_windows(K), ntiles = p.N >> 4;
  const int nt0 = blockIdx.x * NT;
  int row0 = (slab0 + static_cast<int>(blockIdx.y)) * 16, row1 = min(p.M, row0 + 16), e = 0;
  if constexpr (GROUPED) {
    if (!group_tile(p.offsets, p.E, p.M, 16, slab0 + blockIdx.y, e, row0, row1)) return;
  }
  const uint8_t *B = p.B + static_cast<size_t>(e) * ntiles * nb * 1024;
  const uint32_t *BS = p.BS + static_cast<size_t>(e) * ntiles * nw * 64;
  const int row = min(row0 + nl, row1 - 1);   // rows past the end repeat the last; never stored

  f32x4 acc[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int kb = wave; kb < nb; kb += nwaves) {
    u32x4 w[NT];
    uint32_t sw[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int nt = min(nt0 + i, ntiles - 1);
      w[i] = __builtin_nontemporal_load(
          reinterpret_cast<const u32x4 *>(B + (static_cast<size_t>(nt) * nb + kb) * 1024 + lane * 16));
      sw[i] = BS[(static_cast<size_t>(nt) * nw + (kb >> 2)) * 64 + lane] >> (8 * (kb & 3));
    }
    if constexpr (ACT == kMX4) {
      const int rt = row0 >> 4;   // row0 is a multiple of 16 (not grouped)
      const u32x4 a = *reinterpret_cast<const u32x4 *>(
          static_cast<const uint8_t *>(p.A) + (static_cast<size_t>(rt) * nb + kb) * 1024 + lane * 16);
      const uint32_t sa = p.AS[(static_cast<size_t>(rt) * nw + (kb >> 2)) * 64 + lane] >> (8 * (kb & 3));
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[i] = mx4_mfma(w[i], a, acc[i], sw[i], sa);
    } else {
      const uint16_t *ap = static_cast<const uint16_t *>(p.A) + static_cast<size_t>(row) * K + kb * 128 + 32 * j;
      u32x4 a[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) a[t] = *reinterpret_cast<const u32x4 *>(ap + 8 * t);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const float s = mx4_scale_operand(sw[i], 0);
#pragma unroll
        for (int t = 0; t < 4; ++t)
          acc[i] = mfma16x16x32<ACT>(mx4_word_to_operand<ACT>(w[i][t], s), a[t], acc[i]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NT; ++i) *reinterpret_cast<f32x4 *>(red + ((wave * NT + i) * 64 + lane) * 4) = acc[i];
  __syncthreads();
  // Thread (row r, tile i, column quad c): four consecutive columns, the quads
  // of a tile on neighbouring threads.
  for (int q = threadIdx.x; q < NT * 64; q += blockDim.x) {
    const int c = q & 3, i = (q >> 2) % NT, r = q / (4 * NT);
    if (row0 + r >= row1 || nt0 + i >= ntiles) continue;
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    for (int w = 0; w < nwaves; ++w)
      sum += *reinterpret_cast<const f32x4 *>(red + ((w * NT + i) * 64 + 16 * c + r) * 4);
    const int n = (nt0 + i) * 16 + 4 * c;
    float v[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      v[x] = sum[x];
      if (p.bias) v[x] += bits_to_f32_dyn(p.bias[static_cast<size_t>(e) * p.N + n + x], p.bias_dt);
    }
    store4<OUT>(p.C, static_cast<size_t>(row0 + r) * p.N + n, v);
  }
}

// ---------------------------------------------------------------------------
// Tile kernels (mx4_tile16.hpp, mx4_tile4.hpp).
// ---------------------------------------------------------------------------

// Workgroup b runs on XCD b % 8.  Of `count` working workgroups each XCD takes
// a contiguous run of the tile order, so neighbouring tiles share an L2.
__device__ __forceinline__ int xcd_order(int b, int count) {
  const int xcd = b & 7, loc = b >> 3, per = count >> 3, rem = count & 7;
  return (xcd < rem) ? xcd * (per + 1) + loc : rem * (per + 1) + (xcd - rem) * per + loc;
}

// Where a finished sum goes: C, rounded with its bias, or a K slice's partials.
template <int OUT, bool SPLIT>
struct Mx4Store {
  const Mx4Problem &p;
  const uint16_t *bias;   // of the tile's expert
  int slice;
  __device__ __forceinline__ void operator()(int r, int col, const float (&v)[4]) const {
    if constexpr (SPLIT) {
      float *P = p.part + static_cast<size_t>(slice) * p.M * p.N;
      *reinterpret_cast<f32x4 *>(P + static_cast<size_t>(r) * p.N + col) = f32x4{v[0], v[1], v[2], v[3]};
    } else {
      float o[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) o[x] = bias ? v[x] + bits_to_f32_dyn(bias[col + x], p.bias_dt) : v[x];
      store4<OUT>(p.C, static_cast<size_t>(r) * p.N + col, o);
    }
  }
};

// Row tile and column tile of this workgroup.  Dense: bands of four row tiles
// walked column by column, so one weight tile serves the band's row tiles
// while it is in L2.  Grouped: the column tiles of an expert's row tile next
// to each other; the grid is sized for the most row tiles the offsets can
// give, and workgroups past the real count end here.
template <int BM, bool GROUPED>
__device__ __forceinline__ bool mx4_tile_of(const Mx4Problem &p, int tiles_m, int tiles_n, int &tn, int &e,
                                            int &slice, int &row0, int &row1) {
  e = slice = 0;
  if constexpr (GROUPED) {
    const int count = group_tiles(p.offsets, p.E, p.M, BM) * tiles_n;
    if (static_cast<int>(blockIdx.x) >= count) return false;
    const int id = xcd_order(blockIdx.x, count), tm = id / tiles_n;
    tn = id - tm * tiles_n;
    return group_tile(p.offsets, p.E, p.M, BM, tm, e, row0, row1);
  } else {
    constexpr int G = 4;
    int id = xcd_order(blockIdx.x, gridDim.x);
    const int per = tiles_m * tiles_n;
    slice = id / per;
    id -= slice * per;
    const int band = id / (G * tiles_n), first = band * G, gsz = min(G, tiles_m - first);
    const int in = id - band * G * tiles_n;
    tn = in / gsz;
    row0 = (first + in % gsz) * BM;
    row1 = min(p.M, row0 + BM);
    return true;
  }
}

template <class Cfg, int ACT, bool GROUPED, bool SPLIT>
__global__ __launch_bounds__(Cfg::NTHR) void k_mx4_tile16(Mx4Problem p, int tiles_m, int tiles_n) {
  __shared__ __attribute__((aligned(16))) char a0[Cfg::STAGE_A];
  __shared__ __attribute__((aligned(16))) char a1[Cfg::STAGE_A];
  __shared__ __attribute__((aligned(16))) char a2[Cfg::NS > 2 ? Cfg::STAGE_A : 16];
  __shared__ __attribute__((aligned(16))) char a3[Cfg::NS > 2 ? Cfg::STAGE_A : 16];
  __shared__ __attribute__((aligned(16))) char b0[Cfg::STAGE_B];
  __shared__ __attribute__((aligned(16))) char b1[Cfg::STAGE_B];
  __shared__ __attribute__((aligned(16))) char b2[Cfg::NS > 2 ? Cfg::STAGE_B : 16];
  __shared__ __attribute__((aligned(16))) char b3[Cfg::NS > 2 ? Cfg::STAGE_B : 16];
  int tn, e, slice, row0, row1;
  if (!mx4_tile_of<Cfg::BM, GROUPED>(p, tiles_m, tiles_n, tn, e, slice, row0, row1)) return;
  const int nb = p.K >> 7, nw = mx4_scale_windows(p.K), ntiles = p.N >> 4, steps = p.K >> 6;
  const Mx4Tile t{row0, row1 - 1, tn * Cfg::BN, SPLIT ? slice * p.kseg * 8 : 0,
                  SPLIT ? min(steps, (slice + 1) * p.kseg * 8) : steps};
  mx4_tile16<Cfg, ACT>(static_cast<const uint16_t *>(p.A), p.M, p.B + static_cast<size_t>(e) * ntiles * nb * 1024,
                       p.BS + static_cast<size_t>(e) * ntiles * nw * 64, p.N, p.K, t,
                       Mx4Lds{{a0, a1, a2, a3}, {b0, b1, b2, b3}},
                       Mx4Store<ACT, SPLIT>{p, p.bias ? p.bias + static_cast<size_t>(e) * p.N : nullptr, slice});
}

template <class Cfg, int OUT, bool SPLIT>
__global__ __launch_bounds__(Cfg::NTHR) void k_mx4_tile4(Mx4Problem p, int tiles_m, int tiles_n) {
  __shared__ __attribute__((aligned(16))) char a0[Cfg::STAGE_A];
  __shared__ __attribute__((aligned(16))) char a1[Cfg::STAGE_A];
  __shared__ __attribute__((aligned(16))) char a2[Cfg::STAGE_A];
  __shared__ __attribute__((aligned(16))) char a3[Cfg::STAGE_A];
  __shared__ __attribute__((aligned(16))) char b0[Cfg::STAGE_B];
  __shared__ __attribute__((aligned(16))) char b1[Cfg::STAGE_B];
  __shared__ __attribute__((aligned(16))) char b2[Cfg::STAGE_B];
  __shared__ __attribute__((aligned(16))) char b3[Cfg::STAGE_B];
  int tn, e, slice, row0, row1;
  if (!mx4_tile_of<Cfg::BM, false>(p, tiles_m, tiles_n, tn, e, slice, row0, row1)) return;
  const int steps = p.K >> 7;
  const Mx4Tile t{row0, row1 - 1, tn * Cfg::BN, SPLIT ? slice * p.kseg * 4 : 0,
                  SPLIT ? min(steps, (slice + 1) * p.kseg * 4) : steps};
  mx4_tile4<Cfg>(static_cast<const uint8_t *>(p.A), p.AS, p.M, p.B, p.BS, p.N, p.K, t,
                 Mx4Lds{{a0, a1, a2, a3}, {b0, b1, b2, b3}}, Mx4Store<OUT, SPLIT>{p, p.bias, slice});
}

// K slices: C = RNE_out(the slices' partials summed in slice order + bias).
template <int OUT>
__global__ __launch_bounds__(256) void k_mx4_reduce(Mx4Problem p) {
  const size_t mn = static_cast<size_t>(p.M) * p.N, step = static_cast<size_t>(gridDim.x) * 1024;
  for (size_t i = (static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x) * 4; i < mn; i += step) {
    f32x4 s = *reinterpret_cast<const f32x4 *>(p.part + i);
    for (int sl = 1; sl < p.slices; ++sl) s += *reinterpret_cast<const f32x4 *>(p.part + sl * mn + i);
    const int r = static_cast<int>(i / p.N), col = static_cast<int>(i - static_cast<size_t>(r) * p.N);
    const float v[4] = {s[0], s[1], s[2], s[3]};
    Mx4Store<OUT, false>{p, p.bias, 0}(r, col, v);
  }
}

namespace {

constexpr int kMaxSlabs = 65535;   // grid.y

template <int ACT, int OUT, bool GROUPED>
hipError_t run_stream(const Mx4Problem &p, hipStream_t s) {
  constexpr int NT = 2;
  const int nb = p.K >> 7, waves = nb < 8 ? nb : 8;
  const size_t lds = static_cast<size_t>(waves) * NT * 256 * sizeof(float);
  const unsigned cols = static_cast<unsigned>(((p.N >> 4) + NT - 1) / NT);
  // Row slabs: a grouped product has at most one partial slab per expert
  // with rows.
  const long slabs = GROUPED ? p.M / 16 + std::min(p.E, p.M) : (static_cast<long>(p.M) + 15) / 16;
  for (long s0 = 0; s0 < slabs; s0 += kMaxSlabs) {
    const unsigned ny = static_cast<unsigned>(std::min<long>(slabs - s0, kMaxSlabs));
    hipLaunchKernelGGL((k_mx4_stream<ACT, OUT, NT, GROUPED>), dim3(cols, ny), dim3(64 * waves), lds, s, p,
                       static_cast<int>(s0));
  }
  return hipGetLastError();
}

}  // namespace

namespace {

using Cfg16L = Mx4Cfg16<256, 256, 2, 4, 4>;   // waves of 128 x 64
using Cfg16N = Mx4Cfg16<256, 128, 4, 2, 4>;   // waves of 64 x 64
using Cfg16M = Mx4Cfg16<128, 128, 2, 4, 4>;   // waves of 64 x 32
using Cfg16S = Mx4Cfg16<64, 128, 2, 4, 4>;    // waves of 32 x 32
using Cfg4L = Mx4Cfg4<256, 256, 2, 4, 4>;     // waves of 128 x 64
using Cfg4N = Mx4Cfg4<256, 128, 4, 2, 4>;     // waves of 64 x 64
using Cfg4M = Mx4Cfg4<128, 128, 2, 4, 4>;     // waves of 64 x 32
using Cfg4S = Mx4Cfg4<64, 128, 2, 4, 4>;      // waves of 32 x 32

struct Mx4Plan {
  int tile;            // Mx4Tile order below, or kStream
  int kseg, slices;    // K slices in 512-k windows
  size_t bytes;        // partials
};

constexpr int tile_bm(int tile) { return tile == kMx4L || tile == kMx4N ? 256 : tile == kMx4M ? 128 : 64; }
constexpr int tile_bn(int tile) { return tile == kMx4L ? 256 : 128; }

Mx4Plan plan_mx4(int M, int N, int K, bool a4, bool grouped, int E) {
  Mx4Plan pl{kMx4Stream, 0, 1, 0};
  const Override ov = dispatch_override();
  // 32-bit offsets of the tile kernels' buffer loads.
  const uint64_t lim = uint64_t(1) << 31;
  const uint64_t a_bytes = uint64_t((M + 15) / 16 * 16) * K / (a4 ? 2 : 1) * (a4 ? 1 : 2);
  const bool fits = a_bytes < lim && uint64_t(N) * K / 2 < lim;
  if (!fits || ov.mx4_tile == kMx4Stream) return pl;
  if (ov.mx4_tile >= 0) pl.tile = ov.mx4_tile;
  else if (M > 64) pl.tile = kMx4M;
  if (pl.tile == kMx4Stream) return pl;
  if (ov.mx4_split > 1 && !grouped) {
    const int windows = mx4_scale_windows(K), want = std::min(ov.mx4_split, windows);
    pl.kseg = (windows + want - 1) / want;
    pl.slices = (windows + pl.kseg - 1) / pl.kseg;
    if (pl.slices > 1) pl.bytes = static_cast<size_t>(pl.slices) * M * N * sizeof(float);
  }
  return pl;
}

template <int OUT>
hipError_t reduce_mx4(const Mx4Problem &p, hipStream_t s) {
  const size_t blocks = (static_cast<size_t>(p.M) * p.N / 4 + 255) / 256;
  hipLaunchKernelGGL(k_mx4_reduce<OUT>, dim3(static_cast<unsigned>(std::min<size_t>(blocks, 65536))), dim3(256), 0,
                     s, p);
  return hipGetLastError();
}

template <class Cfg, int ACT, bool GROUPED>
hipError_t run_tile16(const Mx4Problem &p, hipStream_t s) {
  const int tn = (p.N + Cfg::BN - 1) / Cfg::BN;
  const int tm = GROUPED ? p.M / Cfg::BM + std::min(p.E, p.M) : (p.M + Cfg::BM - 1) / Cfg::BM;
  const int64_t grid = static_cast<int64_t>(tm) * tn * p.slices;
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  if constexpr (!GROUPED) {
    if (p.slices > 1) {
      hipLaunchKernelGGL((k_mx4_tile16<Cfg, ACT, false, true>), dim3(static_cast<unsigned>(grid)), dim3(Cfg::NTHR),
                         0, s, p, tm, tn);
      return reduce_mx4<ACT>(p, s);
    }
  }
  hipLaunchKernelGGL((k_mx4_tile16<Cfg, ACT, GROUPED, false>), dim3(static_cast<unsigned>(grid)), dim3(Cfg::NTHR), 0,
                     s, p, tm, tn);
  return hipGetLastError();
}

template <class Cfg, int OUT>
hipError_t run_tile4(const Mx4Problem &p, hipStream_t s) {
  const int tn = (p.N + Cfg::BN - 1) / Cfg::BN, tm = (p.M + Cfg::BM - 1) / Cfg::BM;
  const int64_t grid = static_cast<int64_t>(tm) * tn * p.slices;
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  if (p.slices > 1) {
    hipLaunchKernelGGL((k_mx4_tile4<Cfg, OUT, true>), dim3(static_cast<unsigned>(grid)), dim3(Cfg::NTHR), 0, s, p,
                       tm, tn);
    return reduce_mx4<OUT>(p, s);
  }
  hipLaunchKernelGGL((k_mx4_tile4<Cfg, OUT, false>), dim3(static_cast<unsigned>(grid)), dim3(Cfg::NTHR), 0, s, p, tm,
                     tn);
  return hipGetLastError();
}

template <int ACT, bool GROUPED>
hipError_t run_a16(const Mx4Problem &p, int tile, hipStream_t s) {
  switch (tile) {
    case kMx4L: return run_tile16<Cfg16L, ACT, GROUPED>(p, s);
    case kMx4N: return run_tile16<Cfg16N, ACT, GROUPED>(p, s);
    case kMx4M: return run_tile16<Cfg16M, ACT, GROUPED>(p, s);
    case kMx4S: return run_tile16<Cfg16S, ACT, GROUPED>(p, s);
    default: return run_stream<ACT, ACT, GROUPED>(p, s);
  }
}

template <int OUT>
hipError_t run_a4(const Mx4Problem &p, int tile, hipStream_t s) {
  switch (tile) {
    case kMx4L: return run_tile4<Cfg4L, OUT>(p, s);
    case kMx4N: return run_tile4<Cfg4N, OUT>(p, s);
    case kMx4M: return run_tile4<Cfg4M, OUT>(p, s);
    case kMx4S: return run_tile4<Cfg4S, OUT>(p, s);
    default: return run_stream<kMX4, OUT, false>(p, s);
  }
}

}  // namespace

size_t mx4_workspace_bytes(int m, int n, int k, int act_bits) {
  return plan_mx4(m, n, k, act_bits == 4, false, 0).bytes;
}

hipError_t launch_mx4_gemm(const Mx4Args &a, hipStream_t s) {
  Mx4Problem p{a.A, reinterpret_cast<const uint32_t *>(a.AS), a.B, reinterpret_cast<const uint32_t *>(a.BS),
               a.bias, a.C, a.M, a.N, a.K, a.bias_dt, a.offsets, a.E, nullptr, 0, 1};
  const Mx4Plan pl = plan_mx4(a.M, a.N, a.K, a.act == kMX4, a.offsets != nullptr, a.E);
  if (pl.slices > 1 && a.ws && a.ws_bytes >= pl.bytes) {
    p.part = static_cast<float *>(a.ws);
    p.kseg = pl.kseg;
    p.slices = pl.slices;
  }
  if (a.act == kMX4) {
    switch (a.out) {
      case QG_FP32: return run_a4<QG_FP32>(p, pl.tile, s);
      case QG_FP16: return run_a4<QG_FP16>(p, pl.tile, s);
      default: return run_a4<QG_BF16>(p, pl.tile, s);
    }
  }
  if (a.offsets)
    return a.act == kFP16 ? run_a16<kFP16, true>(p, pl.tile, s) : run_a16<kBF16, true>(p, pl.tile, s);
  return a.act == kFP16 ? run_a16<kFP16, false>(p, pl.tile, s) : run_a16<kBF16, false>(p, pl.tile, s);
}

}  // namespace qg

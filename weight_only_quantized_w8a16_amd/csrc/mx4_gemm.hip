// mx4_gemm.hip -- products with MX4 weights:
//   C[m, n] = sum_k A[m, k] * value(B)[n, k] (+ bias[n]),
// A in 16 bits or MX4, dense or grouped by expert (include/qgemm.h).  Sums are
// fp32; the one rounding is the store to C's type (and in fp16 that of a
// weight below 2^-23 or, to infinity, from 65520 on, as the conversion's).
// Subnormal operands, products and sums are kept.
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
#include "mx4_tile.hpp"

namespace qg {

namespace {

// Inclusive prefix sum and maximum over the wave.
__device__ __forceinline__ int wave_scan(int x, int lane) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int y = __shfl_up(x, off);
    if (lane >= off) x += y;
  }
  return x;
}
__device__ __forceinline__ int wave_scan_max(int x, int lane) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int y = __shfl_up(x, off);
    if (lane >= off) x = max(x, y);
  }
  return x;
}

// The row tiles of a grouped product, 64 experts at a time, one a lane.
// Offsets are clamped to [0, M] and never go back: expert e's rows run from
// the largest offset up to e to the largest up to e + 1.  So whatever the
// offsets hold, no row lies outside, none belongs to two experts, and there
// are at most M / BM + min(E, M) row tiles, which is what the grids assume.
struct Mx4Groups {
  const int32_t *offsets;
  int E, M, BM;
  int e0, lo, hi;      // the lane's expert is e0 + lane; its rows [lo, hi)
  int before, upto;    // row tiles before expert e0, and up to the lane's
  __device__ __forceinline__ int bound(int x) const { return min(max(offsets[x], 0), M); }
  __device__ __forceinline__ void load(int start, int from, int tiles) {   // from: the largest offset up to start
    const int lane = threadIdx.x & 63, x = start + lane;
    hi = max(wave_scan_max(x < E ? bound(x + 1) : 0, lane), from);
    lo = __shfl_up(hi, 1);
    if (lane == 0) lo = from;
    e0 = start;
    before = tiles;
    upto = tiles + wave_scan((hi - lo + BM - 1) / BM, lane);
  }
  __device__ __forceinline__ Mx4Groups(const Mx4Problem &p, int bm) : offsets(p.offsets), E(p.E), M(p.M), BM(bm) {
    load(0, bound(0), 0);
  }
  __device__ __forceinline__ int tiles() const { return __builtin_amdgcn_readlane(upto, 63); }   // up to e0 + 63
  __device__ __forceinline__ bool more() const { return e0 + 64 < E; }
  __device__ __forceinline__ void next() { load(e0 + 64, __builtin_amdgcn_readlane(hi, 63), tiles()); }
  // Row tile id, at or after the current 64 experts: expert e, rows
  // [row0, row1); false past the last.
  __device__ __forceinline__ bool find(int id, int &e, int &row0, int &row1) {
    while (id >= tiles()) {
      if (!more()) return false;
      next();
    }
    const int l = __builtin_ctzll(__ballot(id < upto));
    const int first = l == 0 ? before : __builtin_amdgcn_readlane(upto, l - 1);
    e = e0 + l;
    row0 = __builtin_amdgcn_readlane(lo, l) + (id - first) * BM;
    row1 = min(__builtin_amdgcn_readlane(hi, l), row0 + BM);
    return true;
  }
};

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
// Streaming kernel, for few rows: a workgroup owns 16 rows and NT tiles of 16
// columns, and its waves take 128-k blocks in turn, each lane the 16 bytes of
// one 32-value block.  Nothing is shared between waves until their sums meet
// in LDS, so no wave waits for another's loads.  Bound by HBM; row blocks of
// 32 and 64 were slower than the tiles (every wave reads its activations out
// of L2 by itself).  Measured: M = 1, N = 131072, K = 2048 (142.6 MB) 23.6 us,
// 6.0 TB/s; M = 13, N = 18944, K = 3584 (36 MB) 9.7 us; MX4 activations of 8
// rows there 7.6; 48 rows over 64 experts of 2816 x 2048 19.5 (each launch by
// itself; back to back 9.9, 9.1 and 20.0).
// ---------------------------------------------------------------------------
// 4 x 4 transpose over the four 16-lane rows of a wave: a[t] of lane row j and
// a[j] of lane row t trade places.
__device__ __forceinline__ void transpose_rows(u32x4 (&a)[4]) {
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const auto p = __builtin_amdgcn_permlane32_swap(a[0][d], a[2][d], false, false);
    const auto q = __builtin_amdgcn_permlane32_swap(a[1][d], a[3][d], false, false);
    const auto x = __builtin_amdgcn_permlane16_swap(p[0], q[0], false, false);
    const auto y = __builtin_amdgcn_permlane16_swap(p[1], q[1], false, false);
    a[0][d] = x[0];
    a[1][d] = x[1];
    a[2][d] = y[0];
    a[3][d] = y[1];
  }
}

template <int ACT, int NT>
struct Mx4StreamBlock {
  static constexpr int AF = ACT == kMX4 ? 1 : 4;   // fragments of 16 rows and 128 k
  u32x4 w[NT], a[AF];
  uint32_t sw[NT], sa;
};

template <int ACT, int OUT, int NT, bool GROUPED, int DEPTH>
__global__ __launch_bounds__(512) void k_mx4_stream(Mx4Problem p, int slab0) {
  extern __shared__ __attribute__((aligned(16))) float red[];   // [wave][NT][64][4]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, nwaves = blockDim.x >> 6;
  const int nl = lane & 15, j = lane >> 4;
  const int K = p.K, nb = K >> 7, nw = mx4_scale_windows(K), ntiles = p.N >> 4;
  const int nt0 = blockIdx.x * NT;
  int row0 = (slab0 + static_cast<int>(blockIdx.y)) * 16, row1 = min(p.M, row0 + 16), e = 0;
  if constexpr (GROUPED) {
    Mx4Groups groups(p, 16);
    if (!groups.find(slab0 + blockIdx.y, e, row0, row1)) return;
  }
  const uint8_t *B = p.B + static_cast<size_t>(e) * ntiles * nb * 1024;
  const uint32_t *BS = p.BS + static_cast<size_t>(e) * ntiles * nw * 64;
  // Rows, row tiles and column tiles past the end repeat the last; their sums
  // are not stored.
  using Block = Mx4StreamBlock<ACT, NT>;
  const uint8_t *wp[NT];
  const uint32_t *sp[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int nt = min(nt0 + i, ntiles - 1);
    wp[i] = B + static_cast<size_t>(nt) * nb * 1024 + lane * 16;
    sp[i] = BS + static_cast<size_t>(nt) * nw * 64 + lane;
  }
  const uint8_t *ap;
  [[maybe_unused]] const uint32_t *asp = nullptr;
  if constexpr (ACT == kMX4) {   // row0 is a multiple of 16 (not grouped)
    ap = static_cast<const uint8_t *>(p.A) + static_cast<size_t>(row0 >> 4) * nb * 1024 + lane * 16;
    asp = p.AS + static_cast<size_t>(row0 >> 4) * nw * 64 + lane;
  } else {
    const int row = min(row0 + nl, row1 - 1);
    ap = static_cast<const uint8_t *>(p.A) + (static_cast<size_t>(row) * K + 8 * j) * 2;
  }
  auto load = [&](int kb, Block &f) {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      f.w[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(wp[i] + static_cast<size_t>(kb) * 1024));
      f.sw[i] = sp[i][(kb >> 2) * 64];
    }
    if constexpr (ACT == kMX4) {
      f.a[0] = *reinterpret_cast<const u32x4 *>(ap + static_cast<size_t>(kb) * 1024);
      f.sa = asp[(kb >> 2) * 64];
    } else {
      // 64 contiguous bytes of each of 16 rows a load; the lanes trade them
      // into the blocks' order below.
#pragma unroll
      for (int t = 0; t < 4; ++t) f.a[t] = *reinterpret_cast<const u32x4 *>(ap + static_cast<size_t>(kb) * 256 + 64 * t);
    }
  };
  f32x4 acc[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto mma = [&](int kb, Block &f) {
    const int sh = 8 * (kb & 3);
    if constexpr (ACT != kMX4) transpose_rows(f.a);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      if constexpr (ACT == kMX4) {
        acc[i] = mx4_mfma<0>(f.w[i], f.a[0], acc[i], f.sw[i] >> sh, f.sa >> sh);
      } else {
        const float s = mx4_scale_operand(f.sw[i] >> sh, 0);
#pragma unroll
        for (int t = 0; t < 4; ++t)
          acc[i] = mfma16x16x32<ACT>(mx4_word_to_operand<ACT>(f.w[i][t], s), f.a[t], acc[i]);
      }
    }
  };
  // DEPTH blocks at a time, all of their loads on the way before the first is
  // waited for.  nwaves <= nb, so every wave has a block; past its last one a
  // wave loads that one again (a branch around the loads would make every
  // wait a full one) and skips the product.
  Block f[DEPTH];
  for (int kb = wave; kb < nb; kb += DEPTH * nwaves) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) load(kb + d * nwaves < nb ? kb + d * nwaves : kb, f[d]);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
      if (kb + d * nwaves < nb) mma(kb + d * nwaves, f[d]);
  }
  // The waves' sums meet in LDS and are added in wave order; a thread finishes
  // four consecutive columns, the quads of a tile on neighbouring threads.
#pragma unroll
  for (int i = 0; i < NT; ++i) *reinterpret_cast<f32x4 *>(red + ((wave * NT + i) * 64 + lane) * 4) = acc[i];
  __syncthreads();
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
// Tile kernels (mx4_tile.hpp).
// ---------------------------------------------------------------------------

// Which items a workgroup walks.  Workgroup b runs on XCD b % 8; each XCD
// takes a contiguous share of the item order, its workgroups neighbouring items at a
// time, so that the XCD's L2 serves the rows and channels they share.
struct Mx4Share {
  int first, step, end;
  __device__ __forceinline__ explicit Mx4Share(int total) {
    const int b = blockIdx.x, grid = gridDim.x, xcd = b & 7, loc = b >> 3;
    if (grid < 8) {
      first = b; step = grid; end = total;
    } else {
      const int per = grid >> 3, rem = grid & 7;   // workgroups of this XCD: per, or one more
      const int w0 = xcd * per + min(xcd, rem);
      step = per + (xcd < rem ? 1 : 0);
      first = static_cast<int>(static_cast<int64_t>(total) * w0 / grid) + loc;
      end = static_cast<int>(static_cast<int64_t>(total) * (w0 + step) / grid);
    }
  }
};

// Dense: bands of four row tiles walked column by column, so one weight tile
// serves the band's row tiles while it is in L2.
template <class Eng>
struct Mx4DenseWork {
  const Mx4Problem &p;
  const int tiles_m, tiles_n;
  const Mx4Share share;
  __device__ __forceinline__ explicit Mx4DenseWork(const Mx4Problem &pr)
      : p(pr), tiles_m((pr.M + Eng::BM - 1) / Eng::BM), tiles_n((pr.N + Eng::BN - 1) / Eng::BN),
        share(tiles_m * tiles_n * pr.slices) {}
  __device__ __forceinline__ bool get(int n, Mx4Item &t) const {
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
    t.col_lo = tn * Eng::BN;
    t.e = 0;
    const int steps = p.K / Eng::K_STEP, seg = p.kseg * Eng::W;
    t.s0 = p.slices > 1 ? t.slice * seg : 0;
    t.s1 = p.slices > 1 ? min(steps, t.s0 + seg) : steps;
    return true;
  }
};

// Grouped: the column tiles of an expert's row tile next to each other.  Items
// come in increasing order, so the wave moves on to the next 64 experts at
// most E / 64 times.
template <class Eng>
struct Mx4GroupWork {
  const int tiles_n, steps;
  Mx4Groups groups;
  const Mx4Share share;
  static __device__ __forceinline__ int total(const Mx4Problem &p) {
    Mx4Groups g(p, Eng::BM);
    while (g.more()) g.next();
    return g.tiles();
  }
  __device__ __forceinline__ explicit Mx4GroupWork(const Mx4Problem &p)
      : tiles_n((p.N + Eng::BN - 1) / Eng::BN), steps(p.K / Eng::K_STEP), groups(p, Eng::BM),
        share(total(p) * tiles_n) {}
  __device__ __forceinline__ bool get(int n, Mx4Item &t) {
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

// bf16 activations, 2048 x 13312 x 2048: 91 to 97 us (1.15 to 1.23 PFLOP/s) on
// 256 x 256 tiles, 12288 rows over 64 experts of 2816 x 2048 153 to 158 us (0.90
// to 0.93) on 128 x 256; MX4 activations, 4096 x 18944 x 3584: 144 to 150 us
// (3.7 to 3.9).
template <class Eng, class Out, class Work>
__global__ __launch_bounds__(Eng::NTHR, Eng::WAVES) void k_mx4_tiles(Mx4Problem p) {
  __shared__ __attribute__((aligned(16))) char s0[Eng::STAGE];
  __shared__ __attribute__((aligned(16))) char s1[Eng::STAGE];
  __shared__ __attribute__((aligned(16))) char s2[Eng::NS > 2 ? Eng::STAGE : 16];
  __shared__ __attribute__((aligned(16))) char s3[Eng::NS > 2 ? Eng::STAGE : 16];
  __shared__ __attribute__((aligned(16))) char ep[Out::kBytes == 2 ? Eng::EP : 16];
  __shared__ __attribute__((aligned(16))) float bias[Eng::NW * Eng::WTN];
  Work work(p);
  mx4_tiles<Eng, Out>(p, work, Mx4Lds{{s0, s1, s2, s3}, ep, bias});
}

// 100 x 3584 x 3584: 8.8 us back to back (9.5 by itself), against 16.5 on
// 64 x 128 tiles in two K slices.
template <class Eng, int KW, class Out>
__global__ __launch_bounds__(Eng::NTHR * KW) void k_mx4_one_tile(Mx4Problem p) {
  __shared__ __attribute__((aligned(16))) float bias[Eng::NW * Eng::WTN];
  __shared__ __attribute__((aligned(16))) char s0[KW * Eng::STAGE];
  __shared__ __attribute__((aligned(16))) char s1[KW * Eng::STAGE];
  __shared__ __attribute__((aligned(16))) char s2[Eng::NS > 2 ? KW * Eng::STAGE : 16];
  __shared__ __attribute__((aligned(16))) char s3[Eng::NS > 3 ? KW * Eng::STAGE : 16];
  const Mx4DenseWork<Eng> work(p);
  Mx4Item t;
  if (work.get(0, t)) mx4_one_tile<Eng, KW, Out>(p, t, Mx4Lds{{s0, s1, s2, s3}, nullptr, bias});
}

// K slices: C = RNE_out(the slices' partials summed in slice order + bias).
// Bound by the partials' traffic out of MALL: three slices of 333 x 3584
// (14.3 MB) 4.8 to 5.2 us.
template <int OUT>
__global__ __launch_bounds__(256) void k_mx4_reduce(Mx4Problem p) {
  const size_t mn = static_cast<size_t>(p.M) * p.N, step = static_cast<size_t>(gridDim.x) * 1024;
  for (size_t i = (static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x) * 4; i < mn; i += step) {
    f32x4 s = *reinterpret_cast<const f32x4 *>(p.part + i);
    for (int sl = 1; sl < p.slices; ++sl) s += *reinterpret_cast<const f32x4 *>(p.part + sl * mn + i);
    const int r = static_cast<int>(i / p.N), col = static_cast<int>(i - static_cast<size_t>(r) * p.N);
    float v[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) v[x] = p.bias ? s[x] + bits_to_f32_dyn(p.bias[col + x], p.bias_dt) : s[x];
    store4<OUT>(p.C, i, v);
  }
}

namespace {

constexpr int kMaxSlabs = 65535;   // grid.y

template <int ACT, int OUT, int NT, bool GROUPED, int DEPTH>
hipError_t run_stream_as(const Mx4Problem &p, long slabs, hipStream_t s) {
  const int nb = p.K >> 7, waves = nb < 8 ? nb : 8;
  const size_t lds = static_cast<size_t>(waves) * NT * 256 * sizeof(float);
  const unsigned cols = static_cast<unsigned>(((p.N >> 4) + NT - 1) / NT);
  if (static_cast<uint64_t>(cols) * 64 * waves > UINT32_MAX) return hipErrorNotSupported;
  for (long s0 = 0; s0 < slabs; s0 += kMaxSlabs) {
    const unsigned ny = static_cast<unsigned>(std::min<long>(slabs - s0, kMaxSlabs));
    hipLaunchKernelGGL((k_mx4_stream<ACT, OUT, NT, GROUPED, DEPTH>), dim3(cols, ny), dim3(64 * waves), lds, s, p,
                       static_cast<int>(s0));
  }
  return hipGetLastError();
}
// Column tiles a workgroup (NT): as many as let every CU have one workgroup,
// up to six, then half as many (two rounds of workgroups) up to five, then
// four: a round that a few workgroups overhang costs nearly as much as a full
// one.  Measured with NT from 1 on, K = 3584 unless stated:
//   tiles / CUs 1.0  (N = 4096, K = 4096, M = 4)   5.1  5.9  6.7  7.2
//               1.25 (N = 5120, K = 5120, M = 8)  10.2  7.2  8.3  8.8
//               2.5  (N = 10240, K = 2048, M = 1)  5.8  5.8  5.2  5.3  5.7
//               3.25 (N = 13312, K = 2048, M = 12) 9.3  7.1  7.9  6.2  6.7  7.2
//               4.6  (N = 18944, M = 13)          17.7 13.2 12.1 12.9  9.8 10.6
//               6.0  (N = 24576, K = 2048, M = 16) 14.9 10.9  9.1 9.5 10.6  8.5
//               7.0  (N = 28672, K = 4096, M = 1) 18.5 14.0 13.8 12.9 14.8 16.5
//               32   (N = 131072, K = 2048, M = 1) 35 26.4 24.8 23.9 24.4 24.7
// MX4 activations alike (4.6, M = 8: 9.9 9.3 8.9 10.3 8.5 8.7).  One column
// tile keeps two blocks' loads in flight (N = 3584 5.0 -> 4.6 us); with more it
// gains nothing.  A grouped product's workgroups are bounds, most without rows:
// one, two or four (48 rows over 64 experts of 2816 x 2048 29, 20 and 18 us).
template <int ACT, int OUT, bool GROUPED>
hipError_t run_stream(const Mx4Problem &p, hipStream_t s) {
  // Row slabs: a grouped product has at most one partial slab per expert
  // with rows.
  const long slabs = GROUPED ? p.M / 16 + std::min(p.E, p.M) : (p.M + 15) / 16;
  const long cus = device_cus(), rounds = ((p.N >> 4) * slabs + cus - 1) / cus;
  if constexpr (GROUPED) {
    if (rounds <= 2) return run_stream_as<ACT, OUT, 1, true, 2>(p, slabs, s);
    if (rounds <= 4) return run_stream_as<ACT, OUT, 2, true, 1>(p, slabs, s);
    return run_stream_as<ACT, OUT, 4, true, 1>(p, slabs, s);
  } else {
    switch (rounds <= 6 ? rounds : rounds <= 10 ? (rounds + 1) / 2 : 4) {
      case 1: return run_stream_as<ACT, OUT, 1, false, 2>(p, slabs, s);
      case 2: return run_stream_as<ACT, OUT, 2, false, 1>(p, slabs, s);
      case 3: return run_stream_as<ACT, OUT, 3, false, 1>(p, slabs, s);
      case 4: return run_stream_as<ACT, OUT, 4, false, 1>(p, slabs, s);
      case 5: return run_stream_as<ACT, OUT, 5, false, 1>(p, slabs, s);
      default: return run_stream_as<ACT, OUT, 6, false, 1>(p, slabs, s);
    }
  }
}

}  // namespace

namespace {

// The tiles.  T256 .. T64 walk their tiles in a fixed set of workgroups; T32
// runs one tile a workgroup, k dealt out to KW groups of waves.
template <int TILE, int ACT> struct Mx4Tiling;
template <int ACT> struct Mx4Tiling<kMx4T256, ACT> { using Eng = Mx4Engine16<ACT, 256, 256, 2, 4, 2, false>; };
template <int ACT> struct Mx4Tiling<kMx4T256N, ACT> { using Eng = Mx4Engine16<ACT, 128, 256, 2, 4, 4, true>; };
template <int ACT> struct Mx4Tiling<kMx4T128, ACT> { using Eng = Mx4Engine16<ACT, 128, 128, 2, 2, 2, false>; };
template <int ACT> struct Mx4Tiling<kMx4T64, ACT> { using Eng = Mx4Engine16<ACT, 64, 128, 2, 2, 4, true>; };
template <int ACT> struct Mx4Tiling<kMx4T32, ACT> { using Eng = Mx4Engine16<ACT, 32, 64, 1, 2, 3, false>; };
template <> struct Mx4Tiling<kMx4T256, kMX4> { using Eng = Mx4Engine4<256, 256, 2, 4, 4>; };
template <> struct Mx4Tiling<kMx4T256N, kMX4> { using Eng = Mx4Engine4<128, 256, 2, 4, 4>; };
template <> struct Mx4Tiling<kMx4T128, kMX4> { using Eng = Mx4Engine4<128, 128, 2, 2, 4>; };
template <> struct Mx4Tiling<kMx4T64, kMX4> { using Eng = Mx4Engine4<64, 128, 2, 2, 4>; };
template <> struct Mx4Tiling<kMx4T32, kMX4> { using Eng = Mx4Engine4<32, 64, 1, 2, 3>; };
constexpr int kT32Groups = 4;

// What a tile costs, in microseconds: a launch (t0), and per 64 k `full` while
// a CU runs as many workgroups as it does at a time (most), lone + shared * q
// with a mean of q < most (lone: a workgroup's chain of steps; shared: what
// the workgroups take from each other).  Fitted to 2868 timings on MI355X, 17
// to 4096 rows and eight weight shapes of 512 x 2048 to 18944 x 3584, each
// tile and slice count forced (residual 6 to 8 %); the tile it picks is within
// 4 % of the best one on average, 37 % at worst (2048 x 512, k = 2048).
// 32 x 64 tiles, one a workgroup, pay a start (again) for every further round
// (32 x 131072 x 2048: 48 us against 35.6 on 64 x 128 tiles).
struct Mx4Cost {
  int bm, bn, most;
  float t0, lone, shared, full, again;
};
constexpr Mx4Cost kCost16[] = {{256, 256, 1, 10.9f, 0.988f, 0.303f, 1.534f, 0.f},
                               {128, 256, 1, 7.3f, 0.550f, 0.173f, 0.819f, 0.f},
                               {128, 128, 2, 4.8f, 0.394f, 0.221f, 0.880f, 0.f},
                               {64, 128, 2, 5.5f, 0.228f, 0.120f, 0.505f, 0.f},
                               {32, 64, 2, 5.5f, 0.045f, 0.069f, 0.200f, 3.5f}};
constexpr Mx4Cost kCost4[] = {{256, 256, 1, 10.2f, 0.336f, 0.077f, 0.504f, 0.f},
                              {128, 256, 1, 6.8f, 0.218f, 0.077f, 0.302f, 0.f},
                              {128, 128, 2, 6.0f, 0.140f, 0.073f, 0.319f, 0.f},
                              {64, 128, 2, 5.1f, 0.105f, 0.048f, 0.207f, 0.f},
                              {32, 64, 2, 5.6f, 0.029f, 0.037f, 0.123f, 3.5f}};
// K slices: the reduction's launch, and a byte of partials (in the same fit).
constexpr float kSliceLaunch = 2.3f, kSliceByte = 2.8e-7f;

// 32-bit offsets of the tile kernels stay below this, and with MX4 activations
// a launch takes at most so many rows (K from 2^22 on streams: no limit).
constexpr uint64_t kMx4Span = uint64_t(1) << 31;
int mx4_rows_most(int K, bool a4) {
  if (!a4 || K >= 1 << 22) return INT32_MAX;
  return static_cast<int>(std::min<uint64_t>((kMx4Span - 1) / (static_cast<uint64_t>(K) / 2), INT32_MAX)) / 256 * 256;
}

struct Mx4Plan {
  int tile;            // Mx4Kernel
  int kseg, slices;    // K slices in 512-k windows
  size_t bytes;        // partials
};

// Time of `tiles` tiles of `steps` 64-k steps each: full rounds of the
// workgroups the CUs hold, and what is left.
float tiles_time(const Mx4Cost &c, float tiles, float steps) {
  const float q = tiles / static_cast<float>(device_cus()), most = static_cast<float>(c.most);
  const float rounds = static_cast<float>(static_cast<int>(q / most)), rest = q - rounds * most;
  return c.t0 + steps * (rounds * c.full + (rest > 0.f ? c.lone + c.shared * rest : 0.f)) +
         c.again * std::max(0.f, rest > 0.f ? rounds : rounds - 1.f);
}

// The tile, and for few tiles the K slices, with the least time by the
// measured costs; a slice's partials cost another launch and their traffic.
// Up to 16 rows the streaming kernel, which reads each weight once with no
// row padding beyond 16 (bf16, back to back, m = 13, n = 18944, k = 3584: 10.2
// us against 15.2 on 32 x 64 tiles), and up to 32 while its two row slabs still find a CU for
// every five column tiles (m = 32, n = k = 4096: 7.3 against 9.1, MX4
// activations 5.1 against 7.3; n = 11264 13.5 against 11.4), with 16-bit
// activations up to k = 8192 (n = 4096: 11.5 against 11.9 with K slices;
// k = 18944, n = 3584: 23.0 against 18.4; MX4 activations 14.7 against 15.1).
// A grouped product's row tiles
// are not known to the host: it reckons with half a tile too many for every
// expert (on 27 sizes of 12 to 256 rows an expert, 8 to 128 experts, the tile
// so picked is within 1 % of the best on average, 16 % at worst) and takes no
// 32-row tiles (2048 rows over 64 experts, n = 2816, k = 2048: 85.6 us, 64-row
// ones 64.6 then and 56 to 61 now).  It streams up to a mean of 7 rows an expert (64
// experts, n = 2048, k = 1408: 6 rows each 23.7 us against 26.3 on 64-row
// tiles, 8 rows 26.8 against 25.9, 12 rows 31.9 against 27.6), or of 12 up to
// 96 rows in all (8 experts, n = 3584, k = 2560: 8 rows each 12.6 against
// 16.5, 12 rows 17.4 against 17.9).
Mx4Plan plan_mx4(int M, int N, int K, bool a4, bool grouped, int E) {
  Mx4Plan pl{kMx4Stream, 0, 1, 0};
  const Override ov = dispatch_override();
  // The tile kernels' buffer loads and stores have 32-bit offsets.  They span a
  // tile's rows of C (or of fp32 partials), an expert's scales, and with
  // 16-bit activations the tile's rows of A and its channels' codes; with MX4
  // ones all codes of B (and of A: launch_mx4_gemm takes its rows in parts).  So
  // MX4 activations stream against 2^32 and more weights whatever their rows,
  // every 16 rows reading all of them.
  const uint64_t lim = kMx4Span, windows64 = mx4_scale_windows(K) * uint64_t(256);
  if (uint64_t(256) * 4 * N >= lim || (N / 16) * windows64 >= lim || uint64_t(256) * K * 2 >= lim ||
      (a4 && uint64_t(N) * K / 2 >= lim))
    return pl;
  const Mx4Cost *cost = a4 ? kCost4 : kCost16;
  const int windows = mx4_scale_windows(K);
  // A forced 32 x 64 tile fits a dense product whose tiles (and slices of them)
  // one launch covers, a workgroup of 128 * kT32Groups threads each.
  const int64_t t32 = static_cast<int64_t>((M + 31) / 32) * ((N + 63) / 64) * std::max(1, std::min(ov.mx4_split, windows));
  const bool t32_fits = !grouped && t32 * 128 * kT32Groups <= UINT32_MAX;
  if (ov.mx4_tile >= 0 && (ov.mx4_tile != kMx4T32 || t32_fits)) {
    pl.tile = ov.mx4_tile;
  } else if (M > (grouped ? std::max<int64_t>(7 * int64_t(E), std::min<int64_t>(12 * int64_t(E), 96))
                          : N / 16 * 2 <= 5 * device_cus() && (a4 || K <= 8192) ? 32 : 16)) {
    float best = 0.f;
    for (int i = 0; i < (grouped ? 4 : 5); ++i) {
      const int64_t cols = (N + cost[i].bn - 1) / cost[i].bn;
      const float tiles = static_cast<float>(cols) *
                          (grouped ? static_cast<float>(M) / cost[i].bm + 0.5f * E
                                   : static_cast<float>((M + cost[i].bm - 1) / cost[i].bm));
      for (int s = 1; s <= 4 && (s == 1 || (!grouped && s <= windows / 2)); ++s) {
        const int kseg = (windows + s - 1) / s;
        if ((windows + kseg - 1) / kseg != s) continue;
        float t = tiles_time(cost[i], tiles * s, s == 1 ? K / 64.f : kseg * 8.f);
        if (s > 1) t += kSliceLaunch + static_cast<float>(s + 1) * M * N * 4.f * kSliceByte;
        if (best == 0.f || t < best) {
          best = t;
          pl.tile = kMx4T256 + i;
          pl.slices = s;
          pl.kseg = kseg;
        }
      }
    }
  }
  if (pl.tile == kMx4Stream || grouped) {
    pl.slices = 1;
    return pl;
  }
  if (ov.mx4_split > 0) {
    const int want = std::min(ov.mx4_split, windows);
    pl.kseg = (windows + want - 1) / want;
    pl.slices = (windows + pl.kseg - 1) / pl.kseg;
  }
  if (pl.slices > 1) pl.bytes = static_cast<size_t>(pl.slices) * M * N * sizeof(float);
  return pl;
}

template <int OUT>
hipError_t reduce_mx4(const Mx4Problem &p, hipStream_t s) {
  const size_t blocks = (static_cast<size_t>(p.M) * p.N / 4 + 255) / 256;
  hipLaunchKernelGGL(k_mx4_reduce<OUT>, dim3(static_cast<unsigned>(std::min<size_t>(blocks, 65536))), dim3(256), 0,
                     s, p);
  return hipGetLastError();
}

// Workgroups of `Eng` a CU holds: by LDS, and by registers.
template <class Eng>
constexpr int groups_per_cu() {
  const int lds = 160 * 1024 / (Eng::NS * Eng::STAGE + Eng::EP), waves = 4 * Eng::WAVES / Eng::NW;
  return std::max(1, std::min(lds, waves));
}

template <class Eng, int OUT, bool GROUPED>
hipError_t run_tiles(const Mx4Problem &p, hipStream_t s) {
  const int64_t tn = (p.N + Eng::BN - 1) / Eng::BN;
  // A grouped product has at most one partial row tile per expert with rows.
  const int64_t tm = GROUPED ? p.M / Eng::BM + std::min(p.E, p.M) : (p.M + Eng::BM - 1) / Eng::BM;
  const int64_t items = tm * tn * p.slices;
  if (items > INT32_MAX / 2) return hipErrorNotSupported;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(items, device_cus() * groups_per_cu<Eng>()));
  if constexpr (GROUPED) {
    hipLaunchKernelGGL((k_mx4_tiles<Eng, Mx4Out<OUT, false>, Mx4GroupWork<Eng>>), dim3(grid), dim3(Eng::NTHR), 0, s, p);
  } else if (p.slices > 1) {
    hipLaunchKernelGGL((k_mx4_tiles<Eng, Mx4Out<OUT, true>, Mx4DenseWork<Eng>>), dim3(grid), dim3(Eng::NTHR), 0, s, p);
    return reduce_mx4<OUT>(p, s);
  } else {
    hipLaunchKernelGGL((k_mx4_tiles<Eng, Mx4Out<OUT, false>, Mx4DenseWork<Eng>>), dim3(grid), dim3(Eng::NTHR), 0, s, p);
  }
  return hipGetLastError();
}

template <class Eng, int KW, int OUT>
hipError_t run_one_tile(const Mx4Problem &p, hipStream_t s) {
  const int64_t tn = (p.N + Eng::BN - 1) / Eng::BN, tm = (p.M + Eng::BM - 1) / Eng::BM;
  const int64_t items = tm * tn * p.slices;
  if (items * Eng::NTHR * KW > UINT32_MAX) return hipErrorNotSupported;
  const dim3 grid(static_cast<unsigned>(items)), block(Eng::NTHR * KW);
  if (p.slices > 1) {
    hipLaunchKernelGGL((k_mx4_one_tile<Eng, KW, Mx4Out<OUT, true>>), grid, block, 0, s, p);
    return reduce_mx4<OUT>(p, s);
  }
  hipLaunchKernelGGL((k_mx4_one_tile<Eng, KW, Mx4Out<OUT, false>>), grid, block, 0, s, p);
  return hipGetLastError();
}

template <int ACT, bool GROUPED>
hipError_t run_a16(const Mx4Problem &p, int tile, hipStream_t s) {
  switch (tile) {
    case kMx4T256: return run_tiles<typename Mx4Tiling<kMx4T256, ACT>::Eng, ACT, GROUPED>(p, s);
    case kMx4T256N: return run_tiles<typename Mx4Tiling<kMx4T256N, ACT>::Eng, ACT, GROUPED>(p, s);
    case kMx4T128: return run_tiles<typename Mx4Tiling<kMx4T128, ACT>::Eng, ACT, GROUPED>(p, s);
    case kMx4T64: return run_tiles<typename Mx4Tiling<kMx4T64, ACT>::Eng, ACT, GROUPED>(p, s);
    case kMx4T32:
      if constexpr (!GROUPED) return run_one_tile<typename Mx4Tiling<kMx4T32, ACT>::Eng, kT32Groups, ACT>(p, s);
    default: return run_stream<ACT, ACT, GROUPED>(p, s);
  }
}

template <int OUT>
hipError_t run_a4(const Mx4Problem &p, int tile, hipStream_t s) {
  switch (tile) {
    case kMx4T256: return run_tiles<Mx4Tiling<kMx4T256, kMX4>::Eng, OUT, false>(p, s);
    case kMx4T256N: return run_tiles<Mx4Tiling<kMx4T256N, kMX4>::Eng, OUT, false>(p, s);
    case kMx4T128: return run_tiles<Mx4Tiling<kMx4T128, kMX4>::Eng, OUT, false>(p, s);
    case kMx4T64: return run_tiles<Mx4Tiling<kMx4T64, kMX4>::Eng, OUT, false>(p, s);
    case kMx4T32: return run_one_tile<Mx4Tiling<kMx4T32, kMX4>::Eng, kT32Groups, OUT>(p, s);
    default: return run_stream<kMX4, OUT, false>(p, s);
  }
}

hipError_t run_mx4(const Mx4Problem &p, const Mx4Args &a, int tile, hipStream_t s) {
  if (a.act == kMX4) {
    switch (a.out) {
      case QG_FP32: return run_a4<QG_FP32>(p, tile, s);
      case QG_FP16: return run_a4<QG_FP16>(p, tile, s);
      default: return run_a4<QG_BF16>(p, tile, s);
    }
  }
  if (a.offsets) return a.act == kFP16 ? run_a16<kFP16, true>(p, tile, s) : run_a16<kBF16, true>(p, tile, s);
  return a.act == kFP16 ? run_a16<kFP16, false>(p, tile, s) : run_a16<kBF16, false>(p, tile, s);
}

}  // namespace

size_t mx4_workspace_bytes(int m, int n, int k, int act_bits) {
  const bool a4 = act_bits == 4;
  return plan_mx4(std::min(m, mx4_rows_most(k, a4)), n, k, a4, false, 0).bytes;
}

hipError_t launch_mx4_gemm(const Mx4Args &a, hipStream_t s) {
  const bool a4 = a.act == kMX4;
  const int most = mx4_rows_most(a.K, a4);
  for (int64_t m0 = 0; m0 < a.M; m0 += most) {
    const int M = static_cast<int>(std::min<int64_t>(a.M - m0, most));
    const Mx4Plan pl = plan_mx4(M, a.N, a.K, a4, a.offsets != nullptr, a.E);
    Mx4Problem p{a.A, reinterpret_cast<const uint32_t *>(a.AS), a.B, reinterpret_cast<const uint32_t *>(a.BS),
                 a.bias, a.C, M, a.N, a.K, a.bias_dt, a.offsets, a.E, nullptr, 0, 1};
    if (m0) {   // MX4 activations, a multiple of 256 rows in
      p.A = static_cast<const uint8_t *>(a.A) + static_cast<size_t>(m0) * a.K / 2;
      p.AS += static_cast<size_t>(m0 / 16) * mx4_scale_windows(a.K) * 64;
      p.C = static_cast<char *>(a.C) + static_cast<size_t>(m0) * a.N * (a.out == QG_FP32 ? 4 : 2);
    }
    if (pl.slices > 1 && a.ws && a.ws_bytes >= pl.bytes) {
      p.part = static_cast<float *>(a.ws);
      p.kseg = pl.kseg;
      p.slices = pl.slices;
    }
    const hipError_t e = run_mx4(p, a, pl.tile, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace qg

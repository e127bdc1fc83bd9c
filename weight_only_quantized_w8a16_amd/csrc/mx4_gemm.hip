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
#include "mx4_tile.hpp"

namespace qg {

namespace {

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
      for (int i = 0; i < NT; ++i) acc[i] = mx4_mfma<0>(w[i], a, acc[i], sw[i], sa);
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

// Grouped: the column tiles of an expert's row tile next to each other.  The
// wave holds the row tiles of 64 experts at a time (a lane each); items come
// in increasing order, so it moves on to the next 64 at most E / 64 times.
template <class Eng>
struct Mx4GroupWork {
  const Mx4Problem &p;
  const int tiles_n;
  int e0, before, lo, hi, upto;   // before, upto: row tiles up to round e0 / the lane's expert
  __device__ __forceinline__ int bound(int x) const { return min(max(p.offsets[x], 0), p.M); }
  __device__ __forceinline__ void load(int start) {
    const int x = start + (threadIdx.x & 63);
    lo = hi = 0;
    if (x < p.E) {
      lo = bound(x);
      hi = max(bound(x + 1), lo);
    }
    e0 = start;
    upto = before + wave_scan((hi - lo + Eng::BM - 1) / Eng::BM, threadIdx.x & 63);
  }
  static __device__ __forceinline__ int total_tiles(const Mx4Problem &p) {
    int cnt = 0;
    for (int x = threadIdx.x & 63; x < p.E; x += 64) {
      const int a = min(max(p.offsets[x], 0), p.M), b = max(min(max(p.offsets[x + 1], 0), p.M), a);
      cnt += (b - a + Eng::BM - 1) / Eng::BM;
    }
    return __builtin_amdgcn_readlane(wave_scan(cnt, threadIdx.x & 63), 63);
  }
  const Mx4Share share;
  __device__ __forceinline__ explicit Mx4GroupWork(const Mx4Problem &pr)
      : p(pr), tiles_n((pr.N + Eng::BN - 1) / Eng::BN), before(0), share(total_tiles(pr) * tiles_n) {
    load(0);
  }
  __device__ __forceinline__ bool get(int n, Mx4Item &t) {
    const int id = share.first + n * share.step;
    if (id >= share.end) return false;
    const int tm = id / tiles_n;
    int all = __builtin_amdgcn_readlane(upto, 63);
    while (tm >= all) {
      if (e0 + 64 >= p.E) return false;   // never: share counts the same tiles
      before = all;
      load(e0 + 64);
      all = __builtin_amdgcn_readlane(upto, 63);
    }
    const int l = __builtin_ctzll(__ballot(tm < upto));
    const int first = l == 0 ? before : __builtin_amdgcn_readlane(upto, l - 1);
    t.e = e0 + l;
    t.row_lo = __builtin_amdgcn_readlane(lo, l) + (tm - first) * Eng::BM;
    t.row_last = min(__builtin_amdgcn_readlane(hi, l), t.row_lo + Eng::BM) - 1;
    t.col_lo = (id - tm * tiles_n) * Eng::BN;
    t.slice = t.s0 = 0;
    t.s1 = p.K / Eng::K_STEP;
    return true;
  }
};

template <class Eng, class Out, class Work>
__global__ __launch_bounds__(Eng::NTHR, Eng::WAVES) void k_mx4_tiles(Mx4Problem p) {
  __shared__ __attribute__((aligned(16))) char s0[Eng::STAGE];
  __shared__ __attribute__((aligned(16))) char s1[Eng::STAGE];
  __shared__ __attribute__((aligned(16))) char s2[Eng::NS > 2 ? Eng::STAGE : 16];
  __shared__ __attribute__((aligned(16))) char s3[Eng::NS > 2 ? Eng::STAGE : 16];
  __shared__ __attribute__((aligned(16))) char s4[Eng::NS > 4 ? Eng::STAGE : 16];
  __shared__ __attribute__((aligned(16))) char s5[Eng::NS > 4 ? Eng::STAGE : 16];
  __shared__ __attribute__((aligned(16))) char s6[Eng::NS > 4 ? Eng::STAGE : 16];
  __shared__ __attribute__((aligned(16))) char s7[Eng::NS > 4 ? Eng::STAGE : 16];
  Work work(p);
  mx4_tiles<Eng, Out>(p, work, Mx4Lds{{s0, s1, s2, s3, s4, s5, s6, s7}});
}

// K slices: C = RNE_out(the slices' partials summed in slice order + bias).
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

template <int T, int ACT> struct Tile16;
template <int T> struct Tile4;
template <int ACT> struct Tile16<1, ACT> { using Eng = Mx4Engine16<ACT, 256, 256, 2, 4, 4>; };
template <int ACT> struct Tile16<2, ACT> { using Eng = Mx4Engine16<ACT, 128, 256, 2, 2, 2>; };
template <int ACT> struct Tile16<3, ACT> { using Eng = Mx4Engine16<ACT, 128, 256, 2, 4, 4>; };
template <int ACT> struct Tile16<4, ACT> { using Eng = Mx4Engine16<ACT, 128, 128, 2, 4, 4>; };
template <int ACT> struct Tile16<5, ACT> { using Eng = Mx4Engine16<ACT, 128, 128, 2, 2, 4>; };
template <int ACT> struct Tile16<6, ACT> { using Eng = Mx4Engine16<ACT, 64, 128, 2, 2, 8>; };
template <int ACT> struct Tile16<7, ACT> { using Eng = Mx4Engine16<ACT, 64, 128, 2, 2, 4>; };
template <int ACT> struct Tile16<8, ACT> { using Eng = Mx4Engine16<ACT, 64, 64, 2, 2, 8>; };
template <> struct Tile4<1> { using Eng = Mx4Engine4<256, 256, 2, 4, 4>; };
template <> struct Tile4<2> { using Eng = Mx4Engine4<128, 256, 2, 2, 2>; };
template <> struct Tile4<3> { using Eng = Mx4Engine4<128, 256, 2, 4, 4>; };
template <> struct Tile4<4> { using Eng = Mx4Engine4<128, 128, 2, 4, 4>; };
template <> struct Tile4<5> { using Eng = Mx4Engine4<128, 128, 2, 2, 4>; };
template <> struct Tile4<6> { using Eng = Mx4Engine4<64, 128, 2, 4, 4>; };
template <> struct Tile4<7> { using Eng = Mx4Engine4<64, 128, 2, 2, 4>; };
template <> struct Tile4<8> { using Eng = Mx4Engine4<64, 64, 2, 2, 4>; };

struct Mx4Plan {
  int tile;            // Mx4Tile order below, or kStream
  int kseg, slices;    // K slices in 512-k windows
  size_t bytes;        // partials
};

Mx4Plan plan_mx4(int M, int N, int K, bool a4, bool grouped, int E) {
  Mx4Plan pl{kMx4Stream, 0, 1, 0};
  const Override ov = dispatch_override();
  // 32-bit offsets of the tile kernels' buffer loads.
  const uint64_t lim = uint64_t(1) << 31;
  const uint64_t a_bytes = uint64_t((M + 15) / 16 * 16) * K / (a4 ? 2 : 1) * (a4 ? 1 : 2);
  // A tile's rows of C (or of fp32 partials) in one buffer resource.
  const bool fits = a_bytes < lim && uint64_t(N) * K / 2 < lim && uint64_t(N) * 4 * 256 < lim;
  if (!fits || ov.mx4_tile == kMx4Stream) return pl;
  if (ov.mx4_tile >= 0) pl.tile = ov.mx4_tile;
  else if (M > 64) pl.tile = 4;
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

// Workgroups of `Eng` a CU holds: by LDS, and by registers.
template <class Eng>
constexpr int groups_per_cu() {
  const int lds = 160 * 1024 / (Eng::NS * Eng::STAGE), waves = 4 * Eng::WAVES / Eng::NW;
  return std::max(1, std::min(lds, waves));
}

template <class Eng, int OUT, bool GROUPED>
hipError_t run_tiles(const Mx4Problem &p, hipStream_t s) {
  const int64_t tn = (p.N + Eng::BN - 1) / Eng::BN;
  // A grouped product has at most one partial row tile per expert with rows.
  const int64_t tm = GROUPED ? p.M / Eng::BM + std::min(p.E, p.M) : (p.M + Eng::BM - 1) / Eng::BM;
  const int64_t items = tm * tn * p.slices;
  if (items > INT32_MAX / 2) return hipErrorInvalidValue;
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

template <int ACT, bool GROUPED>
hipError_t run_a16(const Mx4Problem &p, int tile, hipStream_t s) {
  switch (tile) {
    case 1: return run_tiles<typename Tile16<1, ACT>::Eng, ACT, GROUPED>(p, s);
    case 2: return run_tiles<typename Tile16<2, ACT>::Eng, ACT, GROUPED>(p, s);
    case 3: return run_tiles<typename Tile16<3, ACT>::Eng, ACT, GROUPED>(p, s);
    case 4: return run_tiles<typename Tile16<4, ACT>::Eng, ACT, GROUPED>(p, s);
    case 5: return run_tiles<typename Tile16<5, ACT>::Eng, ACT, GROUPED>(p, s);
    case 6: return run_tiles<typename Tile16<6, ACT>::Eng, ACT, GROUPED>(p, s);
    case 7: return run_tiles<typename Tile16<7, ACT>::Eng, ACT, GROUPED>(p, s);
    case 8: return run_tiles<typename Tile16<8, ACT>::Eng, ACT, GROUPED>(p, s);
    default: return run_stream<ACT, ACT, GROUPED>(p, s);
  }
}

template <int OUT>
hipError_t run_a4(const Mx4Problem &p, int tile, hipStream_t s) {
  switch (tile) {
    case 1: return run_tiles<Tile4<1>::Eng, OUT, false>(p, s);
    case 2: return run_tiles<Tile4<2>::Eng, OUT, false>(p, s);
    case 3: return run_tiles<Tile4<3>::Eng, OUT, false>(p, s);
    case 4: return run_tiles<Tile4<4>::Eng, OUT, false>(p, s);
    case 5: return run_tiles<Tile4<5>::Eng, OUT, false>(p, s);
    case 6: return run_tiles<Tile4<6>::Eng, OUT, false>(p, s);
    case 7: return run_tiles<Tile4<7>::Eng, OUT, false>(p, s);
    case 8: return run_tiles<Tile4<8>::Eng, OUT, false>(p, s);
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

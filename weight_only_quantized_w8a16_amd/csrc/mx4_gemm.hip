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

size_t mx4_workspace_bytes(int, int, int, int) { return 0; }

hipError_t launch_mx4_gemm(const Mx4Args &a, hipStream_t s) {
  const Mx4Problem p{a.A, reinterpret_cast<const uint32_t *>(a.AS), a.B,
                     reinterpret_cast<const uint32_t *>(a.BS), a.bias, a.C, a.M, a.N, a.K, a.bias_dt,
                     a.offsets, a.E};
  if (a.act == kMX4) {
    switch (a.out) {
      case QG_FP32: return run_stream<kMX4, QG_FP32, false>(p, s);
      case QG_FP16: return run_stream<kMX4, QG_FP16, false>(p, s);
      default: return run_stream<kMX4, QG_BF16, false>(p, s);
    }
  }
  if (a.offsets)
    return a.act == kFP16 ? run_stream<kFP16, QG_FP16, true>(p, s) : run_stream<kBF16, QG_BF16, true>(p, s);
  return a.act == kFP16 ? run_stream<kFP16, QG_FP16, false>(p, s) : run_stream<kBF16, QG_BF16, false>(p, s);
}

}  // namespace qg

// f8.hip -- conversions of the block-scaled 8-bit float format (F8): quantize
// (by rows or by 128 x 128 blocks, transposed as well), read back, and the
// gradient of the gated block's activation and product, quantized both ways
// as the two products of the backward pass read it.  A value is read once and its codes are
// written once each, so all of them are bound by HBM (5.2 TB/s in a large copy) or,
// the smallest, by a launch.  Measured on MI355X, bf16, all but the smallest's values out of the caches:
//     rows 16 x 2048 2.1 us, 4000 x 3600 11.9 us (3.6 TB/s), 4096 x 3584 both ways 16.6 us (3.5),
//     blocks of 18944 x 3584 both ways 55 us (5.0), read back 4096 x 3584 12.1 us (3.6);
// with every call's results over the last one's, which the 256 MB cache then takes in part:
// 11.3, 14.7, 48.5 (5.6 TB/s, past the copy's) and 11.3 us.
// Loads come first, all of a thread's in flight before one is used (both ways 17.4 -> 14.7 us),
// and the division by a scale is part of the conversion instruction.
#include <algorithm>

#include "f8_common.hpp"

namespace qg {

namespace {

// Eight consecutive values of a row, as loaded (zeros unless they are) and as fp32.
// Apart, so that loads behind a bounds check are all in flight before the first is used.
template <int DT>
struct F8Eight {
  u32x4 w[DT == QG_FP32 ? 2 : 1] = {};
  __device__ __forceinline__ void load(const void *X, size_t i) {
    if constexpr (DT == QG_FP32) {
      w[0] = *reinterpret_cast<const u32x4 *>(static_cast<const float *>(X) + i);
      w[1] = *reinterpret_cast<const u32x4 *>(static_cast<const float *>(X) + i + 4);
    } else {
      w[0] = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(X) + i);
    }
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (DT == QG_FP32) v[e] = __uint_as_float(w[e >> 2][e & 3]);
      else v[e] = bits_to_f32<DT>(static_cast<uint16_t>(e & 1 ? w[0][e >> 1] >> 16 : w[0][e >> 1] & 0xFFFFu));
    }
  }
};

// The maximum over the 16 lanes of a DPP row, in all of them (all active).
__device__ __forceinline__ int max16(int x) {
  x = max(x, __builtin_amdgcn_mov_dpp(x, 0xB1, 0xF, 0xF, false));    // quad_perm 1 0 3 2
  x = max(x, __builtin_amdgcn_mov_dpp(x, 0x4E, 0xF, 0xF, false));    // quad_perm 2 3 0 1
  x = max(x, __builtin_amdgcn_mov_dpp(x, 0x141, 0xF, 0xF, false));   // row_half_mirror
  return max(x, __builtin_amdgcn_mov_dpp(x, 0x140, 0xF, 0xF, false)); // row_mirror
}

// Rows alone, one scale per 128 of k: 16 lanes a block, eight values each.
template <int DT>
__global__ __launch_bounds__(256) void k_f8_rows(const void *X, uint8_t *Q, float *S, uint32_t rows, uint32_t k) {
  const uint32_t kb = f8_blocks(static_cast<int>(k)), groups = rows * kb, l = threadIdx.x & 15;
  for (uint32_t g = blockIdx.x * 16 + (threadIdx.x >> 4); g < groups; g += gridDim.x * 16) {
    const uint32_t row = g / kb, b = g - row * kb, col = b * 128 + 8 * l;
    const size_t at = static_cast<size_t>(row) * k + col;
    F8Eight<DT> in;
    float v[8];
    if (col < k) in.load(X, at);
    in.values(v);
    int top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = f8_top(top, v[e]);
    const F8Scale s(max16(top));
    if (col < k) {
      uint32_t lo = f8_pack4(v[0], v[1], v[2], v[3], s.scale);
      uint32_t hi = f8_pack4(v[4], v[5], v[6], v[7], s.scale);
      *reinterpret_cast<u32x2 *>(Q + at) = s.bad ? u32x2{0, 0} : u32x2{lo, hi};
    }
    if (l == 0) S[static_cast<size_t>(b) * rows + row] = s.scale;
  }
}

// One 128 x 128 tile, 512 threads: thread t holds rows 4 (t / 16) .. + 3, columns
// 8 (t % 16) .. + 7.  Writes the codes by rows and, through LDS, transposed, with
// one scale per row (per column, transposed) of the tile, or one for all of it
// (BLOCK).  Values past the matrix are zeros; the transposed rows are padded to a
// multiple of 16 with the zeros' codes.  Called by all threads, again only
// after a barrier.
struct F8TileLds {
  char codes[128 * 128];   // [column][row], 16-byte chunk c of column n at c ^ ((n / 8) % 8)
  int top[128];
  float scale[128];
};
struct F8TileOut {
  uint8_t *Q;       // [rows, ldq] or null
  float *S;         // the tile's row scales (of this block of k), or its one scale
  uint8_t *QT;      // [k, ldqt] or null
  float *ST;        // the tile's column scales, or its one scale
  size_t ldq, ldqt;
};

template <bool BLOCK, bool ROWS, bool COLS>
__device__ __forceinline__ void f8_emit(const float (&v)[4][8], F8TileLds &L, const F8TileOut &o, int row0, int rows,
                                        int col0, int k) {
  const int t = threadIdx.x, r = 4 * (t >> 4), c = 8 * (t & 15);
  int rtop[4] = {0, 0, 0, 0};
#pragma unroll
  for (int p = 0; p < 4; ++p)
#pragma unroll
    for (int e = 0; e < 8; ++e) rtop[p] = f8_top(rtop[p], v[p][e]);
  if (BLOCK || COLS) {
    if (t < 128) L.top[t] = 0;
    __syncthreads();
  }
  if constexpr (BLOCK) {
    const int m = max16(max(max(rtop[0], rtop[1]), max(rtop[2], rtop[3])));
    if ((t & 15) == 0) atomicMax(&L.top[0], m);
    __syncthreads();
  } else if constexpr (COLS) {
    // The wave's 16 rows of a column: lanes 32 and 16 apart trade halves of their
    // columns, which leaves two to a lane, then LDS.
    int m[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) m[e] = f8_top(f8_top(f8_top(f8_top(0, v[0][e]), v[1][e]), v[2][e]), v[3][e]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const auto x = __builtin_amdgcn_permlane32_swap(m[e], m[e + 4], false, false);
      m[e] = max(static_cast<int>(x[0]), static_cast<int>(x[1]));
    }
    const int q = (t >> 4) & 3, at = c + 2 * (q & 1) + 4 * (q >> 1);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const auto x = __builtin_amdgcn_permlane16_swap(m[e], m[e + 2], false, false);
      atomicMax(&L.top[at + e], max(static_cast<int>(x[0]), static_cast<int>(x[1])));
    }
    __syncthreads();
    if (t < 128) {
      const float scale = F8Scale(L.top[t]).scale;
      L.scale[t] = scale;
      if (col0 + t < k) o.ST[t] = scale;
    }
    __syncthreads();
  }
  if constexpr (ROWS) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const F8Scale s(BLOCK ? L.top[0] : max16(rtop[p]));
      const int row = row0 + r + p;
      if (row < rows && col0 + c < k) {
        const uint32_t lo = f8_pack4(v[p][0], v[p][1], v[p][2], v[p][3], s.scale);
        const uint32_t hi = f8_pack4(v[p][4], v[p][5], v[p][6], v[p][7], s.scale);
        *reinterpret_cast<u32x2 *>(o.Q + static_cast<size_t>(row) * o.ldq + col0 + c) =
            s.bad ? u32x2{0, 0} : u32x2{lo, hi};
      }
      if (!BLOCK && (t & 15) == 0 && row < rows) o.S[r + p] = s.scale;
    }
    if (BLOCK && t == 0) o.S[0] = F8Scale(L.top[0]).scale;
  }
  if constexpr (COLS) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float scale = BLOCK ? F8Scale(L.top[0]).scale : L.scale[c + e];
      const uint32_t w = f8_pack4(v[0][e], v[1][e], v[2][e], v[3][e], scale);
      *reinterpret_cast<uint32_t *>(L.codes + (c + e) * 128 + (((r >> 4) ^ (t & 7)) << 4) + (r & 15)) = scale == scale ? w : 0;
    }
    if (BLOCK && t == 0) o.ST[0] = F8Scale(L.top[0]).scale;
    __syncthreads();
    const int padded = f8_pad16(rows);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int n = 64 * i + (t >> 3), q = t & 7;
      if (col0 + n < k && row0 + 16 * q < padded)
        *reinterpret_cast<u32x4 *>(o.QT + static_cast<size_t>(col0 + n) * o.ldqt + row0 + 16 * q) =
            *reinterpret_cast<const u32x4 *>(L.codes + n * 128 + ((q ^ ((n >> 3) & 7)) << 4));
    }
  }
}

// Matrix x, tile (rb, b) of a stack of [rows, k] matrices.
template <int DT, bool BLOCK, bool ROWS, bool COLS>
__global__ __launch_bounds__(512) void k_f8_tile(const void *X, uint8_t *Q, float *S, uint8_t *QT, float *ST, int rows,
                                                 int k) {
  __shared__ __attribute__((aligned(16))) F8TileLds L;
  const uint32_t kb = f8_blocks(k), rb = f8_blocks(rows);
  const uint32_t tiles = rb * kb, x = blockIdx.x / tiles, in = blockIdx.x - x * tiles, ri = in / kb, b = in - ri * kb;
  const int row0 = static_cast<int>(ri) * 128, col0 = static_cast<int>(b) * 128;
  const int r = 4 * (threadIdx.x >> 4), c = 8 * (threadIdx.x & 15);
  const size_t base = static_cast<size_t>(x) * rows * k;
  F8Eight<DT> from[4];
#pragma unroll
  for (int p = 0; p < 4; ++p)
    if (row0 + r + p < rows && col0 + c < k) from[p].load(X, base + static_cast<size_t>(row0 + r + p) * k + col0 + c);
  float v[4][8];
#pragma unroll
  for (int p = 0; p < 4; ++p) from[p].values(v[p]);
  const size_t pad = f8_pad16(rows);
  const F8TileOut o{
      ROWS ? Q + base : nullptr,
      ROWS ? S + (BLOCK ? static_cast<size_t>(x) * tiles + in : static_cast<size_t>(b) * rows + row0) : nullptr,
      COLS ? QT + static_cast<size_t>(x) * k * pad : nullptr,
      COLS ? ST + (BLOCK ? (static_cast<size_t>(x) * kb + b) * rb + ri : static_cast<size_t>(ri) * k + col0) : nullptr,
      static_cast<size_t>(k), pad};
  f8_emit<BLOCK, ROWS, COLS>(v, L, o, row0, rows, col0, k);
}

// D = [dh u act'(g) | dh act(g)] from GU = [g | u], tile (ri, b) of its two halves.
// Workgroups past the tiles (with columns) look through the other scales of the
// weight gradient's product: powers[i] = 0 if the i-th of kF8Flags parts holds normal powers
// of two alone (D's own are).
// 4096 x 18944 moves 776 MB, 150 us at a copy's rate; some 200 here, since one
// workgroup of 8 waves fits a CU (197 registers: both gradients and the loads) and its loading,
// arithmetic (25 instructions a value) and storing overlap with nobody's.  Bounding the registers
// for two spills them (317 -> 584 us with both products of 16 columns).
template <int DT, int ACT, bool ROWS, bool COLS>
__global__ __launch_bounds__(512) void k_f8_gated_grad(const void *dH, const void *GU, uint8_t *D, float *SD,
                                                       uint8_t *DT_, float *SDT, int rows, int inter,
                                                       const float *scales, size_t n_scales, uint32_t *powers,
                                                       int halves) {
  __shared__ __attribute__((aligned(16))) F8TileLds L;
  const uint32_t kb = static_cast<uint32_t>(inter) >> 7;
  if constexpr (COLS) {
    const uint32_t tiles = kb * f8_blocks(rows) * halves;
    if (blockIdx.x >= tiles) {
      const uint32_t part = blockIdx.x - tiles;
      bool bad = false;
      for (size_t i = part * 512 + threadIdx.x; i < n_scales; i += kF8Flags * 512) bad |= !f8_power(scales[i]);
      if (__syncthreads_or(bad) == 0) {
        if (threadIdx.x == 0) powers[part] = 0;
      } else if (threadIdx.x == 0) {
        powers[part] = 1;
      }
      return;
    }
  }
  // halves 2: a workgroup for each half, where there are few (100 x 1408 14 -> 9.6 us, as many
  // loads again).
  const uint32_t tile = blockIdx.x / halves, ri = tile / kb, b = tile - ri * kb;
  const int first = halves == 2 ? static_cast<int>(blockIdx.x & 1) : 0, last = halves == 2 ? first : 1;
  const int row0 = static_cast<int>(ri) * 128, col0 = static_cast<int>(b) * 128;
  const int r = 4 * (threadIdx.x >> 4), c = 8 * (threadIdx.x & 15);
  const size_t wide = 2 * static_cast<size_t>(inter), pad = f8_pad16(rows);
  F8Eight<DT> fh[4], fg[4], fu[4];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const size_t row = static_cast<size_t>(row0 + r + p);
    if (row0 + r + p < rows) {
      fh[p].load(dH, row * inter + col0 + c);
      fg[p].load(GU, row * wide + col0 + c);
      fu[p].load(GU, row * wide + inter + col0 + c);
    }
  }
  float dg[4][8], du[4][8];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    float h[8], g[8], u[8];
    fh[p].values(h);
    fg[p].values(g);
    fu[p].values(u);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float value;
      const float slope = f8_gate_slope(g[e], ACT, value);
      dg[p][e] = h[e] * u[e] * slope;
      du[p][e] = h[e] * value;
    }
  }
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    if (half < first || half > last) continue;
    const int n0 = col0 + half * inter;
    const F8TileOut o{D, ROWS ? SD + static_cast<size_t>(n0 >> 7) * rows + row0 : nullptr, DT_,
                      COLS ? SDT + static_cast<size_t>(ri) * wide + n0 : nullptr, wide, pad};
    if (half) {
      if (first == 0) __syncthreads();
      f8_emit<false, ROWS, COLS>(du, L, o, row0, rows, n0, 2 * inter);
    } else {
      f8_emit<false, ROWS, COLS>(dg, L, o, row0, rows, n0, 2 * inter);
    }
  }
}

// Codes and scales -> values: eight a thread.
template <int DT, bool BLOCK>
__global__ __launch_bounds__(256) void k_f8_dequant(const uint8_t *Q, const float *S, void *out, int stack, int rows,
                                                    int k) {
  const size_t vecs = static_cast<size_t>(stack) * rows * (static_cast<size_t>(k) >> 3), step = static_cast<size_t>(gridDim.x) * 256;
  const uint32_t per = static_cast<uint32_t>(k) >> 3, kb = f8_blocks(k), rb = f8_blocks(rows);
  for (size_t i = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x; i < vecs; i += step) {
    const size_t row = i / per;
    const uint32_t b = static_cast<uint32_t>(i - row * per) >> 4;
    size_t at;
    if constexpr (BLOCK) {
      const size_t x = row / static_cast<uint32_t>(rows);
      at = (x * rb + ((row - x * rows) >> 7)) * kb + b;
    } else {
      at = static_cast<size_t>(b) * rows + row;
    }
    const float s = S[at];
    const u32x2 w = *reinterpret_cast<const u32x2 *>(Q + i * 8);
    float v[8];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const f32x2 lo = f8_unpack2<false>(w[e]), hi = f8_unpack2<true>(w[e]);
      v[4 * e] = lo[0] * s;
      v[4 * e + 1] = lo[1] * s;
      v[4 * e + 2] = hi[0] * s;
      v[4 * e + 3] = hi[1] * s;
    }
    if constexpr (DT == QG_FP32) {
      float *p = static_cast<float *>(out) + i * 8;
      *reinterpret_cast<f32x4 *>(p) = f32x4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4 *>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
    } else {
      *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(out) + i * 8) =
          u32x4{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]), pack2<DT>(v[4], v[5]), pack2<DT>(v[6], v[7])};
    }
  }
}

__global__ __launch_bounds__(256) void k_fill_zero(u32x4 *p, size_t n) {
  const size_t step = static_cast<size_t>(gridDim.x) * 256;
  for (size_t i = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += step) p[i] = u32x4{0, 0, 0, 0};
}

constexpr uint64_t kLaunch = UINT32_MAX;   // threads of a launch

template <int DT>
hipError_t quantize_as(const F8Quantize &q, hipStream_t s) {
  if (q.block == 1 && !q.QT) {
    const uint64_t groups = static_cast<uint64_t>(q.rows) * f8_blocks(q.k);
    if (groups > INT32_MAX) return hipErrorNotSupported;
    const unsigned grid = static_cast<unsigned>(std::min<uint64_t>((groups + 15) / 16, 1u << 20));
    hipLaunchKernelGGL(k_f8_rows<DT>, dim3(grid), dim3(256), 0, s, q.X, q.Q, q.S, static_cast<uint32_t>(q.rows),
                       static_cast<uint32_t>(q.k));
    return hipGetLastError();
  }
  const uint64_t tiles = static_cast<uint64_t>(f8_blocks(q.rows)) * f8_blocks(q.k);
  if (tiles * q.stack * 512 > kLaunch) return hipErrorNotSupported;
  const dim3 grid(static_cast<unsigned>(tiles * q.stack)), block(512);
#define QG_F8_TILE(BLOCK, ROWS, COLS) \
  hipLaunchKernelGGL((k_f8_tile<DT, BLOCK, ROWS, COLS>), grid, block, 0, s, q.X, q.Q, q.S, q.QT, q.ST, q.rows, q.k)
  if (q.block == 1) {
    if (q.Q) QG_F8_TILE(false, true, true);
    else QG_F8_TILE(false, false, true);
  } else if (!q.QT) {
    QG_F8_TILE(true, true, false);
  } else if (q.Q) {
    QG_F8_TILE(true, true, true);
  } else {
    QG_F8_TILE(true, false, true);
  }
#undef QG_F8_TILE
  return hipGetLastError();
}

template <int DT>
hipError_t dequant_as(const uint8_t *Q, const float *S, void *out, int stack, int rows, int k, int block, hipStream_t s) {
  const uint64_t vecs = static_cast<uint64_t>(stack) * rows * (static_cast<uint64_t>(k) >> 3);
  const dim3 grid(static_cast<unsigned>(std::min<uint64_t>((vecs + 255) / 256, 1u << 20)));
  if (block == 1) hipLaunchKernelGGL((k_f8_dequant<DT, false>), grid, dim3(256), 0, s, Q, S, out, stack, rows, k);
  else hipLaunchKernelGGL((k_f8_dequant<DT, true>), grid, dim3(256), 0, s, Q, S, out, stack, rows, k);
  return hipGetLastError();
}

template <int DT, int ACT>
hipError_t grad_as(const F8GatedGrad &g, hipStream_t s) {
  uint64_t tiles = static_cast<uint64_t>(f8_blocks(g.m)) * (g.inter >> 7);
  const int halves = tiles <= static_cast<uint64_t>(device_cus()) ? 2 : 1;
  tiles *= halves;
  if ((tiles + kF8Flags) * 512 > kLaunch) return hipErrorNotSupported;
  const dim3 grid(static_cast<unsigned>(tiles) + (g.DT ? kF8Flags : 0)), block(512);
#define QG_F8_GRAD(ROWS, COLS)                                                                                   \
  hipLaunchKernelGGL((k_f8_gated_grad<DT, ACT, ROWS, COLS>), grid, block, 0, s, g.dH, g.GU, g.D, g.SD, g.DT, g.SDT, g.m, \
                     g.inter, g.scales, g.n_scales, g.powers, halves)
  if (g.D && g.DT) QG_F8_GRAD(true, true);
  else if (g.D) QG_F8_GRAD(true, false);
  else QG_F8_GRAD(false, true);
#undef QG_F8_GRAD
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_f8(const F8Quantize &q, hipStream_t s) {
  switch (q.dt) {
    case QG_FP32: return quantize_as<QG_FP32>(q, s);
    case QG_FP16: return quantize_as<QG_FP16>(q, s);
    default: return quantize_as<QG_BF16>(q, s);
  }
}

hipError_t launch_dequant_f8(const uint8_t *Q, const float *S, void *out, int stack, int rows, int k, int block,
                             int out_dt, hipStream_t s) {
  switch (out_dt) {
    case QG_FP32: return dequant_as<QG_FP32>(Q, S, out, stack, rows, k, block, s);
    case QG_FP16: return dequant_as<QG_FP16>(Q, S, out, stack, rows, k, block, s);
    default: return dequant_as<QG_BF16>(Q, S, out, stack, rows, k, block, s);
  }
}

hipError_t launch_fill_zero(void *p, size_t bytes, hipStream_t s) {
  const size_t n = bytes / 16;
  hipLaunchKernelGGL(k_fill_zero, dim3(static_cast<unsigned>(std::min<size_t>((n + 255) / 256, 4096))), dim3(256), 0, s,
                     static_cast<u32x4 *>(p), n);
  return hipGetLastError();
}

hipError_t launch_gated_f8_grad(const F8GatedGrad &g, hipStream_t s) {
  if (g.act == QG_GATE_GELU) return g.dt == QG_FP16 ? grad_as<QG_FP16, QG_GATE_GELU>(g, s) : grad_as<QG_BF16, QG_GATE_GELU>(g, s);
  return g.dt == QG_FP16 ? grad_as<QG_FP16, QG_GATE_SILU>(g, s) : grad_as<QG_BF16, QG_GATE_SILU>(g, s);
}

}  // namespace qg

// row_groups.hpp -- which tiles a workgroup of a tiled product takes: the row
// tiles of products grouped by expert, and the share of all tiles that falls
// to a workgroup.  Used by the MX4 and the F8 products.
#pragma once

#include "qg_common.hpp"

namespace qg {

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
struct RowGroups {
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
  template <class Problem>
  __device__ __forceinline__ RowGroups(const Problem &p, int bm) : offsets(p.offsets), E(p.E), M(p.M), BM(bm) {
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

// Which items a workgroup walks.  Workgroup b runs on XCD b % 8; each XCD
// takes a contiguous share of the item order, its workgroups neighbouring items at a
// time, so that the XCD's L2 serves the rows and channels they share.
struct WorkShare {
  int first, step, end;
  __device__ __forceinline__ explicit WorkShare(int total) {
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

}  // namespace qg

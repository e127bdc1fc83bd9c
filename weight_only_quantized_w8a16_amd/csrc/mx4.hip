// mx4.hip -- conversions of the microscaled 4-bit format (MX4): quantize,
// read back, and the change between the portable and the tiled layout.  All
// of them are bound by HBM (the smallest by a launch): a value is read or
// written once and everything else happens in registers.  Measured in bf16,
// back to back on inputs in turn (500 MB, or 40 inputs where those are less
// and stay in the caches): 13312 x 2048 (54.5 MB of values, 14.5 MB of codes
// and scales) portable quantize 11.6 us, read back 11.9 us (5.9 TB/s), tiled
// 12.1 and 11.6; 4096 x 18944 28.9 and 29.9 us (6.7 TB/s); 16 x 2048 2.3 and
// 2.2 us.  The layout change of 13312 x 2048 takes 7.7 us.
//
// Four lanes share a 32-value block, eight values each (16 bytes of a 16-bit
// row), so the block's largest magnitude is two quad exchanges away.  The
// magnitudes compare as integers (a float's order is its bit pattern's), so
// infinities and NaNs come out on top and are recognised by the same word.
#include "mx4_common.hpp"

namespace qg {

namespace {

// Eight consecutive values of a row as fp32.
template <int DT>
__device__ __forceinline__ void load8(const void *X, size_t i, float (&v)[8]) {
  if constexpr (DT == QG_FP32) {
    const f32x4 a = *reinterpret_cast<const f32x4 *>(static_cast<const float *>(X) + i);
    const f32x4 b = *reinterpret_cast<const f32x4 *>(static_cast<const float *>(X) + i + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) { v[e] = a[e]; v[4 + e] = b[e]; }
  } else {
    const u32x4 a = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(X) + i);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = bits_to_f32<DT>(static_cast<uint16_t>(a[e] & 0xFFFFu));
      v[2 * e + 1] = bits_to_f32<DT>(static_cast<uint16_t>(a[e] >> 16));
    }
  }
}

// Eight codes (one word) -> eight values of type DT at out[i ..].
template <int DT>
__device__ __forceinline__ void store8(void *out, size_t i, uint32_t w, float scale) {
  if constexpr (DT == QG_FP32) {
    const auto a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 0);
    const auto b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 1);
    const auto c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 2);
    const auto d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 3);
    float *o = static_cast<float *>(out) + i;
    *reinterpret_cast<f32x4 *>(o) = f32x4{a[0], a[1], b[0], b[1]};
    *reinterpret_cast<f32x4 *>(o + 4) = f32x4{c[0], c[1], d[0], d[1]};
  } else {
    *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(out) + i) = mx4_word_to_operand<DT>(w, scale);
  }
}

// The quad's block: scale byte and this lane's word of eight codes.  The four
// lanes of a quad are all active (a block is never split over a tail).
__device__ __forceinline__ uint32_t quantize8(const float (&v)[8], uint32_t &scale) {
  int top = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = max(top, __float_as_int(v[e]) & 0x7FFFFFFF);
  top = max(top, __builtin_amdgcn_update_dpp(top, top, 0xB1, 0xF, 0xF, false));   // quad_perm [1,0,3,2]
  top = max(top, __builtin_amdgcn_update_dpp(top, top, 0x4E, 0xF, 0xF, false));   // quad_perm [2,3,0,1]
  const int field = top >> 23;   // floor(log2) + 127; 0 also for subnormal numbers
  if (field == 255) {            // an infinity or a NaN in the block
    scale = 255u;
    return 0u;
  }
  // The largest magnitude lands in [4, 8); the conversion rounds to nearest
  // even and saturates at 6.  field <= 2: 2^-127, the smallest scale.
  scale = static_cast<uint32_t>(max(field - 2, 0));
  const float s = __uint_as_float(scale << 23);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], s, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], s, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], s, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], s, 3);
  return w;
}

constexpr int kThreads = 256;

}  // namespace

// Portable: thread i takes values 8 i .. 8 i + 7 of the flat matrix (both
// sides of the conversion are then contiguous over a wave).
template <int DT>
__global__ __launch_bounds__(kThreads) void k_mx4_quantize(const void *__restrict__ X,
                                                           uint32_t *__restrict__ codes,
                                                           uint8_t *__restrict__ scales, size_t n8) {
  const size_t step = static_cast<size_t>(gridDim.x) * kThreads;
  for (size_t i = static_cast<size_t>(blockIdx.x) * kThreads + threadIdx.x; i < n8; i += step) {
    float v[8];
    load8<DT>(X, 8 * i, v);
    uint32_t s;
    const uint32_t w = quantize8(v, s);
    codes[i] = w;
    if ((i & 3) == 0) scales[i >> 2] = static_cast<uint8_t>(s);
  }
}

// Tiled: a workgroup takes 16 rows x 512 k (four code blocks and one window
// of scale words); thread 4 * slot + q takes quarter q of lane slot `slot`
// (row slot % 16, block slot / 16) of each of the four code blocks.
template <int DT>
__global__ __launch_bounds__(kThreads) void k_mx4_quantize_tiled(const void *__restrict__ X,
                                                                 uint32_t *__restrict__ codes,
                                                                 uint32_t *__restrict__ scales,
                                                                 int rows, int K) {
  const int nw = mx4_scale_windows(K), nb = K >> 7;
  const int rt = blockIdx.x / nw, win = blockIdx.x - rt * nw;
  const int slot = threadIdx.x >> 2, q = threadIdx.x & 3;
  const int row = 16 * rt + (slot & 15), j = slot >> 4;
  // All four blocks' loads first (past the end the last row and block again),
  // then their conversions: one memory latency instead of four.  8 x 3584 2.6
  // -> 2.3 us, 2048 x 640 3.6 -> 2.9, at 4096 x 3584 7.5 -> 7.8.  A thread per
  // block and eighth (1024 a workgroup) gave 2.3, 2.6 and 8.6.  (Values still in
  // the caches, as an activation just written is; 8 x 3584 behind a product that
  // reads 36 MB, so that they are not: 4.7.)
  float v[4][8];
#pragma unroll
  for (int b = 0; b < 4; ++b)
    load8<DT>(X, static_cast<size_t>(min(row, rows - 1)) * K + min(4 * win + b, nb - 1) * 128 + 32 * j + 8 * q, v[b]);
  uint32_t sw = 0;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const int kb = 4 * win + b;
    uint32_t s, w = quantize8(v[b], s);
    if (kb >= nb) break;
    if (row >= rows) w = s = 0;
    codes[(static_cast<size_t>(rt) * nb + kb) * 256 + threadIdx.x] = w;
    sw |= s << (8 * b);
  }
  if (q == 0) scales[static_cast<size_t>(blockIdx.x) * 64 + slot] = sw;
}

template <int DT>
__global__ __launch_bounds__(kThreads) void k_mx4_dequant(const uint32_t *__restrict__ codes,
                                                          const uint8_t *__restrict__ scales,
                                                          void *__restrict__ out, size_t n8) {
  const size_t step = static_cast<size_t>(gridDim.x) * kThreads;
  for (size_t i = static_cast<size_t>(blockIdx.x) * kThreads + threadIdx.x; i < n8; i += step)
    store8<DT>(out, 8 * i, codes[i], mx4_scale_operand(scales[i >> 2], 0));
}

template <int DT>
__global__ __launch_bounds__(kThreads) void k_mx4_dequant_tiled(const uint32_t *__restrict__ codes,
                                                                const uint32_t *__restrict__ scales,
                                                                void *__restrict__ out, int rows,
                                                                int K) {
  const int nw = mx4_scale_windows(K), nb = K >> 7;
  const int rt = blockIdx.x / nw, win = blockIdx.x - rt * nw;
  const int slot = threadIdx.x >> 2, q = threadIdx.x & 3;
  const int row = 16 * rt + (slot & 15), j = slot >> 4;
  if (row >= rows) return;
  const uint32_t sw = scales[static_cast<size_t>(blockIdx.x) * 64 + slot];
  uint32_t w[4];
#pragma unroll
  for (int b = 0; b < 4; ++b)
    w[b] = codes[(static_cast<size_t>(rt) * nb + min(4 * win + b, nb - 1)) * 256 + threadIdx.x];
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const int kb = 4 * win + b;
    if (kb >= nb) break;
    store8<DT>(out, static_cast<size_t>(row) * K + kb * 128 + 32 * j + 8 * q, w[b], mx4_scale_operand(sw, b));
  }
}

// Layout change: thread 64 * b + slot moves the 16 bytes of lane slot `slot`
// of code block 4 * win + b (one 32-value block of a row); the threads of
// b = 0 also gather (or spread) the slot's scale word.
template <bool TO_TILED>
__global__ __launch_bounds__(kThreads) void k_mx4_relayout(const uint8_t *__restrict__ src_c,
                                                           const uint8_t *__restrict__ src_s,
                                                           uint8_t *__restrict__ dst_c,
                                                           uint8_t *__restrict__ dst_s, int rows,
                                                           int K) {
  const int nw = mx4_scale_windows(K), nb = K >> 7;
  const int rt = blockIdx.x / nw, win = blockIdx.x - rt * nw;
  const int slot = threadIdx.x & 63, b = threadIdx.x >> 6;
  const int row = 16 * rt + (slot & 15), j = slot >> 4, kb = 4 * win + b;
  const size_t tiled = (static_cast<size_t>(rt) * nb + kb) * 1024 + slot * 16;
  const size_t flat = static_cast<size_t>(row) * (K / 2) + kb * 64 + j * 16;
  if (kb < nb) {
    if constexpr (TO_TILED) {
      u32x4 v = {0u, 0u, 0u, 0u};
      if (row < rows) v = *reinterpret_cast<const u32x4 *>(src_c + flat);
      *reinterpret_cast<u32x4 *>(dst_c + tiled) = v;
    } else if (row < rows) {
      *reinterpret_cast<u32x4 *>(dst_c + flat) = *reinterpret_cast<const u32x4 *>(src_c + tiled);
    }
  }
  if (b != 0) return;
  const size_t sflat = static_cast<size_t>(row) * (K / 32) + 16 * win + j;
  const size_t sword = static_cast<size_t>(blockIdx.x) * 64 + slot;
  if constexpr (TO_TILED) {
    uint32_t sw = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (row < rows && 4 * win + i < nb) sw |= static_cast<uint32_t>(src_s[sflat + 4 * i]) << (8 * i);
    reinterpret_cast<uint32_t *>(dst_s)[sword] = sw;
  } else {
    const uint32_t sw = reinterpret_cast<const uint32_t *>(src_s)[sword];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (row < rows && 4 * win + i < nb) dst_s[sflat + 4 * i] = static_cast<uint8_t>(sw >> (8 * i));
  }
}

namespace {

// Workgroups of a flat kernel: at most eight per CU, the rest by its loop.
unsigned flat_grid(size_t n8) {
  const size_t want = (n8 + kThreads - 1) / kThreads, most = static_cast<size_t>(device_cus()) * 8;
  return static_cast<unsigned>(want < most ? want : most);
}

// Workgroups of a tiled kernel: one per (16 rows, 512 k).  A grid has at most
// 2^32 - 1 threads.
constexpr size_t kMostGroups = UINT32_MAX / kThreads;
size_t tiled_grid(int rows, int K) {
  return static_cast<size_t>((rows + 15) / 16) * mx4_scale_windows(K);
}

template <int DT>
hipError_t quantize_dt(const void *X, uint8_t *codes, uint8_t *scales, int rows, int k, int tiled,
                       hipStream_t s) {
  if (tiled) {
    const size_t grid = tiled_grid(rows, k);
    if (grid > kMostGroups) return hipErrorNotSupported;
    hipLaunchKernelGGL(k_mx4_quantize_tiled<DT>, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, s, X,
                       reinterpret_cast<uint32_t *>(codes), reinterpret_cast<uint32_t *>(scales), rows, k);
  } else {
    const size_t n8 = static_cast<size_t>(rows) * k / 8;
    hipLaunchKernelGGL(k_mx4_quantize<DT>, dim3(flat_grid(n8)), dim3(kThreads), 0, s, X,
                       reinterpret_cast<uint32_t *>(codes), scales, n8);
  }
  return hipGetLastError();
}

template <int DT>
hipError_t dequant_dt(const uint8_t *codes, const uint8_t *scales, void *out, int rows, int k, int tiled,
                      hipStream_t s) {
  if (tiled) {
    const size_t grid = tiled_grid(rows, k);
    if (grid > kMostGroups) return hipErrorNotSupported;
    hipLaunchKernelGGL(k_mx4_dequant_tiled<DT>, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, s,
                       reinterpret_cast<const uint32_t *>(codes), reinterpret_cast<const uint32_t *>(scales),
                       out, rows, k);
  } else {
    const size_t n8 = static_cast<size_t>(rows) * k / 8;
    hipLaunchKernelGGL(k_mx4_dequant<DT>, dim3(flat_grid(n8)), dim3(kThreads), 0, s,
                       reinterpret_cast<const uint32_t *>(codes), scales, out, n8);
  }
  return hipGetLastError();
}

template <bool TO_TILED>
hipError_t relayout(const uint8_t *src_c, const uint8_t *src_s, uint8_t *dst_c, uint8_t *dst_s, int rows,
                    int k, hipStream_t s) {
  const size_t grid = tiled_grid(rows, k);
  if (grid > kMostGroups) return hipErrorNotSupported;
  hipLaunchKernelGGL(k_mx4_relayout<TO_TILED>, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, s, src_c,
                     src_s, dst_c, dst_s, rows, k);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_mx4(const void *X, uint8_t *codes, uint8_t *scales, int rows, int k, int tiled,
                               int x_dt, hipStream_t s) {
  switch (x_dt) {
    case QG_FP32: return quantize_dt<QG_FP32>(X, codes, scales, rows, k, tiled, s);
    case QG_FP16: return quantize_dt<QG_FP16>(X, codes, scales, rows, k, tiled, s);
    default: return quantize_dt<QG_BF16>(X, codes, scales, rows, k, tiled, s);
  }
}

hipError_t launch_dequant_mx4(const uint8_t *codes, const uint8_t *scales, void *out, int rows, int k,
                              int tiled, int out_dt, hipStream_t s) {
  switch (out_dt) {
    case QG_FP32: return dequant_dt<QG_FP32>(codes, scales, out, rows, k, tiled, s);
    case QG_FP16: return dequant_dt<QG_FP16>(codes, scales, out, rows, k, tiled, s);
    default: return dequant_dt<QG_BF16>(codes, scales, out, rows, k, tiled, s);
  }
}

hipError_t launch_repack_mx4(const uint8_t *codes, const uint8_t *scales, uint8_t *codes_t,
                             uint8_t *scales_t, int rows, int k, hipStream_t s) {
  return relayout<true>(codes, scales, codes_t, scales_t, rows, k, s);
}

hipError_t launch_unrepack_mx4(const uint8_t *codes_t, const uint8_t *scales_t, uint8_t *codes,
                               uint8_t *scales, int rows, int k, hipStream_t s) {
  return relayout<false>(codes_t, scales_t, codes, scales, rows, k, s);
}

}  // namespace qg

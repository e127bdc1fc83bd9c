// qg_launch.hpp -- host-side launchers implemented in the .hip translation
// units and called by the C ABI layer (api.cpp) after validation.  Every
// launcher assumes its arguments were validated and returns the HIP status
// of the launch.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

namespace qg {

// Raises a kernel's dynamic-LDS limit to `bytes` once per device (the
// attribute belongs to the current device's copy of the kernel): `done`
// holds one bit per device id, set after a successful call.  Concurrent
// first calls may both set it, which is harmless.
template <class Kern>
hipError_t set_lds_limit_once(Kern kern, int bytes, std::atomic<uint64_t> &done) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = (dev >= 0 && dev < 64) ? (uint64_t(1) << dev) : 0;
  if (bit && (done.load(std::memory_order_acquire) & bit)) return hipSuccess;
  e = hipFuncSetAttribute(reinterpret_cast<const void *>(kern),
                          hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == hipSuccess && bit) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// Compute units of the current device (cached per device; 256 if unknown).
inline int device_cus() {
  static std::atomic<int> cus[64] = {};
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
  int c = cus[dev].load(std::memory_order_relaxed);
  if (c == 0) {
    if (hipDeviceGetAttribute(&c, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || c <= 0) c = 256;
    cus[dev].store(c, std::memory_order_relaxed);
  }
  return c;
}

// Dispatch override (qg_set_override): forced choices, or the automatic
// ones (kPathAuto, -1, 0, false).  A forced tile or path that does not fit a
// problem is ignored for that problem.
enum { kPathAuto = 0, kPathDecode = 1, kPathPrefill = 2 };
// Prefill tiles (prefill.hip), in the order qg_set_override names them.
// kP256 .. kP64: the dense tiles of the dequantize-then-dense path.
// kW256 .. kW64: the int8 per-channel tiles that convert codes after the LDS read;
// kWX: 256 x 256 ones for whole rounds of the CUs, 128 x 128 quarters for the rest;
// kDX: fused 256 x 256 tiles for whole rounds, 256 x 128 halves for the rest.
enum PrefillTile { kX, kD8, kD8N, kD64, kD128, kL, kM, kS, kP256, kP128, kP64, kW256, kW256N, kW128, kW64, kWX, kDX };
// W8A8 tiles (w8a8.hip), in the order qg_set_override names them.
enum W8A8Tile { kT256, kT256N, kT128, kT64 };
// MX4 kernels (mx4_gemm.hip), in the order qg_set_override names them: the
// streaming kernel, then tiles of 256 x 256, 128 x 256, 128 x 128, 64 x 128 and
// 32 x 64.
enum Mx4Kernel { kMx4Stream, kMx4T256, kMx4T256N, kMx4T128, kMx4T64, kMx4T32 };
// F8 kernels (f8_gemm.hip), in the order qg_set_override names them: the
// streaming kernel, then tiles of 256 x 256, 128 x 128 and 64 x 128.
enum F8Kernel { kF8Stream, kF8T256, kF8T128, kF8T64 };
struct Override {
  int path = kPathAuto;
  int prefill_tile = -1;       // PrefillTile, or -1
  int splitk = 0;              // prefill K slices (1: none), or 0
  bool moe_small_tile = false; // MoE grouped GEMMs on the 128 x 128 tile
  int w8a8_tile = -1;          // W8A8Tile, or -1
  int w8a8_split = 0;          // W8A8 K slices, or 0
  int mx4_tile = -1;           // Mx4Kernel, or -1
  int mx4_split = 0;           // MX4 K slices, or 0
  int f8_tile = -1;            // F8Kernel, or -1
  int f8_split = 0;            // F8 K slices, or 0
};
Override dispatch_override();

hipError_t launch_repack_w4(const uint8_t *src, uint8_t *dst, int n, int k, hipStream_t s);
hipError_t launch_unrepack_w4(const uint8_t *src, uint8_t *dst, int n, int k, hipStream_t s);
hipError_t launch_repack_w8(const int8_t *src, int8_t *dst, int n, int k, hipStream_t s);
hipError_t launch_unrepack_w8(const int8_t *src, int8_t *dst, int n, int k, hipStream_t s);
hipError_t launch_repack_w8_kn(const int8_t *src, int8_t *dst, int n, int k, hipStream_t s);
hipError_t launch_unrepack_w8_kn(const int8_t *src, int8_t *dst, int n, int k, hipStream_t s);

hipError_t launch_quantize_w4(const void *W, uint8_t *packed, void *scale, void *zero, int n,
                              int k, int group, int w_dt, int sz_dt, hipStream_t s);

hipError_t launch_dequant_w4(const uint8_t *B, const uint16_t *S, const uint16_t *Z, void *W,
                             int n, int k, int group, int act, int out, hipStream_t s);
hipError_t launch_dequant_w8(const int8_t *B, const uint16_t *S, void *W, int n, int k, int group,
                             int act, int out, hipStream_t s);

// Dense GEMM problem as the kernels see it.
struct GemmArgs {
  const uint16_t *A;      // [M, K]
  const void *B;          // tiled codes
  const uint16_t *S;      // scales
  const uint16_t *Z;      // zeros (w4) or null
  const uint16_t *bias;   // [N] or null
  uint16_t *C;            // [M, N]
  int M, N, K, group;     // group: 64/128 (w4; w8 with group scales), 0 = per channel (w8)
  int act, bias_dt;
  void *ws = nullptr;     // caller's workspace (split-K partials), may be null
  size_t ws_bytes = 0;
};

// Decode path: M <= 16, weights streamed once.
hipError_t launch_decode_w4(const GemmArgs &a, hipStream_t s);
hipError_t launch_decode_w8(const GemmArgs &a, hipStream_t s);
// Prefill path: any M, matrix-core tiles with weights dequantized into LDS.
hipError_t launch_prefill_w4(const GemmArgs &a, hipStream_t s);
// Workspace bytes the prefill path would use for split-K on this problem (0:
// none); with less workspace it runs unsplit.
size_t prefill_workspace_bytes(const GemmArgs &a, int wbits);
hipError_t launch_prefill_w8(const GemmArgs &a, hipStream_t s);

// MoE pipeline.
struct MoeArgs {
  const uint16_t *x;
  const float *logits;
  const uint8_t *w1;
  const uint16_t *s1, *z1;
  const uint8_t *w2;
  const uint16_t *s2, *z2;
  uint16_t *out;
  int T, H, I, E, topk, group, act;
  int32_t *ids_out;
  float *w_out;
  void *ws;
  // optional parts of runMoe (null / 1 for the plain call)
  const float *sel_logits = nullptr;    // [T, E] biased logits that choose the experts
  const uint8_t *finished = nullptr;    // [T], nonzero: no expert, zero output
  const uint16_t *b1 = nullptr;         // [E, 2I] fc1 biases
  const uint16_t *b2 = nullptr;         // [E, H] fc2 biases
  int renorm = 1;                       // 1: renormalize over the chosen experts
};
size_t moe_workspace_bytes(int T, int H, int I, int E, int topk);
hipError_t launch_moe(const MoeArgs &a, hipStream_t s);
// Allocation-free MoE: the workspace is the library's device scratch of
// kMoeScratchBytes (moe.hip); callers check the problem fits first.
constexpr size_t kMoeScratchBytes = size_t(64) << 20;
hipError_t launch_moe_noalloc(MoeArgs a, hipStream_t s);

}  // namespace qg

namespace qg {

// W8A8 (int8 activations x int8 weights, fp32 row/column scales).
struct W8A8Args {
  const int8_t *A;          // [M, K]
  const int8_t *B;          // [N, K]
  const float *alpha_row;   // [M] if per_token else [1]
  const float *alpha_col;   // [N] if per_channel else [1]
  void *C;                  // [M, N] in `out`
  int M, N, K;
  int per_token, per_channel;
  int out;                  // QG_BF16, QG_FP16 or QG_FP32
  void *ws;                 // split-K partials, may be null
  size_t ws_bytes;
};
// Workspace bytes the W8A8 kernels would use (split-K), 0 if none; with
// less they run unsplit.
size_t w8a8_workspace_bytes(int m, int n, int k);
hipError_t launch_w8a8(const W8A8Args &a, hipStream_t s);

}  // namespace qg

namespace qg {

// Quantized embedding lookup.
struct EmbedArgs {
  const int32_t *ids;       // [tokens]
  int tokens;
  const void *B;            // table codes, tiled or portable
  int tiled;                // 1: the GEMM's tiled layout; 0: portable
  int bits;                 // 4 or 8
  const uint16_t *S, *Z;    // scales, zeros (int4, may be null)
  void *out;                // [tokens, hidden] in out_dt
  int vocab, hidden;
  int group;                // int4: 64, 128 or hidden; int8: 0 (per row), 64 or 128
  int act, out_dt;
};
hipError_t launch_embed(const EmbedArgs &a, hipStream_t s);

}  // namespace qg

namespace qg {

// Microscaled 4-bit floats (MX4).  hipErrorNotSupported: the sizes need more
// threads than a launch has (2^32 - 1); nothing is enqueued.
hipError_t launch_quantize_mx4(const void *X, uint8_t *codes, uint8_t *scales, int rows, int k,
                               int tiled, int x_dt, hipStream_t s);
hipError_t launch_dequant_mx4(const uint8_t *codes, const uint8_t *scales, void *out, int rows,
                              int k, int tiled, int out_dt, hipStream_t s);
hipError_t launch_repack_mx4(const uint8_t *codes, const uint8_t *scales, uint8_t *codes_t,
                             uint8_t *scales_t, int rows, int k, hipStream_t s);
hipError_t launch_unrepack_mx4(const uint8_t *codes_t, const uint8_t *scales_t, uint8_t *codes,
                               uint8_t *scales, int rows, int k, hipStream_t s);

constexpr int kMX4 = 4;   // activation type code of MX4 activations (next to QG_BF16, QG_FP16)

struct Mx4Args {
  const void *A;             // [M, K] 16-bit, or tiled MX4 codes
  const uint8_t *AS;         // tiled scales of A (MX4 activations), else null
  const uint8_t *B, *BS;     // tiled codes and scales, [N, K] (per expert)
  const uint16_t *bias;      // [N] (per expert) or null
  void *C;                   // [M, N] in `out`
  int M, N, K;
  int act;                   // QG_BF16, QG_FP16 or kMX4
  int out, bias_dt;
  const int32_t *offsets;    // grouped: [E + 1] row offsets, else null
  int E;                     // grouped: experts
  void *ws;                  // split-K partials, may be null
  size_t ws_bytes;
};
size_t mx4_workspace_bytes(int m, int n, int k, int act_bits);
hipError_t launch_mx4_gemm(const Mx4Args &a, hipStream_t s);

}  // namespace qg

namespace qg {

// Block-scaled 8-bit floats (F8).  hipErrorNotSupported: the sizes need more
// threads than a launch has (2^32 - 1); nothing is enqueued.
struct F8Quantize {
  const void *X;            // [stack, rows, k] in dt
  int stack, rows, k, dt;   // stack 1 by rows
  int block;                // 1: a scale per row and 128 k; 128: per 128 x 128
  uint8_t *Q;               // [stack, rows, k], or null
  float *S;
  uint8_t *QT;              // [stack, k, rows padded to 16], or null
  float *ST;
};
hipError_t launch_quantize_f8(const F8Quantize &q, hipStream_t s);
hipError_t launch_dequant_f8(const uint8_t *Q, const float *S, void *out, int stack, int rows, int k, int block,
                             int out_dt, hipStream_t s);

struct F8Args {
  const uint8_t *A;         // [M, K] codes
  const float *SA;          // [blocks of K, M]
  const uint8_t *B;         // [N, K] codes (per expert)
  const float *SB;          // [blocks of N, blocks of K] (per expert), or [blocks of K, N]
  int b_block;              // 128 or 1
  const uint16_t *bias;     // [N] (per expert) or null
  void *C;                  // [M, N] in `out`; gated [M, N / 2]
  int M, N, K;
  int out, bias_dt;
  const int32_t *offsets;   // grouped: [E + 1] row offsets, else null
  int E;                    // grouped: experts
  bool gated;               // B = [gate; up] channels
  int act;                  // gated: qg_gate
  void *GU;                 // gated: [M, N] in `out`, or null
  void *ws;                 // K slices' partials, may be null
  size_t ws_bytes;
  const uint32_t *powers;   // kF8Flags words that are 0 if all scales are normal powers of two, or null
};
size_t f8_workspace_bytes(int m, int n, int k, int b_block);
hipError_t launch_f8_gemm(const F8Args &a, hipStream_t s);

constexpr int kF8Flags = 32;
// Gradient of H = act(g) * u, quantized by rows (D) and transposed (DT).
struct F8GatedGrad {
  const void *dH, *GU;      // [m, inter], [m, 2 inter] in dt
  int m, inter, dt, act;
  uint8_t *D;               // [m, 2 inter], or null
  float *SD;                // [2 inter / 128, m]
  uint8_t *DT;              // [2 inter, m padded to 16], or null
  float *SDT;               // [blocks of m, 2 inter]
  const float *scales;      // other scales of DT's product, n_scales of them, to look through
  size_t n_scales;
  uint32_t *powers;         // kF8Flags words: 0 where all looked at are normal powers of two
};
hipError_t launch_gated_f8_grad(const F8GatedGrad &g, hipStream_t s);
// Zeros (a kernel: it may be captured), a multiple of 16 bytes.
hipError_t launch_fill_zero(void *p, size_t bytes, hipStream_t s);

}  // namespace qg

namespace qg {

// Streaming-read probe (measurement).
size_t read_probe_blocks(size_t bytes);
hipError_t launch_read_probe(const void *buf, size_t bytes, uint32_t *out, hipStream_t s);
hipError_t launch_lds_probe(int waves, int iters, int blocks, unsigned long long *cycles, hipStream_t s);

}  // namespace qg

// The gated feed-forward block's products on the tensor cores: one persistent
// kernel, four uses.  Included by the ffn*.cu files only.
//
//   FORWARD   [g | u] = x [Wg | Wu]^T          epilogue: h = act(g) u, kept copies
//   RECOMPUTE the same product                 epilogue: dg, du from dh
//   DX        dx = dg Wg + du Wu               one sum over both, K = 2 f
//   DW        dWg = dg^T x, dWu = du^T x       K = rows
//
// The gate and up weights enter one tile side by side (half its columns each), so
// both values of an element meet in one thread of the epilogue.  DX and DW read
// the matrices as they are stored, with the K index along rows (MN-major operands),
// so nothing is ever transposed in memory.
//
// Work is split by role: one lane loads 64-deep K slices with TMA into a ring of
// shared-memory stages, one lane issues tcgen05.mma into one of two accumulators
// in TMEM, and eight warps drain the other, so loads, products and
// epilogues overlap across the tiles of a persistent block.
#pragma once

#include "ops.h"
#include "tc.h"

namespace fsdp {
namespace ffn {

enum Mode { FORWARD = 0, RECOMPUTE = 1, DX = 2, DW = 3 };
enum Act { SILU = 0, GELU = 1 };

constexpr int kTileM = 128;  // rows of a block's tile (TMEM lanes)
constexpr int kTileK = 64;   // K values of a stage: one 128-byte swizzled row
constexpr uint32_t kStatusGemm = 16u;  // a wait of this kernel gave up

struct Args {
  CUtensorMap a[2], b[2];
  uint32_t *status;
  uint64_t wait_limit_ns;
  int32_t fault;
  int32_t act;        // Act
  // Tiles: m_tiles x n_tiles, each K loop split into `splits` parts.
  int32_t m_tiles, n_tiles, splits, raster;
  int32_t m_half;     // DW: tiles from here on are the up half
  int32_t k_blocks, k_half;  // K blocks in all; DX: from here on the up half
  int64_t m, n;       // rows and columns of the output (FORWARD, RECOMPUTE: n = f)
  // Outputs, [m, n] with row distance ld.
  void *out[2];       // FORWARD: h; RECOMPUTE: dg, du; DX: dx; DW: dWg, dWu
  int64_t ld_out[2];
  int32_t out_bf16, out_width;  // dtype; row_width() of the outputs
  float *partial;     // splits > 1: [splits][m (DW: 2 m)][n] in binary32 instead of out
  const void *dh;     // RECOMPUTE
  int64_t ld_dh;
  int32_t dh_vec;
  // FORWARD: what is kept for the backward pass.
  int32_t keep;       // 0 nothing, 1 8-bit checkpoints, 2 BF16
  int32_t keep_width;  // row_width() of what is kept, both
  uint8_t *codes[2], *scales[2];
  int64_t groups;
  void *kept[2];
  int64_t ld_kept;
};

// act(g) and its derivative.
//   SiLU: g s with s = 1 / (1 + e^-g);  s + g s (1 - s).
//   GELU: g Phi(g);  Phi(g) + g phi(g), Phi the normal distribution and phi its density.
// For g far below 0 the divisor overflows to infinity and s is 0, as it should be.
template <bool SLOPE>
__device__ __forceinline__ float2 act_of(float g, int act) {
  if (act == SILU) {
    const float s = __fdividef(1.0f, 1.0f + __expf(-g)), y = g * s;
    return make_float2(y, SLOPE ? fmaf(y, 1.0f - s, s) : 0.0f);
  }
  const float p = normcdff(g);
  return make_float2(g * p, SLOPE ? fmaf(g * 0.3989422804014327f, __expf(-0.5f * g * g), p) : 0.0f);
}

// Launches the product kernel of `mode`; `pair`: tiles of two blocks (256 rows).
cudaError_t launch_product(Mode mode, bool pair, Args &a, int sms, cudaStream_t stream);

}  // namespace ffn
}  // namespace fsdp

// The gated feed-forward block's products on the tensor cores: one persistent
// kernel, three uses.  Included by the ffn*.cu files only.
//
//   FORWARD   [g | u] = x [Wg | Wu]^T          epilogue: h = act(g) u, kept copies
//   RECOMPUTE the same product                 epilogue: dg, du from dh
//   BACKWARD  dWg = dg^T x, dWu = du^T x       K = rows
//             dx = dg Wg + du Wu               one sum over both, K = 2 f
//
// The gate and up weights enter one tile side by side (half its columns each), so
// both values of an element meet in one thread of the epilogue.  The backward
// products read the matrices as they are stored, with the K index along rows
// (MN-major operands), so nothing is ever transposed in memory; both are in one
// launch, whose tiles then fill the SMs together.
//
// Bound: the tensor cores, for long products under the power limit: 16384 x 4096 x 12288
// forward takes 1.88 ms (1.76 PFLOP/s; the library's products sustain 1.71), 8192 x 4096 x
// 12288 backward with gate and up computed again 3.13 ms (1.58 PFLOP/s).  Where K is short,
// each tile's start and drain show: 8192 x 1024 x 4096 forward takes 77 us (1.79 PFLOP/s),
// as long as two library products of that size without an epilogue, and with copies of gate
// and up, whose stores hold up the operands' loads, 84 (8 bits) and 87 (BF16); in a graph,
// operands and results rotating past L2.
//
// Work is split by role: one lane loads 64-deep K slices with TMA into a ring of
// shared-memory stages, one lane issues tcgen05.mma into one of two accumulators
// in TMEM, and eight warps drain the other, so loads, products and epilogues
// overlap across the tiles of a persistent block (or of a pair of blocks, whose
// tile has 256 rows and whose tensor cores each read half of the B operand).
#pragma once

#include "ops.h"
#include "tc.h"

namespace fsdp {
namespace ffn {

enum Mode { FORWARD = 0, RECOMPUTE = 1, BACKWARD = 2 };
enum Act { SILU = 0, GELU = 1 };

constexpr int kTileM = 128;  // rows of a block's tile (TMEM lanes)
constexpr int kTileK = 64;   // K values of a stage: one 128-byte swizzled row

// The tiles of one product, m x n of them.  In the order of tile_at, the first `whole`
// are units of work; the K loops of the others are in `splits` parts, each of them a unit.
struct Grid {
  int32_t m, n, whole, splits;
  int32_t raster;    // row tiles of a band (see tile_at)
  int32_t k_blocks;  // of the whole K loop
};

__host__ __device__ __forceinline__ int units_of(const Grid &g) { return g.whole + (g.m * g.n - g.whole) * g.splits; }

// Down a band of `raster` row tiles, then to the next column tile, so that the tiles at
// work at one time share few operand slices, which stay in L2.
__device__ __forceinline__ int2 tile_at(const Grid &g, int t) {
  const int band = g.raster * g.n, b = t / band, first = b * g.raster;
  const int height = min(g.m - first, g.raster), r = t - b * band;
  return make_int2(first + r % height, r / height);
}

struct Args {
  CUtensorMap a[2];   // FORWARD, RECOMPUTE: x; BACKWARD: dg, du
  CUtensorMap b[3];   // Wg, Wu; BACKWARD: also x
  uint32_t *gave_up;  // count of blocks whose waits gave up
  uint64_t wait_limit_ns;
  int32_t fault;
  int32_t act;        // Act
  int32_t turns;      // some rows go through the epilogue warps' buffers
  Grid grid[2];       // BACKWARD: weight gradients, dx; else the first only
  int32_t first, head;  // BACKWARD: whose units come first; see Walk
  int32_t a_rows;     // FORWARD, RECOMPUTE: rows of an x box (see gated())
  int32_t tile_n;     // accumulator columns of a tile (FORWARD, RECOMPUTE: half of them gate;
                      // BACKWARD: 64, 128 or 256)
  int32_t half[2];    // BACKWARD: the row tile / the K block from which on the up half is meant
  int64_t m[2], n;    // rows and columns of the outputs (FORWARD, RECOMPUTE: n = f)
  // Outputs, [m, n] with row distance ld.
  void *out[3];       // FORWARD: h; RECOMPUTE: dg, du; BACKWARD: dWg, dWu, dx
  int64_t ld_out[3];
  int32_t out_bf16[2], out_width[2];  // dtype and row_width(), by product
  float *partial[2];  // by product: [tiles with parts][splits][tile rows][tile columns] in binary32
  int32_t partial_width;  // row_width()
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

// 2^x and 1 / x of two values, to about 2 ulp, with 0 for a result below 2^-126: one
// instruction each, where functions that keep such results take four or five.
constexpr float kLog2E = 1.4426950408889634f;
__device__ __forceinline__ float2 exp2(float2 x) {
  float2 y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y.x) : "f"(x.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y.y) : "f"(x.y));
  return y;
}
__device__ __forceinline__ float2 inverse(float2 x) {
  float2 y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y.x) : "f"(x.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y.y) : "f"(x.y));
  return y;
}

// act(g) and, if SLOPE, act'(g), of two values.
//   SiLU: g s with s = 1 / (1 + e^-g);  s + g s (1 - s).  For g far below 0 the divisor
//   overflows to infinity and s is 0, as it should be.
//   GELU: g Phi(g);  Phi(g) + g phi(g), Phi the normal distribution and phi its density.
//   Phi(-x) = e^(-x^2 / 2) M(x) for x >= 0, where M falls from 1/2 like 1 / x; M is t P(t)
//   with t = 1 / (1 + 0.36 x) and P of degree 8, fitted to erfc's definition over x <= 40
//   for the least relative error, 9e-8 (4e-7 evaluated in binary32).  So the tail keeps its
//   relative precision and phi costs nothing more; one exponential, one reciprocal and
//   nine multiply-adds replace the library's distribution function, whose 60 instructions
//   bound the epilogue.
template <bool SLOPE, int ACT>
__device__ __forceinline__ void act_of(float2 g, float2 &y, float2 &slope) {
  const float2 one = both(1.0f);
  if constexpr (ACT == SILU) {
    const float2 s = inverse(__fadd2_rn(exp2(__fmul2_rn(g, both(-kLog2E))), one));
    y = __fmul2_rn(g, s);
    if constexpr (SLOPE) slope = __ffma2_rn(y, __fadd2_rn(one, make_float2(-s.x, -s.y)), s);
  } else {
    const float2 e = exp2(__fmul2_rn(__fmul2_rn(g, both(-0.5f * kLog2E)), g));
    const float2 x = __ffma2_rn(make_float2(fabsf(g.x), fabsf(g.y)), both(0.36f), one);
    const float2 t = inverse(x);
    float2 p = both(-0.0302381796f);
    p = __ffma2_rn(p, t, both(0.139508076f));
    p = __ffma2_rn(p, t, both(-0.22359911f));
    p = __ffma2_rn(p, t, both(0.107368847f));
    p = __ffma2_rn(p, t, both(-0.000386257331f));
    p = __ffma2_rn(p, t, both(0.0960373353f));
    p = __ffma2_rn(p, t, both(0.124009757f));
    p = __ffma2_rn(p, t, both(0.143681881f));
    p = __ffma2_rn(p, t, both(0.143617665f));
    const float2 tail = __fmul2_rn(__fmul2_rn(p, t), e);
    const float2 phi = make_float2(g.x < 0.0f ? tail.x : 1.0f - tail.x, g.y < 0.0f ? tail.y : 1.0f - tail.y);
    y = __fmul2_rn(g, phi);
    if constexpr (SLOPE) slope = __ffma2_rn(__fmul2_rn(g, both(0.3989422804014327f)), e, phi);
  }
}

// The forward pass of few rows (ffn_rows.cu).
struct RowsArgs {
  const void *x, *w_gate, *w_up;
  void *h;
  int64_t rows, d, f, ld_x, ld_gate, ld_up, ld_h;
  int32_t act, keep;  // as in Args
  uint8_t *codes[2], *scales[2];
  int64_t groups;
  void *kept[2];
  int64_t ld_kept;
};
constexpr int kFewRows = 4;
// When dot products beat the tiles, in us for 1 / 2 / 4 rows (the tiles take the same for
// all): 512 x 1408 2.9 / 3.2 / 4.2 to 5.0; 1024 x 4096 5.5 / 5.9 / 7.4 to 7.4; 2048 x 6144
// 11 / 12 / 17 to 13; 4096 x 12288 33 / 42 / 48 to 35.  One row always; more as long as
// rows x weights stay small, with the border where those meet.
inline bool few_rows(int64_t rows, int64_t d, int64_t f) {
  return rows == 1 || (rows <= kFewRows && rows * d * f <= int64_t(3) << 23);
}
// a.rows in 1 .. kFewRows; `vec`: d is a multiple of 8 and every row of x and the weights
// starts on a 16-byte boundary.
cudaError_t launch_rows(const RowsArgs &a, bool vec, cudaStream_t stream);

// Launch the product kernel for one use; `pair`: tiles of two blocks (256 rows).
cudaError_t launch_forward(bool pair, Args &a, int sms, cudaStream_t stream);
cudaError_t launch_recompute(bool pair, Args &a, int sms, cudaStream_t stream);
cudaError_t launch_backward(bool pair, Args &a, int sms, cudaStream_t stream);

}  // namespace ffn
}  // namespace fsdp

// Gated feed-forward block, forward, for a few rows (single tokens): both
// projections as dot products, without the tensor cores.
//
// With so few rows every weight is used once or a few times, so the bound is HBM:
// 4 d f bytes of weights.  A warp reads whole rows of both weights, 512 bytes of
// each of 8 rows (4 features, gate and up) in flight at a time, which streams better
// than the tile path's 128-byte pieces of many rows (few_rows() has both sides).
// One row through 4096 x 12288 takes 31 us: 201 MB at 6.4 TB/s, 94 % of a plain copy's
// rate.  (A second set of weights in flight spills: 44 us.)
#include "ffn.h"

namespace fsdp {
namespace ffn {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kFeatures = 4;  // of a warp; 32 of a block, a checkpoint's group

template <int ROWS, bool VEC>
__global__ void __launch_bounds__(kThreads, ROWS == 1 ? 3 : 2) rows_kernel(const __grid_constant__ RowsArgs a) {
  __shared__ float gate[ROWS][32], up[ROWS][32];
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int64_t first = (int64_t)blockIdx.x * 32 + warp * kFeatures;
  const uint16_t *w[2 * kFeatures];
#pragma unroll
  for (int i = 0; i < kFeatures; ++i) {  // features past the end read the last one again
    const int64_t row = first + i < a.f ? first + i : a.f - 1;
    w[i] = static_cast<const uint16_t *>(a.w_gate) + row * a.ld_gate;
    w[kFeatures + i] = static_cast<const uint16_t *>(a.w_up) + row * a.ld_up;
  }
  const uint16_t *x = static_cast<const uint16_t *>(a.x);
  float2 sum[ROWS][2 * kFeatures];
#pragma unroll
  for (int t = 0; t < ROWS; ++t)
#pragma unroll
    for (int i = 0; i < 2 * kFeatures; ++i) sum[t][i] = both(0.0f);
  wait_for_previous();
  let_next_start();

  if constexpr (VEC) {
#pragma unroll 1
    for (int64_t k = lane * 8; k < a.d; k += 256) {
      uint4 r[2 * kFeatures];
#pragma unroll
      for (int i = 0; i < 2 * kFeatures; ++i) r[i] = __ldcs(reinterpret_cast<const uint4 *>(w[i] + k));
      float2 v[ROWS][4];
#pragma unroll
      for (int t = 0; t < ROWS; ++t)  // rows past the end read the last one again
        unpack8(__ldg(reinterpret_cast<const uint4 *>(x + (t < a.rows ? t : a.rows - 1) * a.ld_x + k)), v[t]);
#pragma unroll
      for (int i = 0; i < 2 * kFeatures; ++i) {
        float2 q[4];
        unpack8(r[i], q);
#pragma unroll
        for (int t = 0; t < ROWS; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[t][i] = __ffma2_rn(q[e], v[t][e], sum[t][i]);
      }
    }
  } else {
#pragma unroll 2
    for (int64_t k = lane; k < a.d; k += 32) {
      float v[ROWS];
#pragma unroll
      for (int t = 0; t < ROWS; ++t) v[t] = load_any(x, (t < a.rows ? t : a.rows - 1) * a.ld_x + k, true);
#pragma unroll
      for (int i = 0; i < 2 * kFeatures; ++i) {
        const float q = load_any(w[i], k, true);
#pragma unroll
        for (int t = 0; t < ROWS; ++t) sum[t][i].x = fmaf(q, v[t], sum[t][i].x);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < ROWS; ++t)
#pragma unroll
    for (int i = 0; i < 2 * kFeatures; ++i) {
      float s = sum[t][i].x + sum[t][i].y;
#pragma unroll
      for (int m = 16; m > 0; m /= 2) s += __shfl_xor_sync(0xFFFFFFFFu, s, m);
      if (lane == 0) (i < kFeatures ? gate : up)[t][warp * kFeatures + i % kFeatures] = s;
    }
  __syncthreads();

  // One warp to a row, one feature to a lane.
  const int64_t col = (int64_t)blockIdx.x * 32 + lane;
  const bool in = col < a.f;
  for (int t = warp; t < a.rows; t += kWarps) {
    const float g = in ? gate[t][lane] : 0.0f, u = in ? up[t][lane] : 0.0f;
    float2 y, none;
    if (a.act == SILU)
      act_of<false, SILU>(both(g), y, none);
    else
      act_of<false, GELU>(both(g), y, none);
    if (in) store_any(a.h, t * a.ld_h + col, true, y.x * u);
    if (a.keep == 1) {
      const int64_t group = t * a.groups + blockIdx.x;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float v = i == 0 ? g : u;
        const uint32_t s = act8_scale_byte(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v) & 0x7FFFFFFFu));
        a.codes[i][group * kActGroup + lane] = (uint8_t)act8_code(v, s);
        if (lane == 0) a.scales[i][group] = (uint8_t)s;
      }
    } else if (a.keep == 2 && in) {
      store_any(a.kept[0], t * a.ld_kept + col, true, g);
      store_any(a.kept[1], t * a.ld_kept + col, true, u);
    }
  }
}

}  // namespace

cudaError_t launch_rows(const RowsArgs &a, bool vec, cudaStream_t stream) {
  const void *fn = a.rows == 1 ? (vec ? reinterpret_cast<const void *>(&rows_kernel<1, true>)
                                      : reinterpret_cast<const void *>(&rows_kernel<1, false>))
                   : a.rows == 2 ? (vec ? reinterpret_cast<const void *>(&rows_kernel<2, true>)
                                        : reinterpret_cast<const void *>(&rows_kernel<2, false>))
                                 : (vec ? reinterpret_cast<const void *>(&rows_kernel<kFewRows, true>)
                                        : reinterpret_cast<const void *>(&rows_kernel<kFewRows, false>));
  void *args[] = {const_cast<RowsArgs *>(&a)};
  return launch_kernel(fn, dim3((unsigned)((a.f + 31) / 32)), dim3(kThreads), args, 0, stream, true);
}

}  // namespace ffn
}  // namespace fsdp

// Layer norm, forward pass (fsdp_layer_norm_forward), with the 8-bit checkpoint
// of its input written in the same pass.
//
// Mathematics: mean and variance are two sums over values that stay in
// registers, the second over (x - mean)^2, so no cancellation costs digits.
// Bound: HBM; 2 + 2 bytes an element in BF16 (5.03 with the checkpoint) against
// about 10 operations.
#include "norm.h"

namespace fsdp {
namespace {
using namespace norm;

// XK and YB are the dtypes of x and y for vector kernels; other kernels go by the
// flags in Args.
template <int XK, bool YB, bool VEC, int G, int K, bool CLUSTER>
__global__ void __launch_bounds__(G == 32 ? 128 : G) forward_kernel(const __grid_constant__ Args a) {
  constexpr int NT = G == 32 ? 128 : G, RG = NT / G;
  __shared__ Slots slots;
  int turn = 0;
  const int t = threadIdx.x % G, cols = (int)a.cols;
  int base = 0;
  int64_t unit = blockIdx.x, units = gridDim.x;
  if constexpr (CLUSTER) {
    namespace cg = cooperative_groups;
    base = (int)cg::this_cluster().block_rank() * (G * K * 8);
    unit /= cg::this_cluster().num_blocks();
    units /= cg::this_cluster().num_blocks();
  }
  const bool y_bf16 = VEC ? YB : a.y_bf16 != 0;
  wait_for_previous();
  let_next_start();

  int64_t row = unit * RG + threadIdx.x / G;
  const int64_t step = units * RG;
  Raw<XK, VEC, K> raw;
  if (row < a.rows) load_row<XK, VEC, G, K>(raw, a.x, a.x_scales, a.x_kind, row, a.ld_x, a.groups, cols, base, t);
  float w[K][8], b[K][8];
  load_param<VEC, G, K>(w, a.weight, a.param_bf16 != 0, 1.0f, cols, base, t);
  load_param<VEC, G, K>(b, a.bias, a.param_bf16 != 0, 0.0f, cols, base, t);

  for (; row < a.rows; row += step) {
    float v[K][8];
    unpack_row<XK, VEC, K>(raw, v);
    if (row + step < a.rows)
      load_row<XK, VEC, G, K>(raw, a.x, a.x_scales, a.x_kind, row + step, a.ld_x, a.groups, cols, base, t);

    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) s.x += v[k][e];
    const float mean = row_sum<G, CLUSTER>(s, slots, turn).x * a.inv_cols;

    if (a.keep) {  // the checkpoint of the row, from the values as they were read
      uint8_t *codes = a.keep + row * a.groups * kActGroup;
      const int end = (int)(a.groups * kActGroup);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if constexpr (VEC) {
          uint32_t top = 0;
#pragma unroll
          for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[k][e]) & 0x7FFFFFFFu);
          top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
          top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
          const uint32_t sb = act8_scale_byte(top);
          const int j = column<VEC, G>(base, t, k, 0);
          if (j < end) {
            *reinterpret_cast<uint2 *>(codes + j) =
                make_uint2(act8_code4(v[k][0], v[k][1], v[k][2], v[k][3], sb),
                           act8_code4(v[k][4], v[k][5], v[k][6], v[k][7], sb));
            if (t % 4 == 0) a.keep_scales[row * a.groups + j / (int)kActGroup] = (uint8_t)sb;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t sb = act8_scale_byte(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v[k][e]) & 0x7FFFFFFFu));
            const int j = column<VEC, G>(base, t, k, e);
            if (j < end) {
              codes[j] = (uint8_t)act8_code(v[k][e], sb);
              if (t % 32 == 0) a.keep_scales[row * a.groups + j / (int)kActGroup] = (uint8_t)sb;
            }
          }
        }
      }
    }

    s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[k][e] -= mean;
        if (column<VEC, G>(base, t, k, e) < cols) s.x = fmaf(v[k][e], v[k][e], s.x);
      }
    const float rstd = rsqrtf(fmaf(row_sum<G, CLUSTER>(s, slots, turn).x, a.inv_cols, a.eps));
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[k][e] = fmaf(v[k][e] * rstd, w[k][e], b[k][e]);
    store_row<VEC, G, K>(v, a.y, y_bf16, row * a.ld_y, cols, base, t);
    if (t == 0 && base == 0 && a.mean) a.mean[row] = mean, a.rstd[row] = rstd;
  }
  // No block of a cluster leaves while another may still write to its slots.
  if constexpr (CLUSTER) cooperative_groups::this_cluster().sync();
}

template <int XK, bool YB>
const void *vector_kernel(int index) {
  switch (index) {
    case 0: return reinterpret_cast<const void *>(&forward_kernel<XK, YB, true, 32, 2, false>);
    case 1: return reinterpret_cast<const void *>(&forward_kernel<XK, YB, true, 128, 1, false>);
    case 2: return reinterpret_cast<const void *>(&forward_kernel<XK, YB, true, 256, 1, false>);
    case 3: return reinterpret_cast<const void *>(&forward_kernel<XK, YB, true, 256, 2, false>);
    case 4: return reinterpret_cast<const void *>(&forward_kernel<XK, YB, true, 512, 2, false>);
    default: return reinterpret_cast<const void *>(&forward_kernel<XK, YB, true, 512, 2, true>);
  }
}

const void *kernel_for(const Shape &s, bool vec, int kind, bool y_bf16) {
  if (!vec) {
    switch (s.index) {
      case 0: return reinterpret_cast<const void *>(&forward_kernel<X_F32, false, false, 32, 2, false>);
      case 1: return reinterpret_cast<const void *>(&forward_kernel<X_F32, false, false, 128, 2, false>);
      case 4: return reinterpret_cast<const void *>(&forward_kernel<X_F32, false, false, 512, 2, false>);
      default: return reinterpret_cast<const void *>(&forward_kernel<X_F32, false, false, 512, 2, true>);
    }
  }
  switch (kind) {
    case X_F32: return y_bf16 ? vector_kernel<X_F32, true>(s.index) : vector_kernel<X_F32, false>(s.index);
    case X_BF16: return y_bf16 ? vector_kernel<X_BF16, true>(s.index) : vector_kernel<X_BF16, false>(s.index);
    default: return y_bf16 ? vector_kernel<X_ACT8, true>(s.index) : vector_kernel<X_ACT8, false>(s.index);
  }
}

}  // namespace
}  // namespace fsdp

using namespace fsdp;

extern "C" fsdp_status_t fsdp_layer_norm_forward(const fsdp_norm_desc_t *d, const void *x, const void *weight,
                                                 const void *bias, void *y, float *mean, float *rstd, void *keep,
                                                 fsdp_stream_t stream) {
  fsdp_status_t st = check_desc(d);
  if (st != FSDP_OK) return st;
  if (!float_dtype(d->y_dtype)) return fail(FSDP_EINVAL, "unknown y_dtype");
  const bool act8 = d->x_dtype == FSDP_ACT8;
  const int64_t ysize = dtype_bytes(d->y_dtype), psize = dtype_bytes(d->param_dtype);
  if (act8)
    st = check_ptr(x, act8_bytes(d->rows, d->cols), 16, "x", -1);
  else
    st = check_matrix(x, d->rows, d->cols, d->ld_x, dtype_bytes(d->x_dtype), "x");
  if (st != FSDP_OK) return st;
  if ((st = check_matrix(y, d->rows, d->cols, d->ld_y, ysize, "y")) != FSDP_OK) return st;
  if (weight && (st = check_ptr(weight, d->cols * psize, psize, "weight", -1)) != FSDP_OK) return st;
  if (bias && (st = check_ptr(bias, d->cols * psize, psize, "bias", -1)) != FSDP_OK) return st;
  if (!mean != !rstd) return fail(FSDP_EINVAL, "mean and rstd are given together or not at all");
  if (mean && ((st = check_ptr(mean, 4, 4, "mean", -1)) != FSDP_OK || (st = check_ptr(rstd, 4, 4, "rstd", -1)) != FSDP_OK))
    return st;
  if (keep && act8) return fail(FSDP_EINVAL, "keep: x is a checkpoint already");
  if (keep && (st = check_ptr(keep, 1, 16, "keep", -1)) != FSDP_OK) return st;
  if (d->rows == 0) {
    clear_error();
    return FSDP_OK;
  }
  Args a = {};
  a.rows = d->rows, a.cols = d->cols, a.ld_x = d->ld_x, a.ld_y = d->ld_y;
  a.groups = act8_groups(d->cols);
  a.x = x;
  a.x_kind = act8 ? X_ACT8 : d->x_dtype == FSDP_DTYPE_BF16 ? X_BF16 : X_F32;
  if (act8) a.x_scales = static_cast<const uint8_t *>(x) + d->rows * a.groups * kActGroup;
  a.weight = weight, a.bias = bias, a.y = y, a.mean = mean, a.rstd = rstd;
  a.keep = static_cast<uint8_t *>(keep);
  if (keep) a.keep_scales = a.keep + d->rows * a.groups * kActGroup;
  a.y_bf16 = d->y_dtype == FSDP_DTYPE_BF16;
  a.param_bf16 = d->param_dtype == FSDP_DTYPE_BF16;
  a.eps = d->eps;
  a.inv_cols = 1.0f / (float)d->cols;
  auto rows_aligned = [&](const void *p, int64_t ld, int64_t size) {
    return aligned16(p) && (d->rows == 1 || ld * size % 16 == 0);
  };
  const bool vec = d->cols % 8 == 0 && (act8 || rows_aligned(x, d->ld_x, dtype_bytes(d->x_dtype))) &&
                   rows_aligned(y, d->ld_y, ysize) && aligned16(weight) && aligned16(bias);
  const Shape s = shape_of(d->cols, vec);
  const int sms = device_sms();
  const int64_t rows_per_block = s.threads / s.group;
  // As many blocks as are resident (1,024 threads an SM), each then takes its rows in turn.
  int64_t units = (d->rows + rows_per_block - 1) / rows_per_block;
  const int64_t most = (int64_t)(sms > 0 ? sms : 1) * (1024 / s.threads) / s.cluster;
  if (units > most) units = most > 0 ? most : 1;
  void *args[] = {&a};
  st = launched(launch_kernel(kernel_for(s, vec, a.x_kind, a.y_bf16 != 0), dim3((unsigned)(units * s.cluster)),
                              dim3((unsigned)s.threads), args, 0, reinterpret_cast<cudaStream_t>(stream), true, s.cluster));
  if (st != FSDP_OK) return st;
  clear_error();
  return FSDP_OK;
}

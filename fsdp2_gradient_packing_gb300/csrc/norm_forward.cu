// Layer norm, forward pass (fsdp_layer_norm_forward), with the 8-bit checkpoint
// of its input written in the same pass.
//
// Mathematics: mean and variance are two sums over values that stay in
// registers, the second over (x - mean)^2, so no cancellation costs digits.
// Bound: HBM; 2 + 2 bytes an element in BF16 (5.03 with the checkpoint) against
// about 10 operations, 18 instructions issued.  16384 x 4096 in BF16 takes 50.9 us
// (5.3 TB/s), with the checkpoint 60.7 (5.6 TB/s), from the checkpoint 40.5 (5.0 TB/s);
// 8192 x 4096 in FP32 47.3 (5.7 TB/s); 16385 x 1409 in BF16, element by element, 34.2
// (2.7 TB/s).
#include "norm.h"

namespace fsdp {
namespace {
using namespace norm;

constexpr int kMostThreads = 768;  // of a block beside its loading warp, at 80 registers

// XK and YB are the dtypes of x and y for vector kernels; other kernels go by the
// flags in Args.
template <int XK, bool YB, bool VEC, int G, int K, bool CLUSTER>
__global__ void __launch_bounds__(kMostThreads + 32, 1) forward_kernel(const __grid_constant__ Args a) {
  __shared__ Shared sh;
  extern __shared__ __align__(16) uint8_t memory[];
  float *const weight = reinterpret_cast<float *>(memory), *const bias = weight + G * K * 8;
  const int group = threadIdx.x / G, groups = (blockDim.x - 32) / G, t = threadIdx.x % G, cols = (int)a.cols;
  int turn = 0, base = 0;
  int64_t unit = blockIdx.x, units = gridDim.x;
  if constexpr (CLUSTER) {
    base = (int)tc::cluster_rank() * (G * K * 8);
    unit /= cluster_blocks();
    units /= cluster_blocks();
  }
  const bool y_bf16 = VEC ? YB : a.y_bf16 != 0;
  Ring<G, K> ring(a, sh, memory + 2 * G * K * 8 * sizeof(float), group, base);
  begin_block<CLUSTER>(sh, groups, a.stages, 1);
  wait_for_previous();
  let_next_start();
  int64_t row = unit * groups + group;
  const int64_t step = units * groups;
  stage_param<VEC, G, K>(weight, a.weight, a.param_bf16 != 0, 1.0f, cols, base);
  stage_param<VEC, G, K>(bias, a.bias, a.param_bf16 != 0, 0.0f, cols, base);
  __syncthreads();
  const bool loads = (int)threadIdx.x >= groups * G;
  if (loads) load_rows<G, K>(a, sh, memory + 2 * G * K * 8 * sizeof(float), groups, base, unit * groups, step);

  const int mine = columns_of<VEC, G, K>(ring.width, t);
  // Where the row's results go, advanced from row to row.
  const int y_size = y_bf16 ? 2 : 4, end = (int)(a.groups * kActGroup) - base;
  uint8_t *y = static_cast<uint8_t *>(a.y) + (row * a.ld_y + base) * y_size;
  uint8_t *codes = a.keep + row * a.groups * kActGroup + base, *scales = a.keep_scales + row * a.groups + base / (int)kActGroup;
  const int64_t y_step = step * a.ld_y * y_size, code_step = step * a.groups * kActGroup, scale_step = step * a.groups;

  for (; !loads && row < a.rows; row += step, y += y_step, codes += code_step, scales += scale_step) {
    float2 v[K][4];
    float unit[K];
    ring.wait();
    read_row<XK, VEC, G, K>(v, unit, ring.data(0, row, VEC), ring.data(1, row, false), a.x_kind, mine, t, sh.zeros);
    float2 sum = both(0.0f);
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (VEC && XK == X_ACT8) v[k][e] = __fmul2_rn(v[k][e], both(unit[k]));
        sum = __fadd2_rn(sum, v[k][e]);
      }
    float s[1] = {sum.x + sum.y};
    row_sum<1, G, CLUSTER>(s, sh, turn, group, a.wait_limit_ns);
    if (t == 0) ring.release();
    ring.next();
    const float mean = s[0] * a.inv_cols;

    if (a.keep) {  // the checkpoint of the row, from the values as they were read
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if constexpr (VEC) {
          uint32_t top = act8_top(v[k]);
          top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
          top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
          const uint32_t sb = act8_scale_byte(top);
          const int j = column<VEC, G>(0, t, k, 0);
          if (j < end) {
            act8_store<8>(codes + j, v[k], sb);
            if (t % 4 == 0) scales[j / (int)kActGroup] = (uint8_t)sb;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t sb = act8_scale_byte(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(element(v[k], e)) & 0x7FFFFFFFu));
            const int j = column<VEC, G>(0, t, k, e);
            if (j < end) {
              codes[j] = (uint8_t)act8_code(element(v[k], e), sb);
              if (t % 32 == 0) scales[j / (int)kActGroup] = (uint8_t)sb;
            }
          }
        }
      }
    }

    sum = both(0.0f);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (VEC && k >= mine) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[k][e] = __fadd2_rn(v[k][e], both(-mean));
        if (!VEC && k * 8 + 2 * e >= mine) v[k][e].x = 0.0f;
        if (!VEC && k * 8 + 2 * e + 1 >= mine) v[k][e].y = 0.0f;
        sum = __ffma2_rn(v[k][e], v[k][e], sum);
      }
    }
    s[0] = sum.x + sum.y;
    row_sum<1, G, CLUSTER>(s, sh, turn, group, a.wait_limit_ns);
    const float rstd = rsqrtf(fmaf(s[0], a.inv_cols, a.eps));
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float2 w[4], b[4];
      read_param<VEC, G, K>(w, weight, t, k);
      read_param<VEC, G, K>(b, bias, t, k);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[k][e] = __ffma2_rn(__fmul2_rn(v[k][e], both(rstd)), w[e], b[e]);
    }
    store_row<VEC, G, K>(v, y, y_bf16, mine, t);
    if (t == 0 && base == 0 && a.mean) a.mean[row] = mean, a.rstd[row] = rstd;
  }
  // No block of a cluster leaves while another may still write to its slots.
  if constexpr (CLUSTER) {
    __syncwarp();
    tc::cluster_sync();
  }
  end_block(sh, a);
}

// The narrowest shape that holds a row.  Each thread has up to 32 columns: what a row
// costs beside its columns (waits, two sums over the threads, addresses) is about 170
// instructions a warp, as much as 16 columns cost, and these kernels are bound by what
// they issue (67 us with 256 threads x 16 columns at 16384 x 4096 in BF16 with the
// checkpoint kept, where HBM allows 50).
//   columns <=  512   one warp, 2 chunks     <= 1024   one warp, 4 chunks
//           <= 4096   128 threads, 4 chunks (2 up to 2048)
//           <= 8192   256 threads, 4 chunks; above: clusters of 2, 4 or 8 such blocks
Shape shape_of(int64_t cols) {
  if (cols <= 512) return {32, 2, 1, 0};
  if (cols <= 1024) return {32, 4, 1, 1};
  if (cols <= 2048) return {128, 2, 1, 2};
  if (cols <= 4096) return {128, 4, 1, 3};
  const int cluster = cluster_of(cols, 8192);
  return {256, 4, cluster, cluster > 1 ? 5 : 4};
}

template <int XK, bool YB, bool VEC>
const void *kernel_of(int index) {
  switch (index) {
    case 0: return reinterpret_cast<const void *>(&forward_kernel<XK, YB, VEC, 32, 2, false>);
    case 1: return reinterpret_cast<const void *>(&forward_kernel<XK, YB, VEC, 32, 4, false>);
    case 2: return reinterpret_cast<const void *>(&forward_kernel<XK, YB, VEC, 128, 2, false>);
    case 3: return reinterpret_cast<const void *>(&forward_kernel<XK, YB, VEC, 128, 4, false>);
    case 4: return reinterpret_cast<const void *>(&forward_kernel<XK, YB, VEC, 256, 4, false>);
    default: return reinterpret_cast<const void *>(&forward_kernel<XK, YB, VEC, 256, 4, true>);
  }
}

const void *kernel_for(int index, bool vec, int kind, bool y_bf16) {
  if (!vec) return kernel_of<X_F32, false, false>(index);
  switch (kind) {
    case X_F32: return y_bf16 ? kernel_of<X_F32, true, true>(index) : kernel_of<X_F32, false, true>(index);
    case X_BF16: return y_bf16 ? kernel_of<X_BF16, true, true>(index) : kernel_of<X_BF16, false, true>(index);
    default: return y_bf16 ? kernel_of<X_ACT8, true, true>(index) : kernel_of<X_ACT8, false, true>(index);
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
  a.rows = d->rows, a.cols = d->cols, a.ld_y = d->ld_y;
  set_x(a, d, x);
  a.weight = weight, a.bias = bias, a.y = y, a.mean = mean, a.rstd = rstd;
  a.keep = static_cast<uint8_t *>(keep);
  if (keep) a.keep_scales = a.keep + d->rows * a.groups * kActGroup;
  a.y_bf16 = d->y_dtype == FSDP_DTYPE_BF16;
  a.param_bf16 = d->param_dtype == FSDP_DTYPE_BF16;
  a.eps = d->eps;
  a.inv_cols = 1.0f / (float)d->cols;
  const bool vec = d->cols % 8 == 0 && (act8 || rows_aligned(x, d->rows, d->ld_x, dtype_bytes(d->x_dtype))) &&
                   rows_aligned(y, d->rows, d->ld_y, ysize) && aligned16(weight) && aligned16(bias);
  const Shape s = shape_of(d->cols);
  const int sms = device_sms();
  const Launch l = plan_launch(a, s, sms > 0 ? sms : 1, kMostThreads, 0, 2, 0);
  if ((st = run(kernel_for(s.index, vec, a.x_kind, a.y_bf16 != 0), a, l, s, 32, reinterpret_cast<cudaStream_t>(stream))) != FSDP_OK)
    return st;
  clear_error();
  return FSDP_OK;
}

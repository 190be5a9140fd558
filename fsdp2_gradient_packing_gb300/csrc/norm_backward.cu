// Layer norm, backward pass (fsdp_layer_norm_backward), from x or from its 8-bit
// checkpoint, with the weight's and bias's gradients.
//
// Mathematics: with g = dy * weight, dx needs the row's sums of g and g * xh,
// which one reduction gives together; the parameter gradients are column sums.
// A block keeps the column sums of its own rows in registers and writes them
// once, [units][2][cols] in binary32; a second kernel adds the units in order.
// Bound: HBM; 2 + 2 + 2 bytes an element in BF16 (5.03 from the checkpoint).
#include "norm.h"

namespace fsdp {
namespace {
using namespace norm;

template <int XK, bool YB, bool VEC, int G, int K, bool CLUSTER>
__global__ void __launch_bounds__(G == 32 ? 128 : G) backward_kernel(const __grid_constant__ Args a) {
  constexpr int NT = G == 32 ? 128 : G, RG = NT / G;
  constexpr int DK = YB ? X_BF16 : X_F32;
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
  wait_for_previous();

  int64_t row = unit * RG + threadIdx.x / G;
  const int64_t step = units * RG;
  Raw<XK, VEC, K> raw_x;
  Raw<DK, VEC, K> raw_dy;
  const int dy_kind = a.y_bf16 ? X_BF16 : X_F32;
  float mean = 0.0f, rstd = 0.0f;
  if (row < a.rows) {
    load_row<XK, VEC, G, K>(raw_x, a.x, a.x_scales, a.x_kind, row, a.ld_x, a.groups, cols, base, t);
    load_row<DK, VEC, G, K>(raw_dy, a.dy, nullptr, dy_kind, row, a.ld_y, 0, cols, base, t);
    mean = a.mean[row], rstd = a.rstd[row];
  }
  float w[K][8], dw[K][8], db[K][8];
  load_param<VEC, G, K>(w, a.weight, a.param_bf16 != 0, 1.0f, cols, base, t);
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[k][e] = db[k][e] = 0.0f;

  for (; row < a.rows; row += step) {
    float xh[K][8], g[K][8];
    unpack_row<XK, VEC, K>(raw_x, xh);
    unpack_row<DK, VEC, K>(raw_dy, g);
    const float r = rstd, m = mean;
    if (row + step < a.rows) {
      load_row<XK, VEC, G, K>(raw_x, a.x, a.x_scales, a.x_kind, row + step, a.ld_x, a.groups, cols, base, t);
      load_row<DK, VEC, G, K>(raw_dy, a.dy, nullptr, dy_kind, row + step, a.ld_y, 0, cols, base, t);
      mean = a.mean[row + step], rstd = a.rstd[row + step];
    }
    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        xh[k][e] = (xh[k][e] - m) * r;
        db[k][e] += g[k][e];
        dw[k][e] = fmaf(g[k][e], xh[k][e], dw[k][e]);
        g[k][e] *= w[k][e];
        s.x += g[k][e];
        s.y = fmaf(g[k][e], xh[k][e], s.y);
      }
    if (a.dx) {
      s = row_sum<G, CLUSTER>(s, slots, turn);
      const float c2 = s.x * a.inv_cols, c1 = s.y * a.inv_cols;
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) g[k][e] = (g[k][e] - c2 - xh[k][e] * c1) * r;
      store_row<VEC, G, K>(g, a.dx, a.dx_bf16 != 0, row * a.ld_dx, cols, base, t);
    }
  }
  let_next_start();

  // Column sums of the block's row groups, added in order.
  if constexpr (RG > 1) {
    __shared__ float column_sum[2][G * K * 8];
    for (int q = 0; q < RG; ++q) {
      if ((int)threadIdx.x / G == q) {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int j = column<VEC, G>(0, t, k, e);
            if (q > 0) dw[k][e] += column_sum[0][j], db[k][e] += column_sum[1][j];
            if (q < RG - 1) column_sum[0][j] = dw[k][e], column_sum[1][j] = db[k][e];
          }
      }
      __syncthreads();
    }
  }
  if ((int)threadIdx.x / G == RG - 1) {
    if (a.partial) {
      store_row<VEC, G, K>(dw, a.partial, false, unit * 2 * a.cols, cols, base, t);
      store_row<VEC, G, K>(db, a.partial, false, (unit * 2 + 1) * a.cols, cols, base, t);
    } else {  // one unit: its sums are the gradients
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int j = column<VEC, G>(base, t, k, e);
          if (j < cols && a.dweight) store_any(a.dweight, j, a.grad_bf16 != 0, dw[k][e]);
          if (j < cols && a.dbias) store_any(a.dbias, j, a.grad_bf16 != 0, db[k][e]);
        }
    }
  }
  if constexpr (CLUSTER) cooperative_groups::this_cluster().sync();
}

// dweight | dbias [cols] from partial [units][2][cols]: 32 columns of one of the
// two to a block, its 8 warps each adding every eighth unit, then the warps' sums
// in order.
constexpr int kSumThreads = 256;

__global__ void __launch_bounds__(kSumThreads) column_sum_kernel(const float *partial, int64_t units, int64_t cols,
                                                                 void *dweight, void *dbias, int32_t bf16) {
  __shared__ float part[kSumThreads / 32][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int64_t j = (int64_t)blockIdx.x * 32 + lane;
  void *out = blockIdx.y == 0 ? dweight : dbias;
  wait_for_previous();
  let_next_start();
  if (!out) return;
  float s = 0.0f;
  if (j < cols) {
    const float *p = partial + (int64_t)blockIdx.y * cols + j;
#pragma unroll 8
    for (int64_t u = warp; u < units; u += kSumThreads / 32) s += p[u * 2 * cols];
  }
  part[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && j < cols) {
#pragma unroll
    for (int w = 1; w < kSumThreads / 32; ++w) s += part[w][lane];
    store_any(out, j, bf16 != 0, s);
  }
}

template <int XK, bool YB>
const void *vector_kernel(int index) {
  switch (index) {
    case 0: return reinterpret_cast<const void *>(&backward_kernel<XK, YB, true, 32, 2, false>);
    case 1: return reinterpret_cast<const void *>(&backward_kernel<XK, YB, true, 128, 1, false>);
    case 2: return reinterpret_cast<const void *>(&backward_kernel<XK, YB, true, 256, 1, false>);
    case 3: return reinterpret_cast<const void *>(&backward_kernel<XK, YB, true, 256, 2, false>);
    case 4: return reinterpret_cast<const void *>(&backward_kernel<XK, YB, true, 512, 2, false>);
    default: return reinterpret_cast<const void *>(&backward_kernel<XK, YB, true, 512, 2, true>);
  }
}

const void *kernel_for(const Shape &s, bool vec, int kind, bool y_bf16) {
  if (!vec) {
    switch (s.index) {
      case 0: return reinterpret_cast<const void *>(&backward_kernel<X_F32, false, false, 32, 2, false>);
      case 1: return reinterpret_cast<const void *>(&backward_kernel<X_F32, false, false, 128, 2, false>);
      case 4: return reinterpret_cast<const void *>(&backward_kernel<X_F32, false, false, 512, 2, false>);
      default: return reinterpret_cast<const void *>(&backward_kernel<X_F32, false, false, 512, 2, true>);
    }
  }
  switch (kind) {
    case X_F32: return y_bf16 ? vector_kernel<X_F32, true>(s.index) : vector_kernel<X_F32, false>(s.index);
    case X_BF16: return y_bf16 ? vector_kernel<X_BF16, true>(s.index) : vector_kernel<X_BF16, false>(s.index);
    default: return y_bf16 ? vector_kernel<X_ACT8, true>(s.index) : vector_kernel<X_ACT8, false>(s.index);
  }
}

// Units (blocks or clusters) of a call: as many as are resident, about 512
// threads an SM.  An upper bound over both kinds of kernel serves the workspace.
int64_t units_for(int64_t rows, const Shape &s, int sms) {
  const int64_t per_block = s.threads / s.group;
  const int64_t need = (rows + per_block - 1) / per_block;
  int64_t most = (int64_t)sms * (512 / s.threads) / s.cluster;
  if (most < 1) most = 1;
  return need < most ? need : most;
}

int64_t workspace_bytes_for(const fsdp_norm_desc_t *d) {
  const int sms = device_sms() > 0 ? device_sms() : 256;
  int64_t units = 0;
  for (int vec = 0; vec < 2; ++vec) {
    const int64_t n = units_for(d->rows, shape_of(d->cols, vec != 0), sms);
    if (n > units) units = n;
  }
  return units * 2 * d->cols * 4;
}

}  // namespace
}  // namespace fsdp

using namespace fsdp;

extern "C" {

fsdp_status_t fsdp_layer_norm_workspace(const fsdp_norm_desc_t *d, int64_t *bytes) {
  fsdp_status_t st = check_desc(d);
  if (st != FSDP_OK) return st;
  if (!bytes) return fail(FSDP_EINVAL, "bytes is NULL");
  *bytes = workspace_bytes_for(d);
  clear_error();
  return FSDP_OK;
}

fsdp_status_t fsdp_layer_norm_backward(const fsdp_norm_desc_t *d, const void *dy, const void *x, const void *weight,
                                       const float *mean, const float *rstd, void *dx, void *dweight, void *dbias,
                                       void *workspace, int64_t workspace_bytes, fsdp_stream_t stream) {
  fsdp_status_t st = check_desc(d);
  if (st != FSDP_OK) return st;
  if (!float_dtype(d->y_dtype)) return fail(FSDP_EINVAL, "unknown y_dtype");
  if (dx && !float_dtype(d->dx_dtype)) return fail(FSDP_EINVAL, "unknown dx_dtype");
  if ((dweight || dbias) && !float_dtype(d->grad_dtype)) return fail(FSDP_EINVAL, "unknown grad_dtype");
  const bool act8 = d->x_dtype == FSDP_ACT8;
  const int64_t ysize = dtype_bytes(d->y_dtype), psize = dtype_bytes(d->param_dtype);
  if ((st = check_matrix(dy, d->rows, d->cols, d->ld_y, ysize, "dy")) != FSDP_OK) return st;
  if (act8)
    st = check_ptr(x, act8_bytes(d->rows, d->cols), 16, "x", -1);
  else
    st = check_matrix(x, d->rows, d->cols, d->ld_x, dtype_bytes(d->x_dtype), "x");
  if (st != FSDP_OK) return st;
  if (weight && (st = check_ptr(weight, d->cols * psize, psize, "weight", -1)) != FSDP_OK) return st;
  if ((st = check_ptr(mean, d->rows * 4, 4, "mean", -1)) != FSDP_OK) return st;
  if ((st = check_ptr(rstd, d->rows * 4, 4, "rstd", -1)) != FSDP_OK) return st;
  const int64_t dxsize = dx ? dtype_bytes(d->dx_dtype) : 4;
  if (dx && (st = check_matrix(dx, d->rows, d->cols, d->ld_dx, dxsize, "dx")) != FSDP_OK) return st;
  const int64_t gsize = dweight || dbias ? dtype_bytes(d->grad_dtype) : 4;
  if (dweight && (st = check_ptr(dweight, d->cols * gsize, gsize, "dweight", -1)) != FSDP_OK) return st;
  if (dbias && (st = check_ptr(dbias, d->cols * gsize, gsize, "dbias", -1)) != FSDP_OK) return st;
  const int64_t need = workspace_bytes_for(d);
  if (workspace_bytes < need) return fail(FSDP_EINVAL, "workspace_bytes is below fsdp_layer_norm_workspace");
  if ((st = check_ptr(workspace, need, 16, "workspace", -1)) != FSDP_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (d->rows == 0 || (!dx && !dweight && !dbias)) {
    for (void *p : {dweight, dbias})
      if (p) {
        cudaError_t e = cudaMemsetAsync(p, 0, (size_t)(d->cols * gsize), s);
        if (e != cudaSuccess) return fail(FSDP_ECUDA, std::string("cudaMemsetAsync: ") + cudaGetErrorString(e));
      }
    clear_error();
    return FSDP_OK;
  }
  Args a = {};
  a.rows = d->rows, a.cols = d->cols, a.ld_x = d->ld_x, a.ld_y = d->ld_y, a.ld_dx = d->ld_dx;
  a.groups = act8_groups(d->cols);
  a.x = x;
  a.x_kind = act8 ? X_ACT8 : d->x_dtype == FSDP_DTYPE_BF16 ? X_BF16 : X_F32;
  if (act8) a.x_scales = static_cast<const uint8_t *>(x) + d->rows * a.groups * kActGroup;
  a.weight = weight, a.dy = dy, a.dx = dx, a.dweight = dweight, a.dbias = dbias;
  a.mean = const_cast<float *>(mean), a.rstd = const_cast<float *>(rstd);
  a.y_bf16 = d->y_dtype == FSDP_DTYPE_BF16;
  a.dx_bf16 = dx && d->dx_dtype == FSDP_DTYPE_BF16;
  a.param_bf16 = d->param_dtype == FSDP_DTYPE_BF16;
  a.grad_bf16 = gsize == 2;
  a.inv_cols = 1.0f / (float)d->cols;
  auto rows_aligned = [&](const void *p, int64_t ld, int64_t size) {
    return aligned16(p) && (d->rows == 1 || ld * size % 16 == 0);
  };
  const bool vec = d->cols % 8 == 0 && (act8 || rows_aligned(x, d->ld_x, dtype_bytes(d->x_dtype))) &&
                   rows_aligned(dy, d->ld_y, ysize) && (!dx || rows_aligned(dx, d->ld_dx, dxsize)) && aligned16(weight);
  const Shape sh = shape_of(d->cols, vec);
  const int sms = device_sms();
  const int64_t units = units_for(d->rows, sh, sms > 0 ? sms : 1);
  a.partial = units > 1 ? static_cast<float *>(workspace) : nullptr;
  void *args[] = {&a};
  st = launched(launch_kernel(kernel_for(sh, vec, a.x_kind, a.y_bf16 != 0), dim3((unsigned)(units * sh.cluster)),
                              dim3((unsigned)sh.threads), args, 0, s, true, sh.cluster));
  if (st != FSDP_OK) return st;
  if (a.partial && (dweight || dbias)) {
    const float *partial = a.partial;
    int64_t n = units, cols = d->cols;
    int32_t bf16 = a.grad_bf16;
    void *sum_args[] = {&partial, &n, &cols, &dweight, &dbias, &bf16};
    st = launched(launch_kernel(reinterpret_cast<const void *>(&column_sum_kernel), dim3((unsigned)((cols + 31) / 32), 2),
                                dim3(kSumThreads), sum_args, 0, s, true));
    if (st != FSDP_OK) return st;
  }
  clear_error();
  return FSDP_OK;
}

}  // extern "C"

// Layer norm, backward pass (fsdp_layer_norm_backward), from x or from its 8-bit
// checkpoint, with the weight's and bias's gradients.
//
// Mathematics: with g = dy * weight, dx needs the row's sums of g and g * xh,
// which one reduction gives together; the parameter gradients are column sums.
// A block keeps the column sums of its own rows in registers and writes them
// once, [units][2][cols] in binary32; a second kernel adds the units in order.
// Bound: HBM; 2 + 2 + 2 bytes an element in BF16 (5.03 from the checkpoint); what is
// left above it is the latency of a row's sum, which a block hides behind one or two
// more rows.  16384 x 4096 in BF16 takes 69.7 us with its column sums (5.8 TB/s), from
// the checkpoint 67.0 (5.1 TB/s); 8192 x 4096 in FP32 69.3 (5.8 TB/s); 16385 x 1409 in
// FP32, element by element, 52.3 (5.3 TB/s).
#include <algorithm>

#include "norm.h"

namespace fsdp {
namespace {
using namespace norm;

// Threads of a block at most.  A thread's column sums and its values of a row take 128
// registers at 4 chunks, 64 at 2.  (A third group of 128 threads leaves 168 registers and
// spills: 16384 x 4096 takes 91 us from BF16 with it, 70 without; the smallest kernel, from
// the checkpoint, 64.6 and 66.3, but 32768 x 1024 43 and 39.)
constexpr int most_threads(int chunks, bool vec) { return chunks <= 2 ? 512 : vec ? 256 : 384; }
// Up to so many rows a group, one block does them all: its sums are the gradients, and
// neither the second kernel (3 us and as much on the host) nor a workspace is needed.
constexpr int kRowsEach = 4;

template <int XK, bool YB, bool VEC, int G, int K, bool CLUSTER>
__global__ void __launch_bounds__(most_threads(K, VEC), 1) backward_kernel(const __grid_constant__ Args a) {
  constexpr int DK = YB ? X_BF16 : X_F32;
  __shared__ Shared sh;
  extern __shared__ __align__(16) uint8_t memory[];
  float *const weight = reinterpret_cast<float *>(memory);
  uint8_t *const stages = memory + G * K * 8 * sizeof(float);
  const int group = threadIdx.x / G, groups = blockDim.x / G, t = threadIdx.x % G, cols = (int)a.cols;
  int turn = 0, base = 0;
  int64_t unit = blockIdx.x, units = gridDim.x;
  if constexpr (CLUSTER) {
    base = (int)tc::cluster_rank() * (G * K * 8);
    unit /= cluster_blocks();
    units /= cluster_blocks();
  }
  Ring<G, K> ring(a, sh, stages, group, base);
  begin_block<CLUSTER>(sh, groups, a.stages, ring.width > 0 ? 2 + (a.in[1].at >= 0) : 1);
  wait_for_previous();
  int64_t row = unit * groups + group;
  const int64_t step = units * groups;
  const int dy_kind = a.y_bf16 ? X_BF16 : X_F32;
  float mean = 0.0f, rstd = 0.0f;
  if (row < a.rows) mean = a.mean[row], rstd = a.rstd[row];
  stage_param<VEC, G, K>(weight, a.weight, a.param_bf16 != 0, 1.0f, cols, base);
  float2 dw[K][4], db[K][4];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int e = 0; e < 4; ++e) dw[k][e] = db[k][e] = both(0.0f);
  __syncthreads();
  Filler<G, K> filler(a, sh, stages, group, base, row, step);
  for (int i = 0; i < a.stages; ++i)
    if (row + i * step < a.rows) filler.fill(a, i, i == 0 && skips_first(a, group));

  const int mine = columns_of<VEC, G, K>(ring.width, t);
  const int dx_size = a.dx_bf16 ? 2 : 4;
  uint8_t *dx = static_cast<uint8_t *>(a.dx) + (row * a.ld_dx + base) * dx_size;
  const int64_t dx_step = step * a.ld_dx * dx_size;

  for (; row < a.rows; row += step, dx += dx_step) {
    float2 xh[K][4], g[K][4];
    float unit[K], one[K];
    ring.wait();
    read_row<XK, VEC, G, K>(xh, unit, ring.data(0, row, VEC), ring.data(1, row, false), a.x_kind, mine, t, sh.zeros);
    read_row<DK, VEC, G, K>(g, one, ring.data(2, row, VEC), nullptr, dy_kind, mine, t, sh.zeros);
    const float r = rstd, m = -mean;
    if (row + step < a.rows) mean = a.mean[row + step], rstd = a.rstd[row + step];
    float2 s0 = both(0.0f), s1 = both(0.0f);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float2 w[4];
      read_param<VEC, G, K>(w, weight, t, k);
      // The difference first: in x r - mean r the rounded mean r, many times xh where a
      // row is far from 0, would leave its error in xh.
      const float2 by = both(unit[k]), from = both(m);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        xh[k][e] = VEC && XK == X_ACT8 ? __ffma2_rn(xh[k][e], by, from) : __fadd2_rn(xh[k][e], from);
        xh[k][e] = __fmul2_rn(xh[k][e], both(r));
        db[k][e] = __fadd2_rn(db[k][e], g[k][e]);
        dw[k][e] = __ffma2_rn(g[k][e], xh[k][e], dw[k][e]);
        g[k][e] = __fmul2_rn(g[k][e], w[e]);
        s0 = __fadd2_rn(s0, g[k][e]);
        s1 = __ffma2_rn(g[k][e], xh[k][e], s1);
      }
    }
    float s[2] = {s0.x + s0.y, s1.x + s1.y};
    row_sum<2, G, CLUSTER>(s, sh, turn, group, a.wait_limit_ns);
    if (row + a.stages * step < a.rows) filler.fill(a, ring.stage);
    ring.next();
    if (a.dx) {
      const float2 c2 = both(-s[0] * a.inv_cols * r), c1 = both(-s[1] * a.inv_cols * r);
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) g[k][e] = __ffma2_rn(xh[k][e], c1, __ffma2_rn(g[k][e], both(r), c2));
      store_row<VEC, G, K>(g, dx, a.dx_bf16 != 0, mine, t);
    }
  }
  let_next_start();

  // Column sums of the block's row groups, in the ring's memory: each group's to a place
  // of its own, then each thread of the first group adds its columns in order.
  if (groups > 1) {
    float *const sums = reinterpret_cast<float *>(stages);
    __syncthreads();
    if (group > 0) {
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int at = (group - 1) * (2 * G * K * 8) + param_at<VEC, G, K>(t, k, e);
          sums[at] = element(dw[k], e), sums[at + G * K * 8] = element(db[k], e);
        }
    }
    __syncthreads();
    if (group == 0)
#pragma unroll 1
      for (int q = 0; q < groups - 1; ++q)
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int at = q * (2 * G * K * 8) + param_at<VEC, G, K>(t, k, e);
            element(dw[k], e) += sums[at], element(db[k], e) += sums[at + G * K * 8];
          }
  }
  if (group == 0) {
    if (a.partial) {
      float *to = a.partial + unit * 2 * a.cols + base;
      store_row<VEC, G, K>(dw, reinterpret_cast<uint8_t *>(to), false, mine, t);
      store_row<VEC, G, K>(db, reinterpret_cast<uint8_t *>(to + a.cols), false, mine, t);
    } else {  // one unit: its sums are the gradients
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int j = column<VEC, G>(base, t, k, e);
          if (j < cols && a.dweight) store_any(a.dweight, j, a.grad_bf16 != 0, element(dw[k], e));
          if (j < cols && a.dbias) store_any(a.dbias, j, a.grad_bf16 != 0, element(db[k], e));
        }
    }
  }
  if constexpr (CLUSTER) {
    __syncwarp();
    tc::cluster_sync();
  }
  end_block(sh, a);
}

// dweight | dbias [cols] from partial [units][2][cols]: 32 columns of one of the
// two to a block, its 32 warps each adding every 32nd unit, then the warps' sums
// in order.  Bound by latency: a unit's sums are in L2, 152 of them make 5 MB at
// 4096 columns (5 us).
constexpr int kSumThreads = 1024;

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

// The narrowest shape that holds a row.  What a row costs a warp beside its columns is
// about 170 instructions, as much as 16 columns a thread cost, so vector kernels have
// 32 columns a thread (us in BF16, with 16 columns and twice the threads / with 32, where
// xh was one operation less: 32768 x 1024 48.8 / 41.0, 32768 x 2048 74.9 / 70.9, 16384 x
// 4096 72.1 / 69.9, 8192 x 8192 88.6 / 73.2, 4096 x 16384 135 / 118; now 40.7, 70.7, 69.7,
// 74.5 and 119).  Kernels that go element by element are
// bound by their accesses, which want threads, except where a warp has a row to itself
// (16385 x 1409 from the checkpoint 60 / 65, 2048 x 20001 340 / 356; 32769 x 515 77 / 52).
Shape shape_of(int64_t cols, bool vec) {
  if (cols <= 512) return {32, 2, 1, 0};
  if (cols <= 1024) return {32, 4, 1, 1};
  if (cols <= 2048) return vec ? Shape{64, 4, 1, 2} : Shape{128, 2, 1, 2};
  if (cols <= 4096) return vec ? Shape{128, 4, 1, 3} : Shape{256, 2, 1, 3};
  const int cluster = cluster_of(cols, 8192), index = cluster > 1 ? 5 : 4;
  return vec ? Shape{256, 4, cluster, index} : Shape{512, 2, cluster, index};
}

template <int XK, bool YB, bool VEC>
const void *kernel_of(int index) {
  constexpr int K = VEC ? 4 : 2, G = 256 / K;  // of the wider shapes
  switch (index) {
    case 0: return reinterpret_cast<const void *>(&backward_kernel<XK, YB, VEC, 32, 2, false>);
    case 1: return reinterpret_cast<const void *>(&backward_kernel<XK, YB, VEC, 32, 4, false>);
    case 2: return reinterpret_cast<const void *>(&backward_kernel<XK, YB, VEC, G, K, false>);
    case 3: return reinterpret_cast<const void *>(&backward_kernel<XK, YB, VEC, 2 * G, K, false>);
    case 4: return reinterpret_cast<const void *>(&backward_kernel<XK, YB, VEC, 4 * G, K, false>);
    default: return reinterpret_cast<const void *>(&backward_kernel<XK, YB, VEC, 4 * G, K, true>);
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

int64_t workspace_bytes_for(const fsdp_norm_desc_t *d) {
  const int sms = device_sms() > 0 ? device_sms() : 256;
  int64_t units = 0;
  for (bool vec : {false, true}) {  // the pointers, which decide, are not known here
    const Shape s = shape_of(d->cols, vec);
    units = std::max(units, units_of(d->rows, s, sms, most_threads(s.chunks, vec), kRowsEach));
  }
  return units > 1 ? units * 2 * d->cols * 4 : 0;
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
  a.rows = d->rows, a.cols = d->cols, a.ld_dx = d->ld_dx;
  set_x(a, d, x);
  a.in[2] = {static_cast<const uint8_t *>(dy), d->ld_y * ysize, (int32_t)ysize, 0};
  a.weight = weight, a.dx = dx, a.dweight = dweight, a.dbias = dbias;
  a.mean = const_cast<float *>(mean), a.rstd = const_cast<float *>(rstd);
  a.y_bf16 = d->y_dtype == FSDP_DTYPE_BF16;
  a.dx_bf16 = dx && d->dx_dtype == FSDP_DTYPE_BF16;
  a.param_bf16 = d->param_dtype == FSDP_DTYPE_BF16;
  a.grad_bf16 = gsize == 2;
  a.inv_cols = 1.0f / (float)d->cols;
  const bool vec = d->cols % 8 == 0 && (act8 || rows_aligned(x, d->rows, d->ld_x, dtype_bytes(d->x_dtype))) &&
                   rows_aligned(dy, d->rows, d->ld_y, ysize) && (!dx || rows_aligned(dx, d->rows, d->ld_dx, dxsize)) &&
                   aligned16(weight);
  const Shape sh = shape_of(d->cols, vec);
  const int sms = device_sms();
  const Launch l = plan_launch(a, sh, sms > 0 ? sms : 1, most_threads(sh.chunks, vec), kRowsEach, 1, 2);
  a.partial = l.units > 1 ? static_cast<float *>(workspace) : nullptr;
  if ((st = run(kernel_for(sh.index, vec, a.x_kind, a.y_bf16 != 0), a, l, sh, 0, s)) != FSDP_OK) return st;
  if (a.partial && (dweight || dbias)) {
    const float *partial = a.partial;
    int64_t n = l.units, cols = d->cols;
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

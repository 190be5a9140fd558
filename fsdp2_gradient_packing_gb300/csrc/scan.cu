// Gated linear recurrence (fsdp_gated_scan_*): a = sigmoid(gate + bias),
// h_t = a_t h_(t-1) + (1 - a_t) x_t, forward and backward.
//
// A thread to a sequence and a column, row by row.  Backward, the state before each tile
// of kTileRows rows comes from the forward pass and the tile's states are made again.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <string>

#include "layout.h"
#include "ops.h"

namespace fsdp {
namespace scan {
namespace {

constexpr int kTileRows = 128, kThreads = 128;

struct Args {
  const void *x, *gate, *bias, *offsets, *dh;
  const float *initial, *dfinal, *states_in;
  void *h, *dx, *dgate;
  float *final_state, *dinitial, *states, *partial;
  int64_t rows, cols, seqs, seq_len, ld_x, ld_gate, ld_h, ld_dx, ld_dgate;
  int32_t packed, wide, x_bf16, h_bf16, dx_bf16, param_bf16;
};

__device__ __forceinline__ int64_t offset_at(const Args &a, int64_t s) {
  if (!a.packed) return s * a.seq_len;
  const int64_t o = a.wide ? static_cast<const int64_t *>(a.offsets)[s] : static_cast<const int32_t *>(a.offsets)[s];
  return min(max(o, (int64_t)0), a.rows);
}
__device__ __forceinline__ void gates(float z, float &a, float &keep) {
  const float e = expf(-fabsf(z)), big = 1.0f / (1.0f + e), small = e * big;
  a = z >= 0 ? big : small, keep = z >= 0 ? small : big;
}

__global__ void __launch_bounds__(kThreads) forward_kernel(const __grid_constant__ Args a) {
  const int64_t j = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (j >= a.cols) return;
  const float bias = a.bias ? load_any(a.bias, j, a.param_bf16) : 0.0f;
  for (int64_t s = blockIdx.y; s < a.seqs; s += gridDim.y) {
    const int64_t begin = offset_at(a, s), end = offset_at(a, s + 1);
    float h = a.initial ? a.initial[s * a.cols + j] : 0.0f;
    for (int64_t t = begin; t < end; ++t) {
      if (a.states && t % kTileRows == 0) a.states[t / kTileRows * a.cols + j] = h;
      float g, keep;
      gates(load_any(a.gate, t * a.ld_gate + j, a.x_bf16) + bias, g, keep);
      h = fmaf(g, h, keep * load_any(a.x, t * a.ld_x + j, a.x_bf16));
      store_any(a.h, t * a.ld_h + j, a.h_bf16, h);
    }
    if (a.final_state) a.final_state[s * a.cols + j] = h;
  }
}

__global__ void __launch_bounds__(kThreads) backward_kernel(const __grid_constant__ Args a) {
  const int64_t j = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (j >= a.cols) return;
  const float bias = a.bias ? load_any(a.bias, j, a.param_bf16) : 0.0f;
  for (int64_t s = blockIdx.y; s < a.seqs; s += gridDim.y) {
    const int64_t begin = offset_at(a, s), end = offset_at(a, s + 1);
    float d = a.dfinal ? a.dfinal[s * a.cols + j] : 0.0f, db = 0.0f;
    for (int64_t hi = end; hi > begin;) {
      const int64_t lo = max(begin, (hi - 1) / kTileRows * kTileRows);
      float before[kTileRows];
      float h = lo == begin ? (a.initial ? a.initial[s * a.cols + j] : 0.0f) : a.states_in[lo / kTileRows * a.cols + j];
      for (int64_t t = lo; t < hi; ++t) {
        before[t - lo] = h;
        float g, keep;
        gates(load_any(a.gate, t * a.ld_gate + j, a.x_bf16) + bias, g, keep);
        h = fmaf(g, h, keep * load_any(a.x, t * a.ld_x + j, a.x_bf16));
      }
      for (int64_t t = hi - 1; t >= lo; --t) {
        float g, keep;
        gates(load_any(a.gate, t * a.ld_gate + j, a.x_bf16) + bias, g, keep);
        d += load_any(a.dh, t * a.ld_h + j, a.h_bf16);
        const float dz = d * (before[t - lo] - load_any(a.x, t * a.ld_x + j, a.x_bf16)) * (g * keep);
        store_any(a.dx, t * a.ld_dx + j, a.dx_bf16, keep * d);
        store_any(a.dgate, t * a.ld_dgate + j, a.dx_bf16, dz);
        db += dz;
        d *= g;
      }
      hi = lo;
    }
    if (a.dinitial) a.dinitial[s * a.cols + j] = d;
    if (a.partial) a.partial[s * a.cols + j] = db;
  }
}

__global__ void __launch_bounds__(kThreads) column_sum_kernel(const float *partial, int64_t n, int64_t cols, void *out, int32_t bf16) {
  const int64_t j = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (j >= cols) return;
  float s = 0.0f;
  for (int64_t i = 0; i < n; ++i) s += partial[i * cols + j];
  store_any(out, j, bf16, s);
}

fsdp_status_t check(const fsdp_scan_desc_t *d) {
  if (!d) return fail(FSDP_EINVAL, "desc is NULL");
  if (d->rows < 0 || d->cols < 1 || d->seqs < 0) return fail(FSDP_EINVAL, "rows < 0, cols < 1 or seqs < 0");
  if (d->cols > INT64_MAX / 64 / std::max<int64_t>(std::max(d->rows, d->seqs), 1)) return fail(FSDP_EUNSUPPORTED, "the matrices are too large");
  if (d->rows > INT32_MAX - 1024 || d->seqs > INT32_MAX - 1024) return fail(FSDP_EUNSUPPORTED, "2^31 rows or sequences");
  if (d->packed != 0 && d->packed != 1) return fail(FSDP_EINVAL, "packed is neither 0 nor 1");
  if (!d->packed) {
    if (d->seq_len < 0) return fail(FSDP_EINVAL, "seq_len < 0");
    if (d->seqs > 0 && (d->seq_len > d->rows || d->seqs * d->seq_len != d->rows)) return fail(FSDP_EINVAL, "rows is not seqs * seq_len");
    if (d->seqs == 0 && d->rows != 0) return fail(FSDP_EINVAL, "rows is not seqs * seq_len");
  }
  if (d->packed && d->offset_dtype != FSDP_INDEX_I32 && d->offset_dtype != FSDP_INDEX_I64) return fail(FSDP_EINVAL, "unknown offset_dtype");
  if (!float_dtype(d->x_dtype)) return fail(FSDP_EINVAL, "unknown x_dtype");
  if (!float_dtype(d->h_dtype)) return fail(FSDP_EINVAL, "unknown h_dtype");
  if (!float_dtype(d->dx_dtype)) return fail(FSDP_EINVAL, "unknown dx_dtype");
  if (!float_dtype(d->param_dtype)) return fail(FSDP_EINVAL, "unknown param_dtype");
  if (!float_dtype(d->grad_dtype)) return fail(FSDP_EINVAL, "unknown grad_dtype");
  return FSDP_OK;
}

fsdp_status_t check_inputs(const fsdp_scan_desc_t &d, const void *x, const void *gate, const void *bias, const float *initial,
                           const void *offsets) {
  const int64_t size = dtype_bytes(d.x_dtype);
  fsdp_status_t st;
  if ((st = check_matrix(x, d.rows, d.cols, d.ld_x, size, "x")) != FSDP_OK) return st;
  if ((st = check_matrix(gate, d.rows, d.cols, d.ld_gate, size, "gate")) != FSDP_OK) return st;
  const int64_t psize = dtype_bytes(d.param_dtype);
  if (bias && (st = check_ptr(bias, d.cols * psize, psize, "bias", -1)) != FSDP_OK) return st;
  if (initial && (st = check_ptr(initial, d.seqs * d.cols * 4, 4, "initial", -1)) != FSDP_OK) return st;
  const int64_t osize = d.offset_dtype == FSDP_INDEX_I64 ? 8 : 4;
  if (d.packed) return check_ptr(offsets, (d.seqs + 1) * osize, osize, "offsets", -1);
  if (offsets) return fail(FSDP_EINVAL, "offsets are given, but packed is 0");
  return FSDP_OK;
}

fsdp_status_t check_workspace(const void *workspace, int64_t given, int64_t needed) {
  if (given < needed)
    return fail(FSDP_EINVAL, "workspace_bytes is " + std::to_string(given) + ", the call needs " + std::to_string(needed));
  return check_ptr(workspace, needed, 16, "workspace", -1);
}

int64_t workspace_of(const fsdp_scan_desc_t &d, bool backward) { return backward ? d.seqs * d.cols * 4 : 0; }

Args args_of(const fsdp_scan_desc_t &d, const void *x, const void *gate, const void *bias, const float *initial, const void *offsets) {
  Args a = {};
  a.x = x, a.gate = gate, a.bias = bias, a.initial = initial, a.offsets = offsets;
  a.rows = d.rows, a.cols = d.cols, a.seqs = d.seqs, a.seq_len = d.seq_len;
  a.ld_x = d.ld_x, a.ld_gate = d.ld_gate, a.ld_h = d.ld_h, a.ld_dx = d.ld_dx, a.ld_dgate = d.ld_dgate;
  a.packed = d.packed, a.wide = d.offset_dtype == FSDP_INDEX_I64;
  a.x_bf16 = d.x_dtype == FSDP_DTYPE_BF16, a.h_bf16 = d.h_dtype == FSDP_DTYPE_BF16, a.dx_bf16 = d.dx_dtype == FSDP_DTYPE_BF16;
  a.param_bf16 = d.param_dtype == FSDP_DTYPE_BF16;
  return a;
}

}  // namespace
}  // namespace scan
}  // namespace fsdp

using namespace fsdp;
using namespace fsdp::scan;

extern "C" {

fsdp_status_t fsdp_gated_scan_states(int64_t rows, int64_t cols, int64_t *n) {
  if (!n) return fail(FSDP_EINVAL, "n is NULL");
  if (rows < 0 || cols < 1) return fail(FSDP_EINVAL, "rows < 0 or cols < 1");
  *n = (rows + kTileRows - 1) / kTileRows;
  clear_error();
  return FSDP_OK;
}

fsdp_status_t fsdp_gated_scan_workspace(const fsdp_scan_desc_t *desc, int32_t backward, int64_t *bytes) {
  fsdp_status_t st = check(desc);
  if (st != FSDP_OK) return st;
  if (!bytes) return fail(FSDP_EINVAL, "bytes is NULL");
  *bytes = workspace_of(*desc, backward != 0);
  clear_error();
  return FSDP_OK;
}

fsdp_status_t fsdp_gated_scan_forward(const fsdp_scan_desc_t *desc, const void *x, const void *gate, const void *bias,
                                      const float *initial, const void *offsets, void *h, float *final, float *states,
                                      void *workspace, int64_t workspace_bytes, fsdp_stream_t stream) {
  fsdp_status_t st = check(desc);
  if (st != FSDP_OK) return st;
  const fsdp_scan_desc_t &d = *desc;
  if ((st = check_inputs(d, x, gate, bias, initial, offsets)) != FSDP_OK) return st;
  if ((st = check_matrix(h, d.rows, d.cols, d.ld_h, dtype_bytes(d.h_dtype), "h")) != FSDP_OK) return st;
  if (final && (st = check_ptr(final, d.seqs * d.cols * 4, 4, "final", -1)) != FSDP_OK) return st;
  if (states && (st = check_ptr(states, d.rows * 4, 4, "states", -1)) != FSDP_OK) return st;
  if ((st = check_workspace(workspace, workspace_bytes, workspace_of(d, false))) != FSDP_OK) return st;
  if (d.seqs > 0) {
    Args a = args_of(d, x, gate, bias, initial, offsets);
    a.h = h, a.final_state = final, a.states = states;
    void *args[] = {&a};
    st = launched(launch_kernel(reinterpret_cast<const void *>(&forward_kernel),
                                dim3((unsigned)((d.cols + kThreads - 1) / kThreads), (unsigned)std::min<int64_t>(d.seqs, 65535)),
                                dim3(kThreads), args, 0, reinterpret_cast<cudaStream_t>(stream)));
    if (st != FSDP_OK) return st;
  }
  clear_error();
  return FSDP_OK;
}

fsdp_status_t fsdp_gated_scan_backward(const fsdp_scan_desc_t *desc, const void *dh, const void *x, const void *gate,
                                       const void *bias, const float *initial, const void *offsets, const float *states,
                                       const float *dfinal, void *dx, void *dgate, void *dbias, float *dinitial,
                                       void *workspace, int64_t workspace_bytes, fsdp_stream_t stream) {
  fsdp_status_t st = check(desc);
  if (st != FSDP_OK) return st;
  const fsdp_scan_desc_t &d = *desc;
  if ((st = check_inputs(d, x, gate, bias, initial, offsets)) != FSDP_OK) return st;
  if ((st = check_matrix(dh, d.rows, d.cols, d.ld_h, dtype_bytes(d.h_dtype), "dh")) != FSDP_OK) return st;
  if ((st = check_matrix(dx, d.rows, d.cols, d.ld_dx, dtype_bytes(d.dx_dtype), "dx")) != FSDP_OK) return st;
  if ((st = check_matrix(dgate, d.rows, d.cols, d.ld_dgate, dtype_bytes(d.dx_dtype), "dgate")) != FSDP_OK) return st;
  if ((st = check_ptr(states, d.rows * 4, 4, "states", -1)) != FSDP_OK) return st;
  if (dfinal && (st = check_ptr(dfinal, d.seqs * d.cols * 4, 4, "dfinal", -1)) != FSDP_OK) return st;
  const int64_t gsize = dtype_bytes(d.grad_dtype);
  if (dbias && (st = check_ptr(dbias, d.cols * gsize, gsize, "dbias", -1)) != FSDP_OK) return st;
  if (dinitial && (st = check_ptr(dinitial, d.seqs * d.cols * 4, 4, "dinitial", -1)) != FSDP_OK) return st;
  if ((st = check_workspace(workspace, workspace_bytes, workspace_of(d, true))) != FSDP_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const unsigned blocks = (unsigned)((d.cols + kThreads - 1) / kThreads);
  if (d.seqs > 0) {
    Args a = args_of(d, x, gate, bias, initial, offsets);
    a.dh = dh, a.states_in = states, a.dfinal = dfinal, a.dx = dx, a.dgate = dgate, a.dinitial = dinitial;
    a.partial = dbias ? static_cast<float *>(workspace) : nullptr;
    void *args[] = {&a};
    st = launched(launch_kernel(reinterpret_cast<const void *>(&backward_kernel), dim3(blocks, (unsigned)std::min<int64_t>(d.seqs, 65535)),
                                dim3(kThreads), args, 0, s));
    if (st != FSDP_OK) return st;
  }
  if (dbias) {
    const float *partial = static_cast<const float *>(workspace);
    int64_t n = d.seqs, cols = d.cols;
    int32_t bf16 = d.grad_dtype == FSDP_DTYPE_BF16;
    void *args[] = {&partial, &n, &cols, &dbias, &bf16};
    st = launched(launch_kernel(reinterpret_cast<const void *>(&column_sum_kernel), dim3(blocks), dim3(kThreads), args, 0, s));
    if (st != FSDP_OK) return st;
  }
  clear_error();
  return FSDP_OK;
}

}  // extern "C"

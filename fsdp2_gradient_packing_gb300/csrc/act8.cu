// 8-bit activation checkpoints (fsdp_act8_*): store and load.
//
// Both directions move bytes and do a handful of operations per element, so the
// bound is HBM: 2 + 33/32 bytes per BF16 element, 4 + 33/32 per FP32 element.  8192 x
// 12288 in BF16 is stored in 46 us and loaded in 47 (6.6 and 6.5 TB/s, a plain copy's
// rate); 4099 x 1411 in FP32, element by element, in 11.8 and 9.1 (2.5 and 3.2 TB/s).
// A thread holds one 16-byte vector of the matrix (8 BF16 or 4 FP32 elements),
// so a group of 32 is 4 or 8 neighbouring lanes and its maximum 2 or 3
// shuffles; each thread has kUnroll vectors in flight.  Rows that no vector
// divides or that start off a 16-byte boundary go element by element, kUnroll
// groups of a row to a warp, which keeps every load and store of a warp contiguous.
#include <cuda_runtime.h>

#include <cstdint>
#include <string>

#include "act8.h"
#include "layout.h"
#include "ops.h"

namespace fsdp {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;

// Where the codes of one checkpoint are: units of a row (vectors or groups)
// times rows, in row-major order.  A matrix without gaps between rows whose
// columns fill whole groups is one long row.
struct Act8Args {
  const void *x;       // store: source
  void *y;             // load: destination
  uint8_t *codes;
  uint8_t *scales;
  int64_t rows, cols, ld;
  int64_t groups;      // per row
  int64_t units;       // rows * units per row
};

template <class T>
constexpr int kVec = 16 / (int)sizeof(T);  // elements of one vector

template <class T>
__device__ __forceinline__ void unpack_vec(uint4 r, float2 (&v)[kVec<T> / 2]) {
  if constexpr (sizeof(T) == 2) {
    unpack8(r, v);
  } else {
    v[0] = make_float2(__uint_as_float(r.x), __uint_as_float(r.y));
    v[1] = make_float2(__uint_as_float(r.z), __uint_as_float(r.w));
  }
}

// Row and column of unit i, at `per_row` units a row; 32-bit division where it will do.
__device__ __forceinline__ void place(int64_t i, int64_t per_row, int64_t rows, int64_t *row, int64_t *at) {
  if (rows == 1) {
    *row = 0, *at = i;
  } else if (((uint64_t)i | (uint64_t)per_row) >> 32 == 0) {
    const uint32_t q = (uint32_t)i / (uint32_t)per_row;
    *row = q, *at = (uint32_t)i - q * (uint32_t)per_row;
  } else {
    *row = i / per_row, *at = i - *row * per_row;
  }
}

template <class T>
__global__ void __launch_bounds__(kThreads) store_vec_kernel(const __grid_constant__ Act8Args a) {
  constexpr int E = kVec<T>, kLanes = (int)kActGroup / E;
  const int64_t first = (int64_t)blockIdx.x * (kThreads * kUnroll) + threadIdx.x;
  const int64_t per_row = a.groups * kLanes;
  wait_for_previous();
  let_next_start();
  uint4 raw[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t i = first + u * kThreads;
    raw[u] = make_uint4(0, 0, 0, 0);
    int64_t row, at;
    if (i < a.units) {
      place(i, per_row, a.rows, &row, &at);
      if (at * E < a.cols) raw[u] = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const T *>(a.x) + row * a.ld + at * E));
    }
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t i = first + u * kThreads;
    float2 v[E / 2];
    unpack_vec<T>(raw[u], v);
    uint32_t top = act8_top(v);
#pragma unroll
    for (int m = 1; m < kLanes; m *= 2) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, m));
    const uint32_t s = act8_scale_byte(top);
    if (i < a.units) {
      // Units run over whole groups, so unit i's codes are at i * E whatever the row.
      act8_store<E>(a.codes + i * E, v, s);
      if (threadIdx.x % kLanes == 0) a.scales[i / kLanes] = (uint8_t)s;
    }
  }
}

template <class T>
__global__ void __launch_bounds__(kThreads) load_vec_kernel(const __grid_constant__ Act8Args a) {
  constexpr int E = kVec<T>, kLanes = (int)kActGroup / E;
  const int64_t first = (int64_t)blockIdx.x * (kThreads * kUnroll) + threadIdx.x;
  const int64_t per_row = a.groups * kLanes;
  wait_for_previous();
  let_next_start();
  uint32_t code[kUnroll][E / 4], s[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t i = first + u * kThreads;
    if (i < a.units) {
      if constexpr (E == 8) {
        const uint2 c = __ldcs(reinterpret_cast<const uint2 *>(a.codes + i * E));
        code[u][0] = c.x, code[u][1] = c.y;
      } else {
        code[u][0] = __ldcs(reinterpret_cast<const uint32_t *>(a.codes + i * E));
      }
      s[u] = a.scales[i / kLanes];
    }
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t i = first + u * kThreads;
    if (i >= a.units) continue;
    int64_t row, at;
    place(i, per_row, a.rows, &row, &at);
    if (at * E >= a.cols) continue;
    const float2 scale = both(act8_scale(s[u]));
    float2 v[E / 2];
#pragma unroll
    for (int e = 0; e < E / 2; ++e) v[e] = __fmul2_rn(act8_codes_of(act8_biased(code[u][e / 2]), e % 2), scale);
    uint4 r;
    if constexpr (E == 8)
      r = make_uint4(bf16_pair(v[0].x, v[0].y), bf16_pair(v[1].x, v[1].y), bf16_pair(v[2].x, v[2].y), bf16_pair(v[3].x, v[3].y));
    else
      r = make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x), __float_as_uint(v[1].y));
    *reinterpret_cast<uint4 *>(static_cast<T *>(a.y) + row * a.ld + at * E) = r;
  }
}

// kUnroll groups of one row to a warp, one element of each to a lane.
template <class T>
__global__ void __launch_bounds__(kThreads) store_rows_kernel(const __grid_constant__ Act8Args a) {
  const int lane = threadIdx.x & 31;
  const int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32, per_row = (a.groups + kUnroll - 1) / kUnroll;
  wait_for_previous();
  let_next_start();
  if (i >= a.units) return;
  int64_t row, at;
  place(i, per_row, a.rows, &row, &at);
  const int64_t j = at * (kUnroll * kActGroup) + lane, g = row * a.groups + at * kUnroll;
  const T *x = static_cast<const T *>(a.x) + row * a.ld + j;
  float v[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) v[u] = j + u * kActGroup < a.cols ? (float)x[u * kActGroup] : 0.0f;
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    if (at * kUnroll + u >= a.groups) break;
    const uint32_t s = act8_scale_byte(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v[u]) & 0x7FFFFFFFu));
    a.codes[(g + u) * kActGroup + lane] = (uint8_t)act8_code(v[u], s);
    if (lane == 0) a.scales[g + u] = (uint8_t)s;
  }
}

template <class T>
__global__ void __launch_bounds__(kThreads) load_rows_kernel(const __grid_constant__ Act8Args a) {
  const int lane = threadIdx.x & 31;
  const int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32, per_row = (a.groups + kUnroll - 1) / kUnroll;
  wait_for_previous();
  let_next_start();
  if (i >= a.units) return;
  int64_t row, at;
  place(i, per_row, a.rows, &row, &at);
  const int64_t j = at * (kUnroll * kActGroup) + lane, g = row * a.groups + at * kUnroll;
  const uint8_t *codes = a.codes + g * kActGroup + lane, *scales = a.scales + g;
  T *y = static_cast<T *>(a.y) + row * a.ld + j;
  uint32_t code[kUnroll], s[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u)
    if (at * kUnroll + u < a.groups) code[u] = codes[u * kActGroup], s[u] = scales[u];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u)
    if (j + u * kActGroup < a.cols) y[u * kActGroup] = (T)act8_value(act8_biased(code[u]), act8_scale(s[u]));
}

template <class T>
fsdp_status_t run(Act8Args a, bool store, cudaStream_t stream) {
  const void *p = store ? a.x : a.y;
  const bool vec = aligned16(p) && a.cols % kVec<T> == 0 && (a.rows == 1 || a.ld % kVec<T> == 0);
  if (a.cols % kActGroup == 0 && (a.rows == 1 || a.ld == a.cols)) {  // one long row
    a.cols *= a.rows;
    a.groups *= a.rows;
    a.ld = a.cols;
    a.rows = 1;
  }
  a.units = a.rows * (vec ? a.groups * ((int)kActGroup / kVec<T>) : (a.groups + kUnroll - 1) / kUnroll);
  const int64_t per_block = vec ? kThreads * kUnroll : kThreads / 32;
  const int64_t grid = (a.units + per_block - 1) / per_block;
  if (grid > INT32_MAX) return fail(FSDP_EUNSUPPORTED, "the matrix is too large for one launch");
  const void *fn = store ? (vec ? reinterpret_cast<const void *>(&store_vec_kernel<T>)
                                : reinterpret_cast<const void *>(&store_rows_kernel<T>))
                         : (vec ? reinterpret_cast<const void *>(&load_vec_kernel<T>)
                                : reinterpret_cast<const void *>(&load_rows_kernel<T>));
  void *args[] = {&a};
  return launched(launch_kernel(fn, dim3((unsigned)grid), dim3(kThreads), args, 0, stream, true));
}

fsdp_status_t act8(bool store, const void *x, void *y, int32_t dtype, int64_t rows, int64_t cols, int64_t ld,
                   const void *ckpt, cudaStream_t stream) {
  if (!float_dtype(dtype)) return fail(FSDP_EINVAL, "unknown dtype");
  if (rows < 0 || cols < 1) return fail(FSDP_EINVAL, "rows < 0 or cols < 1");
  const int64_t size = dtype_bytes(dtype);
  fsdp_status_t st = check_matrix(store ? x : y, rows, cols, ld, size, store ? "x" : "y");
  if (st != FSDP_OK) return st;
  if ((st = check_ptr(ckpt, act8_bytes(rows, cols), 16, "ckpt", -1)) != FSDP_OK) return st;
  if (rows > 0) {
    Act8Args a = {};
    a.x = x;
    a.y = y;
    a.codes = static_cast<uint8_t *>(const_cast<void *>(ckpt));
    a.groups = act8_groups(cols);
    a.scales = a.codes + rows * a.groups * kActGroup;
    a.rows = rows, a.cols = cols, a.ld = ld;
    st = dtype == FSDP_DTYPE_BF16 ? run<__nv_bfloat16>(a, store, stream) : run<float>(a, store, stream);
    if (st != FSDP_OK) return st;
  }
  clear_error();
  return FSDP_OK;
}

}  // namespace
}  // namespace fsdp

using namespace fsdp;

extern "C" {

fsdp_status_t fsdp_act8_bytes(int64_t rows, int64_t cols, int64_t *bytes) {
  if (!bytes) return fail(FSDP_EINVAL, "bytes is NULL");
  if (rows < 0 || cols < 1) return fail(FSDP_EINVAL, "rows < 0 or cols < 1");
  if (rows > 0 && cols > INT64_MAX / 64 / rows) return fail(FSDP_EUNSUPPORTED, "the matrix is too large");
  *bytes = act8_bytes(rows, cols);
  clear_error();
  return FSDP_OK;
}

fsdp_status_t fsdp_act8_store(const void *x, int32_t dtype, int64_t rows, int64_t cols, int64_t ld, void *ckpt,
                              fsdp_stream_t stream) {
  return act8(true, x, nullptr, dtype, rows, cols, ld, ckpt, reinterpret_cast<cudaStream_t>(stream));
}

fsdp_status_t fsdp_act8_load(const void *ckpt, int64_t rows, int64_t cols, void *y, int32_t dtype, int64_t ld,
                             fsdp_stream_t stream) {
  return act8(false, nullptr, y, dtype, rows, cols, ld, ckpt, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"

// Layer norm: what the forward (norm_forward.cu) and backward
// (norm_backward.cu) kernels share.  Included by those two files only.
//
// A row belongs to one group of G threads, of which each holds K chunks of 8
// columns in registers, so a row is read once whatever the passes over it.
// Groups of one warp share a block; larger groups are a block; a row wider than
// a block holds (512 threads x 16 columns) is split over a cluster of up to 8
// blocks, whose sums meet in distributed shared memory.  Blocks are persistent:
// weight, bias and the parameter gradients' sums stay in registers over all rows
// of a block, and the next row's loads are in flight while a row is worked on.
//
// Vector kernels give a thread 8 consecutive columns (one 16-byte load in
// BF16).  Where rows start off a 16-byte boundary or no vector divides them, a
// thread's 8 columns are G apart instead, which keeps every warp's loads
// contiguous without any alignment; element types are then a run-time flag.
#pragma once

#include <cooperative_groups.h>

#include "ops.h"

namespace fsdp {
namespace norm {

enum XKind { X_F32 = 0, X_BF16 = 1, X_ACT8 = 2 };

struct Args {
  const void *x;             // matrix, or codes of its checkpoint
  const uint8_t *x_scales;   // checkpoint only
  const void *weight, *bias;
  float *mean, *rstd;        // written forward, read backward
  // forward
  void *y;
  uint8_t *keep, *keep_scales;
  // backward
  const void *dy;
  void *dx;
  void *dweight, *dbias;
  float *partial;            // [units][2][cols]
  int64_t rows, cols, ld_x, ld_y, ld_dx;
  int64_t groups;            // of a checkpoint row
  float eps, inv_cols;
  int32_t x_kind, y_bf16, dx_bf16, param_bf16, grad_bf16;
};

constexpr int kMaxCluster = 8;
constexpr int kMaxWarps = 16;

// Sums of two values over the G threads of a row (and over the cluster's blocks
// where CLUSTER), the same in every thread and in a fixed order.  Slots alternate,
// so one barrier a sum is enough: a slot is written again only after every thread
// has passed the barrier of the sum in between.
struct Slots {
  float2 warp[2][kMaxWarps];
  float2 block[2][kMaxCluster];
};

template <int G, bool CLUSTER>
__device__ __forceinline__ float2 row_sum(float2 v, Slots &s, int &turn) {
#pragma unroll
  for (int m = 16; m > 0; m /= 2) {
    v.x += __shfl_xor_sync(0xFFFFFFFFu, v.x, m);
    v.y += __shfl_xor_sync(0xFFFFFFFFu, v.y, m);
  }
  if constexpr (G > 32) {
    const int t = turn & 1;
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) s.warp[t][threadIdx.x / 32] = v;
    __syncthreads();
    v = s.warp[t][0];
#pragma unroll
    for (int w = 1; w < G / 32; ++w) {
      const float2 q = s.warp[t][w];
      v.x += q.x, v.y += q.y;
    }
    if constexpr (CLUSTER) {
      namespace cg = cooperative_groups;
      cg::cluster_group c = cg::this_cluster();
      const unsigned n = c.num_blocks();
      if (threadIdx.x < n) c.map_shared_rank(&s.block[t][0], threadIdx.x)[c.block_rank()] = v;
      c.sync();
      v = s.block[t][0];
      for (unsigned r = 1; r < n; ++r) {
        const float2 q = s.block[t][r];
        v.x += q.x, v.y += q.y;
      }
    }
  }
  return v;
}

// A thread's columns of one row, as loaded: 8 K elements.
template <int XK, bool VEC, int K>
struct Raw {
  static constexpr int kWords = !VEC ? 8 : XK == X_F32 ? 8 : XK == X_BF16 ? 4 : 3;
  uint32_t w[K][kWords];
};

// Column of element e of chunk k (vector: chunk start plus e).
template <bool VEC, int G>
__device__ __forceinline__ int column(int base, int t, int k, int e) {
  return VEC ? base + (k * G + t) * 8 + e : base + (k * 8 + e) * G + t;
}

template <int XK, bool VEC, int G, int K>
__device__ __forceinline__ void load_row(Raw<XK, VEC, K> &r, const void *x, const uint8_t *scales, int kind, int64_t row,
                                         int64_t ld, int64_t groups, int cols, int base, int t) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if constexpr (VEC) {
      const int j = column<VEC, G>(base, t, k, 0);
      const bool in = j < cols;
      if constexpr (XK == X_ACT8) {
        const uint2 c = in ? __ldcs(reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(x) + row * groups * kActGroup + j))
                           : make_uint2(0, 0);
        r.w[k][0] = c.x, r.w[k][1] = c.y;
        r.w[k][2] = in ? scales[row * groups + j / (int)kActGroup] : 127u;
      } else if constexpr (XK == X_BF16) {
        const uint4 c = in ? __ldcs(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(x) + row * ld + j))
                           : make_uint4(0, 0, 0, 0);
        r.w[k][0] = c.x, r.w[k][1] = c.y, r.w[k][2] = c.z, r.w[k][3] = c.w;
      } else {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const float *>(x) + row * ld + j);
        const uint4 z = make_uint4(0, 0, 0, 0), c = in ? __ldcs(p) : z, d = in ? __ldcs(p + 1) : z;
        r.w[k][0] = c.x, r.w[k][1] = c.y, r.w[k][2] = c.z, r.w[k][3] = c.w;
        r.w[k][4] = d.x, r.w[k][5] = d.y, r.w[k][6] = d.z, r.w[k][7] = d.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int j = column<VEC, G>(base, t, k, e);
        float v = 0.0f;
        if (j < cols) {
          if (kind == X_ACT8)
            v = act8_value(static_cast<const uint8_t *>(x)[row * groups * kActGroup + j], 0,
                           act8_scale(scales[row * groups + j / (int)kActGroup]));
          else
            v = load_any(x, row * ld + j, kind == X_BF16);
        }
        r.w[k][e] = __float_as_uint(v);
      }
    }
  }
}

template <int XK, bool VEC, int K>
__device__ __forceinline__ void unpack_row(const Raw<XK, VEC, K> &r, float (&v)[K][8]) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if constexpr (!VEC || XK == X_F32) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[k][e] = __uint_as_float(r.w[k][e]);
    } else if constexpr (XK == X_BF16) {
      unpack8(make_uint4(r.w[k][0], r.w[k][1], r.w[k][2], r.w[k][3]), v[k]);
    } else {
      const float scale = act8_scale(r.w[k][2]);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[k][e] = act8_value(r.w[k][e / 4], e % 4, scale);
    }
  }
}

// A parameter vector's columns of this thread (`fill` where the vector is
// absent), 0 beyond the row.
template <bool VEC, int G, int K>
__device__ __forceinline__ void load_param(float (&v)[K][8], const void *p, bool bf16, float fill, int cols, int base, int t) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if constexpr (VEC) {
      const int j = column<VEC, G>(base, t, k, 0);
      if (p && j < cols) {
        load8(p, j, bf16, v[k]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[k][e] = j < cols ? fill : 0.0f;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int j = column<VEC, G>(base, t, k, e);
        v[k][e] = j >= cols ? 0.0f : p ? load_any(p, j, bf16) : fill;
      }
    }
  }
}

// Store a thread's columns of one row.
template <bool VEC, int G, int K>
__device__ __forceinline__ void store_row(const float (&v)[K][8], void *p, bool bf16, int64_t at, int cols, int base, int t) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if constexpr (VEC) {
      const int j = column<VEC, G>(base, t, k, 0);
      if (j < cols) store8(p, at + j, bf16, v[k]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int j = column<VEC, G>(base, t, k, e);
        if (j < cols) store_any(p, at + j, bf16, v[k][e]);
      }
    }
  }
}

// How a width is laid out: threads of a row, chunks a thread, blocks of a cluster.
struct Shape {
  int threads;   // of a block
  int group;     // threads of a row within the block
  int chunks;
  int cluster;
  int index;     // of the kernel table below
};

// Kernels by width: the narrowest shape that holds a row.
//   columns <=  512   one warp, 2 chunks; 4 rows to a block of 128
//           <= 1024   128 threads, 1 chunk     (vector kernels)
//           <= 2048   256 threads, 1 chunk     (vector)  128 threads, 2 chunks (others)
//           <= 4096   256 threads, 2 chunks    (vector)
//           <= 8192   512 threads, 2 chunks
//           above     clusters of 2, 4 or 8 blocks of 512 threads
// With fewer chunks a thread there is less to keep in flight a thread, with more
// threads a row a longer reduction; both sides of each border are within a few
// percent of one another.
inline Shape shape_of(int64_t cols, bool vec) {
  if (cols <= 512) return {128, 32, 2, 1, 0};
  if (vec) {
    if (cols <= 1024) return {128, 128, 1, 1, 1};
    if (cols <= 2048) return {256, 256, 1, 1, 2};
    if (cols <= 4096) return {256, 256, 2, 1, 3};
  } else if (cols <= 2048) {
    return {128, 128, 2, 1, 1};
  }
  int cluster = 1;
  while (cols > (int64_t)cluster * 8192) cluster *= 2;
  return {512, 512, 2, cluster, cluster > 1 ? 5 : 4};
}

// Host-side checks shared by both directions and the workspace query.
inline fsdp_status_t check_desc(const fsdp_norm_desc_t *d) {
  if (!d) return fail(FSDP_EINVAL, "desc is NULL");
  if (d->rows < 0) return fail(FSDP_EINVAL, "rows < 0");
  if (d->cols < 1) return fail(FSDP_EINVAL, "cols < 1");
  if (d->cols > FSDP_NORM_MAX_COLS) return fail(FSDP_EUNSUPPORTED, "cols > FSDP_NORM_MAX_COLS");
  if (!float_dtype(d->x_dtype) && d->x_dtype != FSDP_ACT8) return fail(FSDP_EINVAL, "unknown x_dtype");
  if (!float_dtype(d->param_dtype)) return fail(FSDP_EINVAL, "unknown param_dtype");
  if (!(d->eps >= 0.0f) || d->eps > 3.0e38f) return fail(FSDP_EINVAL, "eps is negative or not finite");
  return FSDP_OK;
}

}  // namespace norm
}  // namespace fsdp

// Layer norm: what the forward (norm_forward.cu) and backward
// (norm_backward.cu) kernels share.  Included by those two files only.
//
// A row belongs to one group of G threads, of which each holds K chunks of 8
// columns in registers, so a row is read once whatever the passes over it.
// A persistent block per SM has several groups, each with rows of its own; a row
// wider than a block's 8192 columns is split over a cluster of up to 8 blocks, whose
// sums meet in distributed shared memory (three rows at a time forward, one backward;
// 4096 x 16384 in BF16 takes 89 us forward, 168 with one row at a time).
//
// Rows come through a ring of shared-memory stages per group, filled with TMA bulk
// copies several rows ahead: what is in flight then depends neither on registers nor
// on the order in which loads return.  A stage is free once every thread of the group
// has summed its part, which the barrier of the row's first sum shows.  Forward, one
// lane of a warp of its own fills a group's ring; backward the groups need the whole
// register file, 8 warps of up to 255, and a ninth warp would cost each thread 87 of
// them, so a few lanes of each group fill its ring themselves.
//
// Vector kernels give a thread 8 consecutive columns.  Where rows start off a
// 16-byte boundary or no vector divides them, a thread's 8 columns are G apart
// instead, which keeps every access of a warp contiguous; a bulk copy then takes in
// the whole 16-byte units that the row touches, and element types are run-time flags.
#pragma once

#include "ops.h"
#include "tc.h"

namespace fsdp {
namespace norm {

enum XKind { X_F32 = 0, X_BF16 = 1, X_ACT8 = 2 };

constexpr int kMaxCluster = 8;
constexpr int kMaxWarps = 32;
constexpr int kMaxStages = 8;
constexpr int kClusterGroups = 3;  // row groups of a block whose rows are split over a cluster

// One matrix as it passes through the ring: rows of `row_bytes`, `pitch` bytes apart.
struct Stream {
  const uint8_t *p;
  int64_t pitch;
  int32_t elem;    // bytes of a column; 0: a scale byte per 32 columns
  int32_t at;      // offset in a stage; -1: absent
};

struct Args {
  Stream in[3];              // x or its codes; its scales; dy
  int32_t stages, stage_bytes;
  uint32_t *gave_up;         // count of blocks whose waits gave up
  uint64_t wait_limit_ns;
  int32_t fault;             // test hook, see skips_first()
  const void *weight, *bias;
  float *mean, *rstd;        // written forward, read backward
  // forward
  void *y;
  uint8_t *keep, *keep_scales;
  // backward
  void *dx;
  void *dweight, *dbias;
  float *partial;            // [units][2][cols]
  int64_t rows, cols, ld_y, ld_dx;
  int64_t groups;            // of a checkpoint row
  float eps, inv_cols;
  int32_t x_kind, y_bf16, dx_bf16, param_bf16, grad_bf16;
};

struct alignas(16) Shared {
  uint4 zeros[2];
  float warp[2][2][kMaxWarps];
  float block[kClusterGroups][2][2][kMaxCluster];
  uint64_t arrived[kClusterGroups][2];
  uint64_t full[kMaxWarps][kMaxStages], empty[kMaxWarps][kMaxStages];  // one ring to a group
  uint32_t stop;
};

// Test hook: bit 0 makes a row group of block 0 (bits 8 and up say which) leave its
// first stage empty, so that its wait gives up.
__device__ __forceinline__ bool skips_first(const Args &a, int group) {
  return (a.fault & 1) != 0 && blockIdx.x == 0 && group == a.fault >> 8;
}

template <int G>
__device__ __forceinline__ void group_sync(int group) {
  if constexpr (G == 32)
    __syncwarp();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(G) : "memory");
}

__device__ __forceinline__ uint32_t cluster_blocks() {
  uint32_t n;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
  return n;
}

// Sums of N values over the G threads of a row (and over the cluster's blocks where
// CLUSTER), the same in every thread and in a fixed order.  Slots alternate, so one
// barrier a sum is enough: a slot is written again only after every thread has
// passed the barrier of the sum in between.
template <int N, int G, bool CLUSTER>
__device__ __forceinline__ void row_sum(float (&v)[N], Shared &s, int &turn, int group, uint64_t limit_ns) {
  static_assert(N == 1 || N == 2, "one value or two");
  // Two values go down together: the lower half-warp takes the first, the upper the second.
  const int lane = threadIdx.x & 31;
  float w = v[0];
  if constexpr (N == 2) {
    const bool upper = lane >= 16;
    const float other = __shfl_xor_sync(0xFFFFFFFFu, upper ? v[0] : v[1], 16);
    w = (upper ? v[1] : v[0]) + other;
  }
#pragma unroll
  for (int m = N == 2 ? 8 : 16; m > 0; m /= 2) w += __shfl_xor_sync(0xFFFFFFFFu, w, m);
  if constexpr (G == 32) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = N == 1 ? w : __shfl_sync(0xFFFFFFFFu, w, i * 16);
  } else {
    const int q = turn & 1;
    if (lane % (32 / N) == 0) s.warp[q][lane / (32 / N)][threadIdx.x / 32] = w;
    group_sync<G>(group);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float4 *p = reinterpret_cast<const float4 *>(&s.warp[q][i][group * (G / 32)]);
      v[i] = 0.0f;
      if constexpr (G == 64) {
        const float2 a = *reinterpret_cast<const float2 *>(&s.warp[q][i][group * 2]);
        v[i] = a.x + a.y;
      }
#pragma unroll
      for (int w = 0; w < G / 128; ++w) {
        const float4 a = p[w];
        v[i] += (a.x + a.y) + (a.z + a.w);
      }
    }
    if constexpr (CLUSTER) {
      // Thread r sends the block's sums to block r; each block's barrier counts them in.
      // No block can be two sums ahead of another, so two slots do here too.
      const uint32_t n = cluster_blocks(), bar = tc::smem(&s.arrived[group][q]), to = threadIdx.x % G;
      if (to < n) {
        const uint32_t rank = tc::cluster_rank();
#pragma unroll
        for (int i = 0; i < N; ++i)
          asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(tc::at_rank(tc::smem(&s.block[group][q][i][rank]), to)), "f"(v[i])
                       : "memory");
        tc::bar_arrive_cluster(tc::at_rank(bar, to));
      }
      tc::bar_wait(bar, (uint32_t)(turn >> 1) & 1u, limit_ns, &s.stop);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        v[i] = s.block[group][q][i][0];
        for (uint32_t r = 1; r < n; ++r) v[i] += s.block[group][q][i][r];
      }
    }
    ++turn;
  }
}

// Column of element e of chunk k of a thread.
template <bool VEC, int G>
__device__ __forceinline__ int column(int base, int t, int k, int e) {
  return VEC ? base + (k * G + t) * 8 + e : base + (k * 8 + e) * G + t;
}

// The columns of a block, and a group's place in its ring.
template <int G, int K>
struct Ring {
  const Args &a;
  Shared &sh;
  const uint8_t *stages;   // of the group
  int group, base, width;  // first column of the block's part, and how many it has
  int stage = 0;
  uint32_t parity = 0;

  __device__ Ring(const Args &args, Shared &shared, const uint8_t *memory, int which, int first)
      : a(args), sh(shared), stages(memory + (int64_t)which * args.stages * args.stage_bytes), group(which), base(first),
        width(max(0, min((int)args.cols - first, G * K * 8))) {}

  // Waits for the current row; its part of matrix i is then at data(i, row).  A wait
  // that gives up is recorded, and what follows works on whatever is there.
  __device__ __forceinline__ void wait() const {
    if (width > 0) tc::bar_wait(tc::smem(&sh.full[group][stage]), parity, a.wait_limit_ns, &sh.stop);
  }
  // `even`: its rows are known to start on 16-byte boundaries.
  __device__ __forceinline__ const uint8_t *data(int i, int64_t row, bool even) const {
    const uint8_t *p = stages + stage * a.stage_bytes + a.in[i].at;
    if (even) return p;
    const Stream &s = a.in[i];
    return p + (((uint32_t)(uintptr_t)s.p + (uint32_t)row * (uint32_t)s.pitch + (s.elem ? base * s.elem : base / (int)kActGroup)) & 15u);
  }
  // The current row has been read by the whole group; by one thread of it.
  __device__ __forceinline__ void release() const { tc::bar_arrive(tc::smem(&sh.empty[group][stage])); }
  __device__ __forceinline__ void next() {
    if (++stage == a.stages) stage = 0, parity ^= 1u;
  }
};

// The loading warp: lane g fills group g's ring.
template <int G, int K>
__device__ __forceinline__ void load_rows(const Args &a, Shared &sh, uint8_t *memory, int groups, int base, int64_t row,
                                          int64_t step) {
  const int lane = threadIdx.x & 31, width = max(0, min((int)a.cols - base, G * K * 8));
  if (lane >= groups || width == 0) return;
  row += lane;
  uintptr_t from[3];
  uint32_t bytes[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const Stream &s = a.in[i];
    from[i] = (uintptr_t)(s.p + row * s.pitch) + (s.elem ? base * s.elem : base / (int)kActGroup);
    bytes[i] = s.elem ? width * s.elem : (width + (int)kActGroup - 1) / (int)kActGroup;
  }
  const uint32_t ring = tc::smem(memory) + (uint32_t)lane * a.stages * a.stage_bytes;
  bool skip = skips_first(a, lane);
  int stage = 0;
  uint32_t parity = 1;
  for (; row < a.rows; row += step) {
    const uint32_t full = tc::smem(&sh.full[lane][stage]), to = ring + stage * a.stage_bytes;
    if (!tc::bar_wait(tc::smem(&sh.empty[lane][stage]), parity, a.wait_limit_ns, &sh.stop)) break;
    uint32_t n[3], total = 0;
#pragma unroll
    for (int i = 0; i < 3; ++i) {  // whole 16-byte units
      n[i] = a.in[i].at < 0 ? 0u : (((uint32_t)from[i] & 15u) + bytes[i] + 15u) & ~15u;
      total += n[i];
    }
    if (!skip) tc::bar_expect(full, total);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      if (n[i] && !skip)
        asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                         to + a.in[i].at),
                     "l"(from[i] & ~(uintptr_t)15), "r"(n[i]), "r"(full)
                     : "memory");
      from[i] += step * a.in[i].pitch;
    }
    skip = false;
    if (++stage == a.stages) stage = 0, parity ^= 1u;
  }
}

// A group that fills its own ring (every thread has one of these): matrix i by lane
// i / W of warp i % W of the group's W warps.
template <int G, int K>
struct Filler {
  uintptr_t from;
  int64_t step;
  uint32_t bytes, to, full;
  __device__ Filler(const Args &a, Shared &sh, uint8_t *memory, int group, int base, int64_t row, int64_t row_step) {
    const int width = max(0, min((int)a.cols - base, G * K * 8));
    constexpr int W = G / 32;
    const int i = threadIdx.x % 32 * W + threadIdx.x % G / 32;
    const Stream s = a.in[i < 3 ? i : 0];
    from = (uintptr_t)(s.p + row * s.pitch) + (s.elem ? base * s.elem : base / (int)kActGroup);
    step = row_step * s.pitch;
    bytes = s.elem ? width * s.elem : (width + (int)kActGroup - 1) / (int)kActGroup;
    to = tc::smem(memory) + (uint32_t)group * a.stages * a.stage_bytes + s.at;
    full = tc::smem(&sh.full[group][0]);
    if (i >= 3 || s.at < 0) bytes = 0;
  }
  // The next row, whose stage is free.
  __device__ __forceinline__ void fill(const Args &a, int stage, bool skip = false) {
    if (bytes && !skip) {
      const uint32_t n = (((uint32_t)from & 15u) + bytes + 15u) & ~15u;
      tc::bar_expect(full + stage * 8, n);
      asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to + stage * a.stage_bytes),
                   "l"(from & ~(uintptr_t)15), "r"(n), "r"(full + stage * 8)
                   : "memory");
    }
    from += step;
  }
};

// Which of a thread's columns exist, out of the `width` of the block's part: chunks
// (VEC), or elements counted through all chunks.
template <bool VEC, int G, int K>
__device__ __forceinline__ int columns_of(int width, int t) {
  return VEC ? (width - t * 8 + G * 8 - 1) / (G * 8) : (width - t + G - 1) / G;
}

// A thread's columns of one row out of a stage, in binary32 and in pairs; 0 beyond the
// row (vector kernels read such a chunk from `zeros`, so that there is no branch).
// `mine`: columns_of(); `kind`: run-time flag for kernels that are not VEC.  A VEC
// checkpoint gives the codes, and their scale in `unit` (1 for anything else).
template <int XK, bool VEC, int G, int K>
__device__ __forceinline__ void read_row(float2 (&v)[K][4], float (&unit)[K], const uint8_t *p, const uint8_t *scales, int kind,
                                         int mine, int t, const uint4 *zeros) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
    unit[k] = 1.0f;
    if constexpr (VEC) {
      const int j = column<VEC, G>(0, t, k, 0);
      if constexpr (XK == X_ACT8) {
        const uint2 c = *reinterpret_cast<const uint2 *>(k < mine ? p + j : reinterpret_cast<const uint8_t *>(zeros));
        // An absent chunk's scale is 0 too: in a block without columns the stage holds anything.
        unit[k] = k < mine ? act8_scale(scales[j / (int)kActGroup]) : 0.0f;
        const uint32_t lo = act8_biased(c.x), hi = act8_biased(c.y);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[k][e] = act8_codes_of(e < 2 ? lo : hi, e % 2);
      } else {
        load8(k < mine ? p + j * (XK == X_BF16 ? 2 : 4) : reinterpret_cast<const uint8_t *>(zeros), 0, XK == X_BF16, v[k]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int j = column<VEC, G>(0, t, k, e);
        element(v[k], e) = 0.0f;
        if (k * 8 + e < mine)
          element(v[k], e) = kind == X_ACT8 ? act8_value(act8_biased(p[j]), act8_scale(scales[j / (int)kActGroup]))
                                            : load_any(p, j, kind == X_BF16);
      }
    }
  }
}

// A parameter vector's columns of this block in shared memory, in binary32 (`fill`
// where the vector is absent): in registers they would cost 16 a vector.  Vector
// kernels keep the two halves of each thread's 8 columns apart, so that a warp's
// 16-byte reads are contiguous.
template <bool VEC, int G, int K>
__device__ __forceinline__ int param_at(int t, int k, int e) {
  return VEC ? (e / 4) * (G * K * 4) + (k * G + t) * 4 + e % 4 : (k * 8 + e) * G + t;
}
template <bool VEC, int G, int K>
__device__ __forceinline__ void stage_param(float *to, const void *p, bool bf16, float fill, int cols, int base) {
  if ((int)threadIdx.x >= G) return;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    float2 v[4];
    if constexpr (VEC) {
      const int j = column<VEC, G>(base, threadIdx.x, k, 0);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = both(j < cols ? fill : 0.0f);
      if (p && j < cols) load8(p, j, bf16, v);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int j = column<VEC, G>(base, threadIdx.x, k, e);
        element(v, e) = j >= cols ? 0.0f : p ? load_any(p, j, bf16) : fill;
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) to[param_at<VEC, G, K>(threadIdx.x, k, e)] = element(v, e);
  }
}
template <bool VEC, int G, int K>
__device__ __forceinline__ void read_param(float2 (&v)[4], const float *from, int t, int k) {
  if constexpr (VEC) {
    const float4 a = *reinterpret_cast<const float4 *>(from + param_at<VEC, G, K>(t, k, 0));
    const float4 b = *reinterpret_cast<const float4 *>(from + param_at<VEC, G, K>(t, k, 4));
    v[0] = make_float2(a.x, a.y), v[1] = make_float2(a.z, a.w), v[2] = make_float2(b.x, b.y), v[3] = make_float2(b.z, b.w);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) element(v, e) = from[param_at<VEC, G, K>(t, k, e)];
  }
}

// Stores a thread's columns of one row.  `p`: the row's first column of this block's
// part, in bytes; the offsets from there are compile-time multiples of the thread's.
template <bool VEC, int G, int K>
__device__ __forceinline__ void store_row(const float2 (&v)[K][4], uint8_t *p, bool bf16, int mine, int t) {
  void *const q = p + (VEC ? t * 8 : t) * (bf16 ? 2 : 4);
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if constexpr (VEC) {
      if (k < mine) store8(q, k * G * 8, bf16, v[k]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (k * 8 + e < mine) store_any(q, (k * 8 + e) * G, bf16, element(v[k], e));
    }
  }
}

// Barriers (`fills`: threads that fill a stage) and the stop flag; by the whole block, then visible to all of it and to its cluster.
template <bool CLUSTER>
__device__ __forceinline__ void begin_block(Shared &sh, int groups, int stages, int fills) {
  if (threadIdx.x == 0) {
    sh.stop = 0;
    sh.zeros[0] = sh.zeros[1] = make_uint4(0, 0, 0, 0);
    if (CLUSTER)
      for (int q = 0; q < 2 * kClusterGroups; ++q) tc::bar_init(tc::smem(&sh.arrived[q / 2][q % 2]), cluster_blocks());
  }
  for (int i = threadIdx.x; i < groups * stages; i += blockDim.x) {
    tc::bar_init(tc::smem(&sh.full[i / stages][i % stages]), fills);
    tc::bar_init(tc::smem(&sh.empty[i / stages][i % stages]), 1);
  }
  tc::bar_init_fence();
  __syncthreads();
  if (CLUSTER) tc::cluster_sync();
}
// Records a wait that gave up; copies that it did not wait for get a fixed time to
// land before the block leaves its shared memory.  By the whole block: its row groups
// and its loading warp have nothing else in common after their last rows, and any of
// them may be the one whose wait gives up.
__device__ __forceinline__ void end_block(Shared &sh, const Args &a) {
  __syncwarp();  // the loading warp's lanes come from loops of their own
  __syncthreads();
  if (threadIdx.x == 0 && *(volatile uint32_t *)&sh.stop) {
    atomicAdd(a.gave_up, 1u);
    const uint64_t began = tc::now_ns();
    while (tc::now_ns() - began < 1000000) {
    }
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
// How a width is laid out: threads of a row, chunks a thread, blocks of a cluster.
struct Shape {
  int group, chunks, cluster;
  int index;     // of the kernel tables
};

// Blocks of the cluster that a row needs when a block holds `width` columns.
inline int cluster_of(int64_t cols, int64_t width) {
  int cluster = 1;
  while (cols > cluster * width) cluster *= 2;
  return cluster;
}

// Blocks (or clusters), the row groups of each, and its shared memory.
struct Launch {
  int64_t units;
  int groups, smem;
};

constexpr int kSmemBudget = 208 * 1024;

// `rows_each`: so many rows a group may stay with one unit (0: spread over the SMs at once).
inline int groups_of(int64_t rows, const Shape &s, int sms, int most_threads, int rows_each) {
  int64_t most = most_threads / s.group;
  if (s.cluster > 1 && most > kClusterGroups) most = kClusterGroups;
  const int64_t units = sms / s.cluster > 0 ? sms / s.cluster : 1;
  const int64_t want = rows <= most * rows_each ? rows : (rows + units - 1) / units;
  return (int)(want < 1 ? 1 : want < most ? want : most);
}
inline int64_t units_of(int64_t rows, const Shape &s, int sms, int most_threads, int rows_each) {
  const int g = groups_of(rows, s, sms, most_threads, rows_each);
  if (rows <= (int64_t)g * rows_each) return 1;
  const int64_t need = (rows + g - 1) / g, most = sms / s.cluster > 0 ? sms / s.cluster : 1;
  return need < most ? need : most;
}

// Lays out the ring and the rest of shared memory: `params` vectors, then the stages,
// or after them `sums` vectors of each group but one (column sums) in the same place.
inline Launch plan_launch(Args &a, const Shape &s, int sms, int most_threads, int rows_each, int params, int sums) {
  Launch l;
  l.groups = groups_of(a.rows, s, sms, most_threads, rows_each);
  l.units = units_of(a.rows, s, sms, most_threads, rows_each);
  const int width = s.group * s.chunks * 8;
  const int cols = a.cols < width ? (int)a.cols : width;
  int at = 0;
  for (Stream &in : a.in) {
    if (!in.p) {
      in.at = -1;
      continue;
    }
    in.at = at;
    const int bytes = in.elem ? cols * in.elem : (cols + (int)kActGroup - 1) / (int)kActGroup;
    at += (bytes + 15 + 16) / 16 * 16;  // whole 16-byte units around it
  }
  a.stage_bytes = at;
  const int fixed = params * width * 4;
  int64_t stages = (kSmemBudget - fixed) / ((int64_t)l.groups * at);
  const int64_t turns = (a.rows + l.units * l.groups - 1) / (l.units * l.groups);
  if (stages > kMaxStages) stages = kMaxStages;
  if (stages > turns) stages = turns;
  a.stages = (int32_t)(stages > 1 ? stages : 1);
  const int ring = l.groups * a.stages * at, tail = (l.groups - 1) * sums * width * 4;
  l.smem = fixed + (ring > tail ? ring : tail);
  return l;
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

// x as a stream: the matrix, or the codes and scales of its checkpoint.
inline void set_x(Args &a, const fsdp_norm_desc_t *d, const void *x) {
  a.groups = act8_groups(d->cols);
  const uint8_t *p = static_cast<const uint8_t *>(x);
  if (d->x_dtype == FSDP_ACT8) {
    a.x_kind = X_ACT8;
    a.in[0] = {p, a.groups * kActGroup, 1, 0};
    a.in[1] = {p + d->rows * a.groups * kActGroup, a.groups, 0, 0};
  } else {
    const int32_t size = (int32_t)dtype_bytes(d->x_dtype);
    a.x_kind = size == 2 ? X_BF16 : X_F32;
    a.in[0] = {p, d->ld_x * size, size, 0};
  }
}

// `more`: threads of a block beside its row groups (a loading warp's).
inline fsdp_status_t run(const void *fn, Args &a, const Launch &l, const Shape &s, int more, cudaStream_t stream) {
  cudaError_t e = gave_up_count(GAVE_UP_NORM, &a.gave_up);
  if (e != cudaSuccess) return fail(FSDP_ECUDA, std::string("status count: ") + cudaGetErrorString(e));
  a.wait_limit_ns = wait_limit_ns();
  a.fault = wait_fault();
  if (l.smem > 32 * 1024) {
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, l.smem);
    if (e != cudaSuccess) return fail(FSDP_ECUDA, std::string("cudaFuncSetAttribute: ") + cudaGetErrorString(e));
  }
  void *args[] = {&a};
  return launched(launch_kernel(fn, dim3((unsigned)(l.units * s.cluster)), dim3((unsigned)(l.groups * s.group + more)), args,
                                (size_t)l.smem, stream, true, s.cluster));
}

inline bool rows_aligned(const void *p, int64_t rows, int64_t ld, int64_t size) {
  return aligned16(p) && (rows == 1 || ld * size % 16 == 0);
}

}  // namespace norm
}  // namespace fsdp

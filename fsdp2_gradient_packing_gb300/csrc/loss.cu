// Losses over rows of logits (fsdp_distill_loss_*, fsdp_policy_loss_*).
//
// Everything is bound by the logits' bytes: read once for a loss, read once and written once for a gradient
// or both.  A row is cut into slices of whole 16-byte units; a block reads a slice with one TMA bulk copy
// into a ring of shared-memory stages, the next one on its way while it works.
//
//   STATS     a loss alone: a block walks over a row's slices, or with few rows a cluster shares them and its
//             sums meet in distributed shared memory.
//   HELD      a loss with its gradient, of rows of one slice: each thread keeps its elements'
//             exponentials (relative to its own maximum) in registers, and the gradient is a product per element.
//   TWICE     the same of longer rows: a block, or a cluster that shares a row, reads it twice, the second
//             time from L2.
//   GRADIENT  the gradient alone, from lse: slices one by one.
//
// Measured in BF16 against 6.79 TB/s of a copy: distillation's loss alone of 4096 x 131072 153 us (7.0 TB/s), of 8192 x 32768 81
// us (6.6); gradients from lse 327 us (6.6) and 166 (6.5); TWICE 395 us (5.4, bound by L2, which gives each row twice and takes the
// gradient) and 174 us (6.2). Rows of up to 8192 or 16384 logits are another kernel's, further down.
//
// A ninth warp fills the ring, and a tenth prepares what a row has beside its logits: the policy's scalars,
// or the softmax of the teacher's entries, while the other eight are at the row before.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>
#include <string>
#include <type_traits>

#include "layout.h"
#include "ops.h"
#include "tc.h"

namespace fsdp {
namespace loss {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32, kBlock = kThreads + 64, kMaxTop = FSDP_DISTILL_MAX_TOP;
constexpr int kMaxCluster = 8, kMaxStages = 4;
constexpr int kMostUnits = 8;  // 16-byte units of a slice that a thread has
constexpr int kMostSmem = 106 * 1024;  // stages, and what goes with rows: 2 x (32 + 16.1) KB at least
constexpr int kNamed = 32768;
// Bytes of rows at work of which L2 (129 MB) still has what is read a second time; beyond, a row takes more blocks and their sums longer
// (4096 x 50021 FP32 289 us with 80 MB and one block to a row, 319 with 40 MB and two).
constexpr int64_t kL2Rows = 80 << 20;
constexpr float kLog2E = 1.4426950408889634f;

enum Mode { STATS, HELD, TWICE, GRADIENT };
// Blocks of an SM (three of the kernels for slices of up to 512 units), and stages of a ring. Rows that are read twice want deep
// rings (8192 x 32768 BF16: three stages 177 us, two 194, three blocks of half as long slices 188). Gradients alone want few and long
// slices under way, which DRAM's pages like (4096 x 131072 BF16: two blocks of two stages 328 us, three of two 346, two of three
// 369, three of two half as long 372).
constexpr int kBlocks = 2;
constexpr int stages_of_mode(Mode m) { return m == GRADIENT ? 2 : kMaxStages; }

struct Args {
  const void *logits;
  void *dlogits;
  const void *tokens, *teacher;
  const float *old_logp, *ref_logp, *advantage, *weight, *dloss, *lse_in, *logp_in;
  float *loss, *logp, *lse;
  uint32_t *gave_up;
  uint64_t wait_limit_ns;
  int64_t rows, ld_z, ld_g, ld_tokens, ld_teacher;
  int64_t items;       // rows, or rows x slices
  int32_t vocab, top, z_bf16, g_bf16, teacher_bf16, wide, backward, fault;
  int32_t cluster, rounds, slices;  // blocks to a row; slices of a block, one after another; slices as items
  int32_t units;       // of a slice, at most
  int32_t stages, stage_bytes, side_bytes;
  float t, inv_t, scale;  // scale: log2 e / T
  float low, high, kl;
};

// What the tenth warp prepares of a row.  The teacher's entries follow it.
struct alignas(16) Side {
  float up;          // weight x dloss
  float weight;
  float lse;         // backward
  float slope;       // backward
  float old, ref, advantage;
  float mass, q_log_q;  // teacher: sum of q (1 or 0), sum of q log q
  int32_t token;     // policy, -1: none
};

struct alignas(16) Shared {
  float4 warp[2][kWarps];        // maximum and sum of a warp, what it has of the targets, and their mass
  float4 block[2][kMaxCluster];  // the same of the cluster's blocks
  uint64_t arrived[2], full[kMaxStages], empty[kMaxStages];  // of the cluster's sums; of stages
  uint64_t ready[kMaxStages], done[kMaxStages];              // of rows' sides
  uint32_t named[kNamed / 32];   // tokens that the teacher has named
  uint32_t stop;
};

__device__ __forceinline__ void workers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory"); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Maxima are kept as logits and subtracted before a difference is scaled: logits of the type's lowest
// value have no finite multiple, but differences that count do.
// 2^((m - top) scale), 1 where they are equal, infinite or not.
__device__ __forceinline__ float below(float m, float top, float scale) { return ex2(m == top ? 0.0f : (m - top) * scale); }
// Maximum and sum (of 2^((z - maximum) scale)) of two sets, without a NaN for empty ones.
__device__ __forceinline__ void merge(float &m, float &s, float m2, float s2, float scale) {
  const float top = fmaxf(m, m2);
  s = s * below(m, top, scale) + s2 * below(m2, top, scale);
  m = top;
}

// A teacher's targets: sum of q (z - top), with `mass` the sum of q and `top` no less than any of their logits. So all its terms have
// one sign: sum q z against lse would leave nothing of their difference where the logits are large beside it. As of a larger top (in
// halves: the difference of two logits may leave the range that a part of it lies in):
__device__ __forceinline__ float raised(float x, float mass, float top, float to) {
  return top == to || mass == 0.0f ? x : fmaf(2.0f * mass, 0.5f * top - 0.5f * to, x);
}

__device__ __forceinline__ int32_t token_at(const Args &a, int64_t i) {
  const int64_t t = a.wide ? static_cast<const int64_t *>(a.tokens)[i] : static_cast<const int32_t *>(a.tokens)[i];
  return t >= 0 && t < a.vocab ? (int32_t)t : -1;
}

// Where a slice of a row is: its 16-byte units, which begin up to a unit before the row.
template <class T>
struct Slice {
  static constexpr int kPer = 16 / (int)sizeof(T);  // elements of a unit
  int64_t row;
  uintptr_t at;   // of the slice's first unit
  int32_t phase;  // elements between the row's first unit and the row
  int32_t first, units;  // first unit in the row, and how many the slice has of it
  int32_t row_units;
  bool clean;     // all its units lie inside the row
  __device__ __forceinline__ Slice(const Args &a, int64_t r, int32_t index) : row(r) {
    const uintptr_t p = (uintptr_t)a.logits + r * a.ld_z * sizeof(T);
    phase = (int32_t)(p & 15u) / (int)sizeof(T);
    row_units = (phase + a.vocab + kPer - 1) / kPer;
    first = index * a.units;
    units = max(0, min(a.units, row_units - first));
    at = (p & ~(uintptr_t)15) + (int64_t)first * 16;
    clean = (phase == 0 || first > 0) && (row_units * kPer == phase + a.vocab || first + units < row_units);
  }
  // Elements of the row that the slice has.
  __device__ __forceinline__ int32_t begin() const { return max(0, first * kPer - phase); }
  __device__ __forceinline__ int32_t end(const Args &a) const { return min(a.vocab, (first + units) * kPer - phase); }
};

// The policy's loss and its derivative with respect to logp.
__device__ __forceinline__ void policy_of(const Args &a, float logp, const Side &s, float &loss, float &slope) {
  const float r = a.old_logp ? expf(logp - s.old) : 1.0f, held = fminf(fmaxf(r, a.low), a.high);
  const float one = r * s.advantage, two = held * s.advantage;
  loss = -fminf(one, two);
  if (one != one) loss = one;
  slope = one <= two ? -one : one != one ? one : 0.0f;
  if (a.ref_logp) {
    const float gap = s.ref - logp, e = expm1f(gap);
    loss += a.kl * (e - gap);
    slope -= a.kl * e;
  }
}

// ---- the ninth and the tenth warp ------------------------------------------------------------------------
constexpr int kEach = 4;  // teacher's entries that a lane holds in registers: up to 128 in all

// Entries j, j + 32 and so on of a row of the teacher's. Types are asked for once, so that all loads are under way together.
template <int N>
__device__ __forceinline__ void load_entries(const Args &a, int64_t row, int j, int32_t (&id)[N], float (&v)[N]) {
  auto ids = [&](const auto *p) {
    std::remove_cv_t<std::remove_pointer_t<decltype(p)>> t[N];
#pragma unroll
    for (int i = 0; i < N; ++i) t[i] = j + i * 32 < a.top ? p[i * 32] : -1;
#pragma unroll
    for (int i = 0; i < N; ++i) id[i] = t[i] >= 0 && t[i] < a.vocab ? (int32_t)t[i] : -1;
  };
  auto logits = [&](const auto *p) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = j + i * 32 < a.top ? (float)p[i * 32] : 0.0f;
  };
  if (a.teacher_bf16)
    logits(static_cast<const __nv_bfloat16 *>(a.teacher) + row * a.ld_teacher + j);
  else
    logits(static_cast<const float *>(a.teacher) + row * a.ld_teacher + j);
  if (a.wide)
    ids(static_cast<const int64_t *>(a.tokens) + row * a.ld_tokens + j);
  else
    ids(static_cast<const int32_t *>(a.tokens) + row * a.ld_tokens + j);
}

// What a row has beside its logits, on its way while the row before is prepared.
template <bool DISTILL, Mode MODE>
struct Ahead {
  float weight = 1.0f, dloss = 1.0f, lse = 0.0f, logp = 0.0f, old = 0.0f, ref = 0.0f, advantage = 0.0f;
  int32_t token = -1, id[kEach];
  float v[kEach];
  __device__ __forceinline__ void load(const Args &a, int64_t item) {
    if (item >= a.items) return;
    const int64_t row = MODE == GRADIENT ? item / a.slices : item;
    const int lane = threadIdx.x & 31;
    if (a.weight) weight = a.weight[row];
    if (MODE == GRADIENT) {
      lse = a.lse_in[row];
      if (a.dloss) dloss = a.dloss[row];
    }
    if constexpr (DISTILL) {
      if (a.top <= 32 * kEach) {
        load_entries<kEach>(a, row, lane, id, v);
      }
    } else {
      if (MODE == GRADIENT) logp = a.logp_in[row];
      if (a.old_logp) old = a.old_logp[row];
      if (a.ref_logp) ref = a.ref_logp[row];
      advantage = a.advantage[row];
      token = token_at(a, row);
    }
  }
};

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int m = 16; m > 0; m /= 2) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, m));
  return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int m = 16; m > 0; m /= 2) x += __shfl_xor_sync(0xFFFFFFFFu, x, m);
  return x;
}

// The teacher's entries of a row in shared memory: tokens (-1: none), q for the loss, q for the gradient (negative: another
// entry of its token has it), and room for their logits.
struct Teacher {
  int32_t *ids;
  float *q, *gq, *z;
  __device__ __forceinline__ Teacher(Side &side, int top)
      : ids(reinterpret_cast<int32_t *>(&side + 1)), q(reinterpret_cast<float *>(ids + top)), gq(q + top), z(gq + top) {}
};

// Whether an entry's token has been named before; forget() clears that, for a next row.  Tokens from lo on have a bit each where
// kNamed bits are enough for those up to hi, else by a hash, the top of a product with 2^32 over the golden ratio (which spreads
// tokens at equal distances too): then another token may have been named.
struct Names {
  uint32_t *bits;
  int32_t lo;
  bool exact;
  __device__ __forceinline__ Names(uint32_t *named, int32_t l, int32_t hi) : bits(named), lo(l), exact(hi - l <= kNamed) {}
  __device__ __forceinline__ uint32_t at(int32_t id) const {
    return exact ? (uint32_t)(id - lo) : (uint32_t)id * 2654435769u / (0xFFFFFFFFu / kNamed + 1);
  }
  __device__ __forceinline__ bool name(int32_t id) const {
    const uint32_t h = at(id), bit = 1u << (h & 31);
    return (atomicOr(&bits[h / 32], bit) & bit) != 0;
  }
  __device__ __forceinline__ void forget(int32_t id) const { bits[at(id) / 32] = 0; }
};

// Tokens that are named more than once (z is 1 at all but one of a token's entries, and where hashes
// meet): the first entry takes what the others have, in their order.
__device__ __noinline__ void join_entries(int top, const Teacher &e) {
  const int lane = threadIdx.x & 31;
  for (int j0 = 0; j0 < top; j0 += 32) {
    uint32_t which = __ballot_sync(0xFFFFFFFFu, j0 + lane < top && e.z[j0 + lane] == 1.0f);
    for (; which; which &= which - 1) {
      const int at = j0 + __ffs(which) - 1, id = e.ids[at];
      if (e.z[at] != 1.0f) continue;  // its token has been joined
      int first = -1;
      float s = 0.0f;
      for (int k0 = 0; k0 < top; k0 += 32) {
        const int k = k0 + lane;
        const bool same = k < top && e.ids[k] == id;
        const float other = same ? e.q[k] : 0.0f;
        uint32_t more = __ballot_sync(0xFFFFFFFFu, same);
        if (more && first < 0) first = k0 + __ffs(more) - 1;
        for (; more; more &= more - 1) s += __shfl_sync(0xFFFFFFFFu, other, __ffs(more) - 1);
        if (same) e.gq[k] = -1.0f, e.z[k] = 0.0f;
      }
      __syncwarp();
      if (lane == 0) e.gq[first] = s;
      __syncwarp();
    }
  }
}

// The softmax over a row's entries; tokens lo .. hi - 1 are those of this block's gradient.  Their logits, too, are scaled after the
// maximum is subtracted: of the type's lowest value, which counts, a multiple may be -infinity, which does not.  ONCE: the caller has
// this row alone, of up to 32 kEach entries.
template <bool DISTILL, Mode MODE, bool ONCE>
__device__ __forceinline__ void teacher_of(const Args &a, uint32_t *named, Side &side, int64_t row, int32_t lo, int32_t hi,
                                           const Ahead<DISTILL, MODE> &ahead) {
  const int lane = threadIdx.x & 31;
  const Teacher e(side, a.top);
  const Names names(named, lo, hi);
  float top = -INFINITY, sum = 0.0f, total = 0.0f;
  bool nan = false, twice = false;
  if (ONCE || a.top <= 32 * kEach) {
    float v[kEach];
    int32_t id[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      v[i] = ahead.id[i] < 0 ? -INFINITY : ahead.v[i];
      id[i] = v[i] == -INFINITY ? -1 : ahead.id[i];
      top = fmaxf(top, v[i]);
      nan |= v[i] != v[i];
    }
    top = warp_max(top);
    bool again[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const float d = (v[i] - top) * a.inv_t, p = id[i] < 0 ? 0.0f : ex2(d * kLog2E);
      sum += p;
      if (p > 0.0f || p != p) total += p * d;
      v[i] = p;
      again[i] = MODE != STATS && id[i] >= lo && id[i] < hi && names.name(id[i]);
      twice |= again[i];
    }
    sum = warp_sum(sum), total = warp_sum(total);
    const float inv = 1.0f / sum;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int j = i * 32 + lane;
      if (j < a.top) {
        e.ids[j] = id[i];
        e.q[j] = e.gq[j] = id[i] < 0 ? 0.0f : v[i] * inv;
        if (MODE != STATS) {
          e.z[j] = again[i] ? 1.0f : 0.0f;
          if (!ONCE && id[i] >= lo && id[i] < hi) names.forget(id[i]);
        }
      }
    }
  } else {
// Several entries of a lane at a time, all loads before the first store: a store to shared memory may, for all
    // that the compiler knows, be to what the next load reads.
    constexpr int N = 8;
    int32_t id[N];
    float x[N];
    for (int j0 = lane; j0 < a.top; j0 += 32 * N) {
      load_entries<N>(a, row, j0, id, x);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        x[i] = id[i] < 0 ? -INFINITY : x[i];
        if (x[i] == -INFINITY) id[i] = -1;
        top = fmaxf(top, x[i]);
        nan |= x[i] != x[i];
        if (j0 + i * 32 < a.top) e.ids[j0 + i * 32] = id[i], e.z[j0 + i * 32] = x[i];
      }
    }
    top = warp_max(top);
    for (int j0 = lane; j0 < a.top; j0 += 32 * N) {
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = j0 + i * 32 < a.top ? e.z[j0 + i * 32] : -INFINITY;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float d = (x[i] - top) * a.inv_t, p = x[i] == -INFINITY ? 0.0f : ex2(d * kLog2E);
        sum += p;
        if (p > 0.0f || p != p) total += p * d;
        if (j0 + i * 32 < a.top) e.q[j0 + i * 32] = p;
      }
    }
    sum = warp_sum(sum), total = warp_sum(total);
    const float inv = 1.0f / sum;
    for (int j0 = lane; j0 < a.top; j0 += 32 * N) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const bool here = j0 + i * 32 < a.top;
        id[i] = here ? e.ids[j0 + i * 32] : -1, x[i] = here ? e.q[j0 + i * 32] : 0.0f;
      }
      bool again[N];
#pragma unroll
      for (int i = 0; i < N; ++i) again[i] = MODE != STATS && id[i] >= lo && id[i] < hi && names.name(id[i]);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int j = j0 + i * 32;
        twice |= again[i];
        if (j >= a.top) continue;
        e.q[j] = e.gq[j] = id[i] < 0 ? 0.0f : x[i] * inv;
        if (MODE != STATS) e.z[j] = again[i] ? 1.0f : 0.0f;
      }
    }
    if (MODE != STATS) {
      __syncwarp();
#pragma unroll 8
      for (int j = lane; j < a.top; j += 32) {
        const int32_t k = e.ids[j];
        if (k >= lo && k < hi) names.forget(k);
      }
    }
  }
  __syncwarp();
  if (MODE != STATS && __any_sync(0xFFFFFFFFu, twice)) join_entries(a.top, e);
  const bool some = sum > 0.0f || sum != sum || __any_sync(0xFFFFFFFFu, nan);
  // sum q log q, with log q = (v - top) / T - log sum
  if (lane == 0) side.mass = some ? 1.0f : 0.0f, side.q_log_q = some ? total / sum - logf(sum) : 0.0f;
}

// The ninth warp (one lane of it): slices into the ring.
template <class T, Mode MODE>
__device__ __forceinline__ void feed(const Args &a, Shared &sh, uint8_t *stages, uint32_t rank, int64_t first, int64_t step) {
  // What L2 is to make of a row that is read again soon, and of one that is not (4096 x 131072 BF16 with and without, BF16 gradients
  // of rows that are read twice stored as what nothing reads again: loss and gradient 389 / 397 us, gradient alone 328 / 329;
  // 8192 x 32768 174 / 176, 166 / 169).
  uint64_t again, once;
  asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(again));
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
  int stage = 0;
  uint32_t parity = 1;
  auto weight_of = [&](int64_t item) { return item < a.items && a.weight ? a.weight[MODE == GRADIENT ? item / a.slices : item] : 1.0f; };
  float ahead = weight_of(first);
  bool skip = (a.fault & 1) != 0 && blockIdx.x == 0;  // test hook: a first stage that stays empty
  for (int64_t item = first; item < a.items; item += step) {
    const int64_t row = MODE == GRADIENT ? item / a.slices : item;
    const float weight = ahead;
    ahead = weight_of(item + step);
    for (int turn = 0; turn < (MODE == TWICE ? 2 * a.rounds : a.rounds); ++turn) {
      const int round = MODE == TWICE && turn >= a.rounds ? turn - a.rounds : turn;
      const Slice<T> slice(a, row, MODE == GRADIENT ? (int32_t)(item - row * a.slices) : (int32_t)rank * a.rounds + round);
      const uint32_t full = tc::smem(&sh.full[stage]);
      tc::bar_wait(tc::smem(&sh.empty[stage]), parity, a.wait_limit_ns, &sh.stop);
      if (weight != 0.0f && slice.units > 0 && !skip) {
        tc::bar_expect(full, slice.units * 16);
        const uint32_t to = tc::smem(stages + stage * a.stage_bytes), bytes = slice.units * 16;
        if constexpr (MODE == GRADIENT || MODE == TWICE)
          asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(to),
                       "l"(slice.at), "r"(bytes), "r"(full), "l"(MODE == TWICE && turn < a.rounds ? again : once)
                       : "memory");
        else
          asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to), "l"(slice.at),
                       "r"(bytes), "r"(full)
                       : "memory");
      } else if (!skip) {
        tc::bar_arrive(full);
      }
      skip = false;
      if (++stage == a.stages) stage = 0, parity ^= 1u;
    }
  }
}

// What a row, or one of its slices, has beside its logits.
template <bool DISTILL, class T, Mode MODE, bool ONCE>
__device__ __forceinline__ void side_of(const Args &a, uint32_t *named, Side &side, int64_t row, int32_t index, const Ahead<DISTILL, MODE> &ahead) {
  const float up = ahead.weight * ahead.dloss;
  if constexpr (DISTILL) {
    if (ahead.weight != 0.0f) {
      const Slice<T> slice(a, row, index);
      teacher_of<DISTILL, MODE, ONCE>(a, named, side, row, MODE == GRADIENT ? slice.begin() : 0, MODE == GRADIENT ? slice.end(a) : a.vocab, ahead);
    }
  }
  if ((threadIdx.x & 31) == 0) {
    side.weight = ahead.weight, side.up = up, side.lse = ahead.lse;
    if constexpr (DISTILL) {
      side.slope = up * a.t;
    } else {
      side.old = ahead.old, side.ref = ahead.ref, side.advantage = ahead.advantage, side.token = ahead.token;
      side.mass = ahead.token >= 0 ? 1.0f : 0.0f;
      if (MODE == GRADIENT) {
        float l, d;
        policy_of(a, ahead.logp, side, l, d);
        side.slope = -d * up * a.inv_t;
      }
    }
  }
}

// The tenth warp: what rows have beside their logits.
template <bool DISTILL, class T, Mode MODE>
__device__ __forceinline__ void prepare(const Args &a, Shared &sh, uint8_t *stages, int64_t first, int64_t step) {
  const int lane = threadIdx.x & 31;
  int side_at = 0;
  uint32_t parity = 1;
  Ahead<DISTILL, MODE> ahead;
  ahead.load(a, first);
  for (int64_t item = first; item < a.items; item += step) {
    const int64_t row = MODE == GRADIENT ? item / a.slices : item;
    tc::bar_wait(tc::smem(&sh.done[side_at]), parity, a.wait_limit_ns, &sh.stop);
    Side &side = *reinterpret_cast<Side *>(stages + a.stages * a.stage_bytes + side_at * a.side_bytes);
    side_of<DISTILL, T, MODE, false>(a, sh.named, side, row, MODE == GRADIENT ? (int32_t)(item - row * a.slices) : 0, ahead);
    __syncwarp();
    if (lane == 0) tc::bar_arrive(tc::smem(&sh.ready[side_at]));
    if (++side_at == a.stages) side_at = 0, parity ^= 1u;
    ahead.load(a, item + step);
  }
}

// ---- the other eight ----------------------------------------------------------------------
// Element e of unit u of the slice that is in shared memory, as the row's element.
template <class T>
__device__ __forceinline__ float staged(const uint8_t *stage, const Slice<T> &s, int32_t element) {
  return (float)reinterpret_cast<const T *>(stage)[element + s.phase - s.first * Slice<T>::kPer];
}

// A thread's units of a slice, one in N, as they are stored; -infinity behind them.
template <class T, int K, int N>
__device__ __forceinline__ void load_units(const uint8_t *units, const Slice<T> &s, int t, uint4 (&r)[K]) {
  constexpr uint32_t kNone = Slice<T>::kPer == 8 ? 0xFF80FF80u : 0xFF800000u;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int u = k * N + t;
    r[k] = u < s.units ? *reinterpret_cast<const uint4 *>(units + u * 16) : make_uint4(kNone, kNone, kNone, kNone);
  }
}
// -infinity in the first and last unit's elements that lie outside the row.
template <class T, int K, int N>
__device__ __forceinline__ void mask_units(const Args &a, const Slice<T> &s, int t, uint4 (&r)[K]) {
  constexpr int P = Slice<T>::kPer;
  constexpr uint32_t kNone = P == 8 ? 0xFF80FF80u : 0xFF800000u;
  if (s.clean) return;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int32_t g = s.first + k * N + t;
    if (g != 0 && g != s.row_units - 1) continue;
    uint32_t w[4] = {r[k].x, r[k].y, r[k].z, r[k].w};
#pragma unroll
    for (int e = 0; e < P; ++e) {
      const int32_t j = g * P + e - s.phase;
      const uint32_t bits = P == 8 ? 0xFFFFu << (e % 2 * 16) : 0xFFFFFFFFu;
      if (j < 0 || j >= a.vocab) w[e * 4 / P] = (w[e * 4 / P] & ~bits) | (kNone & bits);
    }
    r[k] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
template <class T>
__device__ __forceinline__ void unpack(uint4 r, float2 (&z)[Slice<T>::kPer / 2]) {
  if constexpr (sizeof(T) == 2) {
    unpack8(r, z);
  } else {
    z[0] = make_float2(__uint_as_float(r.x), __uint_as_float(r.y)), z[1] = make_float2(__uint_as_float(r.z), __uint_as_float(r.w));
  }
}
template <class T, int K>
__device__ __forceinline__ float top_of(const uint4 (&r)[K]) {
  if constexpr (sizeof(T) == 2) {
    __nv_bfloat162 m[2];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const __nv_bfloat162 *p = reinterpret_cast<const __nv_bfloat162 *>(&r[k]);
      m[0] = k ? __hmax2(m[0], __hmax2(p[0], p[1])) : __hmax2(p[0], p[1]);
      m[1] = k ? __hmax2(m[1], __hmax2(p[2], p[3])) : __hmax2(p[2], p[3]);
    }
    const float2 v = __bfloat1622float2(__hmax2(m[0], m[1]));
    return fmaxf(fmaxf(v.x, v.y), -INFINITY);  // of NaN alone: as of nothing
  } else {
    float m = -INFINITY;
#pragma unroll
    for (int k = 0; k < K; ++k)
      m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(r[k].x), __uint_as_float(r[k].y)), fmaxf(__uint_as_float(r[k].z), __uint_as_float(r[k].w))));
    return m;
  }
}

// (z - from) scale as z scale + by: one operation, with the rounding of `by` taken back afterwards (`left`, of the
// exponent).  That is at most half an ulp of `by`, and so at most 1 up to 2^25; a mask value of -1e10 would leave hundreds, whose power
// of two is infinite.  Beyond, and where `by` is not finite: a difference and a product.
struct Exponent {
  float from, scale, by, left;
  bool quick;
  __device__ __forceinline__ Exponent(float f, float s) : from(f), scale(s) {
    by = -f * s, left = fmaf(f, s, by);
    quick = fabsf(left) <= 1.0f;  // not of a NaN
  }
  __device__ __forceinline__ float2 quickly(float2 z) const { return __ffma2_rn(z, both(scale), both(by)); }
  __device__ __forceinline__ float2 carefully(float2 z) const { return __fmul2_rn(__fadd2_rn(z, both(-from)), both(scale)); }
};
__device__ __forceinline__ float2 ex2(float2 x) { return make_float2(ex2(x.x), ex2(x.y)); }

// Whether units of the gradient's row begin on their own boundaries.
template <class T>
__device__ __forceinline__ bool even_rows(const Args &a, const Slice<T> &s, const void *g_row) {
  return ((uintptr_t)g_row - s.phase * (a.g_bf16 ? 2 : 4)) % (a.g_bf16 ? Slice<T>::kPer * 2 : 16) == 0;
}
// A unit's gradient.  `even`: units of the gradient's rows begin on their own boundaries.
template <class T, Mode MODE>
__device__ __forceinline__ void put_unit(const Args &a, const Slice<T> &s, void *g_row, bool even, int u, const float2 (&v)[Slice<T>::kPer / 2]) {
  constexpr int P = Slice<T>::kPer;
  const int32_t j = (s.first + u) * P - s.phase;
  if (even && (s.clean || (j >= 0 && j + P <= a.vocab))) {
    if constexpr (P == 8) {
      if (MODE == TWICE && a.g_bf16)
        __stcs(reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(g_row) + j),
               make_uint4(bf16_pair(v[0].x, v[0].y), bf16_pair(v[1].x, v[1].y), bf16_pair(v[2].x, v[2].y), bf16_pair(v[3].x, v[3].y)));
      else
        store8(g_row, j, a.g_bf16 != 0, v);
    } else if (a.g_bf16) {
      *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(g_row) + j) = make_uint2(bf16_pair(v[0].x, v[0].y), bf16_pair(v[1].x, v[1].y));
    } else {
      *reinterpret_cast<float4 *>(static_cast<float *>(g_row) + j) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    }
  } else {
#pragma unroll
    for (int e = 0; e < P; ++e)
      if (j + e >= 0 && j + e < a.vocab) store_any(g_row, j + e, a.g_bf16 != 0, element(v, e));
  }
}

// What a row's gradient is made of: part 2^exponent - slope q.
struct Gradient {
  Exponent x;
  float part, slope;
  bool none;
  __device__ __forceinline__ float of(float z) const { return part * ex2((z - x.from) * x.scale); }
};

// A slice's gradient from its logits: `unit(k, u)` gives unit u, the thread's k-th, of which N threads have one each.
template <bool DISTILL, class T, int K, int N, Mode MODE, class Unit>
__device__ __forceinline__ void write_slice(const Args &a, const Slice<T> &slice, int t, Unit unit, void *g_row, bool even, int32_t token,
                                            const Gradient &g) {
  constexpr int P = Slice<T>::kPer;
  if (g.none) {
    float2 v[P / 2];
#pragma unroll
    for (int i = 0; i < P / 2; ++i) v[i] = both(0.0f);
    for (int u = t; u < slice.units; u += N) put_unit<T, MODE>(a, slice, g_row, even, u, v);
    return;
  }
  const int32_t own = DISTILL ? -1 : (token + slice.phase) / P - slice.first;
  const float2 part = both(g.x.quick ? g.part * ex2(-g.x.left) : g.part);
  auto each = [&](auto quick, auto full) {
#pragma unroll(K < 4 || N < kThreads ? K : 4)
    for (int k = 0; k < K; ++k) {
      const int u = k * N + t;
      if (N < kThreads && k * N >= slice.units) break;
      float2 v[P / 2];
      unpack<T>(full || u < slice.units ? unit(k, u) : make_uint4(0, 0, 0, 0), v);
#pragma unroll
      for (int i = 0; i < P / 2; ++i) v[i] = __fmul2_rn(ex2(quick ? g.x.quickly(v[i]) : g.x.carefully(v[i])), part);
      if (!DISTILL && own == u) {
#pragma unroll
        for (int i = 0; i < P; ++i) element(v, i) -= i == (token + slice.phase) % P ? g.slope : 0.0f;
      }
      if (full || u < slice.units) put_unit<T, MODE>(a, slice, g_row, even, u, v);
    }
  };
  if (!g.x.quick)
    each(std::false_type(), std::false_type());
  else if (N == kThreads && slice.units == K * N)
    each(std::true_type(), std::true_type());
  else
    each(std::true_type(), std::false_type());
}
// Once a slice's units are written: the teacher's tokens in it, once more.
template <class T>
__device__ __forceinline__ void write_named(const Args &a, const Slice<T> &slice, void *g_row, const int32_t *ids, const float *gq,
                                            const float *zt, const Gradient &g) {
  workers_sync();
  const int32_t lo = slice.begin(), hi = slice.end(a);
  for (int j = threadIdx.x; j < a.top; j += kThreads)
    if (ids[j] >= lo && ids[j] < hi && !(gq[j] < 0.0f)) store_any(g_row, ids[j], a.g_bf16 != 0, g.of(zt[j]) - g.slope * gq[j]);
}

// A row's results from its maximum M and sum S and what X its targets make of its logits (a teacher's the sum of q (z - M), the
// policy's token its logit); returns the slope of its gradient.
template <bool DISTILL>
__device__ __forceinline__ float results(const Args &a, const Side &side, int64_t row, float weight, float M, float S, float X, bool write) {
  float loss = 0.0f, logp = 0.0f, lse = 0.0f, slope = 0.0f;
  if (weight != 0.0f) {
    const float log_sum = logf(S);
    lse = fmaf(M, a.inv_t, log_sum);
    if constexpr (DISTILL) {
      if (side.mass != 0.0f) loss = weight * a.t * a.t * (side.q_log_q + (log_sum - a.inv_t * X) + (M - M));  // M infinite: NaN
      slope = side.slope;
    } else if (side.token >= 0) {
      logp = fmaf(X - M, a.inv_t, -log_sum);
      policy_of(a, logp, side, loss, slope);
      loss *= weight;
      slope *= -side.up * a.inv_t;
    }
  }
  if (write) {
    a.loss[row] = loss, a.lse[row] = lse;
    if (!DISTILL) a.logp[row] = logp;
  }
  return slope;
}

template <bool DISTILL, class T, int K, Mode MODE>
__device__ __forceinline__ void work(const Args &a, Shared &sh, uint8_t *stages, uint32_t rank, int64_t first, int64_t step) {
  constexpr int P = Slice<T>::kPer;
  const int t = threadIdx.x, lane = t & 31, warp = t / 32;
  int stage_at = 0, side_at = 0, turn = 0;
  uint32_t parity = 0, side_parity = 0;
  auto staged_unit = [](const uint8_t *stage) { return [stage](int, int u) { return *reinterpret_cast<const uint4 *>(stage + u * 16); }; };
  auto next = [&] {  // the stage has been read
    __syncwarp();
    if (lane == 0) tc::bar_arrive(tc::smem(&sh.empty[stage_at]));
    if (++stage_at == a.stages) stage_at = 0, parity ^= 1u;
  };
  for (int64_t item = first; item < a.items; item += step) {
    const int64_t row = MODE == GRADIENT ? item / a.slices : item;
    Side &side = *reinterpret_cast<Side *>(stages + a.stages * a.stage_bytes + side_at * a.side_bytes);
    const Teacher teacher(side, a.top);
    const int32_t *ids = teacher.ids;
    const float *q = teacher.q, *gq = teacher.gq;
    float *zt = teacher.z;
    tc::bar_wait(tc::smem(&sh.ready[side_at]), side_parity, a.wait_limit_ns, &sh.stop);
    const float weight = side.weight;
    const uint32_t done = tc::smem(&sh.done[side_at]);
    if (++side_at == a.stages) side_at = 0, side_parity ^= 1u;
    auto leave = [&] {  // the row's side has been read
      __syncwarp();
      if (lane == 0) tc::bar_arrive(done);
    };
    uint8_t *g_row = static_cast<uint8_t *>(a.dlogits) + row * a.ld_g * (a.g_bf16 ? 2 : 4);
    float m = -INFINITY, sum = 0.0f;                // of the thread, over the block's slices
    float hit = 0.0f, mass = 0.0f, high = -INFINITY;  // what it has of the targets; of a teacher's, relative to the highest
    float held = 1.0f;               // what the exponentials of a row that is held are still to be multiplied by
    float2 e[MODE == HELD ? K : 1][P / 2];
    for (int round = 0; round < a.rounds; ++round) {
      const Slice<T> slice(a, row, MODE == GRADIENT ? (int32_t)(item - row * a.slices) : (int32_t)rank * a.rounds + round);
      const uint8_t *stage = stages + stage_at * a.stage_bytes;
      tc::bar_wait(tc::smem(&sh.full[stage_at]), parity, a.wait_limit_ns, &sh.stop);
      if (weight != 0.0f) {
        auto targets = [&] {  // their logits
          if constexpr (DISTILL) {
            const int32_t lo = slice.begin(), hi = slice.end(a);
            for (int j = t; j < a.top; j += kThreads)
              if (ids[j] >= lo && ids[j] < hi) {
                const float z = staged(stage, slice, ids[j]);
                if (MODE != STATS) zt[j] = z;
                if (MODE != GRADIENT && (q[j] > 0.0f || q[j] != q[j])) {
                  const float top = fmaxf(high, z);
                  hit = raised(raised(hit, mass, high, top), q[j], z, top);
                  mass += q[j], high = top;
                }
              }
          } else if (MODE != GRADIENT) {
            if (t == 0 && side.token >= slice.begin() && side.token < slice.end(a)) hit += staged(stage, slice, side.token);
          }
        };
        // Rows that are held have few registers while their exponentials are made (8192 x 16384 BF16 distillation with gradient 116 us with the
        // targets first, 112 so); others wait less for targets that come first (8192 x 32768 174 and 177).
        constexpr bool kFirst = MODE != HELD || !DISTILL;
        if constexpr (kFirst) targets();
        if constexpr (MODE != GRADIENT) {
          uint4 raw[K];
          load_units<T, K, kThreads>(stage, slice, t, raw);
          mask_units<T, K, kThreads>(a, slice, t, raw);
          const float top = top_of<T, K>(raw);
          const Exponent x(top == -INFINITY ? 0.0f : top, a.scale);
          float2 s = both(0.0f);
          auto each = [&](auto quick) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
              float2 z[P / 2];
              unpack<T>(raw[k], z);
#pragma unroll
              for (int i = 0; i < P / 2; ++i) {
                const float2 y = ex2(quick ? x.quickly(z[i]) : x.carefully(z[i]));
                s = __fadd2_rn(s, y);
                if constexpr (MODE == HELD) e[k][i] = y;
              }
            }
          };
          float whole = 1.0f;
          if (__all_sync(0xFFFFFFFFu, x.quick)) {
            each(std::true_type());
            whole = ex2(-x.left);
          } else {
            each(std::false_type());
          }
          if constexpr (MODE == HELD) held = whole;
          s = __fmul2_rn(s, both(whole));
          if constexpr (MODE == HELD)
            m = top, sum = s.x + s.y;
          else
            merge(m, sum, top, s.x + s.y, a.scale);
        }
        if constexpr (!kFirst) targets();
      }
      if constexpr (MODE == GRADIENT) {
        // p = 2^((z - lse T) / T log2 e)
        const Gradient g = {Exponent(side.lse * a.t, a.scale), side.slope, side.slope, weight == 0.0f || side.mass == 0.0f};
        write_slice<DISTILL, T, K, kThreads, MODE>(a, slice, t, staged_unit(stage), g_row, even_rows<T>(a, slice, g_row), side.token, g);
        if (DISTILL && !g.none) write_named(a, slice, g_row, ids, gq, zt, g);
      }
      if (MODE != HELD) next();
    }
    if constexpr (MODE == GRADIENT) {
      leave();
      continue;
    }
    // The row's maximum and sum.
    float M = DISTILL ? fmaxf(m, high) : m, S = sum, X = hit, W = mass;
    if (weight != 0.0f) {
      const int slot = turn & 1;
#pragma unroll
      for (int d = 16; d > 0; d /= 2) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, d));
      S = sum * below(m, M, a.scale);
#pragma unroll
      for (int d = 16; d > 0; d /= 2) S += __shfl_xor_sync(0xFFFFFFFFu, S, d);
      if (!DISTILL || __any_sync(0xFFFFFFFFu, mass != 0.0f)) {  // few warps have targets
        if (DISTILL) X = raised(hit, mass, high, M);
#pragma unroll
        for (int d = 16; d > 0; d /= 2) {
          X += __shfl_xor_sync(0xFFFFFFFFu, X, d);
          if (DISTILL) W += __shfl_xor_sync(0xFFFFFFFFu, W, d);
        }
      }
      if (lane == 0) sh.warp[slot][warp] = make_float4(M, S, X, W);
      workers_sync();
      // Of n warps or blocks, a power of two: each lane takes one, and all lanes have what they join to.
      auto join = [&](const float4 *p, int n) {
        const float4 v = p[lane & (n - 1)];
        M = v.x;
        for (int d = n / 2; d > 0; d /= 2) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, d));
        S = v.y * below(v.x, M, a.scale), X = DISTILL ? raised(v.z, v.w, v.x, M) : v.z, W = v.w;
        for (int d = n / 2; d > 0; d /= 2) {
          S += __shfl_xor_sync(0xFFFFFFFFu, S, d), X += __shfl_xor_sync(0xFFFFFFFFu, X, d);
          if (DISTILL) W += __shfl_xor_sync(0xFFFFFFFFu, W, d);
        }
      };
      if (MODE != HELD && a.cluster > 1) {
        const uint32_t bar = tc::smem(&sh.arrived[slot]);
        if (warp == 0) {
          join(sh.warp[slot], kWarps);
          if (t < a.cluster) {
            asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(tc::at_rank(tc::smem(&sh.block[slot][rank]), t)), "f"(M),
                         "f"(S), "f"(X), "f"(W)
                         : "memory");
            tc::bar_arrive_cluster(tc::at_rank(bar, t));
          }
          __syncwarp();
        }
        tc::bar_wait(bar, (uint32_t)(turn >> 1) & 1u, a.wait_limit_ns, &sh.stop);
        __syncwarp();
        join(sh.block[slot], a.cluster);
      } else {
        join(sh.warp[slot], kWarps);
      }
      ++turn;
    }
    const float slope = results<DISTILL>(a, side, row, weight, M, S, X, t == 0 && rank == 0);
    if constexpr (MODE == STATS) {
      leave();
      continue;
    }
    const Gradient g = {Exponent(M, a.scale), slope / S, slope, weight == 0.0f || side.mass == 0.0f};
    if constexpr (MODE == HELD) {
      const Slice<T> slice(a, row, 0);
      if (g.none) {
        write_slice<DISTILL, T, K, kThreads, MODE>(a, slice, t, staged_unit(stages), g_row, even_rows<T>(a, slice, g_row), 0, g);
      } else {
        const float2 by = both(g.part * (held * below(m, M, a.scale)));
        const int32_t own = DISTILL ? -1 : (side.token + slice.phase) / P;  // the token's unit
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
          for (int i = 0; i < P / 2; ++i) e[k][i] = __fmul2_rn(e[k][i], by);
          if (!DISTILL && own == k * kThreads + t) {
#pragma unroll
            for (int i = 0; i < P; ++i) element(e[k], i) -= i == (side.token + slice.phase) % P ? slope : 0.0f;
          }
          if (k * kThreads + t < slice.units) put_unit<T, MODE>(a, slice, g_row, even_rows<T>(a, slice, g_row), k * kThreads + t, e[k]);
        }
        if (DISTILL) write_named(a, slice, g_row, ids, gq, zt, g);
      }
      next();
    } else {
      for (int round = 0; round < a.rounds; ++round) {
        const Slice<T> slice(a, row, (int32_t)rank * a.rounds + round);
        tc::bar_wait(tc::smem(&sh.full[stage_at]), parity, a.wait_limit_ns, &sh.stop);
        write_slice<DISTILL, T, K, kThreads, MODE>(a, slice, t, staged_unit(stages + stage_at * a.stage_bytes), g_row, even_rows<T>(a, slice, g_row), side.token, g);
        if (DISTILL && !g.none) write_named(a, slice, g_row, ids, gq, zt, g);
        next();
      }
    }
    leave();
  }
}

template <bool DISTILL, class T, int K, Mode MODE>
__global__ void __launch_bounds__(kBlock, K > 2 ? kBlocks : 3) row_kernel(const __grid_constant__ Args a) {
  extern __shared__ __align__(128) uint8_t stages[];
  __shared__ Shared sh;
  if (threadIdx.x == 0) {
    sh.stop = 0;
    for (int i = 0; i < kMaxStages; ++i) tc::bar_init(tc::smem(&sh.full[i]), 1), tc::bar_init(tc::smem(&sh.empty[i]), kWarps), tc::bar_init(tc::smem(&sh.ready[i]), 1),
          tc::bar_init(tc::smem(&sh.done[i]), kWarps);
    for (int i = 0; i < 2; ++i) tc::bar_init(tc::smem(&sh.arrived[i]), a.cluster);
    tc::bar_init_fence();
  }
  for (int i = threadIdx.x; i < (int)(sizeof(sh.named) / 4); i += kBlock) sh.named[i] = 0;
  wait_for_previous();
  let_next_start();
  if (a.cluster > 1)
    tc::cluster_sync();
  else
    __syncthreads();
  const uint32_t rank = a.cluster > 1 ? tc::cluster_rank() : 0;
  const int64_t first = blockIdx.x / a.cluster, step = gridDim.x / a.cluster;
  if (threadIdx.x == kThreads)
    feed<T, MODE>(a, sh, stages, rank, first, step);
  else if (threadIdx.x >= kThreads + 32)
    prepare<DISTILL, T, MODE>(a, sh, stages, first, step);
  else if (threadIdx.x < kThreads)
    work<DISTILL, T, K, MODE>(a, sh, stages, rank, first, step);
  __syncthreads();
  if (threadIdx.x == 0 && *(volatile uint32_t *)&sh.stop) {
    atomicAdd(a.gave_up, 1u);
    // What is still on its way must arrive before the block's memory is another's: for the limit, at most.
    const uint64_t began = tc::now_ns();
    while (tc::now_ns() - began < 1000000u) {
    }
  }
  if (a.cluster > 1) tc::cluster_sync();  // no block leaves while another may write to it
}

// Short rows, many of them (16384 x 4096 BF16: policy loss 24 us, 5.6 TB/s, with gradient 49 us, 5.4 TB/s): G warps to each,
// its units in registers from the only read on. No row waits for another: latencies of loads and sums are hidden by the
// other warps of an SM, 16 to 32 by what a row's units take in registers (128 registers for 16 units of a lane and a
// teacher, where 96 would spill: loss and gradient of 16384 x 4096 62 us; it was 76 for 69 when tried).
constexpr int kShortThreads = 128;
constexpr int kShortTop = 32 * kEach;
template <bool DISTILL, class T, int K, int G, Mode MODE>
__global__ void __launch_bounds__(kShortThreads, K > 4 ? (DISTILL ? 4 : 5) : 8) short_kernel(const __grid_constant__ Args a) {
  constexpr int P = Slice<T>::kPer, N = 32 * G, kNames = DISTILL && MODE != STATS ? K * P * G : 0;
  extern __shared__ __align__(16) uint8_t sides[];  // of each row: its side, and a bit for each token
  __shared__ float4 meet[kShortThreads / 32];
  const int t = threadIdx.x % N, lane = t % 32, group = threadIdx.x / N;
  const bool leads = t < 32;  // the warp that deals with what the row has beside its logits
  Side &side = *reinterpret_cast<Side *>(sides + group * (a.side_bytes + kNames * 4));
  uint32_t *named = reinterpret_cast<uint32_t *>(reinterpret_cast<uint8_t *>(&side) + a.side_bytes);
  auto sync = [&] {
    if constexpr (G == 1)
      __syncwarp();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(N) : "memory");
  };
  if (leads) {
    for (int i = lane; i < kNames; i += 32) named[i] = 0;
    __syncwarp();
  }
  wait_for_previous();
  let_next_start();
  const int64_t row = (int64_t)blockIdx.x * (kShortThreads / N) + group;
  if (row >= a.rows) return;
  Ahead<DISTILL, MODE> ahead;
  if (leads)
    ahead.load(a, row);
  else if (a.weight)
    ahead.weight = a.weight[row];
  const Slice<T> slice(a, row, 0);
  const T *z_row = static_cast<const T *>(a.logits) + row * a.ld_z;
  uint8_t *g_row = static_cast<uint8_t *>(a.dlogits) + row * a.ld_g * (a.g_bf16 ? 2 : 4);
  const float weight = ahead.weight;
  uint4 raw[K];
  float zt[kEach];  // the targets' logits
  if (weight != 0.0f) {
    load_units<T, K, N>(reinterpret_cast<const uint8_t *>(slice.at), slice, t, raw);
    if constexpr (DISTILL) {
#pragma unroll
      for (int i = 0; i < kEach; ++i) zt[i] = leads && ahead.id[i] >= 0 ? (float)z_row[ahead.id[i]] : 0.0f;
    } else if (MODE != GRADIENT) {
      zt[0] = leads && ahead.token >= 0 ? (float)z_row[ahead.token] : 0.0f;
    }
  }
  if (leads) {
    side_of<DISTILL, T, MODE, true>(a, named, side, row, 0, ahead);
    __syncwarp();
  }
  const Teacher teacher(side, a.top);
  Gradient g = {Exponent(0.0f, a.scale), 0.0f, 0.0f, true};
  if constexpr (MODE == GRADIENT) {
    sync();
    g = {Exponent(side.lse * a.t, a.scale), side.slope, side.slope, weight == 0.0f || side.mass == 0.0f};
  } else {
    float M = 0.0f, S = 1.0f, X = 0.0f;
    if (weight != 0.0f) {
      mask_units<T, K, N>(a, slice, t, raw);
      const float m = top_of<T, K>(raw);
      const Exponent x(m == -INFINITY ? 0.0f : m, a.scale);
      float2 s = both(0.0f);
      auto each = [&](auto quick) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
          if (k * N >= slice.units) break;
          float2 z[P / 2];
          unpack<T>(raw[k], z);
#pragma unroll
          for (int i = 0; i < P / 2; ++i) s = __fadd2_rn(s, ex2(quick ? x.quickly(z[i]) : x.carefully(z[i])));
        }
      };
      float whole = 1.0f;
      if (__all_sync(0xFFFFFFFFu, x.quick)) {
        each(std::true_type());
        whole = ex2(-x.left);
      } else {
        each(std::false_type());
      }
      if constexpr (!DISTILL) X = zt[0];
      M = warp_max(m);
      S = warp_sum((s.x + s.y) * whole * below(m, M, a.scale));
    }
    if constexpr (G > 1) {
      if (lane == 0) meet[threadIdx.x / 32] = make_float4(M, S, X, 0.0f);
      sync();
      const float4 *v = meet + group * G;
      M = v[0].x, S = v[0].y, X = v[0].z;
#pragma unroll
      for (int w = 1; w < G; ++w) merge(M, S, v[w].x, v[w].y, a.scale);
    }
    if (DISTILL && leads && weight != 0.0f) {
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int j = i * 32 + lane;
        if (j < a.top && teacher.ids[j] >= 0 && (teacher.q[j] > 0.0f || teacher.q[j] != teacher.q[j])) X = raised(X, teacher.q[j], zt[i], M);
      }
      X = warp_sum(X);
    }
    const float slope = results<DISTILL>(a, side, row, weight, M, S, X, t == 0);
    g = {Exponent(M, a.scale), slope / S, slope, weight == 0.0f || side.mass == 0.0f};
  }
  if constexpr (MODE != STATS) {
    write_slice<DISTILL, T, K, N, MODE>(a, slice, t, [&](int k, int) { return raw[k]; }, g_row, even_rows<T>(a, slice, g_row), side.token, g);
    if constexpr (DISTILL) {
      sync();
      if (!leads) return;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int j = i * 32 + lane;
        if (!g.none && j < a.top && teacher.ids[j] >= 0 && !(teacher.gq[j] < 0.0f))
          store_any(g_row, teacher.ids[j], a.g_bf16 != 0, g.of(zt[i]) - g.slope * teacher.gq[j]);
      }
    }
  }
}

// ---- host --------------------------------------------------------------------------------
template <class K>
const void *kernel(K *k) {
  return reinterpret_cast<const void *>(k);
}

// Blocks of a launch that the device holds at once, in whole clusters.
cudaError_t resident(const void *fn, int cluster, int smem, int *clusters) {
  struct Known {
    const void *fn;
    int device, cluster, smem, clusters;
  };
  static std::mutex lock;
  static Known known[64];
  static int n = 0, oldest = 0;
  int device = -1;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  {
    std::lock_guard<std::mutex> hold(lock);
    for (int i = 0; i < n; ++i)
      if (known[i].fn == fn && known[i].device == device && known[i].cluster == cluster && known[i].smem == smem) {
        *clusters = known[i].clusters;
        return cudaSuccess;
      }
  }
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);  // one value: the last one set holds
  if (e != cudaSuccess) return e;
  int most = 0;
  if (cluster > 1) {
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)cluster, at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(cluster * 1024)), cfg.blockDim = dim3(kBlock);
    cfg.dynamicSmemBytes = (size_t)smem, cfg.attrs = &at, cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&most, fn, &cfg);
  } else {
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&most, fn, kBlock, (size_t)smem);
    most *= device_sms();
  }
  if (e != cudaSuccess) return e;
  if (most < 1) return cudaErrorInvalidConfiguration;
  std::lock_guard<std::mutex> hold(lock);
  Known &k = n < 64 ? known[n++] : known[oldest++ & 63];
  k = {fn, device, cluster, smem, most};
  *clusters = most;
  return cudaSuccess;
}

// Units of the longest row, which may begin anywhere in its first.
template <class T>
int64_t units_of(const Args &a) {
  constexpr int P = Slice<T>::kPer;
  return (a.vocab + P - 1) / P + ((uintptr_t)a.logits % 16 != 0 || (a.rows > 1 && a.ld_z % P != 0) ? 1 : 0);
}

template <bool DISTILL, class T, Mode MODE>
cudaError_t launch_rows(Args &a, cudaStream_t s) {
  constexpr int64_t kMost = kThreads * kMostUnits;
  const int64_t row_units = units_of<T>(a);
  a.cluster = a.slices = 1;
  int64_t least = 1;
  if (MODE == GRADIENT) {
    a.slices = (int32_t)((row_units + kMost - 1) / kMost);
  } else if (MODE != HELD) {
    // Few rows: as many blocks to a row as the SMs have room for, with 256 units each at least. Rows that are read twice: as
    // many as it takes for all rows at work to stay in L2. Clusters of three or five leave SMs idle (us, BF16, with a power of
    // two / without: 61 x 131072 loss alone 6.5 / 9.8, 102 x 32768 5.1 / 7.7, 2048 x 200000 with gradient 307 / 480).
    const int64_t blocks = kBlocks * device_sms(), room = std::min<int64_t>(blocks / a.rows, row_units / kThreads);
    if (MODE == TWICE) least = (blocks * row_units * 16 + kL2Rows - 1) / kL2Rows;
    while (a.cluster < kMaxCluster && (a.cluster * 2 <= room || a.cluster < least)) a.cluster *= 2;
  }
  a.items = a.rows * a.slices;
  a.side_bytes = ((int)sizeof(Side) + (DISTILL ? a.top * 16 : 0) + 127) / 128 * 128;
  const void *fn = nullptr;
  int smem = 0, clusters = 0;
  cudaError_t e;
  for (;; a.cluster /= 2) {
    a.rounds = MODE == STATS || MODE == TWICE ? (int32_t)((row_units + kMost * a.cluster - 1) / (kMost * a.cluster)) : 1;
    const int64_t parts = (int64_t)a.cluster * a.rounds * a.slices;
    a.units = (int32_t)((row_units + parts - 1) / parts);
    fn = a.units <= 2 * kThreads ? kernel(&row_kernel<DISTILL, T, 2, MODE>) : kernel(&row_kernel<DISTILL, T, kMostUnits, MODE>);
    a.stage_bytes = (a.units * 16 + 127) / 128 * 128;
    a.stages = stages_of_mode(MODE);  // as many as leave room for the SM's other blocks
    while (a.stages > 2 && a.stages * (a.stage_bytes + a.side_bytes) > kMostSmem) --a.stages;
    smem = a.stages * (a.stage_bytes + a.side_bytes);
    if ((e = resident(fn, a.cluster, smem, &clusters)) != cudaSuccess) return e;
    // Large clusters do not fill all SMs: rather smaller ones than a second turn (us: 76 x 131072 in BF16, loss alone, 7.7 / 9.9).
    if (a.cluster / 2 < least || a.cluster == 1 || a.rows <= clusters) break;
  }
  e = gave_up_count(GAVE_UP_LOSS, &a.gave_up);
  if (e != cudaSuccess) return e;
  a.wait_limit_ns = wait_limit_ns(), a.fault = wait_fault();
  const int64_t grid = std::min<int64_t>(a.items, clusters) * a.cluster;
  void *args[] = {&a};
  return launch_kernel(fn, dim3((unsigned)grid), dim3(kBlock), args, (size_t)smem, s, true, a.cluster);
}

template <bool DISTILL, class T, int K, int G, Mode MODE>
cudaError_t launch_short(Args &a, cudaStream_t s) {
  constexpr int kRows = kShortThreads / (32 * G), kNames = DISTILL && MODE != STATS ? K * G * Slice<T>::kPer * 4 : 0;
  static_assert(kRows * ((int)sizeof(Side) + kShortTop * 16 + kNames) <= 47 * 1024, "more than any kernel may have");
  a.cluster = a.rounds = a.slices = 1;
  a.units = K * G * 32, a.items = a.rows;
  a.side_bytes = ((int)sizeof(Side) + (DISTILL ? a.top * 16 : 0) + 15) / 16 * 16;
  void *args[] = {&a};
  return launch_kernel(kernel(&short_kernel<DISTILL, T, K, G, MODE>), dim3((unsigned)((a.rows + kRows - 1) / kRows)), dim3(kShortThreads), args,
                       (size_t)(kRows * (a.side_bytes + kNames)), s, true);
}

template <bool DISTILL, class T, Mode MODE>
cudaError_t launch_mode(Args &a, cudaStream_t s) {
  // Rows of a block, one after another, are bound by the latency of their sums, and rows of a warp or two by bytes (us by
  // block / so, BF16: distillation loss 16384 x 512 74 / 12, 16384 x 4096 93 / 30, 8192 x 8192 55 / 37, 16 x 4096 4.6 / 3.1; with
  // gradient 93 / 18, 117 / 62, 86 / 67). A gradient's rows have to be enough for all SMs (512 x 4096 6.6 / 6.8, 1024 x 4096
  // 9.4 / 8.0). Four warps to a row wait too long for one's teacher, but not for the policy's scalars (8192 x 16384 distillation
  // 55 / 71, with gradient 113 / 130; policy 55 / 46, 104 / 95).
  const int64_t units = units_of<T>(a);
  if (a.top <= kShortTop && (MODE == STATS || a.rows > 4 * device_sms())) {
    if (units <= 128) return launch_short<DISTILL, T, 4, 1, MODE>(a, s);
    if (units <= 512) return launch_short<DISTILL, T, 16, 1, MODE>(a, s);
    if (units <= 1024) return launch_short<DISTILL, T, 16, 2, MODE>(a, s);
    if constexpr (!DISTILL)
      if (units <= 2048) return launch_short<DISTILL, T, 16, 4, MODE>(a, s);
  }
  if (MODE == HELD && units > kThreads * kMostUnits) return launch_rows<DISTILL, T, TWICE>(a, s);
  return launch_rows<DISTILL, T, MODE>(a, s);
}
template <bool DISTILL, class T>
cudaError_t launch_as(Args &a, cudaStream_t s) {
  if (a.backward) return launch_mode<DISTILL, T, GRADIENT>(a, s);
  return a.dlogits ? launch_mode<DISTILL, T, HELD>(a, s) : launch_mode<DISTILL, T, STATS>(a, s);
}

template <bool DISTILL>
fsdp_status_t run(Args &a, cudaStream_t s) {
  a.scale = a.inv_t * kLog2E;
  return launched(a.z_bf16 ? launch_as<DISTILL, __nv_bfloat16>(a, s) : launch_as<DISTILL, float>(a, s));
}

fsdp_status_t check_rows(const float *p, int64_t rows, bool needed, const char *what) {
  if (!needed && !p) return FSDP_OK;
  return check_ptr(p, rows * 4, 4, what, -1);
}

// What the two losses' descriptors have in common.
template <class D>
fsdp_status_t check(const D *d, const void *logits, void *dlogits, bool backward) {
  if (!d) return fail(FSDP_EINVAL, "desc is NULL");
  if (d->rows < 0 || d->vocab < 1) return fail(FSDP_EINVAL, "rows < 0 or vocab < 1");
  if (d->vocab > INT32_MAX - 63) return fail(FSDP_EUNSUPPORTED, "a vocabulary of 2^31 - 63 or more");  // places in whole units
  if (d->rows > INT64_MAX / 64 / d->vocab) return fail(FSDP_EUNSUPPORTED, "the matrices are too large");
  if (!float_dtype(d->logits_dtype)) return fail(FSDP_EINVAL, "unknown logits_dtype");
  if (d->token_dtype != FSDP_INDEX_I32 && d->token_dtype != FSDP_INDEX_I64) return fail(FSDP_EINVAL, "unknown token_dtype");
  if (!(d->temperature > 0.0f) || !(1.0f / d->temperature > 0.0f) || std::isinf(1.0f / d->temperature))
    return fail(FSDP_EINVAL, "temperature is not a positive number whose inverse is finite");
  fsdp_status_t st = check_matrix(logits, d->rows, d->vocab, d->ld_logits, dtype_bytes(d->logits_dtype), "logits");
  if (st != FSDP_OK || (!dlogits && !backward)) return st;
  if (!float_dtype(d->dlogits_dtype)) return fail(FSDP_EINVAL, "unknown dlogits_dtype");
  if ((st = check_matrix(dlogits, d->rows, d->vocab, d->ld_dlogits, dtype_bytes(d->dlogits_dtype), "dlogits")) != FSDP_OK) return st;
  if (dlogits == logits && d->rows > 0 && (d->logits_dtype != d->dlogits_dtype || (d->rows > 1 && d->ld_logits != d->ld_dlogits)))
    return fail(FSDP_EINVAL, "dlogits is logits, but its dtype or row distance is another");
  return FSDP_OK;
}

template <class D>
Args args_of(const D &d, const void *logits, const void *tokens, const float *weight, void *dlogits) {
  Args a = {};
  a.logits = logits, a.tokens = tokens, a.weight = weight, a.dlogits = dlogits;
  a.rows = d.rows, a.vocab = (int32_t)d.vocab, a.ld_z = d.ld_logits, a.ld_g = d.ld_dlogits;
  a.z_bf16 = d.logits_dtype == FSDP_DTYPE_BF16, a.g_bf16 = d.dlogits_dtype == FSDP_DTYPE_BF16;
  a.wide = d.token_dtype == FSDP_INDEX_I64;
  a.t = d.temperature, a.inv_t = 1.0f / d.temperature;
  return a;
}

fsdp_status_t distill(const fsdp_distill_desc_t *d, Args a, cudaStream_t s) {
  const int64_t tsize = d->token_dtype == FSDP_INDEX_I64 ? 8 : 4;
  fsdp_status_t st;
  if (d->top < 0) return fail(FSDP_EINVAL, "top < 0");
  if (d->top > kMaxTop) return fail(FSDP_EUNSUPPORTED, "top is above FSDP_DISTILL_MAX_TOP");
  if (!float_dtype(d->teacher_dtype)) return fail(FSDP_EINVAL, "unknown teacher_dtype");
  if ((st = check_matrix(a.tokens, d->rows, d->top, d->ld_tokens, tsize, "teacher_tokens")) != FSDP_OK) return st;
  if ((st = check_matrix(a.teacher, d->rows, d->top, d->ld_teacher, dtype_bytes(d->teacher_dtype), "teacher_logits")) != FSDP_OK) return st;
  a.top = (int32_t)d->top, a.ld_tokens = d->ld_tokens, a.ld_teacher = d->ld_teacher;
  a.teacher_bf16 = d->teacher_dtype == FSDP_DTYPE_BF16;
  if (d->rows > 0 && (st = run<true>(a, s)) != FSDP_OK) return st;
  clear_error();
  return FSDP_OK;
}

fsdp_status_t policy(const fsdp_policy_desc_t *d, Args a, cudaStream_t s) {
  const int64_t tsize = d->token_dtype == FSDP_INDEX_I64 ? 8 : 4;
  fsdp_status_t st;
  if (!(d->clip_low >= 0.0f) || !(d->clip_high >= 0.0f)) return fail(FSDP_EINVAL, "clip_low or clip_high is not >= 0");
  if (!(d->kl >= 0.0f) || std::isinf(d->kl)) return fail(FSDP_EINVAL, "kl is not a finite number >= 0");
  if ((st = check_ptr(a.tokens, d->rows * tsize, tsize, "tokens", -1)) != FSDP_OK) return st;
  if ((st = check_rows(a.old_logp, d->rows, false, "old_logp")) != FSDP_OK) return st;
  if ((st = check_rows(a.ref_logp, d->rows, false, "ref_logp")) != FSDP_OK) return st;
  if ((st = check_rows(a.advantage, d->rows, true, "advantage")) != FSDP_OK) return st;
  a.low = 1.0f - d->clip_low, a.high = 1.0f + d->clip_high, a.kl = d->kl;
  if (d->rows > 0 && (st = run<false>(a, s)) != FSDP_OK) return st;
  clear_error();
  return FSDP_OK;
}

}  // namespace
}  // namespace loss
}  // namespace fsdp

using namespace fsdp;
using namespace fsdp::loss;

extern "C" {

fsdp_status_t fsdp_distill_loss_forward(const fsdp_distill_desc_t *desc, const void *logits, const void *teacher_tokens,
                                        const void *teacher_logits, const float *weight, float *loss, float *lse, void *dlogits,
                                        fsdp_stream_t stream) {
  fsdp_status_t st = check(desc, logits, dlogits, false);
  if (st != FSDP_OK) return st;
  if ((st = check_rows(weight, desc->rows, false, "weight")) != FSDP_OK) return st;
  if ((st = check_rows(loss, desc->rows, true, "loss")) != FSDP_OK) return st;
  if ((st = check_rows(lse, desc->rows, true, "lse")) != FSDP_OK) return st;
  Args a = args_of(*desc, logits, teacher_tokens, weight, dlogits);
  a.teacher = teacher_logits, a.loss = loss, a.lse = lse;
  return distill(desc, a, reinterpret_cast<cudaStream_t>(stream));
}

fsdp_status_t fsdp_distill_loss_backward(const fsdp_distill_desc_t *desc, const void *logits, const void *teacher_tokens,
                                         const void *teacher_logits, const float *weight, const float *lse, const float *dloss,
                                         void *dlogits, fsdp_stream_t stream) {
  fsdp_status_t st = check(desc, logits, dlogits, true);
  if (st != FSDP_OK) return st;
  if ((st = check_rows(weight, desc->rows, false, "weight")) != FSDP_OK) return st;
  if ((st = check_rows(lse, desc->rows, true, "lse")) != FSDP_OK) return st;
  if ((st = check_rows(dloss, desc->rows, false, "dloss")) != FSDP_OK) return st;
  Args a = args_of(*desc, logits, teacher_tokens, weight, dlogits);
  a.teacher = teacher_logits, a.lse_in = lse, a.dloss = dloss, a.backward = 1;
  return distill(desc, a, reinterpret_cast<cudaStream_t>(stream));
}

fsdp_status_t fsdp_policy_loss_forward(const fsdp_policy_desc_t *desc, const void *logits, const void *tokens, const float *old_logp,
                                       const float *ref_logp, const float *advantage, const float *weight, float *loss, float *logp,
                                       float *lse, void *dlogits, fsdp_stream_t stream) {
  fsdp_status_t st = check(desc, logits, dlogits, false);
  if (st != FSDP_OK) return st;
  if ((st = check_rows(weight, desc->rows, false, "weight")) != FSDP_OK) return st;
  if ((st = check_rows(loss, desc->rows, true, "loss")) != FSDP_OK) return st;
  if ((st = check_rows(logp, desc->rows, true, "logp")) != FSDP_OK) return st;
  if ((st = check_rows(lse, desc->rows, true, "lse")) != FSDP_OK) return st;
  Args a = args_of(*desc, logits, tokens, weight, dlogits);
  a.old_logp = old_logp, a.ref_logp = ref_logp, a.advantage = advantage, a.loss = loss, a.logp = logp, a.lse = lse;
  return policy(desc, a, reinterpret_cast<cudaStream_t>(stream));
}

fsdp_status_t fsdp_policy_loss_backward(const fsdp_policy_desc_t *desc, const void *logits, const void *tokens, const float *old_logp,
                                        const float *ref_logp, const float *advantage, const float *weight, const float *logp,
                                        const float *lse, const float *dloss, void *dlogits, fsdp_stream_t stream) {
  fsdp_status_t st = check(desc, logits, dlogits, true);
  if (st != FSDP_OK) return st;
  if ((st = check_rows(weight, desc->rows, false, "weight")) != FSDP_OK) return st;
  if ((st = check_rows(logp, desc->rows, true, "logp")) != FSDP_OK) return st;
  if ((st = check_rows(lse, desc->rows, true, "lse")) != FSDP_OK) return st;
  if ((st = check_rows(dloss, desc->rows, false, "dloss")) != FSDP_OK) return st;
  Args a = args_of(*desc, logits, tokens, weight, dlogits);
  a.old_logp = old_logp, a.ref_logp = ref_logp, a.advantage = advantage;
  a.logp_in = logp, a.lse_in = lse, a.dloss = dloss, a.backward = 1;
  return policy(desc, a, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"

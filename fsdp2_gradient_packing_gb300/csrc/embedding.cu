// Embedding lookup with scaling (fsdp_embedding_forward) and its gradient by sorted
// tokens (fsdp_embedding_backward).
//
// The lookup moves rows: a warp takes a run of up to kRowSpan columns of a row, its loads in flight together.
//
// The gradient sorts the tokens with their positions (least significant digit first, so
// equal tokens keep their order), cuts the sorted list into pieces of equal length and
// sums each piece's rows where they lie: a warp to a piece and 256 columns, eight rows of
// loads in flight.  What a token's rows amount to within one piece is written at once;
// where they go on into other pieces, each piece leaves its part in the workspace, and
// the parts are joined in order.  So the work is balanced whatever the frequencies, sums run in
// an order that depends on the sizes alone, and no atomic touches a result.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <string>

#include "layout.h"
#include "ops.h"

namespace fsdp {
namespace embedding {
namespace {

constexpr int kThreads = 256;

// Index i of a list of 32- or 64-bit tokens; anything outside [0, vocab) gives vocab.
__device__ __forceinline__ uint32_t token_at(const void *tokens, int64_t i, bool wide, uint32_t vocab) {
  if (wide) {
    const uint64_t t = (uint64_t)static_cast<const int64_t *>(tokens)[i];
    return t < vocab ? (uint32_t)t : vocab;
  }
  return min(static_cast<const uint32_t *>(tokens)[i], vocab);
}

// ---- lookup ------------------------------------------------------------------
struct LookupArgs {
  const void *tokens, *weight;
  void *out;
  int64_t rows, cols, ld_weight, ld_out;
  int64_t runs;  // of a row
  uint32_t vocab;
  int32_t wide;
  float scale;
};

template <class T>
__device__ __forceinline__ T to(float v) {
  if constexpr (sizeof(T) == 2)
    return __float2bfloat16_rn(v);
  else
    return v;
}

constexpr int kUnroll = 4;

// A warp to a run of 8 * 32 * kUnroll columns (VEC) or 32 * 2 * kUnroll (one by one).
template <class TW, class TO, bool VEC>
__global__ void __launch_bounds__(kThreads) lookup_kernel(const __grid_constant__ LookupArgs a) {
  constexpr int kSpan = VEC ? 256 * kUnroll : 64 * kUnroll;
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  wait_for_previous();
  let_next_start();
  const int64_t row = unit / a.runs, first = (unit - row * a.runs) * kSpan;
  if (row >= a.rows) return;
  const uint32_t token = token_at(a.tokens, row, a.wide != 0, a.vocab);
  const TW *w = static_cast<const TW *>(a.weight) + (int64_t)token * a.ld_weight;
  TO *o = static_cast<TO *>(a.out) + row * a.ld_out;
  const bool there = token < a.vocab;
  if constexpr (VEC) {
    float2 v[kUnroll][4];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t j = first + u * 256 + lane * 8;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[u][e] = both(0.0f);
      if (there && j < a.cols) load8(w, j, sizeof(TW) == 2, v[u]);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t j = first + u * 256 + lane * 8;
      if (j >= a.cols) break;
      if (there) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[u][e] = __fmul2_rn(v[u][e], both(a.scale));
      }
      store8(o, j, sizeof(TO) == 2, v[u]);
    }
  } else {
    float v[2 * kUnroll];
#pragma unroll
    for (int u = 0; u < 2 * kUnroll; ++u) {
      const int64_t j = first + u * 32 + lane;
      v[u] = there && j < a.cols ? (float)w[j] * a.scale : 0.0f;
    }
#pragma unroll
    for (int u = 0; u < 2 * kUnroll; ++u) {
      const int64_t j = first + u * 32 + lane;
      if (j < a.cols) o[j] = to<TO>(v[u]);
    }
  }
}

// ---- sorting -----------------------------------------------------------------
// A pass sorts by one digit of up to kMaxBits bits: each block counts its kTile items by
// digit, then places them behind what the counts of lower digits and earlier blocks say.
// Within a block the order is that of the items: a warp takes consecutive ones, 32 at a
// time, and ranks equal digits by lane, so a pass keeps the order of the one before.
constexpr int kSortThreads = 512, kItems = 8, kTile = kSortThreads * kItems, kMaxBits = 10, kMaxBins = 1 << kMaxBits;
constexpr int kSortWarps = kSortThreads / 32;

struct SortArgs {
  const void *tokens;                        // first pass: the caller's; later passes: keys
  const uint32_t *keys_in, *order_in;
  uint32_t *keys, *order;
  uint32_t *counts;                          // [blocks][bins] of this pass
  int64_t rows;
  uint32_t vocab, blocks;
  int32_t wide, bits, shift;
};

__device__ __forceinline__ uint32_t sort_key(const SortArgs &a, int64_t i) {
  return a.tokens ? token_at(a.tokens, i, a.wide != 0, a.vocab) : a.keys_in[i];
}

__global__ void __launch_bounds__(kSortThreads) count_kernel(const __grid_constant__ SortArgs a) {
  __shared__ uint32_t bin[kMaxBins];
  const int bins = 1 << a.bits;
  for (int d = threadIdx.x; d < bins; d += kSortThreads) bin[d] = 0;
  wait_for_previous();
  let_next_start();
  __syncthreads();
  const int64_t first = (int64_t)blockIdx.x * kTile;
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    const int64_t i = first + k * kSortThreads + threadIdx.x;
    if (i < a.rows) atomicAdd(&bin[(sort_key(a, i) >> a.shift) & (bins - 1)], 1u);
  }
  __syncthreads();
  for (int d = threadIdx.x; d < bins; d += kSortThreads) a.counts[(int64_t)blockIdx.x * bins + d] = bin[d];
}

__global__ void __launch_bounds__(kSortThreads) place_kernel(const __grid_constant__ SortArgs a) {
  __shared__ uint16_t seen[kSortWarps][kMaxBins];  // then: items of earlier warps
  __shared__ uint32_t base[kMaxBins];              // where the block's items of a digit go
  __shared__ uint32_t total[kSortWarps];
  const int bins = 1 << a.bits, lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  for (int i = threadIdx.x; i < kSortWarps * kMaxBins / 2; i += kSortThreads) reinterpret_cast<uint32_t *>(seen)[i] = 0;
  wait_for_previous();
  let_next_start();
  // Where each digit's items start: those of lower digits, then those of earlier blocks.  A
  // thread sums two neighbouring digits (bins are at least 2).
  uint32_t before[2] = {0, 0}, all[2] = {0, 0};
  const int d = threadIdx.x * 2;
  if (d < bins) {
    const uint2 *p = reinterpret_cast<const uint2 *>(a.counts + d);
#pragma unroll 8
    for (uint32_t b = 0; b < a.blocks; ++b) {
      const uint2 c = p[(int64_t)b * (bins / 2)];
      all[0] += c.x, all[1] += c.y;
      if (b < blockIdx.x) before[0] += c.x, before[1] += c.y;
    }
  }
  uint32_t run = all[0] + all[1];
#pragma unroll
  for (int m = 1; m < 32; m *= 2) {
    const uint32_t up = __shfl_up_sync(0xFFFFFFFFu, run, m);
    if (lane >= m) run += up;
  }
  if (lane == 31) total[warp] = run;
  __syncthreads();
  for (int w = 0; w < warp; ++w) run += total[w];
  if (d < bins) {
    base[d] = run - all[0] - all[1] + before[0];
    base[d + 1] = run - all[1] + before[1];
  }
  // Ranks within the warp's items of the same digit.
  const int64_t first = (int64_t)blockIdx.x * kTile + warp * (32 * kItems) + lane;
  uint32_t key[kItems], from[kItems], rank[kItems];
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    const int64_t i = first + k * 32;
    key[k] = i < a.rows ? sort_key(a, i) : 0;
    from[k] = i < a.rows && !a.tokens ? a.order_in[i] : (uint32_t)i;
  }
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    const bool here = first + k * 32 < a.rows;
    const uint32_t digit = (key[k] >> a.shift) & (bins - 1);
    uint32_t same = __ballot_sync(0xFFFFFFFFu, here);
    for (int b = 0; b < a.bits; ++b) {
      const uint32_t ones = __ballot_sync(0xFFFFFFFFu, digit >> b & 1);
      same &= digit >> b & 1 ? ones : ~ones;
    }
    const uint32_t earlier = same & ((1u << lane) - 1);
    rank[k] = here ? seen[warp][digit] + __popc(earlier) : 0;
    __syncwarp();
    if (here && !earlier) seen[warp][digit] = (uint16_t)(rank[k] + __popc(same));
    __syncwarp();
  }
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += kSortThreads) {
    uint32_t sum = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
      const uint32_t n = seen[w][b];
      seen[w][b] = (uint16_t)sum;
      sum += n;
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    if (first + k * 32 >= a.rows) break;
    const uint32_t digit = (key[k] >> a.shift) & (bins - 1), at = base[digit] + seen[warp][digit] + rank[k];
    a.keys[at] = key[k];
    a.order[at] = from[k];
  }
}

// ---- sums --------------------------------------------------------------------
struct SumArgs {
  const uint32_t *keys, *order;
  const void *dout;
  void *grad;
  float *parts;     // [pieces][2][cols]: what a piece has of a token that began before it, and of one that goes on
  int64_t rows, cols, ld_dout, ld_grad;
  int64_t strips;   // of columns
  int64_t pieces;
  int32_t length;   // of a piece
  uint32_t vocab;
  int32_t add;
  float scale;
};

constexpr int kBatch = 8;  // rows of loads in flight

// Eight columns of a lane (VEC: consecutive, 256 columns to a warp), or two 32 apart.
template <bool VEC>
struct Strip {
  static constexpr int kCols = VEC ? 256 : 64;
};

template <class TD, bool VEC>
struct Loaded;
template <>
struct Loaded<__nv_bfloat16, true> {
  uint4 r;
  __device__ void load(const __nv_bfloat16 *p, int64_t j, int64_t cols) {
    r = j < cols ? __ldcs(reinterpret_cast<const uint4 *>(p + j)) : make_uint4(0, 0, 0, 0);
  }
  __device__ void add_to(float2 (&s)[4]) const {
    float2 v[4];
    unpack8(r, v);
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] = __fadd2_rn(s[e], v[e]);
  }
};
template <>
struct Loaded<float, true> {
  float4 a, b;
  __device__ void load(const float *p, int64_t j, int64_t cols) {
    a = b = make_float4(0, 0, 0, 0);
    if (j < cols) a = __ldcs(reinterpret_cast<const float4 *>(p + j)), b = __ldcs(reinterpret_cast<const float4 *>(p + j) + 1);
  }
  __device__ void add_to(float2 (&s)[4]) const {
    s[0] = __fadd2_rn(s[0], make_float2(a.x, a.y)), s[1] = __fadd2_rn(s[1], make_float2(a.z, a.w));
    s[2] = __fadd2_rn(s[2], make_float2(b.x, b.y)), s[3] = __fadd2_rn(s[3], make_float2(b.z, b.w));
  }
};
template <class TD>
struct Loaded<TD, false> {
  float v[2];
  __device__ void load(const TD *p, int64_t j, int64_t cols) {
    v[0] = j < cols ? (float)p[j] : 0.0f;
    v[1] = j + 32 < cols ? (float)p[j + 32] : 0.0f;
  }
  __device__ void add_to(float2 (&s)[4]) const { s[0].x += v[0], s[0].y += v[1]; }
};

// The sum of a token's rows into its row of the gradient.
template <class TG, bool VEC>
__device__ __forceinline__ void write_row(const SumArgs &a, uint32_t token, int64_t j, const float2 (&sum)[4]) {
  TG *g = static_cast<TG *>(a.grad) + (int64_t)token * a.ld_grad;
  if constexpr (VEC) {
    if (j >= a.cols) return;
    float2 v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = __fmul2_rn(sum[e], both(a.scale));
    if (a.add) {
      float2 old[4];
      load8(g, j, sizeof(TG) == 2, old);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = __ffma2_rn(sum[e], both(a.scale), old[e]);
    }
    store8(g, j, sizeof(TG) == 2, v);
  } else {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int64_t c = j + e * 32;
      const float s = e ? sum[0].y : sum[0].x;
      if (c < a.cols) g[c] = to<TG>(a.add ? fmaf(s, a.scale, (float)g[c]) : s * a.scale);
    }
  }
}
template <bool VEC>
__device__ __forceinline__ float *part_of(const SumArgs &a, int64_t piece, int which) {
  return a.parts + (piece * 2 + which) * ((a.cols + 7) / 8 * 8);
}
template <bool VEC>
__device__ __forceinline__ void write_part(const SumArgs &a, int64_t piece, int which, int64_t j, const float2 (&sum)[4]) {
  float *p = part_of<VEC>(a, piece, which);
  if constexpr (VEC) {
    if (j < a.cols) store8(p, j, false, sum);
  } else {
    if (j < a.cols) p[j] = sum[0].x;
    if (j + 32 < a.cols) p[j + 32] = sum[0].y;
  }
}

template <class TD, class TG, bool VEC>
__global__ void __launch_bounds__(kThreads) sum_kernel(const __grid_constant__ SumArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  wait_for_previous();
  let_next_start();
  const int64_t piece = unit / a.strips;
  if (piece >= a.pieces) return;
  const int64_t j = (unit - piece * a.strips) * Strip<VEC>::kCols + lane * (VEC ? 8 : 1);
  const int64_t first = piece * a.length, end = min(first + a.length, a.rows);
  // The first token of the piece began before it; the last one goes on behind it.
  const uint32_t ahead = first > 0 ? a.keys[first - 1] : 0xFFFFFFFFu, behind = end < a.rows ? a.keys[end] : 0xFFFFFFFFu;
  float2 sum[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) sum[e] = both(0.0f);
  bool began = ahead == a.keys[first];
  uint32_t token = a.keys[first];
  for (int64_t at = first; at < end; at += kBatch) {
    // 32 keys and positions could be read at once; lanes 0 .. kBatch - 1 hold a batch's.
    const int64_t mine = at + (lane & (kBatch - 1));
    const uint32_t key = mine < end ? a.keys[mine] : a.vocab, from = mine < end ? a.order[mine] : 0;
    Loaded<TD, VEC> r[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const uint32_t row = __shfl_sync(0xFFFFFFFFu, from, k), t = __shfl_sync(0xFFFFFFFFu, key, k);
      if (at + k < end && t < a.vocab) r[k].load(static_cast<const TD *>(a.dout) + (int64_t)row * a.ld_dout, j, a.cols);
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const uint32_t t = __shfl_sync(0xFFFFFFFFu, key, k);
      if (at + k >= end) break;
      if (t != token) {
        if (began)
          write_part<VEC>(a, piece, 0, j, sum);
        else
          write_row<TG, VEC>(a, token, j, sum);
        began = false;
        token = t;
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] = both(0.0f);
      }
      if (t >= a.vocab) return;  // padding sorts last
      r[k].add_to(sum);
    }
  }
  if (began)
    write_part<VEC>(a, piece, 0, j, sum);
  else if (token == behind)
    write_part<VEC>(a, piece, 1, j, sum);
  else
    write_row<TG, VEC>(a, token, j, sum);
}

// First index whose key is not below k.
__device__ __forceinline__ int64_t lower_bound(const uint32_t *keys, int64_t n, uint32_t k) {
  int64_t lo = 0;
  while (n > 0) {
    const int64_t half = n / 2;
    const bool right = keys[lo + half] < k;
    lo = right ? lo + half + 1 : lo;
    n = right ? n - half - 1 : half;
  }
  return lo;
}

// Tokens whose rows fill more than one piece: a block to the piece where one starts and a
// strip of columns; its warps share out the pieces and meet in order.
template <class TG, bool VEC>
__global__ void __launch_bounds__(kThreads) join_kernel(const __grid_constant__ SumArgs a) {
  __shared__ float2 met[kThreads / 32][32][4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  wait_for_previous();
  let_next_start();
  const int64_t piece = blockIdx.x / a.strips, strip = blockIdx.x - piece * a.strips;
  const int64_t first = piece * a.length, end = first + a.length;
  if (end >= a.rows) return;
  const uint32_t token = a.keys[end - 1];
  if (token >= a.vocab || a.keys[end] != token) return;              // nothing goes on
  if (a.keys[first] == token && first > 0 && a.keys[first - 1] == token) return;  // it began before this piece
  const int64_t last = (lower_bound(a.keys + end, a.rows - end, token + 1) + end - 1) / a.length;
  const int64_t j = strip * Strip<VEC>::kCols + lane * (VEC ? 8 : 1);
  float2 sum[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) sum[e] = both(0.0f);
  // Piece `piece` gives its second part, pieces up to `last` their first.
  const int64_t n = last - piece + 1, share = (n + kThreads / 32 - 1) / (kThreads / 32);
  const int64_t from = piece + warp * share, to_ = min(from + share, last + 1);
#pragma unroll 4
  for (int64_t p = from; p < to_; ++p) {
    const float *q = part_of<VEC>(a, p, p == piece);
    if constexpr (VEC) {
      if (j < a.cols) {
        float2 v[4];
        load8(q, j, false, v);
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] = __fadd2_rn(sum[e], v[e]);
      }
    } else {
      if (j < a.cols) sum[0].x += q[j];
      if (j + 32 < a.cols) sum[0].y += q[j + 32];
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) met[warp][lane][e] = sum[e];
  __syncthreads();
  if (warp > 0) return;
  for (int w = 1; w < kThreads / 32; ++w) {
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] = __fadd2_rn(sum[e], met[w][lane][e]);
  }
  write_row<TG, VEC>(a, token, j, sum);
}

// Rows of the gradient that no token has: zeros.  A block looks for kThreads rows in the
// sorted tokens, one a thread, and writes those that are missing.
template <class TG>
__global__ void __launch_bounds__(kThreads) clear_kernel(const __grid_constant__ SumArgs a) {
  __shared__ uint32_t missing[kThreads];
  __shared__ int32_t n;
  if (threadIdx.x == 0) n = 0;
  wait_for_previous();
  let_next_start();
  __syncthreads();
  const int64_t v = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (v < a.vocab) {
    const int64_t at = lower_bound(a.keys, a.rows, (uint32_t)v);
    if (at >= a.rows || a.keys[at] != (uint32_t)v) missing[atomicAdd(&n, 1)] = (uint32_t)v;
  }
  __syncthreads();
  const int lane = threadIdx.x & 31;
  for (int r = threadIdx.x / 32; r < n; r += kThreads / 32) {
    TG *g = static_cast<TG *>(a.grad) + (int64_t)missing[r] * a.ld_grad;
    // Whole 16-byte units, and what lies before and behind them one by one.
    constexpr int E = 16 / sizeof(TG);
    const int64_t head = min(a.cols, (int64_t)((16 - ((uintptr_t)g & 15)) & 15) / (int64_t)sizeof(TG));
    const int64_t units = (a.cols - head) / E;
    if (lane < head) g[lane] = to<TG>(0.0f);
    for (int64_t u = lane; u < units; u += 32) *reinterpret_cast<uint4 *>(g + head + u * E) = make_uint4(0, 0, 0, 0);
    const int64_t tail = head + units * E + lane;
    if (tail < a.cols) g[tail] = to<TG>(0.0f);
  }
}

// ---- host --------------------------------------------------------------------
fsdp_status_t check(const fsdp_embedding_desc_t *d) {
  if (!d) return fail(FSDP_EINVAL, "desc is NULL");
  if (d->rows < 0 || d->vocab < 1 || d->cols < 1) return fail(FSDP_EINVAL, "rows < 0, vocab < 1 or cols < 1");
  if (d->rows > INT32_MAX || d->vocab > INT32_MAX - 1) return fail(FSDP_EUNSUPPORTED, "rows or vocab of 2^31 or more");
  if (d->cols > INT64_MAX / 64 / std::max<int64_t>(d->vocab, std::max<int64_t>(d->rows, 1)))
    return fail(FSDP_EUNSUPPORTED, "the matrices are too large");
  if (d->token_dtype != FSDP_INDEX_I32 && d->token_dtype != FSDP_INDEX_I64) return fail(FSDP_EINVAL, "unknown token_dtype");
  if (!float_dtype(d->weight_dtype)) return fail(FSDP_EINVAL, "unknown weight_dtype");
  if (!float_dtype(d->out_dtype)) return fail(FSDP_EINVAL, "unknown out_dtype");
  if (d->accumulate != 0 && d->accumulate != 1) return fail(FSDP_EINVAL, "accumulate is neither 0 nor 1");
  if (!(d->scale - d->scale == 0.0f)) return fail(FSDP_EINVAL, "scale is not finite");
  return FSDP_OK;
}

fsdp_status_t check_tokens(const fsdp_embedding_desc_t *d, const void *tokens) {
  const int64_t size = d->token_dtype == FSDP_INDEX_I64 ? 8 : 4;
  return check_ptr(tokens, d->rows * size, size, "tokens", -1);
}

bool rows_aligned(const void *p, int64_t rows, int64_t ld, int64_t size) {
  return aligned16(p) && (rows <= 1 || ld * size % 16 == 0);
}

// How the gradient's work is cut, from the sizes alone.
struct Cut {
  int64_t blocks, pieces, padded_cols;
  int32_t length, passes, bits;
  int64_t keys[2], order[2], counts, parts, bytes;  // offsets in the workspace
};

Cut cut_of(const fsdp_embedding_desc_t &d) {
  Cut c = {};
  c.padded_cols = (d.cols + 7) / 8 * 8;
  c.blocks = (d.rows + kTile - 1) / kTile;
  int bits = 1;
  while ((d.vocab >> bits) != 0) ++bits;  // keys are 0 .. vocab
  c.passes = (bits + kMaxBits - 1) / kMaxBits;
  c.bits = (bits + c.passes - 1) / c.passes;
  // Long pieces leave fewer parts to join, short ones give every SM work.
  const int64_t strips = (c.padded_cols + 255) / 256;
  c.length = 128;
  while (c.length > 8 && (d.rows + c.length - 1) / c.length * strips < 152 * 32) c.length /= 2;
  c.pieces = (d.rows + c.length - 1) / c.length;
  auto take = [&](int64_t bytes) {
    const int64_t at = c.bytes;
    c.bytes += (bytes + 15) / 16 * 16;
    return at;
  };
  for (int k = 0; k < 2; ++k) c.keys[k] = take(d.rows * 4), c.order[k] = take(d.rows * 4);
  c.counts = take(c.blocks * (4ll << c.bits));
  c.parts = take(c.pieces * 2 * c.padded_cols * 4);
  return c;
}

template <class K>
const void *kernel(K *k) {
  return reinterpret_cast<const void *>(k);
}

template <class TD, class TG, bool VEC>
fsdp_status_t sums(SumArgs a, cudaStream_t s) {
  a.strips = (a.cols + Strip<VEC>::kCols - 1) / Strip<VEC>::kCols;
  void *args[] = {&a};
  const int64_t warps = kThreads / 32, units = a.pieces * a.strips;
  const int64_t grid = (units + warps - 1) / warps, joins = (a.pieces - 1) * a.strips;
  if (grid > INT32_MAX || joins > INT32_MAX) return fail(FSDP_EUNSUPPORTED, "the gradient is too large for one launch");
  fsdp_status_t st = launched(launch_kernel(kernel(&sum_kernel<TD, TG, VEC>), dim3((unsigned)grid), dim3(kThreads), args, 0, s, true));
  if (st == FSDP_OK && joins > 0)
    st = launched(launch_kernel(kernel(&join_kernel<TG, VEC>), dim3((unsigned)joins), dim3(kThreads), args, 0, s, true));
  return st;
}

template <class TW, class TO>
fsdp_status_t lookup(LookupArgs a, bool vec, cudaStream_t s) {
  const int64_t span = vec ? 256 * kUnroll : 64 * kUnroll, warps = kThreads / 32;
  a.runs = (a.cols + span - 1) / span;
  const int64_t grid = (a.rows * a.runs + warps - 1) / warps;
  if (grid > INT32_MAX) return fail(FSDP_EUNSUPPORTED, "the lookup is too large for one launch");
  void *args[] = {&a};
  const void *fn = vec ? kernel(&lookup_kernel<TW, TO, true>) : kernel(&lookup_kernel<TW, TO, false>);
  return launched(launch_kernel(fn, dim3((unsigned)grid), dim3(kThreads), args, 0, s, true));
}

}  // namespace
}  // namespace embedding
}  // namespace fsdp

using namespace fsdp;
using namespace fsdp::embedding;

extern "C" {

fsdp_status_t fsdp_embedding_workspace(const fsdp_embedding_desc_t *desc, int64_t *bytes) {
  fsdp_status_t st = check(desc);
  if (st != FSDP_OK) return st;
  if (!bytes) return fail(FSDP_EINVAL, "bytes is NULL");
  *bytes = cut_of(*desc).bytes;
  clear_error();
  return FSDP_OK;
}

fsdp_status_t fsdp_embedding_forward(const fsdp_embedding_desc_t *desc, const void *tokens, const void *weight, void *out,
                                     fsdp_stream_t stream) {
  fsdp_status_t st = check(desc);
  if (st != FSDP_OK) return st;
  const fsdp_embedding_desc_t &d = *desc;
  const int64_t sw = dtype_bytes(d.weight_dtype), so = dtype_bytes(d.out_dtype);
  if ((st = check_tokens(desc, tokens)) != FSDP_OK) return st;
  if ((st = check_matrix(weight, d.vocab, d.cols, d.ld_weight, sw, "weight")) != FSDP_OK) return st;
  if ((st = check_matrix(out, d.rows, d.cols, d.ld_out, so, "out")) != FSDP_OK) return st;
  if (d.rows > 0) {
    LookupArgs a = {};
    a.tokens = tokens, a.weight = weight, a.out = out;
    a.rows = d.rows, a.cols = d.cols, a.ld_weight = d.ld_weight, a.ld_out = d.ld_out;
    a.vocab = (uint32_t)d.vocab, a.wide = d.token_dtype == FSDP_INDEX_I64, a.scale = d.scale;
    const bool vec = d.cols % 8 == 0 && rows_aligned(weight, d.vocab, d.ld_weight, sw) && rows_aligned(out, d.rows, d.ld_out, so);
    const bool wb = d.weight_dtype == FSDP_DTYPE_BF16, ob = d.out_dtype == FSDP_DTYPE_BF16;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    st = wb ? (ob ? lookup<__nv_bfloat16, __nv_bfloat16>(a, vec, s) : lookup<__nv_bfloat16, float>(a, vec, s))
            : (ob ? lookup<float, __nv_bfloat16>(a, vec, s) : lookup<float, float>(a, vec, s));
    if (st != FSDP_OK) return st;
  }
  clear_error();
  return FSDP_OK;
}

fsdp_status_t fsdp_embedding_backward(const fsdp_embedding_desc_t *desc, const void *tokens, const void *dout, void *dweight,
                                      void *workspace, int64_t workspace_bytes, fsdp_stream_t stream) {
  fsdp_status_t st = check(desc);
  if (st != FSDP_OK) return st;
  const fsdp_embedding_desc_t &d = *desc;
  const int64_t sg = dtype_bytes(d.weight_dtype), sd = dtype_bytes(d.out_dtype);
  if ((st = check_tokens(desc, tokens)) != FSDP_OK) return st;
  if ((st = check_matrix(dweight, d.vocab, d.cols, d.ld_weight, sg, "dweight")) != FSDP_OK) return st;
  if ((st = check_matrix(dout, d.rows, d.cols, d.ld_out, sd, "dout")) != FSDP_OK) return st;
  const Cut c = cut_of(d);
  if (workspace_bytes < c.bytes)
    return fail(FSDP_EINVAL, "workspace_bytes is " + std::to_string(workspace_bytes) + ", the call needs " + std::to_string(c.bytes));
  if ((st = check_ptr(workspace, c.bytes, 16, "workspace", -1)) != FSDP_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint8_t *w = static_cast<uint8_t *>(workspace);
  auto words = [&](int64_t at) { return reinterpret_cast<uint32_t *>(w + at); };
  SortArgs q = {};
  q.rows = d.rows, q.vocab = (uint32_t)d.vocab, q.blocks = (uint32_t)c.blocks;
  q.wide = d.token_dtype == FSDP_INDEX_I64, q.bits = c.bits, q.counts = d.rows > 0 ? words(c.counts) : nullptr;
  for (int p = 0; p < c.passes && d.rows > 0; ++p) {
    q.tokens = p == 0 ? tokens : nullptr;
    q.keys_in = words(c.keys[(p + 1) & 1]), q.order_in = words(c.order[(p + 1) & 1]);
    q.keys = words(c.keys[p & 1]), q.order = words(c.order[p & 1]);
    q.shift = p * c.bits;
    void *args[] = {&q};
    for (const void *fn : {kernel(&count_kernel), kernel(&place_kernel)}) {
      st = launched(launch_kernel(fn, dim3((unsigned)c.blocks), dim3(kSortThreads), args, 0, s, true));
      if (st != FSDP_OK) return st;
    }
  }
  SumArgs a = {};
  if (d.rows > 0) a.keys = words(c.keys[(c.passes - 1) & 1]), a.order = words(c.order[(c.passes - 1) & 1]);
  a.dout = dout, a.grad = dweight;
  a.parts = reinterpret_cast<float *>(w + c.parts);
  a.rows = d.rows, a.cols = d.cols, a.ld_dout = d.ld_out, a.ld_grad = d.ld_weight;
  a.pieces = c.pieces, a.length = c.length;
  a.vocab = (uint32_t)d.vocab, a.add = d.accumulate, a.scale = d.scale;
  const bool gb = d.weight_dtype == FSDP_DTYPE_BF16, db = d.out_dtype == FSDP_DTYPE_BF16;
  if (!d.accumulate) {
    void *args[] = {&a};
    st = launched(launch_kernel(gb ? kernel(&clear_kernel<__nv_bfloat16>) : kernel(&clear_kernel<float>),
                                dim3((unsigned)((d.vocab + kThreads - 1) / kThreads)), dim3(kThreads), args, 0, s, true));
    if (st != FSDP_OK) return st;
  }
  if (d.rows > 0) {
    const bool vec = d.cols % 8 == 0 && rows_aligned(dweight, d.vocab, d.ld_weight, sg) && rows_aligned(dout, d.rows, d.ld_out, sd);
    using B = __nv_bfloat16;
    if (vec)
      st = db ? (gb ? sums<B, B, true>(a, s) : sums<B, float, true>(a, s)) : (gb ? sums<float, B, true>(a, s) : sums<float, float, true>(a, s));
    else
      st = db ? (gb ? sums<B, B, false>(a, s) : sums<B, float, false>(a, s))
              : (gb ? sums<float, B, false>(a, s) : sums<float, float, false>(a, s));
    if (st != FSDP_OK) return st;
  }
  clear_error();
  return FSDP_OK;
}

}  // extern "C"

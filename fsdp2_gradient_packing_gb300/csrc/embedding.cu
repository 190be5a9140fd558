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
//
// Measured, 32768 x 4096 in BF16: the lookup of 16,384 tokens (some of them the same) 30 us, 268 MB at 8.9 TB/s of which L2 has
// a part; their gradient 90 us, 403 MB with all zeros at 4.5 TB/s: the sort 21 us, bound by two passes of a cluster's barriers and
// scattered stores, beside which 100 MB are cleared; the sums 54 us at 5.8 TB/s, bound by HBM; the join 10 us, by latency.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <string>

#include "layout.h"
#include "ops.h"
#include "tc.h"

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
// A pass sorts by one digit of up to kMaxBits bits: each block counts its tile's items by
// digit, then places them behind what the counts of lower digits and earlier blocks say.
// Within a block the order is that of the items: a warp takes consecutive ones, 32 at a
// time, and ranks equal digits by lane, so a pass keeps the order of the one before.
constexpr int kSortThreads = 512, kItems = 8, kMaxBits = 10, kMaxBins = 1 << kMaxBits;
constexpr int kSortWarps = kSortThreads / 32;

struct SortArgs {
  const void *tokens;                        // first pass: the caller's; later passes: keys
  const uint2 *pairs_in;                     // tokens and their positions
  uint2 *pairs;
  uint32_t *crossing;                        // two counters that the last pass clears, or nullptr
  uint32_t *counts;                          // [blocks][bins] of this pass; with `totals`, those of earlier tiles
  uint32_t *totals;                          // [bins], or nullptr: tiles sum the counts themselves
  int64_t rows;
  uint32_t vocab, blocks;
  int32_t wide, bits, shift;
  int32_t items;                             // of a thread: 1 .. kItems
};

// Item i: its token, and its position.
__device__ __forceinline__ uint2 sort_item(const SortArgs &a, int64_t i) {
  return a.tokens ? make_uint2(token_at(a.tokens, i, a.wide != 0, a.vocab), (uint32_t)i) : __ldcg(a.pairs_in + i);
}

struct SortShared {
  uint16_t seen[kSortWarps][kMaxBins];  // items of a digit in a warp, then in the warps before it
  uint32_t base[kMaxBins];              // counts of a tile; then where the tile's items of a digit go
  uint32_t total[kSortWarps];
};

// A thread's items of a tile: a warp has consecutive ones, 32 at a time.
struct Items {
  uint2 item[kItems];
  int n;
  __device__ __forceinline__ Items(const SortArgs &a, uint32_t tile) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int64_t first = (int64_t)tile * (a.items * kSortThreads) + warp * (32 * a.items) + lane;
    n = (int)min((int64_t)a.items, (a.rows - first + 31) / 32);
#pragma unroll
    for (int k = 0; k < kItems; ++k) item[k] = k < n ? sort_item(a, first + k * 32) : make_uint2(0, 0);
  }
};

// How many of a tile's items have each digit.
__device__ __forceinline__ void count_tile(const SortArgs &a, SortShared &s, uint32_t tile, const Items &own) {
  const int bins = 1 << a.bits;
  for (int d = threadIdx.x; d < bins; d += kSortThreads) s.base[d] = 0;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kItems; ++k)
    if (k < own.n) atomicAdd(&s.base[(own.item[k].x >> a.shift) & (bins - 1)], 1u);
  __syncthreads();
  for (int d = threadIdx.x; d < bins; d += kSortThreads) a.counts[(int64_t)tile * bins + d] = s.base[d];
}

// A tile's items to their places.
__device__ __forceinline__ void place_tile(const SortArgs &a, SortShared &s, uint32_t tile, const Items &own) {
  const int bins = 1 << a.bits, lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  for (int i = lane; i < bins / 2; i += 32) reinterpret_cast<uint32_t *>(s.seen[warp])[i] = 0;
  uint32_t rank[kItems];
  // Where each digit's items start: behind those of lower digits and those of earlier tiles.  A
  // thread sums two neighbouring digits (bins are at least 2).
  uint32_t before[2] = {0, 0}, all[2] = {0, 0};
  const int d = threadIdx.x * 2;
  if (d < bins && a.totals) {
    const uint2 t = *reinterpret_cast<const uint2 *>(a.totals + d), c = *reinterpret_cast<const uint2 *>(a.counts + (int64_t)tile * bins + d);
    all[0] = t.x, all[1] = t.y, before[0] = c.x, before[1] = c.y;
  } else if (d < bins) {
    const uint2 *p = reinterpret_cast<const uint2 *>(a.counts + d);
#pragma unroll 8
    for (uint32_t b = 0; b < a.blocks; ++b) {
      const uint2 c = __ldcg(p + (int64_t)b * (bins / 2));
      all[0] += c.x, all[1] += c.y;
      if (b < tile) before[0] += c.x, before[1] += c.y;
    }
  }
  uint32_t run = all[0] + all[1];
#pragma unroll
  for (int m = 1; m < 32; m *= 2) {
    const uint32_t up = __shfl_up_sync(0xFFFFFFFFu, run, m);
    if (lane >= m) run += up;
  }
  if (lane == 31) s.total[warp] = run;
  __syncthreads();
  for (int w = 0; w < warp; ++w) run += s.total[w];
  if (d < bins) {
    s.base[d] = run - all[0] - all[1] + before[0];
    s.base[d + 1] = run - all[1] + before[1];
  }
  // Ranks within the warp's items of the same digit.
  __syncwarp();
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    if (k >= a.items) break;
    const bool here = k < own.n;
    const uint32_t digit = (own.item[k].x >> a.shift) & (bins - 1);
    uint32_t same = __ballot_sync(0xFFFFFFFFu, here);
    for (int b = 0; b < a.bits; ++b) {
      const uint32_t ones = __ballot_sync(0xFFFFFFFFu, digit >> b & 1);
      same &= digit >> b & 1 ? ones : ~ones;
    }
    const uint32_t earlier = same & ((1u << lane) - 1);
    rank[k] = here ? s.seen[warp][digit] + __popc(earlier) : 0;
    __syncwarp();
    if (here && !earlier) s.seen[warp][digit] = (uint16_t)(rank[k] + __popc(same));
    __syncwarp();
  }
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += kSortThreads) {
    uint32_t sum = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
      const uint32_t n = s.seen[w][b];
      s.seen[w][b] = (uint16_t)sum;
      sum += n;
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    if (k >= own.n) break;
    const uint32_t digit = (own.item[k].x >> a.shift) & (bins - 1);
    a.pairs[s.base[digit] + s.seen[warp][digit] + rank[k]] = own.item[k];
  }
  if (a.crossing && tile == 0 && threadIdx.x < 2) a.crossing[threadIdx.x] = 0;
}

__global__ void __launch_bounds__(kSortThreads) count_kernel(const __grid_constant__ SortArgs a) {
  __shared__ SortShared s;
  wait_for_previous();
  let_next_start();
  count_tile(a, s, blockIdx.x, Items(a, blockIdx.x));
}
// Many tiles: their counts become those of earlier tiles, and a digit's total.  32 digits to a block, whose warps share out
// the tiles.  (Summing all counts in each tile would cost the square of their number.)
constexpr int kFewTiles = 32;
__global__ void __launch_bounds__(1024) offsets_kernel(const __grid_constant__ SortArgs a) {
  __shared__ uint32_t part[32][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, bins = 1 << a.bits, d = blockIdx.x * 32 + lane;
  wait_for_previous();
  let_next_start();
  const int64_t share = ((int64_t)a.blocks + 31) / 32, begin = min(warp * share, (int64_t)a.blocks), end = min(begin + share, (int64_t)a.blocks);
  uint32_t sum = 0;
  if (d < bins) {
#pragma unroll 8
    for (int64_t b = begin; b < end; ++b) sum += a.counts[b * bins + d];
  }
  part[warp][lane] = sum;
  __syncthreads();
  uint32_t before = 0;
  for (int w = 0; w < warp; ++w) before += part[w][lane];
  if (d >= bins) return;
  if (warp == 31) a.totals[d] = before + sum;
#pragma unroll 8
  for (int64_t b = begin; b < end; ++b) {
    const uint32_t n = a.counts[b * bins + d];
    a.counts[b * bins + d] = before;
    before += n;
  }
}
__global__ void __launch_bounds__(kSortThreads) place_kernel(const __grid_constant__ SortArgs a) {
  __shared__ SortShared s;
  wait_for_previous();
  let_next_start();
  place_tile(a, s, blockIdx.x, Items(a, blockIdx.x));
}

// Zeros to a row, by a warp: whole 16-byte units, and what lies before and behind them one by one.
template <class T>
__device__ __forceinline__ void clear_row(T *g, int64_t cols) {
  constexpr int E = 16 / sizeof(T);
  const int lane = threadIdx.x & 31;
  const int64_t head = min(cols, (int64_t)((16 - ((uintptr_t)g & 15)) & 15) / (int64_t)sizeof(T)), units = (cols - head) / E;
  if (lane < head) g[lane] = to<T>(0.0f);
#pragma unroll 4
  for (int64_t u = lane; u < units; u += 32) *reinterpret_cast<uint4 *>(g + head + u * E) = make_uint4(0, 0, 0, 0);
  const int64_t tail = head + units * E + lane;
  if (tail < cols) g[tail] = to<T>(0.0f);
}

// Few tokens, up to a cluster's kMaxCluster tiles: all passes of the sort in one launch, by the first cluster.  The
// others meanwhile clear the rows of the gradient that no token has, each its share: a cluster's blocks look
// through a part of the tokens each for the rows of all of them.
constexpr int kMaxCluster = 8, kClearBytes = 100 << 20;
struct ShortArgs {
  SortArgs pass[4];
  const void *tokens;
  void *grad;          // nullptr: nothing to clear
  int64_t cols, ld_grad, share, clear_to;  // rows of a clearing cluster; the first row that is not cleared here
  int32_t passes, grad_bf16;
};
template <class T>
__device__ __forceinline__ void clear_share(const ShortArgs &a, SortShared &s, int64_t begin, uint32_t blocks) {
  const SortArgs &q = a.pass[0];
  const uint32_t rank = blocks > 1 ? tc::cluster_rank() : 0;
  uint32_t *mine = s.base, *all = reinterpret_cast<uint32_t *>(s.seen);  // rows that this block's part of the tokens has, and all have
  const int64_t last = min(begin + a.share, a.clear_to);
  constexpr int64_t kRows = kMaxBins * 32;  // rows that are looked for at once
  auto sync = [&] {
    if (blocks > 1)
      tc::cluster_sync();
    else
      __syncthreads();
  };
  for (int64_t lo = begin; lo < last; lo += kRows) {
    const int64_t hi = min(lo + kRows, last);
    const int words = (int)(hi - lo + 31) / 32;
    for (int i = threadIdx.x; i < words; i += kSortThreads) mine[i] = 0;
    __syncthreads();
#pragma unroll 4
    for (int64_t i = (int64_t)rank * kSortThreads + threadIdx.x; i < q.rows; i += (int64_t)blocks * kSortThreads) {
      const int64_t t = token_at(a.tokens, i, q.wide != 0, q.vocab) - lo;
      if (t >= 0 && t < hi - lo) atomicOr(&mine[t / 32], 1u << (t & 31));
    }
    sync();
    for (int i = threadIdx.x; i < words; i += kSortThreads) {
      uint32_t any = mine[i];
      for (uint32_t r = 0; r < blocks && blocks > 1; ++r) {
        uint32_t w;
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(w) : "r"(tc::at_rank(tc::smem(mine + i), r)) : "memory");
        any |= w;
      }
      all[i] = any;
    }
    sync();  // no block begins again, or leaves, while another reads its rows
    for (int64_t r = lo + rank * kSortWarps + threadIdx.x / 32; r < hi; r += blocks * kSortWarps)
      if (!(all[(r - lo) / 32] >> ((r - lo) & 31) & 1)) clear_row(static_cast<T *>(a.grad) + r * a.ld_grad, a.cols);
    __syncthreads();
  }
}
__global__ void __launch_bounds__(kSortThreads) short_kernel(const __grid_constant__ ShortArgs a) {
  __shared__ SortShared s;
  wait_for_previous();
  let_next_start();
  const uint32_t blocks = a.pass[0].blocks;
  if (blockIdx.x < blocks) {
    for (int p = 0; p < a.passes; ++p) {
      const Items own(a.pass[p], blockIdx.x);
      count_tile(a.pass[p], s, blockIdx.x, own);
      if (blocks > 1)
        tc::cluster_sync();
      else
        __syncthreads();
      place_tile(a.pass[p], s, blockIdx.x, own);
      if (blocks > 1)
        tc::cluster_sync();
      else
        __syncthreads();
    }
  } else {
    const uint32_t cluster = max(blocks, 1u);
    const int64_t begin = (int64_t)((blockIdx.x - blocks) / cluster) * a.share;
    if (a.grad_bf16)
      clear_share<__nv_bfloat16>(a, s, begin, cluster);
    else
      clear_share<float>(a, s, begin, cluster);
  }
}

// ---- sums --------------------------------------------------------------------
struct SumArgs {
  const uint2 *pairs;     // sorted tokens and their positions
  // Tokens that go on behind the piece where they begin: how many lie in few and in many pieces; then those
  // pieces, the few from the front and the many from the back.
  uint32_t *crossing;
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
  // Rows from clear_from on are cleared where no token has them: by this many blocks, one in every `every`.
  int64_t clear_from, clear_blocks, every;
};

// Rows of loads at a time, two of them in flight: as many as registers hold.
template <class TD, bool VEC>
constexpr int kBatch = VEC && sizeof(TD) == 2 ? 8 : 4;

// A warp's strip: 256 columns, of which a lane has eight, consecutive (VEC) or 32 apart.
constexpr int kStrip = 256;
constexpr int kManyPieces = 8;  // behind the one where a token begins

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
  TD v[8];
  __device__ void load(const TD *p, int64_t j, int64_t cols) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = j + e * 32 < cols ? p[j + e * 32] : (TD)0.0f;
  }
  __device__ void add_to(float2 (&s)[4]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) element(s, e) += (float)v[e];
  }
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
    TG old[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) old[e] = a.add && j + e * 32 < a.cols ? g[j + e * 32] : (TG)0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (j + e * 32 < a.cols) g[j + e * 32] = to<TG>(fmaf(element(sum, e), a.scale, (float)old[e]));
  }
}
__device__ __forceinline__ float *part_of(const SumArgs &a, int64_t piece, int which) {
  return a.parts + (piece * 2 + which) * ((a.cols + 7) / 8 * 8);
}
template <bool VEC>
__device__ __forceinline__ void write_part(const SumArgs &a, int64_t piece, int which, int64_t j, const float2 (&sum)[4]) {
  float *p = part_of(a, piece, which);
  if constexpr (VEC) {
    if (j < a.cols) store8(p, j, false, sum);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (j + e * 32 < a.cols) p[j + e * 32] = element(sum, e);
  }
}

// First index whose key is not below k.
__device__ __forceinline__ int64_t lower_bound(const uint2 *keys, int64_t n, uint32_t k) {
  int64_t lo = 0;
  while (n > 0) {
    const int64_t half = n / 2;
    const bool right = keys[lo + half].x < k;
    lo = right ? lo + half + 1 : lo;
    n = right ? n - half - 1 : half;
  }
  return lo;
}
// By a warp: the first index whose key is not below k.  Each round takes 32 probes, so 16,384 keys take three.
__device__ __forceinline__ int64_t warp_lower_bound(const uint2 *keys, int64_t n, uint32_t k) {
  const int lane = threadIdx.x & 31;
  int64_t lo = 0;  // keys before lo are below k, those from lo + n on are not
  while (n > 0) {
    const int64_t step = (n + 32) / 33, at = lo + (lane + 1) * step - 1;
    const uint32_t below = __ballot_sync(0xFFFFFFFFu, at < lo + n && keys[at].x < k);
    const int c = __popc(below);  // probes 0 .. c - 1 are below
    const int64_t from = lo + c * step, to = c < 32 ? min(lo + (c + 1) * step - 1, lo + n) : lo + n;
    lo = from, n = max((int64_t)0, to - from);
  }
  return lo;
}

// Rows first .. first + kClearRows - 1 of the gradient, zeros where no token has them: a block looks for them in the part
// of the sorted tokens that has them, one a thread, and writes those that are missing.
constexpr int kClearRows = 64;
template <class TG>
__device__ __forceinline__ void clear_rows(const SumArgs &a, int64_t first) {
  __shared__ uint32_t missing[kClearRows];
  __shared__ int64_t bound[2];
  __shared__ int32_t n;
  const int64_t v = first + threadIdx.x;
  if (threadIdx.x == 0) n = 0;
  if (threadIdx.x < 64) {
    const int64_t at = warp_lower_bound(a.pairs, a.rows, (uint32_t)min(first + threadIdx.x / 32 * kClearRows, (int64_t)a.vocab));
    if (threadIdx.x % 32 == 0) bound[threadIdx.x / 32] = at;
  }
  __syncthreads();
  if (threadIdx.x < kClearRows && v < a.vocab) {
    const int64_t at = bound[0] + lower_bound(a.pairs + bound[0], bound[1] - bound[0], (uint32_t)v);
    if (at >= bound[1] || a.pairs[at].x != (uint32_t)v) missing[atomicAdd(&n, 1)] = (uint32_t)v;
  }
  __syncthreads();
  for (int r = threadIdx.x / 32; r < n; r += kThreads / 32) clear_row(static_cast<TG *>(a.grad) + (int64_t)missing[r] * a.ld_grad, a.cols);
}

template <class TD, class TG, bool VEC>
__global__ void __launch_bounds__(kThreads, 2) sum_kernel(const __grid_constant__ SumArgs a) {
  constexpr int N = kBatch<TD, VEC>;
  const int lane = threadIdx.x & 31;
  wait_for_previous();
  let_next_start();
  int64_t block = blockIdx.x;
  if (a.clear_blocks > 0) {  // every so many blocks, one clears rows
    const int64_t q = block / a.every;
    if (q * a.every == block && q < a.clear_blocks) {
      clear_rows<TG>(a, a.clear_from + q * kClearRows);
      return;
    }
    block -= min(a.clear_blocks, q + 1);
  }
  const int64_t unit = block * (kThreads / 32) + threadIdx.x / 32, piece = unit / a.strips;
  if (piece >= a.pieces) return;
  const int64_t j = (unit - piece * a.strips) * kStrip + lane * (VEC ? 8 : 1);
  const int64_t first = piece * a.length, end = min(first + a.length, a.rows);
  // The first token of the piece may have begun before it; the last one may go on behind it.
  const uint32_t ahead = first > 0 ? a.pairs[first - 1].x : 0xFFFFFFFFu, behind = end < a.rows ? a.pairs[end].x : 0xFFFFFFFFu;
  float2 sum[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) sum[e] = both(0.0f);
  uint32_t token = a.pairs[first].x;
  bool began = ahead == token;
  for (int64_t at = first; at < end; at += 32) {
    // 32 keys and positions, one a lane; padding (keys of vocab) sorts last.
    const uint2 pair = at + lane < end ? a.pairs[at + lane] : make_uint2(a.vocab, 0);
    const uint32_t key = pair.x, from = pair.y;
    const int n = __popc(__ballot_sync(0xFFFFFFFFu, key < a.vocab));  // rows to sum
    Loaded<TD, VEC> r[2][N];
    auto load = [&](int k0, Loaded<TD, VEC> (&to)[N]) {
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const uint32_t row = __shfl_sync(0xFFFFFFFFu, from, (k0 + k) & 31);
        if (k0 + k < n) to[k].load(static_cast<const TD *>(a.dout) + (int64_t)row * a.ld_dout, j, a.cols);
      }
    };
    load(0, r[0]);
#pragma unroll
    for (int b = 0; b < 32 / N; ++b) {
      if (b * N >= n) break;
      if (b + 1 < 32 / N) load((b + 1) * N, r[(b + 1) & 1]);
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const uint32_t t = __shfl_sync(0xFFFFFFFFu, key, b * N + k);
        if (b * N + k >= n) break;
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
        r[b & 1][k].add_to(sum);
      }
    }
  }
  if (token >= a.vocab) return;  // nothing but padding
  if (began) {
    write_part<VEC>(a, piece, 0, j, sum);
  } else if (token == behind) {
    write_part<VEC>(a, piece, 1, j, sum);
    if (unit == piece * a.strips && lane == 0) {
      const int64_t far = end + kManyPieces * (int64_t)a.length;
      const bool many = far < a.rows && a.pairs[far].x == token;
      const uint32_t n = atomicAdd(a.crossing + many, 1u);
      a.crossing[many ? 1 + a.pieces - n : 2 + n] = (uint32_t)piece;
    }
  } else {
    write_row<TG, VEC>(a, token, j, sum);
  }
}

// Tokens whose rows lie in more than one piece (in any order: each has its own row).  A warp to a token of few pieces
// and a strip; a block to one of many, whose warps share out the pieces and meet in order.
template <bool VEC>
__device__ __forceinline__ void add_parts(const SumArgs &a, int64_t piece, int64_t from, int64_t to_, int64_t j, float2 (&sum)[4]) {
#pragma unroll 4
  for (int64_t p = from; p < to_; ++p) {
    const float *q = part_of(a, p, p == piece);  // the piece where the token begins gives its second part
    if constexpr (VEC) {
      if (j < a.cols) {
        float2 v[4];
        load8(q, j, false, v);
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] = __fadd2_rn(sum[e], v[e]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (j + e * 32 < a.cols) element(sum, e) += q[j + e * 32];
    }
  }
}
template <class TG, bool VEC>
__global__ void __launch_bounds__(kThreads) join_kernel(const __grid_constant__ SumArgs a) {
  constexpr int kWarps = kThreads / 32;
  __shared__ float2 met[kWarps][32][4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  wait_for_previous();
  let_next_start();
  const int64_t few = (int64_t)a.crossing[0] * a.strips, many = (int64_t)a.crossing[1] * a.strips;
  float2 sum[4];
  for (int64_t unit = (int64_t)blockIdx.x * kWarps + warp; unit < few; unit += (int64_t)gridDim.x * kWarps) {
    const int64_t at = unit / a.strips, j = (unit - at * a.strips) * kStrip + lane * (VEC ? 8 : 1), piece = a.crossing[2 + at];
    const uint32_t token = a.pairs[(piece + 1) * a.length].x;
    // Where it goes on: lane k looks at piece k behind its first.
    const int64_t next = (piece + 1 + lane) * a.length;
    const int64_t last = piece + __popc(__ballot_sync(0xFFFFFFFFu, lane <= kManyPieces && next < a.rows && a.pairs[min(next, a.rows - 1)].x == token));
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] = both(0.0f);
    add_parts<VEC>(a, piece, piece, last + 1, j, sum);
    write_row<TG, VEC>(a, token, j, sum);
  }
  for (int64_t unit = blockIdx.x; unit < many; unit += gridDim.x) {
    const int64_t at = unit / a.strips, j = (unit - at * a.strips) * kStrip + lane * (VEC ? 8 : 1), piece = a.crossing[1 + a.pieces - at];
    const int64_t end = (piece + 1) * a.length;
    const uint32_t token = a.pairs[end].x;
    const int64_t last = (warp_lower_bound(a.pairs + end, a.rows - end, token + 1) + end - 1) / a.length;  // the piece of its last row
    const int64_t share = (last - piece + kWarps) / kWarps, from = piece + warp * share;
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] = both(0.0f);
    add_parts<VEC>(a, piece, from, min(from + share, last + 1), j, sum);
#pragma unroll
    for (int e = 0; e < 4; ++e) met[warp][lane][e] = sum[e];
    __syncthreads();
    if (warp == 0) {
      for (int w = 1; w < kWarps; ++w) {
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] = __fadd2_rn(sum[e], met[w][lane][e]);
      }
      write_row<TG, VEC>(a, token, j, sum);
    }
    __syncthreads();
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
  int32_t length, passes, bits, items;
  int64_t pairs[2], counts, totals, crossing, parts, bytes;  // offsets in the workspace
};

Cut cut_of(const fsdp_embedding_desc_t &d) {
  Cut c = {};
  c.padded_cols = (d.cols + 7) / 8 * 8;
  // Tiles as small as a cluster's blocks allow, so that all of them have work.
  c.items = (int32_t)std::min<int64_t>(kItems, std::max<int64_t>(1, (d.rows + kMaxCluster * kSortThreads - 1) / (kMaxCluster * kSortThreads)));
  c.blocks = (d.rows + c.items * kSortThreads - 1) / (c.items * kSortThreads);
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
  for (int k = 0; k < 2; ++k) c.pairs[k] = take(d.rows * 8);
  c.counts = take(c.blocks * (4ll << c.bits));
  c.totals = take(c.blocks > kFewTiles ? 4ll << c.bits : 0);
  c.crossing = take(d.rows > 0 ? c.pieces * 4 + 8 : 0);
  c.parts = take(c.pieces * 2 * c.padded_cols * 4);
  return c;
}

template <class K>
const void *kernel(K *k) {
  return reinterpret_cast<const void *>(k);
}

template <class TD, class TG, bool VEC>
fsdp_status_t sums(SumArgs a, cudaStream_t s) {
  a.strips = (a.cols + kStrip - 1) / kStrip;
  void *args[] = {&a};
  const int64_t warps = kThreads / 32, units = a.pieces * a.strips;
  a.clear_blocks = (a.vocab - a.clear_from + kClearRows - 1) / kClearRows;
  const int64_t grid = (units + warps - 1) / warps + a.clear_blocks;
  a.every = a.clear_blocks > 0 ? std::max<int64_t>(1, grid / a.clear_blocks) : 1;
  const int64_t joins = std::min<int64_t>((a.pieces - 1) * a.strips, (int64_t)device_sms() * 4);
  if (grid > INT32_MAX) return fail(FSDP_EUNSUPPORTED, "the gradient is too large for one launch");
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
  const bool gb = d.weight_dtype == FSDP_DTYPE_BF16, db = d.out_dtype == FSDP_DTYPE_BF16;
  auto pass_of = [&](int p) {
    SortArgs r = q;
    r.tokens = p == 0 ? tokens : nullptr;
    r.pairs_in = reinterpret_cast<const uint2 *>(w + c.pairs[(p + 1) & 1]);
    r.pairs = reinterpret_cast<uint2 *>(w + c.pairs[p & 1]);
    r.shift = p * c.bits, r.items = c.items;
    if (p == c.passes - 1) r.crossing = words(c.crossing);
    return r;
  };
  const bool few = c.blocks <= kMaxCluster;
  // Rows that are cleared beside the sort: what it leaves time for, at 5 TB/s and 20 us.  The others are cleared beside
  // the sums, whose reads go well with writes (zeros alone reach 5.8 TB/s, a copy 6.8).
  const int64_t row_bytes = d.cols * sg;
  const int64_t cleared = d.accumulate ? d.vocab : !few ? 0 : d.rows == 0 ? d.vocab : std::min(d.vocab, (int64_t)kClearBytes / row_bytes + 1);
  if (few && (d.rows > 0 || !d.accumulate)) {
    ShortArgs r = {};
    for (int p = 0; p < c.passes; ++p) r.pass[p] = pass_of(p);
    r.passes = c.passes, r.tokens = tokens, r.cols = d.cols, r.ld_grad = d.ld_weight, r.grad_bf16 = gb;
    const int cluster = std::max<int>(1, (int)c.blocks);
    int64_t clearing = 0;
    if (!d.accumulate) {
      // As many clearing blocks as fill the SMs beside the sort (two fit an SM), of 16 rows at least.
      r.grad = dweight;
      clearing = std::max<int64_t>(1, std::min<int64_t>((int64_t)device_sms() * 2 - c.blocks, (cleared + 15) / 16));
      clearing = (clearing + cluster - 1) / cluster * cluster;
      r.share = (cleared + clearing / cluster - 1) / (clearing / cluster);
      r.clear_to = cleared;
    }
    void *args[] = {&r};
    st = launched(launch_kernel(kernel(&short_kernel), dim3((unsigned)(c.blocks + clearing)), dim3(kSortThreads), args, 0, s, true, cluster));
    if (st != FSDP_OK) return st;
  }
  for (int p = 0; p < c.passes && !few; ++p) {
    SortArgs r = pass_of(p);
    void *args[] = {&r};
    st = launched(launch_kernel(kernel(&count_kernel), dim3((unsigned)c.blocks), dim3(kSortThreads), args, 0, s, true));
    if (st == FSDP_OK && c.blocks > kFewTiles) {
      r.totals = words(c.totals);
      st = launched(launch_kernel(kernel(&offsets_kernel), dim3((unsigned)((1 << c.bits) + 31) / 32), dim3(1024), args, 0, s, true));
    }
    if (st == FSDP_OK) st = launched(launch_kernel(kernel(&place_kernel), dim3((unsigned)c.blocks), dim3(kSortThreads), args, 0, s, true));
    if (st != FSDP_OK) return st;
  }
  SumArgs a = {};
  a.pairs = reinterpret_cast<const uint2 *>(w + c.pairs[(c.passes - 1) & 1]), a.crossing = words(c.crossing);
  a.dout = dout, a.grad = dweight;
  a.parts = reinterpret_cast<float *>(w + c.parts);
  a.rows = d.rows, a.cols = d.cols, a.ld_dout = d.ld_out, a.ld_grad = d.ld_weight;
  a.pieces = c.pieces, a.length = c.length;
  a.vocab = (uint32_t)d.vocab, a.add = d.accumulate, a.scale = d.scale, a.clear_from = cleared;
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

// Gated feed-forward block (fsdp_gated_ffn_*): argument checks, operand maps, the
// plan of the launches, and the kernels around the products.
//
// Forward: one launch.  Backward: dg and du (from what was kept, one pass over
// dh, gate and up; or as the epilogue of the forward product), then dx and both
// weight gradients in one launch.  dg and du pass through the workspace in BF16.
#include <cuda.h>

#include <algorithm>
#include <mutex>

#include "ffn.h"

namespace fsdp {
namespace ffn {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxDim = (int64_t(1) << 31) - 512;

int64_t up_to(int64_t n, int64_t m) { return (n + m - 1) / m * m; }
int64_t blocks_of(int64_t n, int64_t m) { return (n + m - 1) / m; }

// ---------------------------------------------------------------------------
// Operands
// ---------------------------------------------------------------------------
using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static std::mutex lock;
  static EncodeFn fn = nullptr;
  std::lock_guard<std::mutex> hold(lock);
  if (!fn) {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) == cudaSuccess &&
        found == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeFn>(p);
    else
      cudaGetLastError();
  }
  return fn;
}

// A BF16 matrix as TMA operand: boxes of 64 columns by `box_rows` rows, 128-byte
// swizzle, zeros outside.
struct Operand {
  const void *p;
  int64_t rows, cols, ld;
};
bool encode(CUtensorMap *map, const Operand &o, int box_rows) {
  EncodeFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)o.cols, (cuuint64_t)o.rows};
  const cuuint64_t strides[1] = {(cuuint64_t)up_to(o.ld, 8) * 2};  // one row: any distance will do
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, steps[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(o.p), dims, strides, box, steps,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Copies of up to three matrices whose rows start anywhere, to rows of `pitch`
// elements: a warp to 256 elements of a row, all of them in flight at once.  The third
// may be a checkpoint (`codes`).  Bound by latency at the sizes that have such rows:
// 3 matrices of 1411 x 515 take 2.5 us.
struct CopyArgs {
  const uint16_t *src[3];
  const uint8_t *codes, *scales;
  uint16_t *dst[3];
  int64_t ld[3], rows[3];
  int64_t pitch, cols;
};
__global__ void __launch_bounds__(kThreads) copy_rows_kernel(const __grid_constant__ CopyArgs a) {
  constexpr int kEach = 8;
  const int lane = threadIdx.x & 31;
  const int64_t pieces = (a.cols + 32 * kEach - 1) / (32 * kEach), all = (a.rows[0] + a.rows[1] + a.rows[2]) * pieces;
  wait_for_previous();
  let_next_start();
  for (int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32; i < all; i += (int64_t)gridDim.x * (kThreads / 32)) {
    int64_t r = i / pieces;
    const int64_t j = (i - r * pieces) * (32 * kEach) + lane;
    int which = 0;
    while (r >= a.rows[which]) r -= a.rows[which++];
    uint16_t *dst = a.dst[which] + r * a.pitch + j, v[kEach];
    if (which == 2 && a.codes) {  // a group to each load of the warp
      const int64_t groups = act8_groups(a.cols), first = r * groups + j / (int)kActGroup;
      const uint8_t *codes = a.codes + first * kActGroup + lane;
#pragma unroll
      for (int u = 0; u < kEach; ++u)
        if (j + u * 32 < a.cols) {
          const float value = act8_value(act8_biased(codes[u * kActGroup]), act8_scale(a.scales[first + u]));
          v[u] = (uint16_t)bf16_pair(value, value);
        }
    } else {
      const uint16_t *src = a.src[which] + r * a.ld[which] + j;
#pragma unroll
      for (int u = 0; u < kEach; ++u)
        if (j + u * 32 < a.cols) v[u] = src[u * 32];
    }
#pragma unroll
    for (int u = 0; u < kEach; ++u)
      if (j + u * 32 < a.cols) dst[u * 32] = v[u];
  }
}

// ---------------------------------------------------------------------------
// dg and du from what was kept
// ---------------------------------------------------------------------------
struct SlopeArgs {
  const void *dh;
  const void *gate, *up;  // BF16, or codes
  const uint8_t *scales[2];
  uint16_t *dg, *du;
  int64_t rows, f, ld_dh, ld_kept, groups, pitch;
  int32_t dh_vec, kept_vec;
};

// Bound: HBM, 2 + 33/16 + 4 bytes an element from 8-bit checkpoints; 8192 x 1408 takes 17
// us from a cold start (5.5 TB/s).  Eight columns make a unit; a thread has kUnits of them
// in flight.  (Sixteen columns at once by whole sectors: the whole backward call 1 %
// faster from the checkpoint, 3 % slower from BF16 and for ragged rows.)
constexpr int kUnits = 2;

template <int ACT, bool ACT8>
__global__ void __launch_bounds__(kThreads) slope_kernel(const __grid_constant__ SlopeArgs a) {
  const int64_t per_row = (a.f + 7) / 8, total = a.rows * per_row;
  wait_for_previous();
  let_next_start();
  const int64_t stride = (int64_t)gridDim.x * (kThreads * kUnits);
  for (int64_t i0 = (int64_t)blockIdx.x * (kThreads * kUnits) + threadIdx.x; i0 < total; i0 += stride) {
    int64_t row[kUnits], col[kUnits];
    uint4 d[kUnits], g[kUnits], u[kUnits];  // eight BF16 values, or of g and u eight codes and the scale byte
#pragma unroll
    for (int q = 0; q < kUnits; ++q) {
      const int64_t i = i0 + q * kThreads;
      if (i >= total) continue;
      if ((uint64_t)total >> 32 == 0)
        row[q] = (uint32_t)i / (uint32_t)per_row, col[q] = (uint32_t)i % (uint32_t)per_row * 8;
      else
        row[q] = i / per_row, col[q] = (i - row[q] * per_row) * 8;
      const int n = (int)(a.f - col[q] < 8 ? a.f - col[q] : 8);
      auto load = [&](const void *p, int64_t ld, bool vec) {
        const uint16_t *from = static_cast<const uint16_t *>(p) + row[q] * ld + col[q];
        if (vec && n == 8) return __ldcs(reinterpret_cast<const uint4 *>(from));
        uint32_t h[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = e < n ? from[e] : 0u;
        return make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
      };
      auto load_codes = [&](const void *p, const uint8_t *scales) {
        const uint2 c = __ldcs(reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(p) + row[q] * a.groups * kActGroup + col[q]));
        return make_uint4(c.x, c.y, scales[row[q] * a.groups + col[q] / (int)kActGroup], 0);
      };
      d[q] = load(a.dh, a.ld_dh, a.dh_vec != 0);
      g[q] = ACT8 ? load_codes(a.gate, a.scales[0]) : load(a.gate, a.ld_kept, a.kept_vec != 0);
      u[q] = ACT8 ? load_codes(a.up, a.scales[1]) : load(a.up, a.ld_kept, a.kept_vec != 0);
    }
#pragma unroll
    for (int q = 0; q < kUnits; ++q) {
      if (i0 + q * kThreads >= total) continue;
      float2 dv[4], gv[4], uv[4];
      unpack8(d[q], dv);
      auto values = [&](float2(&v)[4], const uint4 &r) {
        if (!ACT8) return unpack8(r, v);
        const float2 scale = both(act8_scale(r.z));
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = __fmul2_rn(act8_codes_of(act8_biased(e < 2 ? r.x : r.y), e % 2), scale);
      };
      values(gv, g[q]);
      values(uv, u[q]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float2 act, slope;
        act_of<true, ACT>(gv[e], act, slope);
        gv[e] = __fmul2_rn(__fmul2_rn(dv[e], uv[e]), slope);
        uv[e] = __fmul2_rn(dv[e], act);
      }
      // The pitch holds whole vectors; what lies past the row's end is never read.
      store8(a.dg, row[q] * a.pitch + col[q], true, gv);
      store8(a.du, row[q] * a.pitch + col[q], true, uv);
    }
  }
}

// ---------------------------------------------------------------------------
// The parts of split K loops, added in order
// ---------------------------------------------------------------------------
struct JoinArgs {
  const float *partial;   // Args::partial
  Grid grid;
  int32_t tile_m, tile_n;
  void *out[2];
  int64_t ld[2];
  int64_t rows, cols;     // of one output
  int32_t half;           // row tiles of the first output
  int32_t bf16, vec;
};

// Bound: L2, where the parts still are: 72 parts of 256 x 256 take 7 us.  Four columns of
// a row to a thread; a tile to the blocks of one y.
__global__ void __launch_bounds__(kThreads) join_kernel(const __grid_constant__ JoinArgs a) {
  const int part = a.tile_m * a.tile_n, i = ((int)blockIdx.x * kThreads + (int)threadIdx.x) * 4;
  const int2 tile = tile_at(a.grid, a.grid.whole + (int)blockIdx.y);
  const int second = tile.x >= a.half, r = i / a.tile_n;
  const int64_t row = (int64_t)(tile.x - second * a.half) * a.tile_m + r;
  const int64_t col = (int64_t)tile.y * a.tile_n + (i - r * a.tile_n);
  wait_for_previous();
  let_next_start();
  if (row >= a.rows || col >= a.cols) return;
  const float *p = a.partial + (int64_t)blockIdx.y * a.grid.splits * part + i;
  float4 v = *reinterpret_cast<const float4 *>(p);
#pragma unroll 4
  for (int k = 1; k < a.grid.splits; ++k) {
    const float4 q = *reinterpret_cast<const float4 *>(p + (int64_t)k * part);
    v.x += q.x, v.y += q.y, v.z += q.z, v.w += q.w;
  }
  const int64_t at = row * a.ld[second] + col;
  if (!a.vec || a.cols - col < 4) {
    const float s[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < a.cols - col) store_any(a.out[second], at + e, a.bf16 != 0, s[e]);
  } else if (a.bf16) {
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out[second]) + at) = make_uint2(bf16_pair(v.x, v.y), bf16_pair(v.z, v.w));
  } else {
    *reinterpret_cast<float4 *>(static_cast<float *>(a.out[second]) + at) = v;
  }
}

// ---------------------------------------------------------------------------
// Plan
// ---------------------------------------------------------------------------
// Rows of a tile: one block's 128, or a pair's 256.
bool pairs(int64_t rows) { return rows > kTileM; }
int64_t tile_rows(bool pair) { return pair ? 2 * kTileM : kTileM; }

// Row tiles of a band (see tile_at): 4,096 rows.
int32_t band(int64_t tile_m) { return (int32_t)(4096 / tile_m); }

// The gate / up tile: as many features as fill the workers in the fewest, fullest
// rounds.  A tile costs its features and, for its x slices and its start, about 24
// more; whole groups of 32, so that a checkpoint's groups stay within a tile.
struct GatedTiles {
  bool pair;
  Grid grid;
  int32_t tile_n;
};
GatedTiles gated_tiles(int64_t rows, int64_t f, int64_t d, int sms) {
  GatedTiles t = {};
  t.pair = pairs(rows);
  const int64_t m = blocks_of(rows, tile_rows(t.pair)), workers = t.pair ? sms / 2 : sms;
  int64_t best = INT64_MAX;
  for (int64_t features = 128; features >= 32; features -= 32) {
    const int64_t n = blocks_of(f, features), cost = blocks_of(m * n, workers) * (features + 24);
    if (cost >= best) continue;
    best = cost;
    t.tile_n = (int32_t)(2 * features);
    t.grid = {(int32_t)m, (int32_t)n, 0, 1, band(tile_rows(t.pair)), (int32_t)blocks_of(d, kTileK)};
  }
  return t;
}

// The backward products: tiles of 256 columns, or fewer where those would be mostly
// empty.  K loops are split where that shortens the longest worker's share: those of all
// tiles of a product, or of the tiles that are left after whole rounds (8192 x 1024 x
// 4096: 256 tiles of 128 K blocks on 76 workers; three rounds and 28 tiles in two parts
// each).  Costs are in hundredths of a K block of a full tile (which takes a pair about
// 0.33 us): a narrower tile's K block costs less, though not in proportion, for A is the
// same; a unit its K blocks, but an epilogue at least; joining parts a launch and the
// parts' bytes, at about 1.5 MB a K block.  The weight gradients come first unless the
// other order saves a twentieth: their operands wait in L2, dx reads the weights from HBM
// (2048 x 2048 x 6144 took 144 us with dx first, 140 with it last, for all that the
// shares were 337 and 358 K blocks).  A call that wants only some of the gradients splits
// as if it wanted all.
struct BackwardTiles {
  bool pair;
  int32_t tile_n, first, head;  // as in Args
  Grid grid[2];       // weight gradients, dx
  int64_t half[2];    // tiles of one weight's rows; K blocks of one half of dx
};

// A product's units in a plan: `whole` of cost `cost`, then `parts` of cost `part`.
struct Units {
  int64_t whole, parts, cost, part;
  int64_t all() const { return whole + parts; }
  int64_t longest() const { return whole > 0 ? cost : part; }
};
// The longest share of a worker (see Walk, whose steps this follows).
int64_t longest_share(const Units &a, const Units &b, int64_t head, int64_t workers) {
  const int64_t rem = a.all() % workers, others = workers - rem;
  auto count = [](int64_t from, int64_t step, int64_t below) { return from < below ? (below - from + step - 1) / step : 0; };
  // Shares change at few workers: where the long units end, and where the rounds of the
  // others' whole units and parts end.
  const int64_t rest = head * others;
  const int64_t ends[] = {0, rem, a.whole % workers, (b.whole > rest ? b.whole - rest : 0) % workers,
                          (b.all() > rest ? b.all() - rest : 0) % workers};
  int64_t longest = 0;
  for (int64_t w : ends) {
    const int64_t wholes = count(w, workers, a.whole), mine = count(w, workers, a.all());
    int64_t share = wholes * a.cost + (mine - wholes) * a.part, got[2];
    const int64_t below[2] = {b.whole, b.all()};
    for (int i = 0; i < 2; ++i) {
      got[i] = count(rest + w, workers, below[i]);
      if (w >= rem) got[i] += std::min(head, count(w - rem, others, below[i]));
    }
    share += got[0] * b.cost + (got[1] - got[0]) * b.part;
    longest = std::max(longest, share);
  }
  return longest;
}

BackwardTiles find_backward_tiles(int64_t rows, int64_t d, int64_t f, int sms) {
  BackwardTiles t = {};
  t.pair = pairs(rows);
  const int64_t tile_m = tile_rows(t.pair), workers = t.pair ? sms / 2 : sms;
  t.half[0] = blocks_of(f, tile_m), t.half[1] = blocks_of(f, kTileK);
  const int64_t m[2] = {2 * t.half[0], blocks_of(rows, tile_m)};
  const int64_t k[2] = {blocks_of(rows, kTileK), 2 * t.half[1]};
  constexpr int kChoices = 8;
  const int64_t by[kChoices] = {1, 2, 3, 4, 6, 8, 12, 16};
  int64_t best = INT64_MAX;
  for (int64_t width = 256; width >= (t.pair ? 128 : 64); width /= 2) {
    const int64_t n = blocks_of(d, width), block = width == 256 ? 100 : width == 128 ? 80 : 65;
    auto cost = [&](int64_t blocks) { return std::max<int64_t>(blocks, 10) * block + 100; };
    auto join = [&](int64_t parts) { return parts == 0 ? 0 : 900 + parts * (tile_m * width * 4) / 15000; };
    // Product w with its tiles from `whole` on in by[c] parts; none where parts would be too short, or empty.
    auto units = [&](int w, int64_t whole, int c) {
      const int64_t per = blocks_of(k[w], by[c]), tiles = m[w] * n;
      if (c == 0) return Units{tiles, 0, cost(k[w]), 0};
      if (per < 4 || blocks_of(k[w], per) != by[c]) return Units{};
      return Units{whole, (tiles - whole) * by[c], cost(k[w]), cost(per)};
    };
    const bool many = (m[0] + m[1]) * n > 8 * workers;
    for (int p = 0; p < kChoices; ++p)
      for (int q = 0; q < kChoices; ++q) {
        // All of a product's tiles in parts, then (leaving the first product's whole) those left after whole rounds.
        for (int left = 0; left < (p == 0 && q > 0 ? 2 : 1); ++left)
          for (int first = 0; first < 2; ++first) {
            if (many && (p > 0 || (q > 0 && !left))) continue;
            const int second = first ^ 1;
            const Units a = units(first, 0, p), one = units(second, 0, 0);
            const int64_t other = left || q == 0 ? one.cost : units(second, 0, q).part;
            if (a.all() == 0 || other == 0 || (first == 1 && a.longest() < other)) continue;
            const int64_t others = workers - a.all() % workers, ratio = std::max<int64_t>(1, a.longest() / other);
            for (int64_t head = ratio; head <= ratio + 1; ++head) {
              int64_t whole = 0;
              if (left) {
                if (one.whole < head * others) continue;
                whole = head * others + (one.whole - head * others) / workers * workers;
              }
              const Units b = units(second, whole, q);
              if (b.all() == 0 || (left && b.parts == 0)) continue;
              int64_t total = longest_share(a, b, head, workers) + join(a.parts) + join(b.parts);
              if (first == 1) total += total / 20;
              if (total >= best) continue;
              best = total;
              t.tile_n = (int32_t)width, t.first = first, t.head = (int32_t)head;
              for (int w = 0; w < 2; ++w) {
                const Units &u = w == first ? a : b;
                t.grid[w] = {(int32_t)m[w], (int32_t)n, (int32_t)u.whole, (int32_t)by[w == first ? p : q], band(tile_m), (int32_t)k[w]};
              }
            }
          }
      }
  }
  return t;
}

// A thread's last plans: a program has few sizes, and finding one takes longer than a launch.
BackwardTiles backward_tiles(int64_t rows, int64_t d, int64_t f, int sms) {
  struct Found {
    int64_t rows, d, f;
    int sms;
    BackwardTiles tiles;
  };
  constexpr int kFound = 8;
  static thread_local Found found[kFound] = {};
  static thread_local int next = 0;
  for (const Found &e : found)
    if (e.rows == rows && e.d == d && e.f == f && e.sms == sms) return e.tiles;
  Found &e = found[next++ % kFound];
  e = {rows, d, f, sms, find_backward_tiles(rows, d, f, sms)};
  return e.tiles;
}

struct Plan {
  int sms;
  bool stage_x, stage_wg, stage_wu;
  int64_t d_pitch, f_pitch;
  BackwardTiles tiles;
  int64_t at_x, at_wg, at_wu, at_dg, at_du, at_partial[2], bytes;
};

bool rows_off(int64_t rows, int64_t ld, bool base) { return base || (rows > 1 && ld % 8 != 0); }

Plan plan_of(const fsdp_ffn_desc_t *d, bool backward) {
  Plan p = {};
  p.sms = device_sms() > 0 ? device_sms() : 160;
  p.d_pitch = up_to(d->d, 8), p.f_pitch = up_to(d->f, 16);
  if (!backward && few_rows(d->rows, d->d, d->f)) return p;  // reads its operands where they are
  p.stage_x = d->x_dtype == FSDP_ACT8 || rows_off(d->rows, d->ld_x, d->unaligned & 1);
  p.stage_wg = rows_off(d->f, d->ld_w_gate, d->unaligned & 2);
  p.stage_wu = rows_off(d->f, d->ld_w_up, d->unaligned & 4);
  int64_t at = 0;
  auto take = [&](bool want, int64_t bytes) {
    const int64_t here = at;
    if (want) at += up_to(bytes, 256);
    return here;
  };
  p.at_x = take(p.stage_x, d->rows * p.d_pitch * 2);
  p.at_wg = take(p.stage_wg, d->f * p.d_pitch * 2);
  p.at_wu = take(p.stage_wu, d->f * p.d_pitch * 2);
  if (backward && d->rows > 0) {
    p.at_dg = take(true, d->rows * p.f_pitch * 2);
    p.at_du = take(true, d->rows * p.f_pitch * 2);
    p.tiles = backward_tiles(d->rows, d->d, d->f, p.sms);
    for (int w = 0; w < 2; ++w) {
      const int64_t parts = units_of(p.tiles.grid[w]) - p.tiles.grid[w].whole;
      p.at_partial[w] = take(parts > 0, parts * tile_rows(p.tiles.pair) * p.tiles.tile_n * 4);
    }
  }
  p.bytes = at;
  return p;
}

fsdp_status_t check_desc(const fsdp_ffn_desc_t *d, bool backward) {
  if (!d) return fail(FSDP_EINVAL, "desc is NULL");
  if (d->rows < 0) return fail(FSDP_EINVAL, "rows < 0");
  if (d->d < 1 || d->f < 1) return fail(FSDP_EINVAL, "d < 1 or f < 1");
  if (d->rows > kMaxDim || d->d > kMaxDim || d->f > kMaxDim)
    return fail(FSDP_EUNSUPPORTED, "rows, d or f is above 2^31 - 512");
  if (blocks_of(d->rows, kTileM) * blocks_of(d->f, kTileM) > (int64_t(1) << 24) ||
      blocks_of(d->rows, kTileM) * blocks_of(d->d, kTileM) > (int64_t(1) << 24) ||
      blocks_of(d->f, kTileM) * blocks_of(d->d, kTileM) > (int64_t(1) << 24))
    return fail(FSDP_EUNSUPPORTED, "a product has more than 2^24 tiles of 128 x 128");
  if (d->activation != FSDP_ACT_SILU && d->activation != FSDP_ACT_GELU) return fail(FSDP_EINVAL, "unknown activation");
  if (d->keep != FSDP_KEEP_NONE && d->keep != FSDP_KEEP_ACT8 && d->keep != FSDP_KEEP_BF16)
    return fail(FSDP_EINVAL, "unknown keep");
  if (d->x_dtype != FSDP_DTYPE_BF16 && !(backward && d->x_dtype == FSDP_ACT8))
    return fail(d->x_dtype == FSDP_DTYPE_F32 ? FSDP_EUNSUPPORTED : FSDP_EINVAL,
                backward ? "x_dtype is neither BF16 nor FSDP_ACT8" : "x_dtype is not BF16");
  if (backward && !float_dtype(d->dx_dtype)) return fail(FSDP_EINVAL, "unknown dx_dtype");
  if (backward && !float_dtype(d->dw_dtype)) return fail(FSDP_EINVAL, "unknown dw_dtype");
  if (d->unaligned & ~7) return fail(FSDP_EINVAL, "unknown bits in unaligned");
  return FSDP_OK;
}

fsdp_status_t check_operand(const void *p, int64_t rows, int64_t cols, int64_t ld, bool declared, const char *what) {
  fsdp_status_t st = check_matrix(p, rows, cols, ld, 2, what);
  if (st != FSDP_OK) return st;
  if (ld >= (int64_t(1) << 38)) return fail(FSDP_EUNSUPPORTED, std::string(what) + ": row distance above 2^38");
  if (rows > 0 && !aligned16(p) && !declared)
    return fail(FSDP_EINVAL, std::string(what) + " starts off a 16-byte boundary: say so in desc.unaligned");
  return FSDP_OK;
}

fsdp_status_t check_kept(const fsdp_ffn_desc_t *d, const void *gate, const void *up) {
  fsdp_status_t st = FSDP_OK;
  if (d->keep == FSDP_KEEP_NONE) {
    if (gate || up) return fail(FSDP_EINVAL, "gate or up given, but keep is FSDP_KEEP_NONE");
  } else if (d->keep == FSDP_KEEP_ACT8) {
    const int64_t bytes = act8_bytes(d->rows, d->f);
    if ((st = check_ptr(gate, bytes, 16, "gate", -1)) != FSDP_OK) return st;
    if ((st = check_ptr(up, bytes, 16, "up", -1)) != FSDP_OK) return st;
  } else {
    if ((st = check_matrix(gate, d->rows, d->f, d->ld_kept, 2, "gate")) != FSDP_OK) return st;
    if ((st = check_matrix(up, d->rows, d->f, d->ld_kept, 2, "up")) != FSDP_OK) return st;
  }
  return st;
}

bool vec_rows(const void *p, int64_t rows, int64_t ld, int64_t size) {
  return aligned16(p) && (rows <= 1 || ld * size % 16 == 0);
}

// A call's state: its operands, staged where they have to be.
struct Call {
  const fsdp_ffn_desc_t *d;
  Plan plan;
  uint8_t *ws;
  cudaStream_t stream;
  Operand x, wg, wu;

  fsdp_status_t stage(const void *px, const void *pwg, const void *pwu) {
    wg = {pwg, d->f, d->d, d->ld_w_gate};
    wu = {pwu, d->f, d->d, d->ld_w_up};
    x = {px, d->rows, d->d, d->ld_x};
    CopyArgs a = {};
    a.pitch = plan.d_pitch, a.cols = d->d;
    auto copy = [&](Operand &o, bool want, int64_t at, int i) {
      if (!want || o.rows == 0) return;
      a.src[i] = static_cast<const uint16_t *>(o.p), a.dst[i] = reinterpret_cast<uint16_t *>(ws + at);
      a.ld[i] = o.ld, a.rows[i] = o.rows;
      o.p = a.dst[i], o.ld = plan.d_pitch;
    };
    copy(wg, plan.stage_wg, plan.at_wg, 0);
    copy(wu, plan.stage_wu, plan.at_wu, 1);
    if (d->x_dtype == FSDP_ACT8 && a.rows[0] + a.rows[1] > 0) {  // with the weights, one launch less
      const int64_t groups = act8_groups(d->d);
      a.codes = static_cast<const uint8_t *>(px), a.scales = a.codes + d->rows * groups * kActGroup;
      copy(x, true, plan.at_x, 2);
    } else if (d->x_dtype == FSDP_ACT8) {
      x.p = ws + plan.at_x, x.ld = plan.d_pitch;
      fsdp_status_t st = fsdp_act8_load(px, d->rows, d->d, ws + plan.at_x, FSDP_DTYPE_BF16, plan.d_pitch,
                                        reinterpret_cast<fsdp_stream_t>(stream));
      if (st != FSDP_OK) return st;
    } else {
      copy(x, plan.stage_x, plan.at_x, 2);
    }
    const int64_t rows = a.rows[0] + a.rows[1] + a.rows[2];
    if (rows == 0) return FSDP_OK;
    int64_t grid = blocks_of(rows * blocks_of(a.cols, 256), kThreads / 32);
    if (grid > plan.sms * 16) grid = plan.sms * 16;
    void *args[] = {&a};
    return launched(launch_kernel(reinterpret_cast<const void *>(&copy_rows_kernel), dim3((unsigned)grid), dim3(kThreads),
                                  args, 0, stream, true));
  }

  bool operands(Args &a, const Operand (&left)[2], int left_rows, const Operand (&right)[3], int right_rows) {
    // One after the other, an operand given twice has one map.
    auto all = [](CUtensorMap *maps, const Operand *o, int n, int rows) {
      for (int i = 0; i < n; ++i) {
        if (i > 0 && o[i].p == o[i - 1].p && o[i].ld == o[i - 1].ld && o[i].rows == o[i - 1].rows)
          maps[i] = maps[i - 1];
        else if (!encode(&maps[i], o[i], rows))
          return false;
      }
      return true;
    };
    return all(a.a, left, 2, left_rows) && all(a.b, right, 3, right_rows);
  }

  // Launches one product; args' operands, tiles and outputs are set.
  fsdp_status_t launch(Mode mode, bool pair, Args &a) {
    cudaError_t e = gave_up_count(GAVE_UP_PRODUCT, &a.gave_up);
    if (e != cudaSuccess) return fail(FSDP_ECUDA, std::string("status count: ") + cudaGetErrorString(e));
    a.wait_limit_ns = wait_limit_ns();
    a.fault = wait_fault();
    a.act = d->activation == FSDP_ACT_SILU ? SILU : GELU;
    return launched((mode == FORWARD     ? launch_forward
                     : mode == RECOMPUTE ? launch_recompute
                                         : launch_backward)(pair, a, plan.sms, stream));
  }

  // FORWARD or RECOMPUTE.
  fsdp_status_t gated(Mode mode, Args &a) {
    const GatedTiles t = gated_tiles(d->rows, d->f, d->d, plan.sms);
    // Boxes of x no higher than x: rows that a box has to fill with zeros are slow (5 to 15
    // rows through 4096 x 12288 took 48 to 68 us with boxes of 128, 35 with these).  What the
    // rest of a stage holds meets only rows that are not stored.
    a.a_rows = (int32_t)(d->rows < kTileM ? up_to(d->rows, 8) : kTileM);
    if (!operands(a, {x, x}, a.a_rows, {wg, wu, wu}, t.tile_n / 2))
      return fail(FSDP_ECUDA, "cuTensorMapEncodeTiled failed or is missing");
    a.grid[0] = t.grid;
    a.tile_n = t.tile_n;
    a.m[0] = d->rows, a.n = d->f;
    return launch(mode, t.pair, a);
  }

  // Adds up the parts of product w, if there are any.
  fsdp_status_t join(const Args &a, int w) {
    const Grid &g = a.grid[w];
    if (units_of(g) == g.whole) return FSDP_OK;
    JoinArgs j = {};
    j.partial = a.partial[w], j.grid = g;
    j.tile_m = (int32_t)tile_rows(plan.tiles.pair), j.tile_n = a.tile_n;
    for (int i = 0; i < 2; ++i) j.out[i] = a.out[w == 1 ? 2 : i], j.ld[i] = a.ld_out[w == 1 ? 2 : i];
    j.rows = a.m[w], j.cols = a.n;
    j.half = w == 0 ? a.half[0] : g.m;
    j.bf16 = a.out_bf16[w], j.vec = a.out_width[w] >= 16;
    void *args[] = {&j};
    return launched(launch_kernel(reinterpret_cast<const void *>(&join_kernel),
                                  dim3((unsigned)(j.tile_m * j.tile_n / (4 * kThreads)), (unsigned)(g.m * g.n - g.whole)),
                                  dim3(kThreads), args, 0, stream, true));
  }
};

template <class A>
void kept_into(const fsdp_ffn_desc_t *d, void *gate, void *up, A &a) {
  a.keep = d->keep;
  a.groups = act8_groups(d->f);
  void *p[2] = {gate, up};
  for (int i = 0; i < 2; ++i) {
    a.codes[i] = static_cast<uint8_t *>(p[i]);
    a.scales[i] = a.codes[i] ? a.codes[i] + d->rows * a.groups * kActGroup : nullptr;
    a.kept[i] = p[i];
  }
  a.ld_kept = d->ld_kept;
}

}  // namespace
}  // namespace ffn
}  // namespace fsdp

using namespace fsdp;
using namespace fsdp::ffn;

extern "C" {

fsdp_status_t fsdp_gated_ffn_workspace(const fsdp_ffn_desc_t *d, int32_t backward, int64_t *bytes) {
  fsdp_status_t st = check_desc(d, backward != 0);
  if (st != FSDP_OK) return st;
  if (!bytes) return fail(FSDP_EINVAL, "bytes is NULL");
  *bytes = plan_of(d, backward != 0).bytes;
  clear_error();
  return FSDP_OK;
}

fsdp_status_t fsdp_gated_ffn_forward(const fsdp_ffn_desc_t *d, const void *x, const void *w_gate, const void *w_up,
                                     void *h, void *gate, void *up, void *workspace, int64_t workspace_bytes,
                                     fsdp_stream_t stream) {
  fsdp_status_t st = check_desc(d, false);
  if (st != FSDP_OK) return st;
  if ((st = check_operand(x, d->rows, d->d, d->ld_x, d->unaligned & 1, "x")) != FSDP_OK) return st;
  if ((st = check_operand(w_gate, d->f, d->d, d->ld_w_gate, d->unaligned & 2, "w_gate")) != FSDP_OK) return st;
  if ((st = check_operand(w_up, d->f, d->d, d->ld_w_up, d->unaligned & 4, "w_up")) != FSDP_OK) return st;
  if ((st = check_matrix(h, d->rows, d->f, d->ld_h, 2, "h")) != FSDP_OK) return st;
  if ((st = check_kept(d, gate, up)) != FSDP_OK) return st;
  Call c = {d, plan_of(d, false), static_cast<uint8_t *>(workspace), reinterpret_cast<cudaStream_t>(stream), {}, {}, {}};
  if (workspace_bytes < c.plan.bytes) return fail(FSDP_EINVAL, "workspace_bytes is below fsdp_gated_ffn_workspace");
  if ((st = check_ptr(workspace, c.plan.bytes, 16, "workspace", -1)) != FSDP_OK) return st;
  if (d->rows > 0 && few_rows(d->rows, d->d, d->f)) {
    RowsArgs a = {};
    a.x = x, a.w_gate = w_gate, a.w_up = w_up, a.h = h;
    a.rows = d->rows, a.d = d->d, a.f = d->f;
    a.ld_x = d->ld_x, a.ld_gate = d->ld_w_gate, a.ld_up = d->ld_w_up, a.ld_h = d->ld_h;
    a.act = d->activation == FSDP_ACT_SILU ? SILU : GELU;
    kept_into(d, gate, up, a);
    const bool vec = d->d % 8 == 0 && vec_rows(x, d->rows, d->ld_x, 2) && vec_rows(w_gate, d->f, d->ld_w_gate, 2) &&
                     vec_rows(w_up, d->f, d->ld_w_up, 2);
    if ((st = launched(launch_rows(a, vec, c.stream))) != FSDP_OK) return st;
  } else if (d->rows > 0) {
    if ((st = c.stage(x, w_gate, w_up)) != FSDP_OK) return st;
    Args a = {};
    a.out[0] = h, a.ld_out[0] = d->ld_h;
    a.out_width[0] = row_width(h, d->rows, d->ld_h, 2);
    kept_into(d, gate, up, a);
    const int64_t ld = d->keep == FSDP_KEEP_ACT8 ? 16 : d->ld_kept;  // a checkpoint's groups are 32 bytes each
    const int wg = row_width(gate, d->rows, ld, 2), wu = row_width(up, d->rows, ld, 2);
    a.keep_width = wg < wu ? wg : wu;
    if ((st = c.gated(FORWARD, a)) != FSDP_OK) return st;
  }
  clear_error();
  return FSDP_OK;
}

fsdp_status_t fsdp_gated_ffn_backward(const fsdp_ffn_desc_t *d, const void *dh, const void *x, const void *w_gate,
                                      const void *w_up, const void *gate, const void *up, void *dx, void *dw_gate,
                                      void *dw_up, void *workspace, int64_t workspace_bytes, fsdp_stream_t stream) {
  fsdp_status_t st = check_desc(d, true);
  if (st != FSDP_OK) return st;
  if ((st = check_matrix(dh, d->rows, d->f, d->ld_h, 2, "dh")) != FSDP_OK) return st;
  if (d->x_dtype == FSDP_ACT8)
    st = check_ptr(x, act8_bytes(d->rows, d->d), 16, "x", -1);
  else
    st = check_operand(x, d->rows, d->d, d->ld_x, d->unaligned & 1, "x");
  if (st != FSDP_OK) return st;
  if ((st = check_operand(w_gate, d->f, d->d, d->ld_w_gate, d->unaligned & 2, "w_gate")) != FSDP_OK) return st;
  if ((st = check_operand(w_up, d->f, d->d, d->ld_w_up, d->unaligned & 4, "w_up")) != FSDP_OK) return st;
  if ((st = check_kept(d, gate, up)) != FSDP_OK) return st;
  const int64_t xsize = dtype_bytes(d->dx_dtype), wsize = dtype_bytes(d->dw_dtype);
  if (dx && (st = check_matrix(dx, d->rows, d->d, d->ld_dx, xsize, "dx")) != FSDP_OK) return st;
  if (!dw_gate != !dw_up) return fail(FSDP_EINVAL, "dw_gate and dw_up are given together or not at all");
  if (dw_gate && (st = check_matrix(dw_gate, d->f, d->d, d->ld_dw_gate, wsize, "dw_gate")) != FSDP_OK) return st;
  if (dw_up && (st = check_matrix(dw_up, d->f, d->d, d->ld_dw_up, wsize, "dw_up")) != FSDP_OK) return st;
  Call c = {d, plan_of(d, true), static_cast<uint8_t *>(workspace), reinterpret_cast<cudaStream_t>(stream), {}, {}, {}};
  if (workspace_bytes < c.plan.bytes) return fail(FSDP_EINVAL, "workspace_bytes is below fsdp_gated_ffn_workspace");
  if ((st = check_ptr(workspace, c.plan.bytes, 16, "workspace", -1)) != FSDP_OK) return st;
  if (d->rows == 0) {
    void *p[2] = {dw_gate, dw_up};
    const int64_t ld[2] = {d->ld_dw_gate, d->ld_dw_up};
    for (int i = 0; i < 2; ++i)
      if (p[i]) {
        cudaError_t e = cudaMemset2DAsync(p[i], (size_t)(ld[i] * wsize), 0, (size_t)(d->d * wsize), (size_t)d->f, c.stream);
        if (e != cudaSuccess) return fail(FSDP_ECUDA, std::string("cudaMemset2DAsync: ") + cudaGetErrorString(e));
      }
    clear_error();
    return FSDP_OK;
  }
  if (!dx && !dw_gate) {
    clear_error();
    return FSDP_OK;
  }
  if ((st = c.stage(x, w_gate, w_up)) != FSDP_OK) return st;
  uint16_t *dg = reinterpret_cast<uint16_t *>(c.ws + c.plan.at_dg), *du = reinterpret_cast<uint16_t *>(c.ws + c.plan.at_du);
  if (d->keep == FSDP_KEEP_NONE) {
    Args a = {};
    a.out[0] = dg, a.out[1] = du;
    a.ld_out[0] = a.ld_out[1] = c.plan.f_pitch;
    a.out_width[0] = row_width(c.ws, d->rows, c.plan.f_pitch, 2);
    a.dh = dh, a.ld_dh = d->ld_h, a.dh_vec = vec_rows(dh, d->rows, d->ld_h, 2);
    if ((st = c.gated(RECOMPUTE, a)) != FSDP_OK) return st;
  } else {
    SlopeArgs s = {};
    s.dh = dh, s.gate = gate, s.up = up;
    s.groups = act8_groups(d->f);
    const void *p[2] = {gate, up};
    for (int i = 0; i < 2; ++i) s.scales[i] = static_cast<const uint8_t *>(p[i]) + d->rows * s.groups * kActGroup;
    s.dg = dg, s.du = du;
    s.rows = d->rows, s.f = d->f, s.ld_dh = d->ld_h, s.ld_kept = d->ld_kept, s.pitch = c.plan.f_pitch;
    s.dh_vec = vec_rows(dh, d->rows, d->ld_h, 2);
    s.kept_vec = vec_rows(gate, d->rows, d->ld_kept, 2) && vec_rows(up, d->rows, d->ld_kept, 2);
    int64_t grid = blocks_of(d->rows * blocks_of(d->f, 8), kThreads * kUnits);
    if (grid > (int64_t)c.plan.sms * 64) grid = (int64_t)c.plan.sms * 64;
    const bool silu = d->activation == FSDP_ACT_SILU, act8 = d->keep == FSDP_KEEP_ACT8;
    const void *fn = silu ? (act8 ? reinterpret_cast<const void *>(&slope_kernel<SILU, true>)
                                  : reinterpret_cast<const void *>(&slope_kernel<SILU, false>))
                          : (act8 ? reinterpret_cast<const void *>(&slope_kernel<GELU, true>)
                                  : reinterpret_cast<const void *>(&slope_kernel<GELU, false>));
    void *args[] = {&s};
    st = launched(launch_kernel(fn, dim3((unsigned)grid), dim3(kThreads), args, 0,
                                c.stream, true));
    if (st != FSDP_OK) return st;
  }
  const Operand og = {dg, d->rows, d->f, c.plan.f_pitch}, ou = {du, d->rows, d->f, c.plan.f_pitch};
  Args a = {};
  if (!c.operands(a, {og, ou}, 64, {c.wg, c.wu, c.x}, 64))
    return fail(FSDP_ECUDA, "cuTensorMapEncodeTiled failed or is missing");
  const BackwardTiles &t = c.plan.tiles;
  a.tile_n = t.tile_n;
  a.out[0] = dw_gate, a.out[1] = dw_up, a.out[2] = dx;
  a.ld_out[0] = d->ld_dw_gate, a.ld_out[1] = d->ld_dw_up, a.ld_out[2] = d->ld_dx;
  a.m[0] = d->f, a.m[1] = d->rows, a.n = d->d;
  a.out_bf16[0] = d->dw_dtype == FSDP_DTYPE_BF16, a.out_bf16[1] = d->dx_dtype == FSDP_DTYPE_BF16;
  const int rg = row_width(dw_gate, d->f, d->ld_dw_gate, wsize), ru = row_width(dw_up, d->f, d->ld_dw_up, wsize);
  a.out_width[0] = rg < ru ? rg : ru, a.out_width[1] = row_width(dx, d->rows, d->ld_dx, xsize);
  for (int w = 0; w < 2; ++w) {
    a.grid[w] = t.grid[w], a.half[w] = (int32_t)t.half[w];
    a.partial[w] = reinterpret_cast<float *>(c.ws + c.plan.at_partial[w]);
  }
  a.partial_width = row_width(c.ws, 2, t.tile_n, 4);
  a.first = t.first, a.head = t.head;
  if (!dw_gate) a.grid[0].m = a.grid[0].whole = 0;  // no tiles
  if (!dx) a.grid[1].m = a.grid[1].whole = 0;
  if ((st = c.launch(BACKWARD, t.pair, a)) != FSDP_OK) return st;
  for (int w = 0; w < 2; ++w)
    if (a.grid[w].m > 0 && (st = c.join(a, w)) != FSDP_OK) return st;
  clear_error();
  return FSDP_OK;
}

}  // extern "C"

// The tensor-core kernel of the gated feed-forward block (see ffn.h).  Included by the
// files that instantiate it, one to a use, which compile side by side.
#pragma once

#include "ffn.h"

namespace fsdp {
namespace ffn {
namespace {

// Two epilogue warps to each quarter of TMEM's lanes, one warp that loads and one that
// issues MMAs.  (Sixteen epilogue warps, which the registers would allow, take 5 % longer
// at 8192 x 1024 x 4096: the MMAs bound it, and more warps slow the thread that issues them.)
constexpr int kEpilogueWarps = 8;
constexpr int kThreads = 64 + 32 * kEpilogueWarps;
constexpr int kTileN = 256;       // most accumulator columns of a tile
constexpr int kAccumulators = 2;  // 2 x 256 columns: all of TMEM
constexpr int kTmemColumns = kTileN * kAccumulators;

// Each epilogue warp's buffer for 32 rows x 16 columns that change from a row to a
// thread to a row to half a warp, for rows that no vector store fits.
constexpr int kTurnPitch = 17;
constexpr int kTurnBytes = 32 * kTurnPitch * 4;

constexpr int kA = kTileM * kTileK * 2;  // bytes of a block's A in a stage; B follows
constexpr int kMostStages = 8;
// Shared memory of the stages and, only where some rows take no vectors, of the warps'
// buffers after them; the stages begin on a 1,024-byte boundary.
constexpr int kDynamic = 226 * 1024;
__host__ __device__ __forceinline__ int ring_bytes(bool turns) {
  return kDynamic - 1024 - (turns ? kEpilogueWarps * kTurnBytes : 0);
}

// Bytes of a block's stage, and how many fit: narrow tiles get more, so that as many bytes
// are in flight (with four stages for all, 16 rows through 2048 x 6144 took 22 us, not 13).
__host__ __device__ __forceinline__ int stage_bytes(int columns, int cg) { return kA + columns / cg * (kTileK * 2); }
__host__ __device__ __forceinline__ int stages_of(int ring, int bytes) { return min(ring / bytes, kMostStages); }

struct Shared {
  uint64_t full[kMostStages], empty[kMostStages], tmem_full[kAccumulators], tmem_empty[kAccumulators], drain;
  uint32_t tmem, stop, filled;
};

// A unit of work: one tile, or one part of its K loop.
struct Unit {
  int which;           // of Args::grid
  int m, n;            // tile indices
  int part;            // place among the product's parts; -1: a whole tile
  int k0, k1;          // K blocks
};

// The units of one worker.  The units of the product with the longer ones come first,
// every W-th of them to a worker.  What is left over, `rem` units, makes the first `rem`
// workers one long unit later than the others, which therefore go `head` rounds of the
// short ones ahead (as many as a long one takes); then all go on together.  Workers at
// work at one time have units side by side throughout, which share operands in L2.
// (4096 x 1024 x 4096: 64 units of 128 K blocks and 128 of 64 for 76 workers, of which 12
// go two short units ahead.)
template <int MODE>
struct Walk {
  int i, end, step;
  int first, others, ahead, late;

  __device__ Walk(const Args &a, int worker, int workers) : i(worker), step(workers) {
    end = first = units_of(a.grid[MODE == BACKWARD ? a.first : 0]);
    if constexpr (MODE == BACKWARD) {
      end += units_of(a.grid[a.first ^ 1]);
      const int rem = first % workers;
      others = workers - rem;
      ahead = worker >= rem ? a.head - 1 : 0;
      late = worker < rem ? (a.head - 1) * others : 0;
    }
  }
  __device__ __forceinline__ bool more() const { return i < end; }
  __device__ __forceinline__ void next() {
    if (MODE == BACKWARD && i >= first && ahead > 0) {
      i += others, --ahead;
    } else {
      const bool was = i < first;
      i += step;
      if (MODE == BACKWARD && was && i >= first) i += late;
    }
  }
};

// Unit i as the product it belongs to and its place there.
template <int MODE>
__device__ __forceinline__ int product_of(const Args &a, int &i) {
  if constexpr (MODE != BACKWARD) return 0;
  const int units = units_of(a.grid[a.first]);
  if (i < units) return a.first;
  i -= units;
  return a.first ^ 1;
}

// The K blocks of unit i, all that issuing its MMAs takes: worked out by one thread while
// the tensor cores run dry, so without the divisions that find the tile.
struct Span {
  int which, k0, k1;
};
__device__ __forceinline__ void part_of(const Grid &g, int split, int &k0, int &k1) {
  const int per = (g.k_blocks + g.splits - 1) / g.splits;
  k0 = min(split * per, g.k_blocks);
  k1 = min(k0 + per, g.k_blocks);
}
template <int MODE>
__device__ __forceinline__ Span span_at(const Args &a, int i) {
  Span s;
  s.which = product_of<MODE>(a, i);
  const Grid &g = a.grid[s.which];
  s.k0 = 0, s.k1 = g.k_blocks;
  if (MODE == BACKWARD && i >= g.whole) part_of(g, (i - g.whole) % g.splits, s.k0, s.k1);
  return s;
}

template <int MODE>
__device__ __forceinline__ Unit unit_at(const Args &a, int i) {
  Unit u;
  u.which = product_of<MODE>(a, i);
  const Grid &g = a.grid[u.which];
  u.part = -1;
  u.k0 = 0, u.k1 = g.k_blocks;
  int t = i;
  if (MODE == BACKWARD && i >= g.whole) {
    u.part = i - g.whole;
    t = g.whole + u.part / g.splits;
    part_of(g, u.part % g.splits, u.k0, u.k1);
  }
  const int2 at = tile_at(g, t);
  u.m = at.x, u.n = at.y;
  return u;
}

// How a tile's K blocks are loaded: boxes at (x, y) of two maps, advanced by (kx, ky) from
// K block to K block.  One thread loads and one issues MMAs, about 500 cycles to a K
// block, so what they do for each is worked out once a tile.
template <int MODE, int CG, int COLS>
struct Loader {
  const CUtensorMap *ma, *mb, *mb2;
  int ax, ay, bx, by;        // next box of A and of B
  int acx, acy;              // from one box of A to the next in the stage
  int kax, kay, kby;         // K block to K block: A along x or y, B (not FORWARD) along y

  __device__ Loader(const Args &a, const Unit &u, int rank) {
    if constexpr (MODE != BACKWARD) {
      const int half = a.tile_n / 2;
      ma = &a.a[0], mb = &a.b[CG == 1 ? 0 : rank], mb2 = &a.b[1];
      ax = u.k0 * kTileK, ay = (u.m * CG + rank) * kTileM;
      bx = ax, by = u.n * half;
    } else {
      // Boxes of 64 x 64 throughout.  Along K in a row (A of dx): two boxes of 64 rows lie
      // one after the other; along M or N in a row: one box to 64 of them.
      bx = u.n * COLS + rank * (COLS / CG);
      if (u.which == 1) {
        go_to(a, u.k0);
        ay = (u.m * CG + rank) * kTileM;
        acx = 0, acy = 64, kax = kTileK, kay = 0;
      } else {
        const int up = u.m >= a.half[0];
        ma = &a.a[up], mb = &a.b[2];
        ax = ((u.m - up * a.half[0]) * CG + rank) * kTileM, ay = by = u.k0 * kTileK;
        acx = 64, acy = 0, kax = 0, kay = kTileK;
      }
      kby = kTileK;
    }
  }
  // dx: the K block `kb` of the sum over gate and up.
  __device__ __forceinline__ void go_to(const Args &a, int kb) {
    const int up = kb >= a.half[1];
    ma = &a.a[up], mb = &a.b[up];
    ax = by = (kb - up * a.half[1]) * kTileK;
  }
  __device__ __forceinline__ void load(const Args &a, uint32_t at, uint32_t bar) const {
    const uint32_t sb = at + kA;
    if constexpr (MODE != BACKWARD) {
      tc::tma_load<CG>(at, ma, ax, ay, bar);
      tc::tma_load<CG>(sb, mb, bx, by, bar);
      if constexpr (CG == 1) tc::tma_load<CG>(sb + a.tile_n / 2 * (kTileK * 2), mb2, bx, by, bar);
    } else {
#pragma unroll
      for (int c = 0; c < kTileM / 64; ++c) tc::tma_load<CG>(at + c * 8192, ma, ax + c * acx, ay + c * acy, bar);
#pragma unroll
      for (int c = 0; c < COLS / CG / 64; ++c) tc::tma_load<CG>(sb + c * 8192, mb, bx + c * 64, by, bar);
    }
  }
  __device__ __forceinline__ void advance() {
    if constexpr (MODE != BACKWARD)
      ax += kTileK, bx += kTileK;
    else
      ax += kax, ay += kay, by += kby;
  }
};

// A warp's 32 x 32 part of a tile: one row to a thread.
struct Part {
  int64_t col;   // first column
  int n;         // columns that exist, at most 32
  int rows;      // rows that exist (lanes below it), at most 32
  int64_t row;   // this thread's row
  float *turn;   // the warp's buffer
};

// The part to memory; `width`: row_width().  Stores of a row to a thread go to 32 rows at
// a time; whole 32-byte sectors keep that from costing two writes a sector.  Rows that no
// vector fits go through the warp's buffer, half a warp to a row (element by element from
// a row to a thread, a store instruction would touch 32 sectors for 64 bytes).
__device__ __forceinline__ bool whole(int width, const Part &q) { return width >= 16 && q.n >= 32; }

// 32 columns as 16 or 32 words of a row of whole vectors.
template <int WORDS>
__device__ __forceinline__ void store_words(void *row, int width, const uint32_t (&w)[WORDS]) {
  uint4 *to = static_cast<uint4 *>(row);
#pragma unroll
  for (int i = 0; i < WORDS / 8; ++i) {
    const uint32_t(&h)[8] = reinterpret_cast<const uint32_t(&)[8]>(w[8 * i]);
    if (width == 32)
      store32(to + 2 * i, h);
    else
      to[2 * i] = make_uint4(h[0], h[1], h[2], h[3]), to[2 * i + 1] = make_uint4(h[4], h[5], h[6], h[7]);
  }
}

// Sixteen columns from `side` on, through the buffer.
template <class F>
__device__ __forceinline__ void store_turned(void *p, int64_t ld, bool bf16, const Part &q, F &&value) {
  const int lane = threadIdx.x & 31;
  const int64_t first = q.row - lane;
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 16; ++e) q.turn[lane * kTurnPitch + e] = value(side * 16 + e);
    __syncwarp();
    const int c = side * 16 + lane % 16;
    if (c < q.n)
      for (int r = lane / 16; r < q.rows; r += 2)
        store_any(p, (first + r) * ld + q.col + c, bf16, q.turn[r * kTurnPitch + lane % 16]);
  }
}

// 64 bytes of each row, from a row to a thread, as two threads to a row: neighbours
// exchange halves and store first the even one's row, then the odd one's, so that a row's
// two sectors leave together (forward 8192 x 1024 x 4096 80 us without the exchange, 78.5
// with it; with 8-bit copies 98 and 95.5: measured in turn as single calls among others).  `row`: this thread's; `pitch`: bytes.
__device__ __forceinline__ void store_pairs(void *row, int64_t pitch, const uint32_t (&w)[16], int rows) {
  const int lane = threadIdx.x & 31;
  const bool odd = lane & 1;
  uint32_t a[8], b[8];  // for the even row, the odd row
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, odd ? w[i] : w[8 + i], 1);
    a[i] = odd ? other : w[i];
    b[i] = odd ? w[8 + i] : other;
  }
  uint8_t *const even = static_cast<uint8_t *>(row) - (odd ? pitch - 32 : 0);
  if ((lane & ~1) < rows) store32(even, a);
  if ((lane | 1) < rows) store32(even + pitch, b);
}

// Binary32 values (as bits), or BF16 pairs, in memory.
__device__ __forceinline__ void store_part(void *p, int64_t ld, bool bf16, int width, const uint32_t (&v)[32], const Part &q) {
  if (!whole(width, q))
    return store_turned(p, ld, bf16, q, [&](int e) { return __uint_as_float(v[e]); });
  const int64_t at = q.row * ld + q.col;
  if (bf16) {
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = bf16_pair(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
    if (width == 32)
      store_pairs(static_cast<uint16_t *>(p) + at, ld * 2, w, q.rows);
    else if ((int)(threadIdx.x & 31) < q.rows)
      store_words(static_cast<uint16_t *>(p) + at, width, w);
  } else if (width == 32) {
#pragma unroll
    for (int half = 0; half < 2; ++half)
      store_pairs(static_cast<float *>(p) + at + 16 * half, ld * 4, reinterpret_cast<const uint32_t(&)[16]>(v[16 * half]), q.rows);
  } else if ((int)(threadIdx.x & 31) < q.rows) {
    store_words(static_cast<float *>(p) + at, width, v);
  }
}
__device__ __forceinline__ void store_part(void *p, int64_t ld, int width, const uint32_t (&w)[16], const Part &q) {
  if (!whole(width, q))
    return store_turned(p, ld, true, q, [&](int e) { return e % 2 ? bf16_high(w[e / 2]) : bf16_low(w[e / 2]); });
  if (width == 32)
    store_pairs(static_cast<uint16_t *>(p) + q.row * ld + q.col, ld * 2, w, q.rows);
  else if ((int)(threadIdx.x & 31) < q.rows)
    store_words(static_cast<uint16_t *>(p) + q.row * ld + q.col, width, w);
}

// The part of a BF16 matrix as pairs, 0 where there is none; `vec`: its rows start on
// 16-byte boundaries.
__device__ __forceinline__ void load_part(const uint16_t *p, int64_t ld, bool vec, uint32_t (&w)[16], const Part &q) {
  const int lane = threadIdx.x & 31;
  if (vec && q.n >= 32) {
    const uint4 *from = reinterpret_cast<const uint4 *>(p + q.row * ld + q.col);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 r = lane < q.rows ? from[i] : make_uint4(0, 0, 0, 0);
      w[4 * i] = r.x, w[4 * i + 1] = r.y, w[4 * i + 2] = r.z, w[4 * i + 3] = r.w;
    }
    return;
  }
  const int64_t first = q.row - lane;
  uint32_t *const turn = reinterpret_cast<uint32_t *>(q.turn);
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const int c = side * 16 + lane % 16;
    __syncwarp();
    for (int r = lane / 16; r < 32; r += 2)
      turn[r * kTurnPitch + lane % 16] = c < q.n && r < q.rows ? p[(first + r) * ld + q.col + c] : 0u;
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 8; ++e)
      w[side * 8 + e] = turn[lane * kTurnPitch + 2 * e] | turn[lane * kTurnPitch + 2 * e + 1] << 16;
  }
}

__device__ __forceinline__ float2 pair_at(const uint32_t (&r)[32], int i) {
  return make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
}

// The codes of 32 consecutive elements, one whole group; its scale byte is returned.
__device__ __forceinline__ uint32_t keep_group(uint8_t *codes, const uint32_t (&r)[32], bool sector) {
  float2 v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = pair_at(r, i);
  const uint32_t s = act8_scale_byte(act8_top(v));
  act8_store<32>(codes, v, s, sector);
  return s;
}

// A warp's part of a gate / up tile.  What is kept goes first, and results are packed as
// they are made, so that few values live beside g and u.  `next`: the warp has the 32
// columns after these too; `held`: scale bytes that wait for theirs (0: none).
template <int MODE, int ACT, int KEEP>
__device__ __forceinline__ void gated_part(const Args &a, uint32_t (&gr)[32], uint32_t (&ur)[32], const Part &q, bool next,
                                           uint32_t &held) {
  if constexpr (MODE == FORWARD) {
    if constexpr (KEEP == 1) {
      if (q.n < 32) {  // a row's last group: its missing elements are 0
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (i >= q.n) gr[i] = ur[i] = 0u;
      }
      if ((int)(threadIdx.x & 31) < q.rows) {
        const int64_t group = q.row * a.groups + q.col / (int)kActGroup;
        const uint32_t s = keep_group(a.codes[0] + group * kActGroup, gr, a.keep_width == 32) |
                           keep_group(a.codes[1] + group * kActGroup, ur, a.keep_width == 32) << 16;
        // Scale bytes of two groups leave together: one by one they are as many sectors
        // for L2 as the codes (96 and 92 us at 8192 x 1024 x 4096).
        if (group % 2 == 0 && next && a.groups % 2 == 0) {
          held = s;
        } else {
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const uint32_t mine = s >> 16 * w & 0xFFu;
            if (held != 0)
              *reinterpret_cast<uint16_t *>(a.scales[w] + group - 1) = (uint16_t)((held >> 16 * w & 0xFFu) | mine << 8);
            else
              a.scales[w][group] = (uint8_t)mine;
          }
          held = 0;
        }
      }
    } else if constexpr (KEEP == 2) {
      store_part(a.kept[0], a.ld_kept, true, a.keep_width, gr, q);
      store_part(a.kept[1], a.ld_kept, true, a.keep_width, ur, q);
    }
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float2 y, none;
      act_of<false, ACT>(pair_at(gr, i), y, none);
      y = __fmul2_rn(y, pair_at(ur, i));
      w[i] = bf16_pair(y.x, y.y);
    }
    store_part(a.out[0], a.ld_out[0], a.out_width[0], w, q);
  } else {
    uint32_t d[16];
    load_part(static_cast<const uint16_t *>(a.dh), a.ld_dh, a.dh_vec != 0, d, q);
    uint32_t dg[16], du[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 dh = make_float2(bf16_low(d[i]), bf16_high(d[i]));
      float2 act, slope;
      act_of<true, ACT>(pair_at(gr, i), act, slope);
      slope = __fmul2_rn(__fmul2_rn(dh, pair_at(ur, i)), slope);
      act = __fmul2_rn(dh, act);
      dg[i] = bf16_pair(slope.x, slope.y), du[i] = bf16_pair(act.x, act.y);
    }
    store_part(a.out[0], a.ld_out[0], a.out_width[0], dg, q);
    store_part(a.out[1], a.ld_out[1], a.out_width[0], du, q);
  }
}

// Test hook: the first worker leaves its first stage empty, so the wait for it gives up.
__device__ __forceinline__ bool skips_first(const Args &a, int worker) { return a.fault != 0 && worker == 0; }

// After a wait that gave up, by one thread once every role has left its loop: wait
// (again for a limited time) until the copies in flight have landed.  The leader's
// barriers count both blocks' bytes; what the other block of a pair sent to a stage
// that the leader never armed is not counted anywhere and gets a fixed time.
__device__ __noinline__ void land_copies(Shared &sh, const Args &a, uint32_t stages, int rank, bool skipped) {
  if (rank == 0) {
    uint32_t f = sh.filled > stages ? sh.filled - stages : 0;
    if (f == 0 && skipped) f = 1;
    for (; f < sh.filled; ++f) {
      uint32_t never = 0;
      tc::bar_wait(tc::smem(&sh.full[f % stages]), (f / stages) & 1u, a.wait_limit_ns, &never);
    }
  } else {
    const uint64_t began = tc::now_ns();
    while (tc::now_ns() - began < 1000000) {
    }
  }
}

// COLS: columns of a BACKWARD tile (other uses go by Args).
template <int MODE, int CG, int ACT, int KEEP, int COLS>
__global__ void __launch_bounds__(kThreads, 1) product_kernel(const __grid_constant__ Args a) {
  extern __shared__ uint8_t dynamic[];
  __shared__ Shared sh;
  const int columns = MODE == BACKWARD ? COLS : a.tile_n;
  const uint32_t stage_size = stage_bytes(columns, CG), stage_count = stages_of(ring_bytes(a.turns != 0), (int)stage_size);
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const uint32_t stages = (tc::smem(dynamic) + 1023u) & ~1023u;
  const int rank = CG == 1 ? 0 : (int)tc::cluster_rank();
  const int worker = blockIdx.x / CG, workers = gridDim.x / CG;
  volatile uint32_t *stop = &sh.stop;

  if (warp == 0 && lane == 0) {
    for (uint32_t s = 0; s < stage_count; ++s) {
      tc::bar_init(tc::smem(&sh.full[s]), 1);
      tc::bar_init(tc::smem(&sh.empty[s]), 1);
    }
    for (int s = 0; s < kAccumulators; ++s) {
      tc::bar_init(tc::smem(&sh.tmem_full[s]), 1);
      tc::bar_init(tc::smem(&sh.tmem_empty[s]), kEpilogueWarps * CG);
    }
    tc::bar_init(tc::smem(&sh.drain), 1);
    sh.stop = sh.filled = 0;
    tc::bar_init_fence();
    tc::tma_prefetch_map(&a.a[0]);
    tc::tma_prefetch_map(&a.b[0]);
  }
  if (warp == 1) {
    tc::tmem_alloc<CG>(tc::smem(&sh.tmem), kTmemColumns);
    tc::fence_before();
  }
  __syncthreads();
  if constexpr (CG == 2) tc::cluster_sync();
  tc::fence_after();
  const uint32_t tmem = sh.tmem;
  wait_for_previous();
  let_next_start();

  bool ok = true;
  if (warp == 0) {
    // ---- loads ---------------------------------------------------------------
    if (lane == 0) {
      uint32_t stage = 0, phase = 0, filled = 0;
      const uint32_t bytes = CG * stage_size - (MODE == BACKWARD ? 0 : (kTileM - a.a_rows) * (kTileK * 2));
      const uint32_t full = tc::smem(&sh.full[0]), empty = tc::smem(&sh.empty[0]);
      const uint32_t leader = CG == 1 ? full : tc::at_rank(full, 0);
      const bool skip = skips_first(a, worker);
      const int half = MODE == BACKWARD ? a.half[1] : 0;
      for (Walk<MODE> walk(a, worker, workers); walk.more() && ok; walk.next()) {
        const Unit u = unit_at<MODE>(a, walk.i);
        Loader<MODE, CG, COLS> from(a, u, rank);
        const int k0 = u.k0, k1 = u.k1, which = u.which;
        for (int kb = k0; kb < k1; ++kb) {
          if (!(ok = tc::bar_wait(empty + stage * 8, phase ^ 1u, a.wait_limit_ns, stop))) break;
          if (MODE == BACKWARD && which == 1 && kb == half) from.go_to(a, kb);
          if (!skip || filled > 0) {
            if (rank == 0) tc::bar_expect(full + stage * 8, bytes);
            from.load(a, stages + stage * stage_size, leader + stage * 8);
          }
          from.advance();
          ++filled;
          if (++stage == stage_count) stage = 0, phase ^= 1u;
        }
      }
      // The last products hand their stages back before this block leaves: the other
      // block of a pair must not signal into shared memory that is no longer its own.
      for (uint32_t s = 0; ok && s < stage_count; ++s) {
        ok = tc::bar_wait(tc::smem(&sh.empty[stage]), phase ^ 1u, a.wait_limit_ns, stop);
        if (++stage == stage_count) stage = 0, phase ^= 1u;
      }
      sh.filled = filled;
    }
  } else if (warp == 1) {
    // ---- products ------------------------------------------------------------
    if (lane == 0 && rank == 0) {
      uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0;
      bool issued = false;
      const uint32_t full = tc::smem(&sh.full[0]), empty = tc::smem(&sh.empty[0]);
      for (Walk<MODE> walk(a, worker, workers); walk.more() && ok; walk.next()) {
        const Span u = span_at<MODE>(a, walk.i);
        if (!(ok = tc::bar_wait(tc::smem(&sh.tmem_empty[acc]), acc_phase ^ 1u, a.wait_limit_ns, stop))) break;
        tc::fence_after();
        const uint32_t d = tmem + acc * kTileN;
        // Majors by use.  Descriptors advance by 16 K values: 32 bytes within a row, or 16
        // rows of 128 bytes (in units of 16 bytes).
        const bool a_mn = MODE == BACKWARD && u.which == 0, b_mn = MODE == BACKWARD;
        const uint32_t idesc = tc::instruction(kTileM * CG, columns, a_mn, b_mn);
        const uint32_t a0 = tc::operand_low(stages, a_mn ? 8192 : 16), b0 = tc::operand_low(stages + kA, b_mn ? 8192 : 16);
        const uint32_t a_step = a_mn ? 128 : 2, b_step = b_mn ? 128 : 2;
        constexpr uint32_t kHigh = tc::operand_high(1024);
        uint32_t add = 0;
        for (int kb = u.k0; kb < u.k1; ++kb) {
          if (!(ok = tc::bar_wait(full + stage * 8, phase, a.wait_limit_ns, stop))) break;
          tc::fence_after();
          uint32_t al = a0 + stage * (stage_size / 16), bl = b0 + stage * (stage_size / 16);
#pragma unroll
          for (int k = 0; k < kTileK / 16; ++k) {
            tc::mma<CG>(d, al, kHigh, bl, kHigh, idesc, add);
            al += a_step, bl += b_step, add = 1;
          }
          issued = true;
          tc::mma_commit<CG>(empty + stage * 8);
          if (++stage == stage_count) stage = 0, phase ^= 1u;
        }
        if (!ok) break;
        tc::mma_commit<CG>(tc::smem(&sh.tmem_full[acc]));
        if (++acc == kAccumulators) acc = 0, acc_phase ^= 1u;
      }
      // After a wait that gave up: products in flight end before TMEM is freed.
      if (!ok && issued) {
        uint32_t never = 0;
        tc::mma_commit<CG>(tc::smem(&sh.drain));
        tc::bar_wait(tc::smem(&sh.drain), 0, a.wait_limit_ns, &never);
      }
    }
  } else {
    // ---- epilogue ------------------------------------------------------------
    const int quarter = warp & 3;          // the lanes of TMEM that this warp may read
    const int side = (warp - 2) / 4;       // and its part of the columns, of `sides`
    constexpr int sides = kEpilogueWarps / 4;
    float *const turn = reinterpret_cast<float *>(dynamic + kDynamic - kEpilogueWarps * kTurnBytes) +
                        (warp - 2) * (kTurnBytes / 4);
    uint32_t acc = 0, acc_phase = 0;
    for (Walk<MODE> walk(a, worker, workers); walk.more(); walk.next()) {
      const Unit u = unit_at<MODE>(a, walk.i);
      if (!(ok = tc::bar_wait(tc::smem(&sh.tmem_full[acc]), acc_phase, a.wait_limit_ns, stop))) break;
      tc::fence_after();
      const uint32_t from = tmem + acc * kTileN + ((uint32_t)quarter * 32u << 16);
      // This warp has read its part of the accumulator: the next tile may overwrite it
      // while this one's results are still being worked out and stored.
      auto drained = [&] {
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::bar_arrive_relaxed(tc::at_rank(tc::smem(&sh.tmem_empty[acc]), 0));
      };
      const bool some = u.k1 > u.k0;  // an empty part of a K loop: the sum is 0
      if constexpr (MODE == FORWARD || MODE == RECOMPUTE) {
        const int64_t row = ((int64_t)u.m * CG + rank) * kTileM + quarter * 32 + lane;
        const int half = a.tile_n / 2, runs = half / 32;
        const int begin = side * runs / sides, end = (side + 1) * runs / sides;
        uint32_t held = 0;
        if (begin == end) drained();
#pragma unroll 1
        for (int c = begin; c < end; ++c) {
          const int64_t col = (int64_t)u.n * half + c * 32;
          uint32_t g[32], up[32];
          __syncwarp();
          tc::tmem_load32(from + c * 32, g);
          tc::tmem_load32(from + half + c * 32, up);
          tc::tmem_load_wait();
          if (c + 1 == end) drained();
          const int64_t rows = a.m[0] - (row - lane);
          if (rows > 0 && col < a.n)
            gated_part<MODE, ACT, KEEP>(a, g, up, {col, (int)min((int64_t)32, a.n - col), (int)min((int64_t)32, rows), row, turn},
                                        c + 1 < end && col + 32 < a.n, held);
        }
      } else {
        const int which = u.which, up = which == 0 && u.m >= a.half[0] ? 1 : 0, to = which == 1 ? 2 : up;
        const int64_t row = ((int64_t)(u.m - up * a.half[0]) * CG + rank) * kTileM + quarter * 32 + lane, m = a.m[which];
        constexpr int runs = COLS / 32;
        const int begin = side * runs / sides, end = (side + 1) * runs / sides;
        if (begin == end) drained();
#pragma unroll 1
        for (int c = begin; c < end; ++c) {
          const int64_t col = (int64_t)u.n * COLS + c * 32;
          uint32_t r[32];
          __syncwarp();
          tc::tmem_load32(from + c * 32, r);
          tc::tmem_load_wait();
          if (c + 1 == end) drained();
          const int64_t rows = m - (row - lane);
          if (rows > 0 && col < a.n) {
            const Part q = {col, (int)min((int64_t)32, a.n - col), (int)min((int64_t)32, rows), row, turn};
            if (!some) {
#pragma unroll
              for (int e = 0; e < 32; ++e) r[e] = 0u;
            }
            if (u.part >= 0) {
              const Part in = {c * 32, 32, q.rows, rank * kTileM + quarter * 32 + lane, turn};
              store_part(a.partial[which] + (int64_t)u.part * (kTileM * CG * COLS), COLS, false, a.partial_width, r, in);
            } else {
              store_part(a.out[to], a.ld_out[to], a.out_bf16[which] != 0, a.out_width[which], r, q);
            }
          }
        }
      }
      if (++acc == kAccumulators) acc = 0, acc_phase ^= 1u;
    }
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && sh.stop) {
    atomicAdd(a.gave_up, 1u);
    land_copies(sh, a, stage_count, rank, skips_first(a, worker));
  }
  __syncthreads();
  if constexpr (CG == 2) tc::cluster_sync();
  tc::fence_after();
  if (warp == 1) tc::tmem_free<CG>(tmem, kTmemColumns);
}

template <int MODE, int CG, int ACT, int KEEP, int COLS>
cudaError_t launch(Args &a, int sms, cudaStream_t stream) {
  const void *fn = reinterpret_cast<const void *>(&product_kernel<MODE, CG, ACT, KEEP, COLS>);
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kDynamic);
  if (e != cudaSuccess) return e;
  int64_t units = 0;
  for (int w = 0; w < (MODE == BACKWARD ? 2 : 1); ++w) units += units_of(a.grid[w]);
  int64_t workers = sms / CG;
  if (workers > units) workers = units;
  // Rows through the warps' buffers: those that no vector fits, and a row's last columns.
  auto odd = [](int width) { return width < 16; };
  if (MODE == BACKWARD) {
    a.turns = 0;
    for (int w = 0; w < 2; ++w) a.turns |= a.grid[w].whole > 0 && (a.n % 32 != 0 || odd(a.out_width[w]));
  } else {
    a.turns = a.n % 32 != 0 || odd(a.out_width[0]) || (MODE == FORWARD && KEEP == 2 && odd(a.keep_width)) || (MODE == RECOMPUTE && !a.dh_vec);
  }
  void *args[] = {&a};
  return launch_kernel(fn, dim3((unsigned)(workers * CG)), dim3(kThreads), args, kDynamic, stream, true, CG);
}

// FORWARD and RECOMPUTE, by activation and by what is kept.
template <int MODE, int CG, int ACT>
cudaError_t launch_gated(Args &a, int sms, cudaStream_t stream) {
  if constexpr (MODE == FORWARD) {
    if (a.keep == 1) return launch<MODE, CG, ACT, 1, 0>(a, sms, stream);
    if (a.keep == 2) return launch<MODE, CG, ACT, 2, 0>(a, sms, stream);
  }
  return launch<MODE, CG, ACT, 0, 0>(a, sms, stream);
}
template <int MODE>
cudaError_t launch_gated(bool pair, Args &a, int sms, cudaStream_t stream) {
  if (a.act == SILU) return pair ? launch_gated<MODE, 2, SILU>(a, sms, stream) : launch_gated<MODE, 1, SILU>(a, sms, stream);
  return pair ? launch_gated<MODE, 2, GELU>(a, sms, stream) : launch_gated<MODE, 1, GELU>(a, sms, stream);
}

// BACKWARD, by the tile's columns.
inline cudaError_t launch_columns(bool pair, Args &a, int sms, cudaStream_t stream) {
  if (pair)
    return a.tile_n == 256 ? launch<BACKWARD, 2, SILU, 0, 256>(a, sms, stream) : launch<BACKWARD, 2, SILU, 0, 128>(a, sms, stream);
  if (a.tile_n == 256) return launch<BACKWARD, 1, SILU, 0, 256>(a, sms, stream);
  return a.tile_n == 128 ? launch<BACKWARD, 1, SILU, 0, 128>(a, sms, stream) : launch<BACKWARD, 1, SILU, 0, 64>(a, sms, stream);
}

}  // namespace

}  // namespace ffn
}  // namespace fsdp

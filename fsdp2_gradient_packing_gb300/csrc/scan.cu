// Gated linear recurrence (fsdp_gated_scan_*): a = sigmoid(gate + bias),
// h_t = a_t h_(t-1) + (1 - a_t) x_t, forward and backward.
//
// Rows are cut into tiles of 128 (BF16) or 64 rows and 64 columns, whatever sequences they belong to;
// where one begins, the state before it is its own initial one.  A thread has two columns and
// 16 or 8 rows.  Its rows take a state h to A h + B; so do a warp's, one behind the other, and a
// tile's.  A tile makes its A and B known, then looks back over the tiles before it for the
// nearest one whose state behind its last row is known, and comes from there to its own start by
// the A and B in between.  So every matrix is read and written once and long sequences keep all
// SMs busy.  Tiles are handed out in the order of their rows, so what a tile waits for has begun;
// a wait is bounded.  Whatever a tile finds known when it looks back, the state at its start is the
// same chain of A h + B from the sequence's start, so results are the same bits on every run.
//
// Measured in BF16: 65536 x 1024 in one sequence 110 us forward (403 MB at 3.7 TB/s) and 185 backward (671 MB at 3.6); 32768 x
// 4096 in four 169 us (806 MB at 4.8 TB/s) and 321 (1342 MB at 4.2). A copy without the look back took 74 us for 107 at 32768 x 2048.
//
// What bounds it is the time from a tile's rows to its carry, so that is kept short: the next
// tile's rows are on their way into shared memory meanwhile (cp.async, two stages), and the values
// that tiles leave for one another are their own flags (all ones: not there yet), which costs no
// fence and one trip to L2 instead of two.
//
// Backward the same goes from the last row to the first, with a_t D_t in place of the state.
// The states are made again from those that the forward pass keeps every kStateRows rows:
// 4 bytes a column instead of a read of h, and in binary32.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <string>

#include "layout.h"
#include "ops.h"
#include "tc.h"

namespace fsdp {
namespace scan {
namespace {

constexpr int kCols = 64, kWarps = 8, kThreads = kWarps * 32;
constexpr int kStateRows = 64;
constexpr int kWindow = 2 * kWarps;  // tiles that a look back takes in at once, at most
// Rows of a warp.  What a tile costs a warp beside its rows is about 400 instructions, 30 to 60 a row: 1 x 65536 x 1024 in
// BF16 with 16 rows 121 us, with 8 197.  Of FP32 rows, two stages and two blocks of an SM hold 64.
constexpr int steps_of(int64_t size) { return size == 4 ? 8 : 16; }

struct Args {
  const void *x, *gate, *bias, *offsets, *dh;
  const float *initial, *dfinal, *states_in;
  void *h, *dx, *dgate;
  float *final_state, *dinitial, *states, *partial;
  uint2 *parts;        // [time tiles][padded columns]: A and B
  uint32_t *carried;   // [time tiles][padded columns]: the state behind the tile
  uint32_t *ticket;
  int32_t *begins, *ends;  // packed: the sequence that begins or ends at a row, or -1
  uint32_t *gave_up;
  uint64_t wait_limit_ns;
  int64_t rows, cols, seqs, seq_len, ld_x, ld_gate, ld_h, ld_dx, ld_dgate;
  int64_t padded_cols;  // whole column tiles
  uint32_t column_tiles, time_tiles, tiles;
  int32_t packed, wide, h_bf16, dx_bf16, param_bf16, fault;
  int32_t window;  // tiles that a look back takes in at once
  uint32_t aside;  // sequences that go side by side
};

__device__ __forceinline__ int64_t offset_at(const Args &a, int64_t s) {
  const int64_t o = a.wide ? static_cast<const int64_t *>(a.offsets)[s] : static_cast<const int32_t *>(a.offsets)[s];
  return min(max(o, (int64_t)0), a.rows);
}

// A gate is held as its odds o = (1 - a) / a = e^-z, from which a = 1 / (1 + o) and 1 - a = o a both come to a few ulp of their own
// sizes; one made from the other would lose the bits of the lesser.
__device__ __forceinline__ float2 ex2(float2 t) {
  float2 e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
  return e;
}
__device__ __forceinline__ float2 odds(float2 z) { return ex2(__fmul2_rn(z, both(-1.4426950408889634f))); }
__device__ __forceinline__ float2 gate_of(float2 o) {
  const float2 d = __fadd2_rn(o, both(1.0f));
  float2 a;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(a.x) : "f"(d.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(a.y) : "f"(d.y));
  return a;
}
// Of any odds, up to infinity, whose product with an a of 0 would be a NaN: held to 2^125, which stand for a gate that is shut.
// 1 - a is then 1, and a, less 2^-125, 0.  A NaN stays one.
__device__ __forceinline__ float2 held_odds(float2 z) {
  float2 t = __fmul2_rn(z, both(-1.4426950408889634f));
  asm("min.NaN.f32 %0, %0, 0f42FA0000;" : "+f"(t.x));
  asm("min.NaN.f32 %0, %0, 0f42FA0000;" : "+f"(t.y));
  return ex2(t);
}
__device__ __forceinline__ void gates(float2 o, float2 &a, float2 &keep) {
  a = gate_of(o), keep = __fmul2_rn(o, a);
  a = __fadd2_rn(a, both(-0x1p-125f));
}
// How a warp goes over its rows.  SHORT: inside one sequence, taking h to a (h + o x), which is right for odds of up to 2^100.  A row
// beyond makes K, of which kMuch times as much is held, infinite or a NaN, and so do o x beyond all bounds the state; the warp then
// takes its rows once more as HELD, with odds that are held and an h that is multiplied by a before anything is added to it.  The
// later passes go so, too, where a state beyond 2^100 comes in.  MARKED: as HELD, with borders of sequences.  (us in BF16, 32768 x 4096,
// forward and backward: 169 and 321, HELD alone 176 and 317; with a gate that is shut every 512 rows 174 and 321, every 16 rows, so
// that every warp meets one, 216 and 370.)
enum Path { SHORT, HELD, MARKED };
constexpr float kMuch = 0x1p28f;

// How a tile comes and goes.  DIRECT: each value by its own load and store, of any types, a lane's columns 32 apart (backward, where dh
// is of another type than x).  ANY: x, gate and dh, of one type, staged wherever rows begin, otherwise as DIRECT.  UNITS: all matrices of one
// type, staged by 16 bytes, a lane's columns neighbours, results stored in pairs.
enum Way { DIRECT, ANY, UNITS };

template <Way WAY>
__device__ __forceinline__ void put(void *p, bool bf16, bool second, float2 v) {
  if constexpr (WAY == UNITS) {
    if (bf16)
      *static_cast<uint32_t *>(p) = bf16_pair(v.x, v.y);
    else
      *static_cast<float2 *>(p) = v;
  } else {
    store_any(p, 0, bf16, v.x);
    if (second) store_any(p, 32, bf16, v.y);
  }
}
// Two columns of a matrix of binary32 values that is aligned to nothing more.
template <Way WAY>
__device__ __forceinline__ float2 get_f32(const float *p, bool second) {
  return make_float2(p[0], second ? p[WAY == UNITS ? 1 : 32] : 0.0f);
}
template <Way WAY>
__device__ __forceinline__ void put_f32(float *p, bool second, float2 v) {
  p[0] = v.x;
  if (second) p[WAY == UNITS ? 1 : 32] = v.y;
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

// One tensor's rows of a tile on their way into shared memory: rows of kCols elements, 16-byte
// units, zeros outside the matrix.
template <int ROWS, int SIZE>
__device__ __forceinline__ void fetch(uint8_t *to, const void *from, int64_t ld, int64_t first, int64_t column, const Args &a) {
  constexpr int kUnits = kCols * SIZE / 16, kStep = kThreads / kUnits;  // 16-byte units of a row; rows of a round
  const int r = threadIdx.x / kUnits, u = threadIdx.x % kUnits;
  const int64_t j = column + u * (16 / SIZE);
  const bool in = j < a.cols;
  const int64_t left = a.rows - first - r;
  const uint8_t *src = static_cast<const uint8_t *>(from) + (in ? ((first + r) * ld + j) * SIZE : 0);
  const int64_t pitch = ld * SIZE * kStep;
  const uint32_t dst = tc::smem(to) + threadIdx.x * 16;
#pragma unroll
  for (int k = 0; k < ROWS / kStep; ++k) {
    const bool there = in && k * kStep < left;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + k * (kThreads * 16)), "l"(there ? src : static_cast<const uint8_t *>(from)),
                 "r"(there ? 16 : 0)
                 : "memory");
    src += pitch;
  }
}

// The same whatever the rows' alignment: the units of GRAIN bytes that a row's 64 columns lie in, which begin up to a unit before
// them.  A warp takes the rows that it works on.
constexpr int row_units(int size, int grain) { return (kCols * size + 2 * grain - size - 1) / grain; }
template <int STEPS, int SIZE, int GRAIN>
__device__ __forceinline__ void fetch_any(uint8_t *to, const void *from, int64_t ld, int64_t tile_first, int64_t column, const Args &a) {
  constexpr int kUnits = row_units(SIZE, GRAIN);
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int64_t first = tile_first + warp * STEPS, cols = a.cols - column;
  const int rows = (int)min((int64_t)STEPS, a.rows - first);
  const uintptr_t base = (uintptr_t)from + column * SIZE;
  const uint32_t dst = tc::smem(to) + warp * (STEPS * kUnits * GRAIN);
#pragma unroll 4
  for (int u = lane; u < STEPS * kUnits; u += 32) {
    const int r = u / kUnits, k = u - r * kUnits;
    const uintptr_t p = base + (r < rows ? (first + r) * ld * SIZE : 0);
    const int phase = (int)(p & (GRAIN - 1)) / SIZE;  // elements of the first unit that lie before the columns
    const bool there = r < rows && k * (GRAIN / SIZE) - phase < cols;
    const uintptr_t at = (p & ~(uintptr_t)(GRAIN - 1)) + (there ? k * GRAIN : 0);
    if constexpr (GRAIN == 16)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + u * 16), "l"(at), "r"(there ? 16 : 0) : "memory");
    else
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst + u * 4), "l"(at), "r"(there ? 4 : 0) : "memory");
  }
}

// Where a tile is, found by one thread: its time tile and first column; and without packing, the sequence
// of its first row, that row's place in it, and whether all its rows lie inside that sequence.
struct Spot {
  int64_t tile, left;
  uint32_t reach;  // tiles before it (behind it, backward) that a look back may wait for: those that come earlier in the order
  int32_t sequence;
  uint32_t place;
  bool inside;
};
template <int ROWS>
__device__ __forceinline__ Spot spot_of(const Args &a, uint32_t ticket, bool backward) {
  Spot p = {};
  const uint32_t q = ticket / a.column_tiles;
  uint32_t tile = q;
  p.reach = q;
  if (a.aside > 1) {  // sequences side by side: the same tile of each, then the next
    const uint32_t k = q / a.aside;
    tile = (q - k * a.aside) * (a.time_tiles / a.aside) + k;
    p.reach = k;
  }
  p.tile = backward ? a.time_tiles - 1 - tile : tile;
  p.left = (int64_t)(ticket - q * a.column_tiles) * kCols;
  if (!a.packed) {
    const uint32_t t = (uint32_t)p.tile * ROWS, n = (uint32_t)a.seq_len;
    p.sequence = t / n, p.place = t - p.sequence * n;
    p.inside = p.place > 0 && p.place + ROWS < n;
  }
  return p;
}

struct Warps {
  float2 a[kWarps][32], b[kWarps][32];
  uint32_t cut[kWarps], found[kWindow];
};
template <bool BACKWARD, Way WAY>
struct Shared {
  Warps warps;
  uint32_t ticket[2];  // of the next tile, by turns: one may still be read while the next one is written
  Spot spot[2];
  float2 forward[BACKWARD ? kWarps : 0][32];  // backward pass: B of the states
  uint4 look[WAY == DIRECT ? kWindow : 0][32];          // what other tiles have left: A and B, or the state
  uint32_t stop;
};
// Bits of `cut`: nothing passes a warp's rows downwards, or upwards; a sequence begins at their
// first row; one ends at their last.
enum Cut : uint32_t { CUT_DOWN = 1, CUT_UP = 2, CUT_FIRST = 4, CUT_LAST = 8 };

// This lane's columns and this warp's rows.
template <int STEPS, Way WAY>
struct Place {
  int64_t tile, column, first;  // time tile; first column of the lane; first row of the warp
  uint32_t reach;
  int64_t at0;                  // of the lane among the values that tiles leave
  bool in, second;              // whether the lane's columns exist
  __device__ __forceinline__ Place(const Args &a, const Spot &p) {
    const int lane = threadIdx.x & 31;
    tile = p.tile, reach = p.reach;
    column = p.left + (WAY == UNITS ? 2 * lane : lane);
    at0 = p.left + 2 * lane;
    first = tile * (kWarps * STEPS) + threadIdx.x / 32 * STEPS;
    in = column < a.cols, second = column + (WAY == UNITS ? 1 : 32) < a.cols;
  }
};

// Boundaries in a warp's rows: bit i for row first + i; lane i has the sequence.
template <int STEPS>
struct Marks {
  int32_t begin, end;
  uint32_t begins, ends, valid;
  __device__ __forceinline__ Marks(const Args &a, const Spot &p, int64_t first, int64_t lo, int64_t hi) {
    begin = end = -1, begins = ends = 0, valid = (1u << STEPS) - 1;
    if (p.inside) return;
    const int lane = threadIdx.x & 31;
    const int64_t t = first + lane;
    if (a.packed) {
      const bool there = lane < STEPS && t < a.rows;
      if (there) begin = a.begins[t], end = a.ends[t];
      begins = __ballot_sync(0xFFFFFFFFu, begin >= 0), ends = __ballot_sync(0xFFFFFFFFu, end >= 0);
    } else {  // one ends where the next one begins
      const uint32_t n = (uint32_t)a.seq_len, u = p.place + threadIdx.x / 32 * STEPS + lane, q = u / n;
      begin = end = p.sequence + (int32_t)q;
      const uint32_t on = __ballot_sync(0xFFFFFFFFu, lane <= STEPS && t <= a.rows && q * n == u);
      begins = on & __ballot_sync(0xFFFFFFFFu, lane < STEPS && t < a.rows), ends = on >> 1;
    }
    valid = __ballot_sync(0xFFFFFFFFu, lane < STEPS && t >= lo && t < hi);
  }
  // Rows that are not in the middle of a sequence.
  __device__ __forceinline__ uint32_t odd() const { return (begins | ends | ~valid) & ((1u << STEPS) - 1); }
  __device__ __forceinline__ uint32_t cut() const {
    return (begins ? CUT_DOWN : 0u) | (begins | ends ? CUT_UP : 0u) | (begins & 1 ? CUT_FIRST : 0u) | (ends >> (STEPS - 1) & 1 ? CUT_LAST : 0u);
  }
};

// Values that tiles leave for others.  All ones means not there yet; the NaN of that pattern
// is left as another one.
__device__ __forceinline__ uint32_t as_left(float v) {
  const uint32_t u = __float_as_uint(v);
  return u == 0xFFFFFFFFu ? 0x7FFFFFFFu : u;
}
__device__ __forceinline__ void leave_part(const Args &a, int64_t at, float2 A, float2 B) {
  asm volatile("st.relaxed.gpu.global.v2.b64 [%0], {%1, %2};" ::"l"(a.parts + at),
               "l"((uint64_t)as_left(B.x) << 32 | as_left(A.x)), "l"((uint64_t)as_left(B.y) << 32 | as_left(A.y))
               : "memory");
}
__device__ __forceinline__ void leave_state(const Args &a, int64_t at, float2 s) {
  asm volatile("st.relaxed.gpu.global.v2.b32 [%0], {%1, %2};" ::"l"(a.carried + at), "r"(as_left(s.x)), "r"(as_left(s.y)) : "memory");
}

// Whether a warp has waited for longer than it may, since it first asked.
__device__ __forceinline__ bool too_late(const Args &a, uint64_t &began) {
  const uint64_t now = __shfl_sync(0xFFFFFFFFu, tc::now_ns(), 0);
  if (began == 0) began = now;
  return now - began > a.wait_limit_ns;
}

// All warps: the state that comes into a tile from `towards` (-1: the tiles before it, 1: those
// behind).  A warp reads what one or two of the nearest tiles have left.
__device__ __forceinline__ float2 look_back(const Args &a, Warps &s, uint32_t &stop, uint4 *look, int64_t tile, uint32_t reach, int towards, int64_t at0) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  uint64_t began = 0;
  bool late = false;
  for (;;) {
    for (int slot = warp; slot < a.window; slot += kWarps) {
      const int64_t other = tile + (int64_t)towards * (1 + slot);
      const bool exists = (uint32_t)slot < reach;
      const int64_t at = other * a.padded_cols + at0;
      uint32_t found = 0;  // 1: A and B, 2: the state
      uint64_t p0 = 0, p1 = 0;
      uint32_t c0 = 0, c1 = 0;
      for (uint32_t n = 1; exists; ++n) {
        asm volatile("ld.relaxed.gpu.global.v2.b64 {%0, %1}, [%2];" : "=l"(p0), "=l"(p1) : "l"(a.parts + at) : "memory");
        asm volatile("ld.relaxed.gpu.global.v2.b32 {%0, %1}, [%2];" : "=r"(c0), "=r"(c1) : "l"(a.carried + at) : "memory");
        const bool state = c0 != 0xFFFFFFFFu && c1 != 0xFFFFFFFFu;
        const bool part = (uint32_t)p0 != 0xFFFFFFFFu && (uint32_t)p1 != 0xFFFFFFFFu && p0 >> 32 != 0xFFFFFFFFu && p1 >> 32 != 0xFFFFFFFFu;
        found = __all_sync(0xFFFFFFFFu, state) ? 2 : __all_sync(0xFFFFFFFFu, part) ? 1 : 0;
        if (found) break;
        if ((n & 15u) == 0 && (late = too_late(a, began))) break;
      }
      look[slot * 32 + lane] = found == 2 ? make_uint4(c0, 0, c1, 0) : make_uint4((uint32_t)p0, (uint32_t)(p0 >> 32), (uint32_t)p1, (uint32_t)(p1 >> 32));
      if (lane == 0) s.found[slot] = found;
    }
    if (late) stop = 1;  // before the barrier: all threads see the same
    __syncthreads();
    const uint32_t states = __ballot_sync(0xFFFFFFFFu, lane < a.window && s.found[lane % kWindow] == 2);
    float2 carry = make_float2(0, 0);
    if (*(volatile uint32_t *)&stop) return carry;
    if (states) {
      const int back = __ffs(states) - 1;
      const uint4 r = look[back * 32 + lane];
      carry = make_float2(__uint_as_float(r.x), __uint_as_float(r.z));
#pragma unroll 4
      for (int w = back - 1; w >= 0; --w) {
        const uint4 q = look[w * 32 + lane];
        carry = fma2(make_float2(__uint_as_float(q.x), __uint_as_float(q.z)), carry, make_float2(__uint_as_float(q.y), __uint_as_float(q.w)));
      }
      return carry;
    }
    __syncthreads();  // none of them knows its state yet
    late = too_late(a, began);
  }
}

// A tile's A and B (from its first warp to its last, or backward the other way), left for other tiles by
// warp 0, which keeps them.
struct Whole {
  float2 A, B;
  bool cut, alone, last;  // nothing passes; nothing comes in; nothing goes out
};
template <bool BACKWARD>
__device__ __forceinline__ Whole leave(const Args &a, const Warps &s, int64_t tile, int64_t at0) {
  constexpr uint32_t kBit = BACKWARD ? CUT_UP : CUT_DOWN;
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  Whole t = {both(1.0f), both(0.0f), false, true, true};
  if (a.time_tiles > 1) {
    t.alone = BACKWARD ? tile == a.time_tiles - 1 || (s.cut[kWarps - 1] & CUT_LAST) : tile == 0 || (s.cut[0] & CUT_FIRST);
    t.last = tile == (BACKWARD ? 0 : a.time_tiles - 1);
    if (warp == 0 && !t.last) {
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const int w = BACKWARD ? kWarps - 1 - k : k;
        const bool c = s.cut[w] & kBit;
        t.A = __fmul2_rn(t.A, s.a[w][lane]);
        t.B = c ? s.b[w][lane] : fma2(s.a[w][lane], t.B, s.b[w][lane]);
        t.cut |= c;
      }
      const int64_t at = tile * a.padded_cols + at0;
      if (!t.cut && !t.alone)
        leave_part(a, at, t.A, t.B);
      else if (!(a.fault & 1) || tile != (BACKWARD ? a.time_tiles - 1 : 0))  // the test hook leaves out the first
        leave_state(a, at, t.B);
    }
  }
  return t;
}
// The state that comes into the tile.
template <bool BACKWARD>
__device__ __forceinline__ float2 take(const Args &a, Warps &s, uint32_t &stop, uint4 *look, const Whole &t, int64_t tile, uint32_t reach, int64_t at0) {
  if (t.alone) return both(0.0f);
  const float2 carry = look_back(a, s, stop, look, tile, reach, BACKWARD ? 1 : -1, at0);
  if (threadIdx.x < 32 && !t.last && !t.cut) leave_state(a, tile * a.padded_cols + at0, fma2(t.A, carry, t.B));
  return carry;
}

template <class T, Way WAY, bool BACKWARD>
struct Tile {
  static constexpr int kSteps = steps_of(sizeof(T)), kRows = kWarps * kSteps, kSize = (int)sizeof(T);
  using At = Place<kSteps, WAY>;
  using Block = Shared<BACKWARD, WAY>;
  static constexpr bool kBf16 = kSize == 2;
  // Bytes of a row of x or gate in a stage.  The three BF16 matrices of a backward tile leave no room for rows' first and
  // last units of 16 bytes, only of 4.
  static constexpr int kGrain = BACKWARD && kBf16 ? 4 : 16;
  static constexpr int kPitch = WAY == ANY ? row_units(kSize, kGrain) * kGrain : kCols * kSize;
  static constexpr int kMatrix = kRows * kPitch;
  static constexpr int kStage = WAY == DIRECT ? 0 : (BACKWARD ? 3 : 2) * kMatrix;
  static constexpr int kSmem = 2 * kStage;
  static constexpr int kBlocks = BACKWARD || (WAY == ANY && kBf16) ? 2 : 3;  // of an SM
  // Where all matrices have x's type, that of the results is known.
  __device__ __forceinline__ static bool out_bf16(int32_t bf16) { return WAY == UNITS ? kBf16 : bf16 != 0; }
  __device__ __forceinline__ static int64_t out_size(int32_t bf16) { return out_bf16(bf16) ? 2 : 4; }

  __device__ __forceinline__ static void fetch_matrix(uint8_t *to, const void *from, int64_t ld, const Spot &p, const Args &a) {
    if constexpr (WAY == UNITS)
      fetch<kRows, kSize>(to, from, ld, p.tile * kRows, p.left, a);
    else
      fetch_any<kSteps, kSize, kGrain>(to, from, ld, p.tile * kRows, p.left, a);
  }
  __device__ __forceinline__ static void start(const Args &a, uint8_t *stage, uint32_t ticket, const Spot &p) {
    if constexpr (WAY != DIRECT) {
      if (ticket < a.tiles) {
        fetch_matrix(stage, a.x, a.ld_x, p, a);
        fetch_matrix(stage + kMatrix, a.gate, a.ld_gate, p, a);
        if constexpr (BACKWARD) fetch_matrix(stage + 2 * kMatrix, a.dh, a.ld_h, p, a);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  }
  // Once a tile's gates have been computed, their place holds what other tiles have left.
  static_assert(WAY == DIRECT || kMatrix >= kWindow * 32 * 16, "no room to look back");
  __device__ __forceinline__ static uint4 *look_at(Block &all, uint8_t *stage) {
    if constexpr (WAY != DIRECT)
      return reinterpret_cast<uint4 *>(stage + kMatrix);
    else
      return &all.look[0][0];
  }
  // Row i of the warp's in x, gate or dh (m 0, 1, 2).
  __device__ __forceinline__ static float2 row(const Args &a, const uint8_t *stage, const At &at, int m, int i) {
    const int lane = threadIdx.x & 31;
    const void *p = m == 0 ? a.x : m == 1 ? a.gate : a.dh;
    const int64_t ld = m == 0 ? a.ld_x : m == 1 ? a.ld_gate : a.ld_h;
    if constexpr (WAY == DIRECT) {
      const bool bf16 = m == 2 ? a.h_bf16 != 0 : kBf16;
      const int64_t t = at.first + i, k = t * ld + at.column;
      if (!at.in || t >= a.rows) return both(0.0f);
      return make_float2(load_any(p, k, bf16), at.second ? load_any(p, k + 32, bf16) : 0.0f);
    } else {
      const uint8_t *r = stage + m * kMatrix + (threadIdx.x / 32 * kSteps + i) * kPitch;
      if constexpr (WAY == ANY) {
        const uint32_t first = (uint32_t)(uintptr_t)p / kSize + (uint32_t)(at.first + i) * (uint32_t)ld + (uint32_t)(at.column - lane);
        const T *q = reinterpret_cast<const T *>(r) + lane + first % (kGrain / kSize);
        return make_float2((float)q[0], (float)q[32]);
      } else if constexpr (kBf16) {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(r + lane * 4);
        return make_float2(bf16_low(w), bf16_high(w));
      } else {
        return *reinterpret_cast<const float2 *>(r + lane * 8);
      }
    }
  }
  __device__ static float2 bias(const Args &a, const At &at) {
    if (!a.bias || !at.in) return make_float2(0, 0);
    return make_float2(load_any(a.bias, at.column, a.param_bf16),
                       at.second ? load_any(a.bias, at.column + (WAY == UNITS ? 1 : 32), a.param_bf16) : 0.0f);
  }
  // A lane's columns of row s of `initial` or `dfinal`.
  __device__ __forceinline__ static float2 given(const Args &a, const float *p, int32_t s, const At &at) {
    return p && at.in ? get_f32<WAY>(p + (int64_t)s * a.cols + at.column, at.second) : both(0.0f);
  }
  // Whether a warp's rows went well as SHORT, from what they amount to (staged by units, columns that do not exist are 0).  If not,
  // the gates are read once more, from where a barrier lets no register keep them (without it 193 us for 169).
  __device__ __forceinline__ static bool went_well(float2 B, float2 K, const At &at) {
    bool well = fabsf(B.x) + fabsf(B.y) + (K.x + K.y) < INFINITY;
    if constexpr (WAY != UNITS) well = !at.in || (at.second ? well : fabsf(B.x) + K.x < INFINITY);
    well = __all_sync(0xFFFFFFFFu, well);
    if (!well) __syncwarp();
    return well;
  }
  __device__ __forceinline__ static Path second_path(Path path, float2 h) {
    return path == SHORT && __any_sync(0xFFFFFFFFu, fmaxf(fabsf(h.x), fabsf(h.y)) > 0x1p100f) ? HELD : path;
  }
  // A row's state.
  template <Path PATH>
  __device__ __forceinline__ static float2 state_step(float2 x, float2 o, float2 h) {
    if constexpr (PATH == SHORT) return __fmul2_rn(gate_of(o), fma2(o, x, h));
    float2 f, keep;
    gates(o, f, keep);
    return fma2(f, h, __fmul2_rn(keep, x));
  }
  // One row of the second and of the third pass over a backward tile.
  template <Path PATH>
  __device__ __forceinline__ static void slope_step(float2 x, float2 o, float2 &h, float2 &slope) {
    float2 f, keep;
    if constexpr (PATH == SHORT) {
      f = gate_of(o), keep = __fmul2_rn(o, f);
      slope = __fmul2_rn(fma2(x, both(-1.0f), h), __fmul2_rn(f, keep));
      h = __fmul2_rn(f, fma2(o, x, h));
    } else {  // the difference may be beyond all bounds where a quarter of it, which a (1 - a) is at most, is not
      gates(o, f, keep);
      slope = __fmul2_rn(fma2(x, both(-0.25f), __fmul2_rn(h, both(0.25f))), __fmul2_rn(__fmul2_rn(f, both(4.0f)), keep));
      h = fma2(f, h, __fmul2_rn(keep, x));
    }
  }
  template <Path PATH>
  __device__ __forceinline__ static float2 gradient_step(const Args &a, float2 dh, float2 o, float2 slope, const At &at, void *dx,
                                                         void *dgate, float2 &e) {
    float2 f, keep;
    if constexpr (PATH == SHORT)
      f = gate_of(o), keep = __fmul2_rn(o, f);
    else
      gates(o, f, keep);
    const float2 d = __fadd2_rn(dh, e), dz = __fmul2_rn(d, slope);
    if (at.in) {
      put<WAY>(dx, out_bf16(a.dx_bf16), at.second, __fmul2_rn(keep, d));
      put<WAY>(dgate, out_bf16(a.dx_bf16), at.second, dz);
    }
    e = __fmul2_rn(f, d);
    return dz;
  }
  // One tile, from its stage; starts the next one's loads into the other stage, and gives its ticket and its place.
  __device__ static uint32_t forward(const Args &a, Block &all, int turn, uint8_t *stage, uint8_t *other, Spot &p, int64_t lo, int64_t hi);
  __device__ static uint32_t backward(const Args &a, Block &all, int turn, uint8_t *stage, uint8_t *other, Spot &p, int64_t lo, int64_t hi);
};

// A warp's A: 1 - K, where K is the recurrence's answer to inputs of 1, or the rows' product where that is
// the smaller: near 1, as a slow column's is, a product of rounded factors would lose a rounding a row.
__device__ __forceinline__ float2 factor(float2 product, float2 K) {
  return make_float2(K.x < 0.5f ? 1.0f - K.x : product.x, K.y < 0.5f ? 1.0f - K.y : product.y);
}

template <class T, Way WAY, bool BACKWARD>
__device__ __forceinline__ uint32_t Tile<T, WAY, BACKWARD>::forward(const Args &a, Block &all, int turn, uint8_t *stage, uint8_t *other,
    Spot &p, int64_t lo, int64_t hi) {
  const At at(a, p);
  Warps &sh = all.warps;
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const float2 shift = bias(a, at);
  const Marks<kSteps> m(a, p, at.first, lo, hi);
  // A row takes h to f h + b.  Only its odds stay in registers, from which both come again: a third block fits the SM.
  float2 o[kSteps], A = both(1.0f), B = both(0.0f), K = both(0.0f);
  Path path = m.odd() == 0 ? SHORT : MARKED;
  if (__builtin_expect(path == SHORT, 1)) {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      o[i] = odds(__fadd2_rn(row(a, stage, at, 1, i), shift));
      const float2 f = gate_of(o[i]);
      A = __fmul2_rn(A, f), B = __fmul2_rn(f, fma2(o[i], row(a, stage, at, 0, i), B)), K = __fmul2_rn(f, fma2(o[i], both(kMuch), K));
    }
    if (__builtin_expect(!went_well(B, K, at), 0)) {
      path = HELD;
      A = both(1.0f), B = K = both(0.0f);
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        float2 f, keep;
        o[i] = held_odds(__fadd2_rn(row(a, stage, at, 1, i), shift));
        gates(o[i], f, keep);
        A = __fmul2_rn(A, f), B = fma2(f, B, __fmul2_rn(keep, row(a, stage, at, 0, i))), K = fma2(f, K, keep);
      }
    } else {
      K = __fmul2_rn(K, both(1.0f / kMuch));
    }
  } else {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      float2 f, keep;
      o[i] = held_odds(__fadd2_rn(row(a, stage, at, 1, i), shift));
      gates(o[i], f, keep);
      float2 b = __fmul2_rn(keep, row(a, stage, at, 0, i));
      if (!(m.valid >> i & 1)) f = both(1.0f), keep = b = both(0.0f);
      if (m.begins >> i & 1) {
        // The row's state itself, kept in place of the odds: `initial` may be `final`, which a later tile may write
        // as soon as this one has left its own state.
        o[i] = B = fma2(f, given(a, a.initial, __shfl_sync(0xFFFFFFFFu, m.begin, i), at), b);
      } else {
        A = __fmul2_rn(A, f), B = fma2(f, B, b), K = fma2(f, K, keep);
      }
    }
  }
  sh.a[warp][lane] = factor(A, K);
  sh.b[warp][lane] = B;
  if (lane == 0) sh.cut[warp] = m.cut();
  __syncthreads();
  const uint32_t next = all.ticket[turn];
  p = all.spot[turn];
  start(a, other, next, p);
  const Whole whole = leave<false>(a, sh, at.tile, at.at0);
  float2 h = take<false>(a, sh, all.stop, look_at(all, stage), whole, at.tile, at.reach, at.at0);
  for (int w = 0; w < warp; ++w) h = sh.cut[w] & CUT_DOWN ? sh.b[w][lane] : fma2(sh.a[w][lane], h, sh.b[w][lane]);
  if (a.states && at.in && at.first % kStateRows == 0 && at.first < a.rows)
    put_f32<WAY>(a.states + at.first / kStateRows * a.cols + at.column, at.second, h);
  path = second_path(path, h);
  const int64_t pitch = a.ld_h * out_size(a.h_bf16);
  uint8_t *out = static_cast<uint8_t *>(a.h) + (at.first * a.ld_h + at.column) * out_size(a.h_bf16);
  auto rows = [&](auto step) {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      h = step(row(a, stage, at, 0, i), o[i], h);
      if (at.in) put<WAY>(out, out_bf16(a.h_bf16), at.second, h);
      out += pitch;
    }
  };
  if (__builtin_expect(path == SHORT, 1)) {
    rows([](float2 x, float2 o, float2 h) { return state_step<SHORT>(x, o, h); });
  } else if (path == HELD) {
    rows([](float2 x, float2 o, float2 h) { return state_step<HELD>(x, o, h); });
  } else {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      if (m.valid >> i & 1) {
        h = m.begins >> i & 1 ? o[i] : state_step<MARKED>(row(a, stage, at, 0, i), o[i], h);
        if (at.in) put<WAY>(out, out_bf16(a.h_bf16), at.second, h);
      }
      out += pitch;
      if (m.ends >> i & 1) {
        const int32_t s = __shfl_sync(0xFFFFFFFFu, m.end, i);
        if (at.in && a.final_state) put_f32<WAY>(a.final_state + (int64_t)s * a.cols + at.column, at.second, h);
      }
    }
  }
  return next;
}

template <class T, Way WAY, bool BACKWARD>
__device__ __forceinline__ uint32_t Tile<T, WAY, BACKWARD>::backward(const Args &a, Block &all, int turn, uint8_t *stage, uint8_t *other,
    Spot &p, int64_t lo, int64_t hi) {
  const At at(a, p);
  Warps &sh = all.warps;
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const float2 shift = bias(a, at);
  const Marks<kSteps> m(a, p, at.first, lo, hi);
  // The state before the warp's rows comes from the nearest kept one above.
  constexpr int kPer = kStateRows / kSteps;  // warps to a kept state
  const int64_t kept = (at.tile * kRows + warp / kPer * kStateRows) / kStateRows;
  float2 h = at.in && kept * kStateRows < a.rows ? get_f32<WAY>(a.states_in + kept * a.cols + at.column, at.second) : both(0.0f);
  // States go A h + B over the warp's rows; e = a_(t+1) D_(t+1) comes in from below and leaves as
  // A e + C.
  float2 A = both(1.0f), B = both(0.0f), C = both(0.0f), K = both(0.0f), o[kSteps], slope[kSteps];
  Path path = m.odd() == 0 ? SHORT : MARKED;
  if (__builtin_expect(path == SHORT, 1)) {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      o[i] = odds(__fadd2_rn(row(a, stage, at, 1, i), shift));
      const float2 f = gate_of(o[i]);
      A = __fmul2_rn(A, f), B = __fmul2_rn(f, fma2(o[i], row(a, stage, at, 0, i), B)), K = __fmul2_rn(f, fma2(o[i], both(kMuch), K));
      C = fma2(A, row(a, stage, at, 2, i), C);
    }
    if (__builtin_expect(!went_well(B, K, at), 0)) {
      path = HELD;
      A = both(1.0f), B = C = K = both(0.0f);
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        float2 f, keep;
        o[i] = held_odds(__fadd2_rn(row(a, stage, at, 1, i), shift));
        gates(o[i], f, keep);
        A = __fmul2_rn(A, f), B = fma2(f, B, __fmul2_rn(keep, row(a, stage, at, 0, i))), K = fma2(f, K, keep);
        C = fma2(A, row(a, stage, at, 2, i), C);
      }
    } else {
      K = __fmul2_rn(K, both(1.0f / kMuch));
    }
  } else {
    bool open = true;  // whether what comes from this row on reaches the warp's first row
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      float2 f, keep, d = row(a, stage, at, 2, i);
      o[i] = held_odds(__fadd2_rn(row(a, stage, at, 1, i), shift));
      gates(o[i], f, keep);
      float2 b = __fmul2_rn(keep, row(a, stage, at, 0, i));
      if (!(m.valid >> i & 1)) f = both(1.0f), keep = b = d = both(0.0f);
      if (m.begins >> i & 1) {
        B = fma2(f, given(a, a.initial, __shfl_sync(0xFFFFFFFFu, m.begin, i), at), b);
        open = false;
      } else {
        B = fma2(f, B, b);
      }
      if (m.ends >> i & 1) d = __fadd2_rn(d, given(a, a.dfinal, __shfl_sync(0xFFFFFFFFu, m.end, i), at));
      A = __fmul2_rn(A, f), K = fma2(f, K, keep);
      if (open) C = fma2(A, d, C);
      if (m.ends >> i & 1) open = false;
    }
  }
  sh.a[warp][lane] = factor(A, K);
  sh.b[warp][lane] = C, all.forward[warp][lane] = B;
  if (lane == 0) sh.cut[warp] = m.cut();
  __syncthreads();
  const uint32_t next = all.ticket[turn];
  p = all.spot[turn];
  start(a, other, next, p);
  const Whole whole = leave<true>(a, sh, at.tile, at.at0);
  // Rows' slopes (h_(t-1) - x_t) a_t (1 - a_t), downwards from the warp's state.
  for (int w = warp / kPer * kPer; w < warp; ++w) h = sh.cut[w] & CUT_DOWN ? all.forward[w][lane] : fma2(sh.a[w][lane], h, all.forward[w][lane]);
  path = second_path(path, h);
  if (__builtin_expect(path == SHORT, 1)) {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) slope_step<SHORT>(row(a, stage, at, 0, i), o[i], h, slope[i]);
  } else if (path == HELD) {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) slope_step<HELD>(row(a, stage, at, 0, i), o[i], h, slope[i]);
  } else {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      if (m.begins >> i & 1) h = given(a, a.initial, __shfl_sync(0xFFFFFFFFu, m.begin, i), at);
      slope_step<MARKED>(row(a, stage, at, 0, i), o[i], h, slope[i]);
    }
  }
  float2 e = take<true>(a, sh, all.stop, look_at(all, stage), whole, at.tile, at.reach, at.at0), db = both(0.0f);
  for (int w = kWarps - 1; w > warp; --w) e = sh.cut[w] & CUT_UP ? sh.b[w][lane] : fma2(sh.a[w][lane], e, sh.b[w][lane]);
  const int64_t size = out_size(a.dx_bf16), pitch_x = a.ld_dx * size, pitch_g = a.ld_dgate * size;
  uint8_t *dx = static_cast<uint8_t *>(a.dx) + ((at.first + kSteps - 1) * a.ld_dx + at.column) * size;
  uint8_t *dgate = static_cast<uint8_t *>(a.dgate) + ((at.first + kSteps - 1) * a.ld_dgate + at.column) * size;
  auto rows = [&](auto step) {
#pragma unroll
    for (int i = kSteps - 1; i >= 0; --i) {
      db = __fadd2_rn(db, step(row(a, stage, at, 2, i), o[i], slope[i]));
      dx -= pitch_x, dgate -= pitch_g;
    }
  };
  if (__builtin_expect(path == SHORT, 1)) {
    rows([&](float2 dh, float2 o, float2 slope) { return gradient_step<SHORT>(a, dh, o, slope, at, dx, dgate, e); });
  } else if (path == HELD) {
    rows([&](float2 dh, float2 o, float2 slope) { return gradient_step<HELD>(a, dh, o, slope, at, dx, dgate, e); });
  } else {
#pragma unroll
    for (int i = kSteps - 1; i >= 0; --i) {
      if (m.ends >> i & 1) e = given(a, a.dfinal, __shfl_sync(0xFFFFFFFFu, m.end, i), at);
      if (m.valid >> i & 1) {  // else e passes
        const float2 dz = gradient_step<MARKED>(a, row(a, stage, at, 2, i), o[i], slope[i], at, dx, dgate, e);
        db = __fadd2_rn(db, dz);
      }
      dx -= pitch_x, dgate -= pitch_g;
      if (m.begins >> i & 1) {
        const int32_t s = __shfl_sync(0xFFFFFFFFu, m.begin, i);
        if (at.in && a.dinitial) put_f32<WAY>(a.dinitial + (int64_t)s * a.cols + at.column, at.second, e);
      }
    }
  }
  if (a.partial) {
    __syncthreads();
    sh.a[warp][lane] = db;
    __syncthreads();
    if (warp == 0 && at.in) {
      for (int w = 1; w < kWarps; ++w) db = __fadd2_rn(db, sh.a[w][lane]);
      put_f32<WAY>(a.partial + at.tile * a.cols + at.column, at.second, db);
    }
  }
  return next;
}

template <class T, Way WAY, bool BACKWARD>
__global__ void __launch_bounds__(kThreads, Tile<T, WAY, BACKWARD>::kBlocks) tile_kernel(const __grid_constant__ Args a) {
  using Work = Tile<T, WAY, BACKWARD>;
  extern __shared__ __align__(128) uint8_t stages[];
  __shared__ typename Work::Block sh;
  if (threadIdx.x == 0) sh.stop = 0;
  wait_for_previous();
  // Tiles by ticket where they wait for one another, else by block.  A ticket is taken when the tile
  // before it is under way, so that tiles begin in the order of their tickets.
  const bool by_ticket = a.time_tiles > 1;
  uint32_t now = blockIdx.x;
  if (threadIdx.x == 0) {
    sh.ticket[1] = by_ticket ? atomicAdd(a.ticket, 1u) + 1 : now;
    sh.spot[1] = spot_of<Work::kRows>(a, sh.ticket[1], BACKWARD);
  }
  __syncthreads();
  now = sh.ticket[1];
  Spot p = sh.spot[1];
  let_next_start();
  int64_t lo = 0, hi = a.rows;
  if (a.packed) lo = offset_at(a, 0), hi = offset_at(a, a.seqs);
  Work::start(a, stages, now, p);
  for (uint32_t n = 0; now < a.tiles; ++n) {
    uint8_t *stage = stages + (n & 1) * Work::kStage, *other = stages + (~n & 1) * Work::kStage;
    if (threadIdx.x == 0) {
      const uint32_t t = by_ticket ? atomicAdd(a.ticket, 1u) + 1 : now + gridDim.x;
      sh.ticket[n & 1] = t, sh.spot[n & 1] = spot_of<Work::kRows>(a, t, BACKWARD);
    }
    if constexpr (WAY != DIRECT) asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();  // the stage is whole, and every warp has left the tile before
    now = BACKWARD ? Work::backward(a, sh, n & 1, stage, other, p, lo, hi) : Work::forward(a, sh, n & 1, stage, other, p, lo, hi);
  }
  if constexpr (WAY != DIRECT) asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();
  if (threadIdx.x == 0 && sh.stop) atomicAdd(a.gave_up, 1u);
}

// Sequences of one row each, a step of generation: nothing to scan.  A lane to 4 columns of a row (PAIRS: in pairs, whose
// addresses all matrices align; else 32 apart), a warp to 128.  The states kept for the backward pass are initial ones.
template <class T, bool PAIRS>
__global__ void __launch_bounds__(kThreads) step_kernel(const __grid_constant__ Args a) {
  const int lane = threadIdx.x & 31;
  const int64_t strips = (a.cols + 127) / 128, unit = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32;
  const int64_t t = unit / strips, left = (unit - t * strips) * 128;
  wait_for_previous();
  let_next_start();
  if (t >= a.rows) return;
  const T *x = static_cast<const T *>(a.x) + t * a.ld_x, *gate = static_cast<const T *>(a.gate) + t * a.ld_gate;
  const int64_t s = t * a.cols;
  float *kept = a.states && t % kStateRows == 0 ? a.states + t / kStateRows * a.cols : nullptr;
  if constexpr (PAIRS) {
    float2 u[2], z[2], b[2], h0[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t j = left + i * 64 + lane * 2;
      u[i] = z[i] = b[i] = h0[i] = both(0.0f);
      if (j >= a.cols) continue;
      if constexpr (sizeof(T) == 2) {
        const uint32_t p = *reinterpret_cast<const uint32_t *>(x + j), q = *reinterpret_cast<const uint32_t *>(gate + j);
        u[i] = make_float2(bf16_low(p), bf16_high(p)), z[i] = make_float2(bf16_low(q), bf16_high(q));
      } else {
        u[i] = *reinterpret_cast<const float2 *>(x + j), z[i] = *reinterpret_cast<const float2 *>(gate + j);
      }
      if (a.bias) b[i] = make_float2(load_any(a.bias, j, a.param_bf16), load_any(a.bias, j + 1, a.param_bf16));
      if (a.initial) h0[i] = make_float2(a.initial[s + j], a.initial[s + j + 1]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t j = left + i * 64 + lane * 2;
      if (j >= a.cols) continue;
      float2 f, keep;
      gates(held_odds(__fadd2_rn(z[i], b[i])), f, keep);
      const float2 h = fma2(f, h0[i], __fmul2_rn(keep, u[i]));
      put<UNITS>(static_cast<uint8_t *>(a.h) + (t * a.ld_h + j) * (a.h_bf16 ? 2 : 4), a.h_bf16 != 0, true, h);
      if (kept) kept[j] = h0[i].x, kept[j + 1] = h0[i].y;
      if (a.final_state) a.final_state[s + j] = h.x, a.final_state[s + j + 1] = h.y;
    }
  } else {
    float u[4], z[4], b[4], h0[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t j = left + i * 32 + lane;
      const bool in = j < a.cols;
      u[i] = in ? (float)x[j] : 0.0f, z[i] = in ? (float)gate[j] : 0.0f;
      b[i] = in && a.bias ? load_any(a.bias, j, a.param_bf16) : 0.0f, h0[i] = in && a.initial ? a.initial[s + j] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t j = left + i * 32 + lane;
      if (j >= a.cols) continue;
      float2 f, keep;
      gates(held_odds(both(z[i] + b[i])), f, keep);
      const float h = fmaf(f.x, h0[i], keep.x * u[i]);
      store_any(a.h, t * a.ld_h + j, a.h_bf16 != 0, h);
      if (kept) kept[j] = h0[i];
      if (a.final_state) a.final_state[s + j] = h;
    }
  }
}

// Packed sequences: marks where they begin and end, and the states of those without rows.
// A warp to a sequence.
__global__ void __launch_bounds__(256) mark_kernel(const __grid_constant__ Args a) {
  const int lane = threadIdx.x & 31;
  const int64_t s = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
  wait_for_previous();
  let_next_start();
  if (s >= a.seqs) return;
  const int64_t begin = offset_at(a, s), end = offset_at(a, s + 1);
  if (begin < end) {
    if (lane == 0) a.begins[begin] = (int32_t)s, a.ends[end - 1] = (int32_t)s;
    return;
  }
  for (int64_t j = lane; j < a.cols; j += 32) {
    if (a.final_state) a.final_state[s * a.cols + j] = a.initial ? a.initial[s * a.cols + j] : 0.0f;
    if (a.dinitial) a.dinitial[s * a.cols + j] = a.dfinal ? a.dfinal[s * a.cols + j] : 0.0f;
  }
}

// Sums of the tiles' parts of dbias, in a fixed order: 32 columns to a block.
constexpr int kSumThreads = 1024;
__global__ void __launch_bounds__(kSumThreads) column_sum_kernel(const float *partial, int64_t n, int64_t cols, void *out, int32_t bf16) {
  __shared__ float part[kSumThreads / 32][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int64_t j = (int64_t)blockIdx.x * 32 + lane;
  wait_for_previous();
  let_next_start();
  float s = 0.0f;
  if (j < cols) {
#pragma unroll 8
    for (int64_t i = warp; i < n; i += kSumThreads / 32) s += partial[i * cols + j];
  }
  part[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && j < cols) {
    for (int w = 1; w < kSumThreads / 32; ++w) s += part[w][lane];
    store_any(out, j, bf16 != 0, s);
  }
}

fsdp_status_t check(const fsdp_scan_desc_t *d) {
  if (!d) return fail(FSDP_EINVAL, "desc is NULL");
  if (d->rows < 0 || d->cols < 1 || d->seqs < 0) return fail(FSDP_EINVAL, "rows < 0, cols < 1 or seqs < 0");
  if (d->cols > INT64_MAX / 64 / std::max<int64_t>(std::max(d->rows, d->seqs), 1)) return fail(FSDP_EUNSUPPORTED, "the matrices are too large");
  if (d->rows > INT32_MAX - 1024 || d->seqs > INT32_MAX - 1024) return fail(FSDP_EUNSUPPORTED, "2^31 rows or sequences");
  if (d->packed != 0 && d->packed != 1) return fail(FSDP_EINVAL, "packed is neither 0 nor 1");
  if (!d->packed) {
    if (d->seq_len < 1) return fail(FSDP_EINVAL, "seq_len < 1 (sequences without rows come packed)");
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

// The workspace: parts of dbias, then what has to be 0xFF: what tiles leave for one another,
// the ticket, and the marks of packed sequences.
struct Plan {
  int64_t column_tiles, time_tiles, padded_cols;
  int64_t partial, clear, carried, ticket, parts, begins, ends, bytes;
};
Plan plan_of(const fsdp_scan_desc_t &d, bool backward) {
  Plan p = {};
  const int64_t tile = kWarps * steps_of(dtype_bytes(d.x_dtype));
  p.column_tiles = (d.cols + kCols - 1) / kCols;
  p.time_tiles = (d.rows + tile - 1) / tile;
  p.padded_cols = p.column_tiles * kCols;
  auto take = [&](int64_t bytes) {
    const int64_t at = p.bytes;
    p.bytes += (bytes + 15) / 16 * 16;
    return at;
  };
  const bool several = p.time_tiles > 1 && (backward || d.packed || d.seq_len != 1);
  p.partial = take(backward ? p.time_tiles * d.cols * 4 : 0);
  p.clear = p.bytes;
  p.parts = take(several ? p.time_tiles * p.padded_cols * 8 : 0);
  p.carried = take(several ? p.time_tiles * p.padded_cols * 4 : 0);
  p.ticket = take(several ? 4 : 0);
  p.begins = take(d.packed ? d.rows * 4 : 0);
  p.ends = take(d.packed ? d.rows * 4 : 0);
  return p;
}

template <class K>
const void *kernel(K *k) {
  return reinterpret_cast<const void *>(k);
}

template <class Work>
cudaError_t launch_tiles(void (*fn)(Args), Args &a, cudaStream_t s) {
  static_assert((Work::kSmem + (int)sizeof(typename Work::Block) + 1024) * Work::kBlocks <= 228 * 1024, "an SM's blocks");
  static std::atomic<uint64_t> ready{0};  // devices on which this kernel may have its shared memory
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (device & 63);
  if (Work::kSmem > 0 && (device > 63 || !(ready.load(std::memory_order_relaxed) & bit))) {
    e = cudaFuncSetAttribute(kernel(fn), cudaFuncAttributeMaxDynamicSharedMemorySize, Work::kSmem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  // Few chains are bound by their carries, which a third block of an SM delays (us with two / three blocks, BF16 forward: 65536 rows
  // of one sequence, 64 columns 41 / 46, 256 50 / 51, 384 62 / 59, 1024 127 / 109; of sequences of 2048, 64 14.6 / 14.8, 256 34 / 29).
  const int blocks = a.column_tiles * a.aside <= 4 ? std::min(2, Work::kBlocks) : Work::kBlocks;
  const int64_t grid = std::min<int64_t>(a.tiles, (int64_t)device_sms() * blocks);
  void *args[] = {&a};
  return launch_kernel(kernel(fn), dim3((unsigned)grid), dim3(kThreads), args, Work::kSmem, s, true);
}
template <bool BACKWARD, class T>
cudaError_t launch_as(Way way, Args &a, cudaStream_t s) {
  if (way == UNITS) return launch_tiles<Tile<T, UNITS, BACKWARD>>(&tile_kernel<T, UNITS, BACKWARD>, a, s);
  if (way == ANY) return launch_tiles<Tile<T, ANY, BACKWARD>>(&tile_kernel<T, ANY, BACKWARD>, a, s);
  if constexpr (BACKWARD) return launch_tiles<Tile<T, DIRECT, true>>(&tile_kernel<T, DIRECT, true>, a, s);
  return cudaErrorInvalidValue;  // forward, x and gate are always of one type
}

// Whether pairs of columns, and the 16-byte units of staged rows, fit all matrices.
struct Fit {
  bool pairs = true, units = true;
  void matrix(const void *p, int64_t rows, int64_t cols, int64_t ld, int64_t size) {
    pairs &= cols % 2 == 0 && (uintptr_t)p % (2 * size) == 0 && (rows <= 1 || ld % 2 == 0);
    units &= cols * size % 16 == 0 && aligned16(p) && (rows <= 1 || ld * size % 16 == 0);
  }
};

// Fill the marks and the values to come, mark packed sequences, and launch the tiles.
template <bool BACKWARD>
fsdp_status_t run(const fsdp_scan_desc_t &d, Args &a, const Plan &p, void *workspace, const Fit &fit, cudaStream_t s) {
  uint8_t *w = static_cast<uint8_t *>(workspace);
  if (!BACKWARD && !d.packed && d.seq_len == 1) {
    // A tile's rows would each begin and end a sequence (64 x 4096 in BF16 5.4 us, here 1.9).
    const int64_t blocks = (d.rows * ((d.cols + 127) / 128) + kWarps - 1) / kWarps;
    if (blocks > INT32_MAX) return fail(FSDP_EUNSUPPORTED, "the step is too large for one launch");
    using B = __nv_bfloat16;
    const bool bf16 = d.x_dtype == FSDP_DTYPE_BF16;
    const void *fn = fit.pairs ? (bf16 ? kernel(&step_kernel<B, true>) : kernel(&step_kernel<float, true>))
                               : (bf16 ? kernel(&step_kernel<B, false>) : kernel(&step_kernel<float, false>));
    void *args[] = {&a};
    return launched(launch_kernel(fn, dim3((unsigned)blocks), dim3(kThreads), args, 0, s, true));
  }
  if (p.time_tiles * p.column_tiles > INT32_MAX / 2) return fail(FSDP_EUNSUPPORTED, "more than 2^30 tiles");
  if (p.bytes > p.clear) {
    const cudaError_t e = cudaMemsetAsync(w + p.clear, 0xFF, p.bytes - p.clear, s);
    if (e != cudaSuccess) return fail(FSDP_ECUDA, std::string("memset: ") + cudaGetErrorString(e));
  }
  a.parts = reinterpret_cast<uint2 *>(w + p.parts), a.carried = reinterpret_cast<uint32_t *>(w + p.carried);
  a.ticket = reinterpret_cast<uint32_t *>(w + p.ticket);
  a.begins = reinterpret_cast<int32_t *>(w + p.begins), a.ends = reinterpret_cast<int32_t *>(w + p.ends);
  a.column_tiles = (uint32_t)p.column_tiles, a.time_tiles = (uint32_t)p.time_tiles, a.padded_cols = p.padded_cols;
  a.tiles = a.column_tiles * a.time_tiles;
  // Where tiles do not cross sequences, these go side by side: the tile before one is then further back in the order and has
  // mostly been done when it is looked for (us one behind the other / side by side, forward: 4 x 8192 x 4096 BF16 182 / 174,
  // 16 x 2048 x 2048 FP32 159 / 141).
  a.aside = !d.packed && d.seqs > 1 && a.time_tiles > 1 && d.seq_len % (kWarps * steps_of(dtype_bytes(d.x_dtype))) == 0 ? (uint32_t)d.seqs : 1;
  // Few chains of tiles are long ones at work, which want a wide look back; many are short, and the look back costs what it
  // reads (us with 2 / 8 / 16 tiles, BF16 forward: 131072 x 64 - / 119 / 75, 65536 x 1024 - / 123 / 110, 32768 x 4096 in one
  // sequence after another - / 182 / 205, four side by side 168 / 174 / -).
  const uint32_t chains = a.column_tiles * a.aside;
  a.window = chains <= 16 ? kWindow : chains < 256 ? kWindow / 2 : 2;
  a.fault = wait_fault(), a.wait_limit_ns = wait_limit_ns();
  cudaError_t e = gave_up_count(GAVE_UP_SCAN, &a.gave_up);
  if (e != cudaSuccess) return fail(FSDP_ECUDA, std::string("status: ") + cudaGetErrorString(e));
  if (d.packed) {
    void *args[] = {&a};
    e = launch_kernel(kernel(&mark_kernel), dim3((unsigned)((d.seqs + 7) / 8)), dim3(256), args, 0, s);
  }
  const bool alike = d.h_dtype == d.x_dtype;
  const Way way = BACKWARD && !alike ? DIRECT : fit.units && alike && (!BACKWARD || d.dx_dtype == d.x_dtype) ? UNITS : ANY;
  if (e == cudaSuccess && a.tiles > 0)
    e = d.x_dtype == FSDP_DTYPE_BF16 ? launch_as<BACKWARD, __nv_bfloat16>(way, a, s)
                                     : launch_as<BACKWARD, float>(way, a, s);
  return launched(e);
}

Args args_of(const fsdp_scan_desc_t &d, const void *x, const void *gate, const void *bias, const float *initial, const void *offsets) {
  Args a = {};
  a.x = x, a.gate = gate, a.bias = bias, a.initial = initial, a.offsets = offsets;
  a.rows = d.rows, a.cols = d.cols, a.seqs = d.seqs, a.seq_len = d.seq_len;
  a.ld_x = d.ld_x, a.ld_gate = d.ld_gate, a.ld_h = d.ld_h, a.ld_dx = d.ld_dx, a.ld_dgate = d.ld_dgate;
  a.packed = d.packed, a.wide = d.offset_dtype == FSDP_INDEX_I64;
  a.h_bf16 = d.h_dtype == FSDP_DTYPE_BF16, a.dx_bf16 = d.dx_dtype == FSDP_DTYPE_BF16;
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
  *n = (rows + kStateRows - 1) / kStateRows;
  clear_error();
  return FSDP_OK;
}

fsdp_status_t fsdp_gated_scan_workspace(const fsdp_scan_desc_t *desc, int32_t backward, int64_t *bytes) {
  fsdp_status_t st = check(desc);
  if (st != FSDP_OK) return st;
  if (!bytes) return fail(FSDP_EINVAL, "bytes is NULL");
  *bytes = plan_of(*desc, backward != 0).bytes;
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
  const Plan plan = plan_of(d, false);
  if ((st = check_workspace(workspace, workspace_bytes, plan.bytes)) != FSDP_OK) return st;
  if (d.seqs > 0) {
    Args a = args_of(d, x, gate, bias, initial, offsets);
    a.h = h, a.final_state = final, a.states = states;
    const int64_t sx = dtype_bytes(d.x_dtype);
    Fit fit;
    fit.matrix(x, d.rows, d.cols, d.ld_x, sx), fit.matrix(gate, d.rows, d.cols, d.ld_gate, sx);
    fit.matrix(h, d.rows, d.cols, d.ld_h, dtype_bytes(d.h_dtype));
    st = run<false>(d, a, plan, workspace, fit, reinterpret_cast<cudaStream_t>(stream));
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
  if (dinitial && dinitial == dfinal) return fail(FSDP_EINVAL, "dinitial is dfinal");
  const Plan plan = plan_of(d, true);
  if ((st = check_workspace(workspace, workspace_bytes, plan.bytes)) != FSDP_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  float *partial = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + plan.partial);
  if (d.seqs > 0) {
    Args a = args_of(d, x, gate, bias, initial, offsets);
    a.dh = dh, a.states_in = states, a.dfinal = dfinal, a.dx = dx, a.dgate = dgate, a.dinitial = dinitial;
    a.partial = dbias ? partial : nullptr;
    const int64_t sx = dtype_bytes(d.x_dtype), sd = dtype_bytes(d.dx_dtype);
    Fit fit;
    fit.matrix(x, d.rows, d.cols, d.ld_x, sx), fit.matrix(gate, d.rows, d.cols, d.ld_gate, sx);
    fit.matrix(dh, d.rows, d.cols, d.ld_h, dtype_bytes(d.h_dtype));
    fit.matrix(dx, d.rows, d.cols, d.ld_dx, sd), fit.matrix(dgate, d.rows, d.cols, d.ld_dgate, sd);
    st = run<true>(d, a, plan, workspace, fit, s);
    if (st != FSDP_OK) return st;
  }
  if (dbias) {
    int64_t n = d.seqs > 0 ? plan.time_tiles : 0, cols = d.cols;
    int32_t bf16 = d.grad_dtype == FSDP_DTYPE_BF16;
    void *args[] = {&partial, &n, &cols, &dbias, &bf16};
    st = launched(launch_kernel(reinterpret_cast<const void *>(&column_sum_kernel), dim3((unsigned)((d.cols + 31) / 32)), dim3(kSumThreads), args, 0, s, true));
    if (st != FSDP_OK) return st;
  }
  clear_error();
  return FSDP_OK;
}

}  // extern "C"

// The tensor-core kernel of the gated feed-forward block (see ffn.h).
#include "ffn.h"

namespace fsdp {
namespace ffn {
namespace {

constexpr int kEpilogueWarps = 8; // two to each quarter of TMEM's lanes
constexpr int kThreads = 64 + 32 * kEpilogueWarps;  // and a TMA and an MMA warp
constexpr int kTileN = 256;       // accumulator columns
constexpr int kAccumulators = 2;  // 2 x 256 columns: all of TMEM
constexpr int kTmemColumns = kTileN * kAccumulators;

template <int CG>
struct Shape {
  static constexpr int kA = kTileM * kTileK * 2;        // bytes of a block's A stage
  static constexpr int kB = kTileN / CG * kTileK * 2;   // bytes of a block's B stage
  static constexpr int kStage = kA + kB;
  static constexpr int kStages = CG == 1 ? 4 : 6;
  static constexpr int kSmem = kStages * kStage + 1024;  // stages start on 1,024-byte boundaries
};

struct Shared {
  uint64_t full[6], empty[6], tmem_full[kAccumulators], tmem_empty[kAccumulators], drain;
  uint32_t tmem, stop, filled;
};

// A unit of work: one tile and one part of its K loop.
struct Unit {
  int m, n, split;     // tile indices
  int k0, k1;          // K blocks
};

__device__ __forceinline__ Unit unit_at(const Args &a, int i) {
  Unit u;
  u.split = i % a.splits;
  const int t = i / a.splits;
  // Down a band of `raster` row tiles, then to the next column tile, so that the
  // tiles at work at one time share few operand slices, which stay in L2.
  const int band = a.raster * a.n_tiles, b = t / band, first = b * a.raster;
  const int height = min(a.m_tiles - first, a.raster), r = t - b * band;
  u.m = first + r % height;
  u.n = r / height;
  const int per = (a.k_blocks + a.splits - 1) / a.splits;
  u.k0 = min(u.split * per, a.k_blocks);
  u.k1 = min(u.k0 + per, a.k_blocks);
  return u;
}

// Loads one K block of a tile into a stage.  `rank`: this block's place in its pair.
template <int MODE, int CG>
__device__ __forceinline__ void load_stage(const Args &a, const Unit &u, int kb, int rank, uint32_t at, uint32_t bar) {
  using S = Shape<CG>;
  const uint32_t sa = at, sb = at + S::kA;
  if constexpr (MODE == FORWARD || MODE == RECOMPUTE) {
    tc::tma_load<CG>(sa, &a.a[0], kb * kTileK, (u.m * CG + rank) * kTileM, bar);
    const int n0 = u.n * (kTileN / 2);
    if constexpr (CG == 1) {
      tc::tma_load<CG>(sb, &a.b[0], kb * kTileK, n0, bar);
      tc::tma_load<CG>(sb + S::kB / 2, &a.b[1], kb * kTileK, n0, bar);
    } else {
      tc::tma_load<CG>(sb, &a.b[rank], kb * kTileK, n0, bar);
    }
  } else if constexpr (MODE == DX) {
    const int half = kb >= a.k_half ? 1 : 0, k0 = (half ? kb - a.k_half : kb) * kTileK;
    tc::tma_load<CG>(sa, &a.a[half], k0, (u.m * CG + rank) * kTileM, bar);
#pragma unroll
    for (int c = 0; c < kTileN / CG / 64; ++c)
      tc::tma_load<CG>(sb + c * 8192, &a.b[half], u.n * kTileN + rank * (kTileN / CG) + c * 64, k0, bar);
  } else {
    const int half = u.m >= a.m_half ? 1 : 0, m0 = ((half ? u.m - a.m_half : u.m) * CG + rank) * kTileM;
#pragma unroll
    for (int c = 0; c < kTileM / 64; ++c) tc::tma_load<CG>(sa + c * 8192, &a.a[half], m0 + c * 64, kb * kTileK, bar);
#pragma unroll
    for (int c = 0; c < kTileN / CG / 64; ++c)
      tc::tma_load<CG>(sb + c * 8192, &a.b[0], u.n * kTileN + rank * (kTileN / CG) + c * 64, kb * kTileK, bar);
  }
}

// 32 consecutive elements of a row to memory: `n` of them exist; `width`: row_width().
// A thread has a row of its own, so a store instruction of a warp goes to 32 rows;
// whole 32-byte sectors keep that from costing two writes a sector.
__device__ __forceinline__ void store_run(void *p, int64_t at, bool bf16, int width, const float2 (&v)[16], int n) {
  if (width >= 16 && n >= 32) {
    if (bf16) {
      uint32_t w[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = bf16_pair(v[i].x, v[i].y);
      uint4 *q = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p) + at);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t(&h)[8] = reinterpret_cast<const uint32_t(&)[8]>(w[8 * i]);
        if (width == 32)
          store32(q + 2 * i, h);
        else
          q[2 * i] = make_uint4(h[0], h[1], h[2], h[3]), q[2 * i + 1] = make_uint4(h[4], h[5], h[6], h[7]);
      }
    } else {
      float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(p) + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (width == 32) {
          uint32_t h[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) h[e] = __float_as_uint(element(v, 8 * i + e));
          store32(q + 2 * i, h);
        } else {
          q[2 * i] = make_float4(v[4 * i].x, v[4 * i].y, v[4 * i + 1].x, v[4 * i + 1].y);
          q[2 * i + 1] = make_float4(v[4 * i + 2].x, v[4 * i + 2].y, v[4 * i + 3].x, v[4 * i + 3].y);
        }
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (i < n) store_any(p, at + i, bf16, element(v, i));
}

// The 8-bit checkpoint of 32 consecutive elements, one whole group; elements from n on are 0.
__device__ __forceinline__ void keep_group(uint8_t *codes, uint8_t *scale, float2 (&v)[16], int n, bool sector) {
  if (n < 32) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i >= n) element(v, i) = 0.0f;
  }
  const uint32_t s = act8_scale_byte(act8_top(v));
  act8_store<32>(codes, v, s, sector);
  *scale = (uint8_t)s;
}

__device__ __forceinline__ float2 pair_at(const uint32_t (&r)[32], int i) {
  return make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
}

// One thread's part of a gate / up tile: 32 columns of one row.
template <int MODE>
__device__ __forceinline__ void gated_run(const Args &a, const uint32_t (&gr)[32], const uint32_t (&ur)[32], int64_t row,
                                          int64_t col) {
  const int n = (int)min((int64_t)32, a.n - col);
  float2 x[16], y[16];
  if constexpr (MODE == FORWARD) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 g = pair_at(gr, i);
      x[i] = __fmul2_rn(make_float2(act_of<false>(g.x, a.act).x, act_of<false>(g.y, a.act).x), pair_at(ur, i));
    }
    store_run(a.out[0], row * a.ld_out[0] + col, true, a.out_width, x, n);
    if (a.keep) {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = pair_at(gr, i), y[i] = pair_at(ur, i);
      if (a.keep == 1) {
        const int64_t group = row * a.groups + col / (int)kActGroup;
        keep_group(a.codes[0] + group * kActGroup, a.scales[0] + group, x, n, a.keep_width == 32);
        keep_group(a.codes[1] + group * kActGroup, a.scales[1] + group, y, n, a.keep_width == 32);
      } else {
        store_run(a.kept[0], row * a.ld_kept + col, true, a.keep_width, x, n);
        store_run(a.kept[1], row * a.ld_kept + col, true, a.keep_width, y, n);
      }
    }
  } else {
    const __nv_bfloat16 *dh = static_cast<const __nv_bfloat16 *>(a.dh) + row * a.ld_dh + col;
    float2 d[16];
    if (a.dh_vec && n >= 32) {
#pragma unroll
      for (int i = 0; i < 4; ++i) load8(dh, 8 * i, true, reinterpret_cast<float2(&)[4]>(d[4 * i]));
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) element(d, i) = i < n ? __bfloat162float(dh[i]) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 g = pair_at(gr, i), p = act_of<true>(g.x, a.act), q = act_of<true>(g.y, a.act);
      x[i] = __fmul2_rn(__fmul2_rn(d[i], pair_at(ur, i)), make_float2(p.y, q.y));
      y[i] = __fmul2_rn(d[i], make_float2(p.x, q.x));
    }
    store_run(a.out[0], row * a.ld_out[0] + col, true, a.out_width, x, n);
    store_run(a.out[1], row * a.ld_out[1] + col, true, a.out_width, y, n);
  }
}

// Test hook: the first worker leaves its first stage empty, so the wait for it gives up.
__device__ __forceinline__ bool skips_first(const Args &a, int worker) { return a.fault != 0 && worker == 0; }

// After a wait that gave up, by one thread once every role has left its loop: wait
// (again for a limited time) until the copies in flight have landed.  The leader's
// barriers count both blocks' bytes; what the other block of a pair sent to a stage
// that the leader never armed is not counted anywhere and gets a fixed time.
template <int CG>
__device__ __noinline__ void land_copies(Shared &sh, const Args &a, int rank, bool skipped) {
  using S = Shape<CG>;
  if (rank == 0) {
    uint32_t f = sh.filled > (uint32_t)S::kStages ? sh.filled - S::kStages : 0;
    if (f == 0 && skipped) f = 1;
    for (; f < sh.filled; ++f) {
      uint32_t never = 0;
      tc::bar_wait(tc::smem(&sh.full[f % S::kStages]), (f / S::kStages) & 1u, a.wait_limit_ns, &never);
    }
  } else {
    const uint64_t began = tc::now_ns();
    while (tc::now_ns() - began < 1000000) {
    }
  }
}

template <int MODE, int CG>
__global__ void __launch_bounds__(kThreads, 1) product_kernel(const __grid_constant__ Args a) {
  using S = Shape<CG>;
  extern __shared__ uint8_t dynamic[];
  __shared__ Shared sh;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const uint32_t stages = (tc::smem(dynamic) + 1023u) & ~1023u;
  const int rank = CG == 1 ? 0 : (int)tc::cluster_rank();
  const int worker = blockIdx.x / CG, workers = gridDim.x / CG;
  const int units = a.m_tiles * a.n_tiles * a.splits;
  volatile uint32_t *stop = &sh.stop;

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < S::kStages; ++s) {
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
      for (int i = worker; i < units && ok; i += workers) {
        const Unit u = unit_at(a, i);
        for (int kb = u.k0; kb < u.k1; ++kb) {
          const uint32_t full = tc::smem(&sh.full[stage]), full_leader = CG == 1 ? full : tc::at_rank(full, 0);
          if (!(ok = tc::bar_wait(tc::smem(&sh.empty[stage]), phase ^ 1u, a.wait_limit_ns, stop))) break;
          if (!skips_first(a, worker) || filled > 0) {
            if (rank == 0) tc::bar_expect(full, CG * S::kStage);
            load_stage<MODE, CG>(a, u, kb, rank, stages + stage * S::kStage, full_leader);
          }
          ++filled;
          if (++stage == S::kStages) stage = 0, phase ^= 1u;
        }
      }
      sh.filled = filled;
    }
  } else if (warp == 1) {
    // ---- products ------------------------------------------------------------
    if (lane == 0 && rank == 0) {
      constexpr bool kAMn = MODE == DW, kBMn = MODE == DX || MODE == DW;
      constexpr uint32_t idesc = tc::instruction(kTileM * CG, kTileN, kAMn, kBMn);
      // Descriptors advance by 16 K values: 32 bytes within a row, or 16 rows of 128 bytes.
      constexpr uint32_t kStepA = kAMn ? 2048 : 32, kStepB = kBMn ? 2048 : 32;
      uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0;
      bool issued = false;
      for (int i = worker; i < units && ok; i += workers) {
        const Unit u = unit_at(a, i);
        if (!(ok = tc::bar_wait(tc::smem(&sh.tmem_empty[acc]), acc_phase ^ 1u, a.wait_limit_ns, stop))) break;
        tc::fence_after();
        const uint32_t d = tmem + acc * kTileN;
        for (int kb = u.k0; kb < u.k1; ++kb) {
          if (!(ok = tc::bar_wait(tc::smem(&sh.full[stage]), phase, a.wait_limit_ns, stop))) break;
          tc::fence_after();
          const uint32_t sa = stages + stage * S::kStage, sb = sa + S::kA;
#pragma unroll
          for (int k = 0; k < kTileK / 16; ++k)
            tc::mma<CG>(d, tc::operand(sa + k * kStepA, kAMn ? 8192 : 16, 1024),
                        tc::operand(sb + k * kStepB, kBMn ? 8192 : 16, 1024), idesc, kb > u.k0 || k > 0);
          issued = true;
          tc::mma_commit<CG>(tc::smem(&sh.empty[stage]));
          if (++stage == S::kStages) stage = 0, phase ^= 1u;
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
    const int side = (warp - 2) / 4;       // and its half of the columns
    uint32_t acc = 0, acc_phase = 0;
    for (int i = worker; i < units; i += workers) {
      const Unit u = unit_at(a, i);
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
#pragma unroll 1
        for (int c = side * (kTileN / 4); c < (side + 1) * (kTileN / 4); c += 32) {
          const int64_t col = (int64_t)u.n * (kTileN / 2) + c;
          uint32_t g[32], up[32];
          __syncwarp();
          tc::tmem_load32(from + c, g);
          tc::tmem_load32(from + kTileN / 2 + c, up);
          tc::tmem_load_wait();
          if (c + 32 == (side + 1) * (kTileN / 4)) drained();
          if (col >= a.n) continue;
          if (row < a.m) gated_run<MODE>(a, g, up, row, col);
        }
      } else {
        const int half = MODE == DW && u.m >= a.m_half ? 1 : 0;
        const int64_t row = ((int64_t)(half ? u.m - a.m_half : u.m) * CG + rank) * kTileM + quarter * 32 + lane;
#pragma unroll 1
        for (int c = side * (kTileN / 2); c < (side + 1) * (kTileN / 2); c += 32) {
          const int64_t col = (int64_t)u.n * kTileN + c;
          uint32_t r[32];
          __syncwarp();
          tc::tmem_load32(from + c, r);
          tc::tmem_load_wait();
          if (c + 32 == (side + 1) * (kTileN / 2)) drained();
          if (col >= a.n) continue;
          float2 v[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = some ? pair_at(r, e) : both(0.0f);
          if (row < a.m) {
            const int n = (int)min((int64_t)32, a.n - col);
            if (a.splits > 1) {
              const int64_t rows = MODE == DW ? 2 * a.m : a.m;
              store_run(a.partial, ((int64_t)u.split * rows + half * a.m + row) * a.n + col, false, a.n % 8 == 0 ? 32 : a.n % 4 == 0 ? 16 : 0, v, n);
            } else {
              store_run(a.out[half], row * a.ld_out[half] + col, a.out_bf16 != 0, a.out_width, v, n);
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
    atomicOr(a.status, kStatusGemm);
    land_copies<CG>(sh, a, rank, skips_first(a, worker));
  }
  __syncthreads();
  if constexpr (CG == 2) tc::cluster_sync();
  tc::fence_after();
  if (warp == 1) tc::tmem_free<CG>(tmem, kTmemColumns);
}

template <int MODE, int CG>
cudaError_t launch(Args &a, int sms, cudaStream_t stream) {
  using S = Shape<CG>;
  const void *fn = reinterpret_cast<const void *>(&product_kernel<MODE, CG>);
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t units = (int64_t)a.m_tiles * a.n_tiles * a.splits;
  int64_t workers = sms / CG;
  if (workers > units) workers = units;
  void *args[] = {&a};
  return launch_kernel(fn, dim3((unsigned)(workers * CG)), dim3(kThreads), args, S::kSmem, stream, true, CG);
}

}  // namespace

cudaError_t launch_product(Mode mode, bool pair, Args &a, int sms, cudaStream_t stream) {
  switch (mode) {
    case FORWARD: return pair ? launch<FORWARD, 2>(a, sms, stream) : launch<FORWARD, 1>(a, sms, stream);
    case RECOMPUTE: return pair ? launch<RECOMPUTE, 2>(a, sms, stream) : launch<RECOMPUTE, 1>(a, sms, stream);
    case DX: return pair ? launch<DX, 2>(a, sms, stream) : launch<DX, 1>(a, sms, stream);
    default: return pair ? launch<DW, 2>(a, sms, stream) : launch<DW, 1>(a, sms, stream);
  }
}

}  // namespace ffn
}  // namespace fsdp

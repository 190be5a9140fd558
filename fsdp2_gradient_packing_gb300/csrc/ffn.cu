// Gated feed-forward block (fsdp_gated_ffn_*): argument checks, operand maps, the
// plan of the launches, and the kernels around the products.
//
// Forward: one launch.  Backward: dg and du (from what was kept, one pass over
// dh, gate and up; or as the epilogue of the forward product), then dx, then both
// weight gradients.  dg and du pass through the workspace in BF16.
#include <cuda.h>

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

// Copy of a matrix whose rows start anywhere, to rows of `pitch` elements.
__global__ void __launch_bounds__(kThreads) copy_rows_kernel(const uint16_t *src, int64_t ld, uint16_t *dst, int64_t pitch,
                                                             int64_t rows, int64_t cols) {
  wait_for_previous();
  let_next_start();
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
    for (int64_t j = threadIdx.x; j < cols; j += kThreads) dst[r * pitch + j] = src[r * ld + j];
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
  int32_t act, act8, dh_vec, kept_vec;
};

// Bound: HBM, 2 + 33/16 + 4 bytes an element from 8-bit checkpoints.  Eight columns
// to a thread.
__global__ void __launch_bounds__(kThreads) slope_kernel(const __grid_constant__ SlopeArgs a) {
  const int64_t per_row = (a.f + 7) / 8, total = a.rows * per_row;
  wait_for_previous();
  let_next_start();
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThreads) {
    int64_t row, at;
    if ((uint64_t)total >> 32 == 0)
      row = (uint32_t)i / (uint32_t)per_row, at = (uint32_t)i % (uint32_t)per_row;
    else
      row = i / per_row, at = i % per_row;
    const int64_t j = at * 8;
    const bool whole = j + 8 <= a.f;
    float2 d[4], g[4], u[4];
    auto load = [&](float2(&v)[4], const void *p, int64_t at, bool vec) {
      if (whole && vec) {
        load8(p, at, true, v);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) element(v, e) = j + e < a.f ? load_any(p, at + e, true) : 0.0f;
      }
    };
    load(d, a.dh, row * a.ld_dh + j, a.dh_vec != 0);
    if (a.act8) {
      const int64_t c = row * a.groups * kActGroup + j, s = row * a.groups + j / (int)kActGroup;
      const uint2 p = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(a.gate) + c);
      const uint2 q = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(a.up) + c);
      const float2 sg = both(act8_scale(a.scales[0][s])), su = both(act8_scale(a.scales[1][s]));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        g[e] = __fmul2_rn(act8_codes_of(act8_biased(e < 2 ? p.x : p.y), e % 2), sg);
        u[e] = __fmul2_rn(act8_codes_of(act8_biased(e < 2 ? q.x : q.y), e % 2), su);
      }
    } else {
      load(g, a.gate, row * a.ld_kept + j, a.kept_vec != 0);
      load(u, a.up, row * a.ld_kept + j, a.kept_vec != 0);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 p = act_of<true>(g[e].x, a.act), q = act_of<true>(g[e].y, a.act);
      g[e] = __fmul2_rn(__fmul2_rn(d[e], u[e]), make_float2(p.y, q.y));
      u[e] = __fmul2_rn(d[e], make_float2(p.x, q.x));
    }
    // The pitch holds whole vectors; what lies past the row's end is never read.
    store8(a.dg, row * a.pitch + j, true, g);
    store8(a.du, row * a.pitch + j, true, u);
  }
}

// ---------------------------------------------------------------------------
// The parts of split K loops, added in order
// ---------------------------------------------------------------------------
struct JoinArgs {
  const float *partial;   // [splits][rows][cols]
  void *out[2];
  int64_t ld[2];
  int64_t rows, half, cols;  // rows from `half` on belong to out[1]
  int32_t splits, bf16, vec;
};

// Bound: L2, where the parts still are.  VEC columns to a thread, one row to a block
// at a time.
template <int VEC>
__global__ void __launch_bounds__(kThreads) join_kernel(const __grid_constant__ JoinArgs a) {
  const int64_t total = a.rows * a.cols;
  wait_for_previous();
  let_next_start();
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const bool second = r >= a.half;
    const int64_t row = second ? r - a.half : r;
    for (int64_t col = ((int64_t)blockIdx.y * kThreads + threadIdx.x) * VEC; col < a.cols; col += (int64_t)gridDim.y * kThreads * VEC) {
      const float *p = a.partial + r * a.cols + col;
      float s[VEC];
      if constexpr (VEC == 4) {
        float4 v = *reinterpret_cast<const float4 *>(p);
#pragma unroll 4
        for (int k = 1; k < a.splits; ++k) {
          const float4 q = *reinterpret_cast<const float4 *>(p + k * total);
          v.x += q.x, v.y += q.y, v.z += q.z, v.w += q.w;
        }
        s[0] = v.x, s[1] = v.y, s[2] = v.z, s[3] = v.w;
        if (a.vec) {
          const int64_t at = row * a.ld[second] + col;
          if (a.bf16)
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out[second]) + at) =
                make_uint2(bf16_pair(s[0], s[1]), bf16_pair(s[2], s[3]));
          else
            *reinterpret_cast<float4 *>(static_cast<float *>(a.out[second]) + at) = v;
          continue;
        }
      } else {
        s[0] = p[0];
#pragma unroll 4
        for (int k = 1; k < a.splits; ++k) s[0] += p[k * total];
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) store_any(a.out[second], row * a.ld[second] + col + e, a.bf16 != 0, s[e]);
    }
  }
}

// ---------------------------------------------------------------------------
// Plan
// ---------------------------------------------------------------------------
struct Tiling {
  bool pair;
  int64_t m_tiles, n_tiles, m_half, k_blocks, splits;
};

// The tiles of one product, and how often its K loop is split so that there is
// work for every SM.
Tiling tiling(Mode mode, int64_t m, int64_t n, int64_t k, int sms) {
  Tiling t = {};
  t.pair = true;
  const int64_t tile_m = t.pair ? 2 * kTileM : kTileM, tile_n = mode == FORWARD || mode == RECOMPUTE ? 128 : 256;
  t.m_half = blocks_of(m, tile_m);
  t.m_tiles = mode == DW ? 2 * t.m_half : t.m_half;
  t.n_tiles = blocks_of(n, tile_n);
  t.k_blocks = mode == DX ? 2 * blocks_of(k, kTileK) : blocks_of(k, kTileK);
  t.splits = 1;
  if (mode == DX || mode == DW) {
    const int64_t workers = t.pair ? sms / 2 : sms, tiles = t.m_tiles * t.n_tiles;
    int64_t s = workers / tiles;
    if (s > t.k_blocks / 8) s = t.k_blocks / 8;
    if (s > 16) s = 16;
    if (s > 1) t.splits = blocks_of(t.k_blocks, blocks_of(t.k_blocks, s));  // no part is empty
  }
  return t;
}

struct Plan {
  int sms;
  bool stage_x, stage_wg, stage_wu;
  int64_t d_pitch, f_pitch;
  int64_t at_x, at_wg, at_wu, at_dg, at_du, at_partial, bytes;
};

bool rows_off(int64_t rows, int64_t ld, bool base) { return base || (rows > 1 && ld % 8 != 0); }

Plan plan_of(const fsdp_ffn_desc_t *d, bool backward) {
  Plan p = {};
  p.sms = device_sms() > 0 ? device_sms() : 160;
  p.d_pitch = up_to(d->d, 8), p.f_pitch = up_to(d->f, 16);
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
    const Tiling x = tiling(DX, d->rows, d->d, d->f, p.sms), w = tiling(DW, d->f, d->d, d->rows, p.sms);
    const int64_t px = x.splits > 1 ? x.splits * d->rows * d->d * 4 : 0;
    const int64_t pw = w.splits > 1 ? w.splits * 2 * d->f * d->d * 4 : 0;
    p.at_partial = take(true, px > pw ? px : pw);
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

  fsdp_status_t copy(Operand &o, bool want, int64_t at) {
    if (!want || o.rows == 0) return FSDP_OK;
    const uint16_t *src = static_cast<const uint16_t *>(o.p);
    uint16_t *dst = reinterpret_cast<uint16_t *>(ws + at);
    int64_t ld = o.ld, pitch = plan.d_pitch, rows = o.rows, cols = o.cols;
    void *args[] = {&src, &ld, &dst, &pitch, &rows, &cols};
    const int64_t grid = rows < plan.sms * 8 ? rows : plan.sms * 8;
    o.p = dst, o.ld = pitch;
    return launched(launch_kernel(reinterpret_cast<const void *>(&copy_rows_kernel), dim3((unsigned)grid), dim3(kThreads),
                                  args, 0, stream, true));
  }

  fsdp_status_t stage(const void *px, const void *pwg, const void *pwu) {
    wg = {pwg, d->f, d->d, d->ld_w_gate};
    wu = {pwu, d->f, d->d, d->ld_w_up};
    x = {px, d->rows, d->d, d->ld_x};
    fsdp_status_t st = copy(wg, plan.stage_wg, plan.at_wg);
    if (st == FSDP_OK) st = copy(wu, plan.stage_wu, plan.at_wu);
    if (st != FSDP_OK) return st;
    if (d->x_dtype == FSDP_ACT8) {
      x.p = ws + plan.at_x, x.ld = plan.d_pitch;
      return fsdp_act8_load(px, d->rows, d->d, ws + plan.at_x, FSDP_DTYPE_BF16, plan.d_pitch,
                            reinterpret_cast<fsdp_stream_t>(stream));
    }
    return copy(x, plan.stage_x, plan.at_x);
  }

  // One product; args' outputs and flags are set by the caller.
  fsdp_status_t product(Mode mode, int64_t m, int64_t n, int64_t k, const Operand &a0, const Operand &a1,
                        const Operand &b0, const Operand &b1, Args &a) {
    const Tiling t = tiling(mode, m, n, k, plan.sms);
    const int a_rows = mode == DW ? 64 : 128, b_rows = mode == FORWARD || mode == RECOMPUTE ? 128 : 64;
    if (!encode(&a.a[0], a0, a_rows) || !encode(&a.a[1], a1, a_rows) || !encode(&a.b[0], b0, b_rows) ||
        !encode(&a.b[1], b1, b_rows))
      return fail(FSDP_ECUDA, "cuTensorMapEncodeTiled failed or is missing");
    cudaError_t e = status_word(&a.status);
    if (e != cudaSuccess) return fail(FSDP_ECUDA, std::string("status word: ") + cudaGetErrorString(e));
    a.wait_limit_ns = wait_limit_ns();
    a.fault = wait_fault();
    a.act = d->activation == FSDP_ACT_SILU ? SILU : GELU;
    a.m_tiles = (int32_t)t.m_tiles, a.n_tiles = (int32_t)t.n_tiles, a.splits = (int32_t)t.splits;
    a.raster = 16;
    a.m_half = (int32_t)t.m_half;
    a.k_blocks = (int32_t)t.k_blocks, a.k_half = (int32_t)(t.k_blocks / 2);
    a.m = m, a.n = n;
    if (t.splits > 1) a.partial = reinterpret_cast<float *>(ws + plan.at_partial);
    fsdp_status_t st = launched(launch_product(mode, t.pair, a, plan.sms, stream));
    if (st != FSDP_OK || t.splits == 1) return st;
    JoinArgs j = {};
    j.partial = a.partial;
    j.out[0] = a.out[0], j.out[1] = a.out[1];
    j.ld[0] = a.ld_out[0], j.ld[1] = a.ld_out[1];
    j.rows = mode == DW ? 2 * m : m, j.half = m, j.cols = n;
    j.splits = (int32_t)t.splits, j.bf16 = a.out_bf16;
    j.vec = a.out_width >= 16;
    void *args[] = {&j};
    const int vec = n % 4 == 0 ? 4 : 1;
    int64_t across = blocks_of(n, (int64_t)kThreads * vec), down = j.rows;
    if (across > 64) across = 64;
    if (down > plan.sms * 64) down = plan.sms * 64;
    return launched(launch_kernel(vec == 4 ? reinterpret_cast<const void *>(&join_kernel<4>)
                                           : reinterpret_cast<const void *>(&join_kernel<1>),
                                  dim3((unsigned)down, (unsigned)across), dim3(kThreads), args, 0, stream, true));
  }
};

void kept_into(const fsdp_ffn_desc_t *d, void *gate, void *up, Args &a) {
  a.keep = d->keep;
  a.groups = act8_groups(d->f);
  void *p[2] = {gate, up};
  for (int i = 0; i < 2; ++i) {
    a.codes[i] = static_cast<uint8_t *>(p[i]);
    a.scales[i] = a.codes[i] ? a.codes[i] + d->rows * a.groups * kActGroup : nullptr;
    a.kept[i] = p[i];
  }
  a.ld_kept = d->ld_kept;
  const int64_t ld = d->keep == FSDP_KEEP_ACT8 ? 16 : d->ld_kept;  // a checkpoint's groups are 32 bytes each
  const int wg = row_width(gate, d->rows, ld, 2), wu = row_width(up, d->rows, ld, 2);
  a.keep_width = wg < wu ? wg : wu;
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
  if (d->rows > 0) {
    if ((st = c.stage(x, w_gate, w_up)) != FSDP_OK) return st;
    Args a = {};
    a.out[0] = h, a.ld_out[0] = d->ld_h;
    a.out_bf16 = 1, a.out_width = row_width(h, d->rows, d->ld_h, 2);
    kept_into(d, gate, up, a);
    if ((st = c.product(FORWARD, d->rows, d->f, d->d, c.x, c.x, c.wg, c.wu, a)) != FSDP_OK) return st;
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
    a.out_bf16 = 1, a.out_width = row_width(c.ws, d->rows, c.plan.f_pitch, 2);
    a.dh = dh, a.ld_dh = d->ld_h, a.dh_vec = vec_rows(dh, d->rows, d->ld_h, 2);
    if ((st = c.product(RECOMPUTE, d->rows, d->f, d->d, c.x, c.x, c.wg, c.wu, a)) != FSDP_OK) return st;
  } else {
    SlopeArgs s = {};
    s.dh = dh, s.gate = gate, s.up = up;
    s.groups = act8_groups(d->f);
    s.act8 = d->keep == FSDP_KEEP_ACT8;
    const void *p[2] = {gate, up};
    for (int i = 0; i < 2; ++i) s.scales[i] = static_cast<const uint8_t *>(p[i]) + d->rows * s.groups * kActGroup;
    s.dg = dg, s.du = du;
    s.rows = d->rows, s.f = d->f, s.ld_dh = d->ld_h, s.ld_kept = d->ld_kept, s.pitch = c.plan.f_pitch;
    s.act = d->activation == FSDP_ACT_SILU ? SILU : GELU;
    s.dh_vec = vec_rows(dh, d->rows, d->ld_h, 2);
    s.kept_vec = vec_rows(gate, d->rows, d->ld_kept, 2) && vec_rows(up, d->rows, d->ld_kept, 2);
    int64_t grid = blocks_of(d->rows * blocks_of(d->f, 8), kThreads);
    if (grid > (int64_t)c.plan.sms * 64) grid = (int64_t)c.plan.sms * 64;
    void *args[] = {&s};
    st = launched(launch_kernel(reinterpret_cast<const void *>(&slope_kernel), dim3((unsigned)grid), dim3(kThreads), args, 0,
                                c.stream, true));
    if (st != FSDP_OK) return st;
  }
  const Operand og = {dg, d->rows, d->f, c.plan.f_pitch}, ou = {du, d->rows, d->f, c.plan.f_pitch};
  if (dx) {
    Args a = {};
    a.out[0] = a.out[1] = dx;
    a.ld_out[0] = a.ld_out[1] = d->ld_dx;
    a.out_bf16 = d->dx_dtype == FSDP_DTYPE_BF16;
    a.out_width = row_width(dx, d->rows, d->ld_dx, xsize);
    if ((st = c.product(DX, d->rows, d->d, d->f, og, ou, c.wg, c.wu, a)) != FSDP_OK) return st;
  }
  if (dw_gate) {
    Args a = {};
    a.out[0] = dw_gate, a.out[1] = dw_up;
    a.ld_out[0] = d->ld_dw_gate, a.ld_out[1] = d->ld_dw_up;
    a.out_bf16 = d->dw_dtype == FSDP_DTYPE_BF16;
    const int rg = row_width(dw_gate, d->f, d->ld_dw_gate, wsize), ru = row_width(dw_up, d->f, d->ld_dw_up, wsize);
    a.out_width = rg < ru ? rg : ru;
    if ((st = c.product(DW, d->f, d->d, d->rows, og, ou, c.x, c.x, a)) != FSDP_OK) return st;
  }
  clear_error();
  return FSDP_OK;
}

}  // extern "C"

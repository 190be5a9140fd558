// Losses over rows of logits (fsdp_distill_loss_*, fsdp_policy_loss_*).
//
// A block to a row, which it reads once for the sum of exponentials and once more for the
// gradient.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <string>

#include "layout.h"
#include "ops.h"

namespace fsdp {
namespace loss {
namespace {

constexpr int kThreads = 256, kMaxTop = FSDP_DISTILL_MAX_TOP;

struct Args {
  const void *logits;
  void *dlogits;
  const void *tokens, *teacher;
  const float *old_logp, *ref_logp, *advantage, *weight, *dloss, *lse_in, *logp_in;
  float *loss, *logp, *lse;
  int64_t rows, ld_z, ld_g, ld_tokens, ld_teacher;
  int32_t vocab, top, z_bf16, g_bf16, teacher_bf16, wide, backward;
  float t, inv_t, low, high, kl;
};

__device__ __forceinline__ float block_sum(float v, bool take_max, float *part) {
  for (int m = 16; m > 0; m /= 2) {
    const float o = __shfl_xor_sync(0xFFFFFFFFu, v, m);
    v = take_max ? fmaxf(v, o) : v + o;
  }
  __syncthreads();
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
  __syncthreads();
  v = part[0];
  for (int w = 1; w < kThreads / 32; ++w) v = take_max ? fmaxf(v, part[w]) : v + part[w];
  return v;
}

__device__ __forceinline__ int64_t token_at(const Args &a, int64_t i) {
  const int64_t t = a.wide ? static_cast<const int64_t *>(a.tokens)[i] : static_cast<const int32_t *>(a.tokens)[i];
  return t >= 0 && t < a.vocab ? t : -1;
}

template <bool DISTILL>
__global__ void __launch_bounds__(kThreads) row_kernel(const __grid_constant__ Args a) {
  __shared__ float part[kThreads / 32];
  __shared__ int32_t ids[DISTILL ? kMaxTop : 1];
  __shared__ float q[DISTILL ? kMaxTop : 1], zt[DISTILL ? kMaxTop : 1];
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const float w = a.weight ? a.weight[row] : 1.0f;
    const int64_t z0 = row * a.ld_z, g0 = row * a.ld_g;
    if (w == 0.0f) {
      if (threadIdx.x == 0 && !a.backward) {
        a.loss[row] = 0.0f, a.lse[row] = 0.0f;
        if (!DISTILL) a.logp[row] = 0.0f;
      }
      for (int32_t i = threadIdx.x; a.dlogits && i < a.vocab; i += kThreads) store_any(a.dlogits, g0 + i, a.g_bf16, 0.0f);
      continue;
    }
    float lse;
    if (a.backward) {
      lse = a.lse_in[row];
    } else {
      float top = -INFINITY;
      bool nan = false;
      for (int32_t i = threadIdx.x; i < a.vocab; i += kThreads) {
        const float z = load_any(a.logits, z0 + i, a.z_bf16) * a.inv_t;
        top = fmaxf(top, z);
        nan |= z != z;
      }
      top = block_sum(top, true, part);
      float sum = nan ? NAN : 0.0f;
      const float nans = block_sum(sum, false, part);
      for (int32_t i = threadIdx.x; i < a.vocab; i += kThreads) sum += expf(load_any(a.logits, z0 + i, a.z_bf16) * a.inv_t - top);
      sum = block_sum(sum, false, part);
      lse = nans != nans ? nans : top == -INFINITY ? top : top + logf(sum);
      if (threadIdx.x == 0) a.lse[row] = lse;
    }
    float slope = 0.0f, mass = 0.0f;  // dz_i = slope (mass p_i - q_i)
    int64_t token = -1;
    float zq = 0.0f;
    const float up = w * (a.backward && a.dloss ? a.dloss[row] : 1.0f);
    if constexpr (DISTILL) {
      float top = -INFINITY;
      __syncthreads();
      for (int k = threadIdx.x; k < a.top; k += kThreads) {
        const int64_t t = token_at(a, row * a.ld_tokens + k);
        const float v = t < 0 ? -INFINITY : load_any(a.teacher, row * a.ld_teacher + k, a.teacher_bf16) * a.inv_t;
        ids[k] = v == -INFINITY ? -1 : (int32_t)t;
        q[k] = v;
        zt[k] = ids[k] < 0 ? 0.0f : load_any(a.logits, z0 + t, a.z_bf16) * a.inv_t;
        top = fmaxf(top, v);
      }
      top = block_sum(top, true, part);
      float sum = 0.0f;
      for (int k = threadIdx.x; k < a.top; k += kThreads)
        if (ids[k] >= 0) sum += expf(q[k] - top);
      sum = block_sum(sum, false, part);
      float l = 0.0f;
      for (int k = threadIdx.x; k < a.top; k += kThreads)
        if (ids[k] >= 0) {
          const float lq = q[k] - top - logf(sum), p = expf(lq);
          q[k] = p;
          if (p > 0.0f || p != p) l += p * (lq - zt[k] + lse);
        }
      l = block_sum(l, false, part);
      if (threadIdx.x == 0 && !a.backward) a.loss[row] = w * a.t * a.t * l;
      mass = sum > 0.0f || sum != sum ? 1.0f : 0.0f;
      slope = up * a.t;
    } else {
      token = token_at(a, row);
      if (token >= 0) {
        zq = load_any(a.logits, z0 + token, a.z_bf16) * a.inv_t;
        const float logp = a.backward ? a.logp_in[row] : zq - lse;
        const float r = a.old_logp ? expf(logp - a.old_logp[row]) : 1.0f, adv = a.advantage[row];
        const float held = fminf(fmaxf(r, a.low), a.high);
        const float gap = a.ref_logp ? a.ref_logp[row] - logp : 0.0f;
        if (threadIdx.x == 0 && !a.backward) {
          a.logp[row] = logp;
          a.loss[row] = w * (-fminf(r * adv, held * adv) + (a.ref_logp ? a.kl * (expm1f(gap) - gap) : 0.0f));
        }
        slope = -((r * adv <= held * adv ? -r * adv : 0.0f) + (a.ref_logp ? -a.kl * expm1f(gap) : 0.0f)) * up * a.inv_t;
        mass = 1.0f;
      } else if (threadIdx.x == 0 && !a.backward) {
        a.logp[row] = 0.0f, a.loss[row] = 0.0f;
      }
    }
    if (!a.dlogits) continue;
    __syncthreads();  // every thread has read what it needs of a row that may be overwritten
    for (int32_t i = threadIdx.x; i < a.vocab; i += kThreads) {
      const float p = mass != 0.0f ? expf(load_any(a.logits, z0 + i, a.z_bf16) * a.inv_t - lse) : 0.0f;
      store_any(a.dlogits, g0 + i, a.g_bf16, mass != 0.0f ? slope * (p - (i == token ? 1.0f : 0.0f)) : 0.0f);
    }
    if constexpr (DISTILL) {
      __syncthreads();
      for (int k = threadIdx.x; k < a.top; k += kThreads) {
        if (ids[k] < 0) continue;
        float s = 0.0f;
        bool first = true;
        for (int m = 0; m < a.top; ++m)
          if (ids[m] == ids[k]) {
            first &= m >= k;
            s += q[m];
          }
        if (first) store_any(a.dlogits, g0 + ids[k], a.g_bf16, slope * (expf(zt[k] - lse) - s));
      }
    }
  }
}

template <bool DISTILL>
fsdp_status_t run(Args &a, cudaStream_t s) {
  void *args[] = {&a};
  const int64_t grid = std::min<int64_t>(a.rows, 1 << 20);
  return launched(launch_kernel(reinterpret_cast<const void *>(&row_kernel<DISTILL>), dim3((unsigned)grid), dim3(kThreads), args, 0, s));
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
  if (d->vocab > INT32_MAX) return fail(FSDP_EUNSUPPORTED, "a vocabulary of 2^31 or more");
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

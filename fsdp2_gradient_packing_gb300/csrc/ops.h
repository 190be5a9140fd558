// Host and device helpers shared by the training operators (fsdp_ops.h).
// Included by .cu files only; not part of the C ABI.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <string>

#include "act8.h"
#include "layout.h"

namespace fsdp {

// The current device's word in which kernels record waits that gave up.
cudaError_t status_word(uint32_t **word);

// SMs of the current device (cached per device); 0 if there is none.
int device_sms();

inline bool float_dtype(int32_t dt) { return dt == FSDP_DTYPE_F32 || dt == FSDP_DTYPE_BF16; }

// A matrix argument: `bytes` 0 stands for an empty one.
fsdp_status_t check_matrix(const void *p, int64_t rows, int64_t cols, int64_t ld, int64_t size, const char *what);

inline fsdp_status_t launched(cudaError_t e) {
  if (e != cudaSuccess) return fail(FSDP_ECUDA, std::string("kernel launch failed: ") + cudaGetErrorString(e));
  return FSDP_OK;
}

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

// Launch, optionally letting it start while the previous kernel on the stream
// drains (such kernels call wait_for_previous() before they touch memory), and
// optionally in clusters along x.
cudaError_t launch_kernel(const void *fn, dim3 grid, dim3 block, void **args, size_t smem, cudaStream_t stream,
                          bool overlap = false, int cluster = 1);

#ifdef __CUDACC__
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ float bf16_low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_high(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Two binary32 values rounded to BF16 (nearest, ties to even), a in the low half.
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
  return d;
}

// Element j of a vector or matrix row whose dtype is known at run time.
__device__ __forceinline__ float load_any(const void *p, int64_t j, bool bf16) {
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[j]) : static_cast<const float *>(p)[j];
}
__device__ __forceinline__ void store_any(void *p, int64_t j, bool bf16, float v) {
  if (bf16)
    static_cast<__nv_bfloat16 *>(p)[j] = __float2bfloat16_rn(v);
  else
    static_cast<float *>(p)[j] = v;
}

// Eight consecutive elements, 16-byte aligned, of either dtype.
__device__ __forceinline__ void store8(void *p, int64_t j, bool bf16, const float (&v)[8]) {
  if (bf16) {
    *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p) + j) =
        make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7]));
  } else {
    float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(p) + j);
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}
__device__ __forceinline__ void unpack8(uint4 r, float (&v)[8]) {
  v[0] = bf16_low(r.x), v[1] = bf16_high(r.x), v[2] = bf16_low(r.y), v[3] = bf16_high(r.y);
  v[4] = bf16_low(r.z), v[5] = bf16_high(r.z), v[6] = bf16_low(r.w), v[7] = bf16_high(r.w);
}
__device__ __forceinline__ void load8(const void *p, int64_t j, bool bf16, float (&v)[8]) {
  if (bf16) {
    unpack8(*reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p) + j), v);
  } else {
    const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + j);
    const float4 a = q[0], b = q[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
}
#endif

}  // namespace fsdp

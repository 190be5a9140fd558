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

// The current device's counts of blocks whose waits gave up, by kind of kernel.  Kernels
// add to them and nothing takes away, so no failure is lost between a read and a reset;
// who asks (fsdp_ops_sync_status) remembers what it has seen.
enum GaveUp { GAVE_UP_PRODUCT = 0, GAVE_UP_NORM = 1, GAVE_UP_KINDS = 2 };
cudaError_t gave_up_count(GaveUp kind, uint32_t **count);

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

// Widest store that every row's start allows: 32, 16 or 0 bytes (elements one by one).
inline int row_width(const void *p, int64_t rows, int64_t ld, int64_t size) {
  for (int w = 32; w >= 16; w /= 2)
    if ((uintptr_t)p % w == 0 && (rows <= 1 || ld * size % w == 0)) return w;
  return 0;
}

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

// One whole 32-byte sector.
__device__ __forceinline__ void store32(void *p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Eight consecutive elements as four pairs, 16-byte aligned, of either dtype.
__device__ __forceinline__ void store8(void *p, int64_t j, bool bf16, const float2 (&v)[4]) {
  if (bf16) {
    *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p) + j) =
        make_uint4(bf16_pair(v[0].x, v[0].y), bf16_pair(v[1].x, v[1].y), bf16_pair(v[2].x, v[2].y), bf16_pair(v[3].x, v[3].y));
  } else {
    float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(p) + j);
    q[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    q[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
  }
}
__device__ __forceinline__ void unpack8(uint4 r, float2 (&v)[4]) {
  v[0] = make_float2(bf16_low(r.x), bf16_high(r.x)), v[1] = make_float2(bf16_low(r.y), bf16_high(r.y));
  v[2] = make_float2(bf16_low(r.z), bf16_high(r.z)), v[3] = make_float2(bf16_low(r.w), bf16_high(r.w));
}
__device__ __forceinline__ void load8(const void *p, int64_t j, bool bf16, float2 (&v)[4]) {
  if (bf16) {
    unpack8(*reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p) + j), v);
  } else {
    const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + j);
    const float4 a = q[0], b = q[1];
    v[0] = make_float2(a.x, a.y), v[1] = make_float2(a.z, a.w), v[2] = make_float2(b.x, b.y), v[3] = make_float2(b.z, b.w);
  }
}
// Element e of pairs, for code that goes element by element.
template <int N>
__device__ __forceinline__ float &element(float2 (&v)[N], int e) {
  return e % 2 ? v[e / 2].y : v[e / 2].x;
}
template <int N>
__device__ __forceinline__ float element(const float2 (&v)[N], int e) {
  return e % 2 ? v[e / 2].y : v[e / 2].x;
}
#endif

}  // namespace fsdp

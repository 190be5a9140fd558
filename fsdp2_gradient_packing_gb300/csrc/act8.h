// Device side of the 8-bit activation checkpoint format (fsdp_ops.h), shared
// by the store / load kernels (act8.cu), the layer norm (norm_*.cu) and the
// gated feed-forward block (ffn*.cu).  Included by .cu files only.
#pragma once

#include <cstdint>

#include "fsdp_ops.h"

namespace fsdp {

constexpr int64_t kActGroup = FSDP_ACT8_GROUP;
inline __host__ __device__ int64_t act8_groups(int64_t cols) { return (cols + kActGroup - 1) / kActGroup; }
inline int64_t act8_bytes(int64_t rows, int64_t cols) { return rows * act8_groups(cols) * (kActGroup + 1); }

#ifdef __CUDACC__
// Scale byte of a group from the bits of its largest magnitude.  A binary32
// m * 2^k with m in [1, 2) is at most 127 * 2^e = (127/64) * 2^(e+6) when
// e >= k - 6 and m <= 127/64, whose mantissa field is 0x7E0000: adding 0x1FFFF
// carries into the exponent exactly when the field is above that.  The largest
// of the bits with the sign off orders NaN above infinity above every finite
// value, so one integer maximum also finds a group that is not finite.
__device__ __forceinline__ uint32_t act8_scale_byte(uint32_t top_bits) {
  if (top_bits >= 0x7F800000u) return 255u;
  const int s = (int)((top_bits + 0x1FFFFu) >> 23) - 6;
  return (uint32_t)(s < 1 ? 1 : s);
}

// 2^-e for the scale byte e + 127 (at most 249 for a finite group); 0 for 255,
// which leaves the codes to act8_code's own test.
__device__ __forceinline__ float act8_inverse(uint32_t s) {
  return s == 255u ? 0.0f : __uint_as_float((254u - s) << 23);
}

// 2^e for the scale byte; infinity for 255, whose product with a code 0 is NaN.
__device__ __forceinline__ float act8_scale(uint32_t s) { return __uint_as_float(s << 23); }

// The two scale bytes whose codes need care: 255 (a group that is not finite),
// and 249 (2^122, the largest of a finite group), where 64 * 2^122 would read
// back as infinity.
constexpr uint32_t kActTopScale = 249u;

// Code of x in its group's scale: the product with a power of two is exact (or so
// far below one half that its rounding is 0 either way), so this is the one
// rounding.  Adding and subtracting 1.5 * 2^23 would round a binary32 below 2^22
// to the nearest integer, ties to even; the sum alone already holds that integer
// in its low bits, and so the code in two's complement in its low byte.
__device__ __forceinline__ uint32_t act8_code(float x, uint32_t s) {
  uint32_t c = __float_as_uint(__fadd_rn(__fmul_rn(x, act8_inverse(s)), 12582912.0f)) & 0xFFu;
  if (s >= kActTopScale) {
    const int v = (int)(int8_t)c;
    c = s == kActTopScale ? (uint32_t)(v > 63 ? 63 : v < -63 ? -63 : v) & 0xFFu : 0u;
  }
  return c;
}

// Four codes as the bytes of one word, element 0 lowest.
__device__ __forceinline__ uint32_t act8_code4(float a, float b, float c, float d, uint32_t s) {
  return act8_code(a, s) | act8_code(b, s) << 8 | act8_code(c, s) << 16 | act8_code(d, s) << 24;
}

// Value of the code in byte `i` of a word.
__device__ __forceinline__ float act8_value(uint32_t word, int i, float scale) {
  return __fmul_rn((float)(int8_t)(word >> (8 * i)), scale);
}
#endif

}  // namespace fsdp

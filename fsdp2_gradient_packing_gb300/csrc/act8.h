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

// Codes of four elements as the bytes of one word, element 0 lowest.  x * 2^-e is
// exact (or so far below one half that its rounding is 0 either way), so the fused
// sum with 1.5 * 2^23 rounds once: to the nearest integer, ties to even, which it
// holds in its low bits, and so the code in two's complement in its low byte.
// Arithmetic here and in the kernels is on pairs: the SM issues one instruction for
// the two, and these kernels are bound by what they issue before they are by HBM.
__device__ __forceinline__ uint32_t act8_code4(float2 a, float2 b, float inverse) {
  const float2 i = make_float2(inverse, inverse), shift = make_float2(12582912.0f, 12582912.0f);
  const float2 p = __ffma2_rn(a, i, shift), q = __ffma2_rn(b, i, shift);
  return __byte_perm(__byte_perm(__float_as_uint(p.x), __float_as_uint(p.y), 0x0040),
                     __byte_perm(__float_as_uint(q.x), __float_as_uint(q.y), 0x0040), 0x5410);
}

// What scale bytes 249 and 255 make of a word of codes (see kActTopScale).
__device__ __forceinline__ uint32_t act8_limit4(uint32_t codes, uint32_t s) {
  uint32_t w = 0;
  if (s == kActTopScale)
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
      const int v = (int)(int8_t)(codes >> (8 * i));
      w |= ((uint32_t)(v > 63 ? 63 : v < -63 ? -63 : v) & 0xFFu) << (8 * i);
    }
  return w;
}

// Stores the codes of N consecutive elements (4, 8 or 32) in their group's scale.
// The two special scales mend what was stored, in a loop: kept inline in the main
// path, their code cost the tensor-core epilogue two thirds of its speed.
template <int N>
__device__ __forceinline__ void act8_store(uint8_t *to, const float2 (&v)[N / 2], uint32_t s, bool sector = false) {
  const float inverse = act8_inverse(s);
  uint32_t w[N / 4];
#pragma unroll
  for (int i = 0; i < N / 4; ++i) w[i] = act8_code4(v[2 * i], v[2 * i + 1], inverse);
  if constexpr (N == 4) {
    *reinterpret_cast<uint32_t *>(to) = w[0];
  } else if constexpr (N == 8) {
    *reinterpret_cast<uint2 *>(to) = make_uint2(w[0], w[1]);
  } else if (sector) {  // 32-byte aligned
    static_assert(N == 4 || N == 8 || N == 32, "4, 8 or 32 codes");
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < N / 16; ++i)
      reinterpret_cast<uint4 *>(to)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
  if (s >= kActTopScale) {
    volatile uint32_t *p = reinterpret_cast<volatile uint32_t *>(to);
#pragma unroll 1
    for (int i = 0; i < N / 4; ++i) p[i] = act8_limit4(p[i], s);
  }
}
__device__ __forceinline__ uint32_t act8_code(float x, uint32_t s) {
  const uint32_t c = act8_code4(make_float2(x, 0.0f), make_float2(0.0f, 0.0f), act8_inverse(s));
  return (s >= kActTopScale ? act8_limit4(c, s) : c) & 0xFFu;
}

// Bits of the largest magnitude, a NaN's where there is one.
template <int PAIRS>
__device__ __forceinline__ uint32_t act8_top(const float2 (&v)[PAIRS]) {
  constexpr int kChains = PAIRS < 4 ? 1 : PAIRS < 16 ? 2 : 4;  // side by side, each step waits for the one before
  float top[kChains] = {};
#pragma unroll
  for (int i = 0; i < PAIRS; ++i) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(top[i % kChains]), "f"(fabsf(v[i].x)), "f"(fabsf(v[i].y)));
    top[i % kChains] = r;
  }
#pragma unroll
  for (int i = 1; i < kChains; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(top[0]) : "f"(top[i]));
  return __float_as_uint(top[0]);
}

// Codes of a word, made unsigned once for act8_value: code + 128 in each byte.
__device__ __forceinline__ uint32_t act8_biased(uint32_t codes) { return codes ^ 0x80808080u; }

// Codes 2 i and 2 i + 1 of a biased word: a byte becomes the low mantissa of 2^23, whose
// difference to 2^23 + 128 is the code, exactly.
__device__ __forceinline__ float2 act8_codes_of(uint32_t biased, int i) {
  return __fadd2_rn(make_float2(__uint_as_float(__byte_perm(biased, 0x4B000000u, 0x7440 + 2 * i)),
                                __uint_as_float(__byte_perm(biased, 0x4B000000u, 0x7441 + 2 * i))),
                    make_float2(-8388736.0f, -8388736.0f));
}
// Value of code 0 of a biased word; the product with a power of two is exact.
__device__ __forceinline__ float act8_value(uint32_t biased, float scale) { return act8_codes_of(biased, 0).x * scale; }
#endif

}  // namespace fsdp

// i8.hpp -- rounding to 8-bit codes, shared by the activation quantizer and
// the cache append.
#pragma once

#include "common.hpp"

namespace md {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// rint(x / s) for finite x and s > 0 with |x / s| < 256, ties to even, clamped
// to -127..127, exactly: a product with 1 / s gives the integer or its
// neighbour, and the sign of the fused x - (n +- 1/2) s (one rounding, so never
// wrong) says on which side of the two borders x lies.  s is at least 2^-100
// here (tiny magnitudes are scaled up first), so nothing underflows.
MD_DEV int code_of(float x, float s, float inv) {
  float n = rintf(x * inv);
  const float hi = fmaf(-(n + 0.5f), s, x), lo = fmaf(-(n - 0.5f), s, x);
  const bool odd = ((int)n) & 1;
  if (hi > 0.0f || (hi == 0.0f && odd)) n += 1.0f;
  else if (lo < 0.0f || (lo == 0.0f && odd)) n -= 1.0f;
  return (int)fminf(fmaxf(n, -127.0f), 127.0f);
}

// Values whose largest magnitude is below 2^-60 are scaled by 2^80 before
// their codes are formed (their step may be subnormal).
constexpr float kTiny = 0x1p-60f, kTinyUp = 0x1p80f;

template <int XT>
MD_DEV void load8(const void* x, int64_t i, float (&v)[8]) {
  if constexpr (XT == XF32) {
    const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(x) + i);
    const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(x) + i + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const u32x4 a = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(x) + i);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      v[2 * m] = __uint_as_float(a[m] << 16);
      v[2 * m + 1] = __uint_as_float(a[m] & 0xFFFF0000u);
    }
  }
}

MD_DEV uint16_t to_bf16(float f) {  // to nearest, ties to even; NaN stays NaN
  const uint32_t u = __float_as_uint(f);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0x7FC0;
  return (uint16_t)((u + 0x7FFFu + ((u >> 16) & 1u)) >> 16);
}

}  // namespace md

// i8.hpp -- rounding to 8-bit codes, shared by the activation quantizer and
// the cache append.
#pragma once

#include "common.hpp"

namespace md {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// Values whose largest magnitude is below 2^-60 are scaled by 2^80 before
// their codes are formed (their step may be subnormal).
constexpr float kTiny = 0x1p-60f, kTinyUp = 0x1p80f;

// A scale s as what turns values of magnitudes up to amax into codes.  s that
// is zero or NaN gives codes 0.
struct Step {
  float up, s, inv;
  bool none;
};
MD_DEV Step step_of(float s, float amax) {
  Step o;
  o.up = amax < kTiny && s < 1.0f ? kTinyUp : 1.0f;
  o.none = !(s > 0.0f);
  o.s = o.none ? 1.0f : s * o.up;
  o.inv = 1.0f / o.s;
  return o;
}

// x / s to the nearest integer, ties to even, clamped to -127..127, for eight
// finite x with |x / s| < 256, exactly: x (1 / s) is within 2^-15 of the
// quotient, so its integer is the one sought unless it lies next to a border
// k + 1/2.  There (one value in 5000) the sign of the fused x - (n +- 1/2) s,
// one rounding and so never wrong, says on which side of the borders x lies.
// s is at least 2^-100 here, so nothing underflows.
MD_DEV uint2 codes8(const float (&v)[8], const Step& s) {
  uint32_t w[2] = {0, 0};
  if (s.none) return make_uint2(0, 0);
  float n[8], far = 0.0f;
#pragma unroll
  for (int m = 0; m < 8; ++m) {
    const float r = v[m] * s.up * s.inv;
    n[m] = rintf(r);
    far = fmaxf(far, fabsf(r - n[m]));
  }
  if (far > 0.4999f) {
#pragma unroll
    for (int m = 0; m < 8; ++m) {
      const float x = v[m] * s.up, hi = fmaf(-(n[m] + 0.5f), s.s, x), lo = fmaf(-(n[m] - 0.5f), s.s, x);
      const bool odd = ((int)n[m]) & 1;
      if (hi > 0.0f || (hi == 0.0f && odd)) n[m] += 1.0f;
      else if (lo < 0.0f || (lo == 0.0f && odd)) n[m] -= 1.0f;
    }
  }
#pragma unroll
  for (int m = 0; m < 8; ++m)
    w[m >> 2] |= (uint32_t)((int)fminf(fmaxf(n[m], -127.0f), 127.0f) & 255) << (8 * (m & 3));
  return make_uint2(w[0], w[1]);
}

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

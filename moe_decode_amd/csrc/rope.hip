// rope.hip -- norms of queries and keys for each head and their rotation by
// position, in one pass over them.
//
//   z = x / sqrt(mean x^2 + eps) * w,  (y_a, y_b) = R(t) (z_a, z_b),  t = position * inv_freq
//
// Bound by memory: every value is read once and written once.  A wave takes one
// row and 64 / L of its heads at a time, L lanes a head and eight channels a
// lane, four pairs of them, so that a pair never leaves its lane and the sines
// and cosines, which all heads of a row share, are formed once for the lane's
// pairs and kept in registers over the row's heads.
//
// Measured: 8191 rows of 64 + 8 heads of 128, bf16, 62 us (302 MB, 4.9 TB/s, what a
// large copy reaches); one row of 32 + 4 heads of 64 3 us, its heads shared out over
// five workgroups.
#include <hip/hip_runtime.h>

#include "common.hpp"
#include "i8.hpp"
#include "kernels.hpp"

namespace md {

// cos and sin of r turns, r in 64 bits: whole quarter turns are taken off there
// (the angle of a position near 2^31 has 28 bits before its point, so fp32 would
// be lost), the rest, within an eighth of a turn, goes to the Taylor series in
// fp32: their next terms are below 2^-28.
MD_DEV void cos_sin(double r, float& c, float& s) {
  const double q = r * 4.0, n = rint(q);
  const float x = (float)((q - n) * 1.5707963267948966), x2 = x * x;
  const float sn = fmaf(x * x2, fmaf(x2, fmaf(x2, fmaf(x2, 2.7557319e-6f, -1.9841270e-4f), 8.3333333e-3f), -0.16666667f), x);
  const float cs = fmaf(x2, fmaf(x2, fmaf(x2, fmaf(x2, fmaf(x2, -2.7557319e-7f, 2.4801587e-5f), -1.3888889e-3f),
                                          4.1666667e-2f), -0.5f), 1.0f);
  const int k = (int)(int64_t)n & 3;
  const float a = k & 1 ? sn : cs, b = k & 1 ? cs : sn;
  c = k == 1 || k == 2 ? -a : a;
  s = k >= 2 ? -b : b;
}

template <int XT>
MD_DEV void load4(const void* p, int64_t i, float* v) {
  if constexpr (XT == XF32) {
    const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  } else {
    const uint2 a = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
    v[0] = __uint_as_float(a.x << 16); v[1] = __uint_as_float(a.x & 0xFFFF0000u);
    v[2] = __uint_as_float(a.y << 16); v[3] = __uint_as_float(a.y & 0xFFFF0000u);
  }
}

template <int YT>
MD_DEV void store4(void* p, int64_t i, float a, float b, float c, float d) {
  if constexpr (YT == XF32) *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(a, b, c, d);
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) =
        make_uint2(to_bf16(a) | (uint32_t)to_bf16(b) << 16, to_bf16(c) | (uint32_t)to_bf16(d) << 16);
}

// PAIRS: pairs of neighbours, the lane's channels 8 c .. 8 c + 7; else its four
// pairs p = 4 c .. are (p, p + rot / 2) below rot / 2, and behind the turned
// channels the rest is split into halves the same way (rot and the width are
// multiples of 8, so a lane's four stay together).
template <int L, bool PAIRS, int XT, int YT>
__global__ __launch_bounds__(256) void k_qk_norm_rope(RopeArgs g) {
  constexpr int HP = 64 / L;  // heads of a wave at a time
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row = (int64_t)blockIdx.x * 4 + wave;
  if (row >= g.rows) return;
  const int c = lane % L, hs = lane / L;
  const int D = g.D, rot = g.rot, heads = g.Hq + g.Hkv;
  const bool live = 8 * c < D;
  const int cc = live ? c : 0;
  int at_a, at_b;
  bool turned;
  if constexpr (PAIRS) {
    at_a = 8 * cc;
    at_b = at_a + 4;
    turned = 8 * cc < rot;
  } else {
    const int p = 4 * cc, t = p - rot / 2;
    turned = t < 0;
    at_a = turned ? p : rot + t;
    at_b = turned ? p + rot / 2 : rot + t + (D - rot) / 2;
  }
  float cs[4], sn[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) cs[i] = 1.0f, sn[i] = 0.0f;
  if (turned) {
    const double pos = (double)g.positions[row] * 0.15915494309189535;  // turns per radian
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      cos_sin(pos * (double)g.inv_freq[4 * cc + i], cs[i], sn[i]);
      cs[i] *= g.factor;
      sn[i] *= g.factor;
    }
  }
  const float inv_d = 1.0f / (float)D;
  const int per = (heads + HP - 1) / HP, each = (per + gridDim.y - 1) / gridDim.y;
  const int s0 = blockIdx.y * each, s1 = min(s0 + each, per);
  for (int st = s0; st < s1; ++st) {
    const int h = st * HP + hs;
    const bool here = live && h < heads, is_q = h < g.Hq;
    const int hh = is_q ? h : h - g.Hq;
    const void* x = is_q ? g.q : g.k;
    const int64_t at = row * (is_q ? g.q_stride : g.k_stride) + (int64_t)hh * D;
    float a[4] = {0.0f, 0.0f, 0.0f, 0.0f}, b[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (here) {
      load4<XT>(x, at + at_a, a);
      load4<XT>(x, at + at_b, b);
    }
    const float* w = is_q ? g.q_weight : g.k_weight;
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) ss = fmaf(a[i], a[i], fmaf(b[i], b[i], ss));
    ss = group_sum<L>(ss);
    if (here) {
      if (w) {
        const float r = 1.0f / sqrtf(fmaf(ss, inv_d, g.eps));
        float wa[4], wb[4];
        load4<XF32>(w, at_a, wa);
        load4<XF32>(w, at_b, wb);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[i] *= r * wa[i];
          b[i] *= r * wb[i];
        }
      }
      if constexpr (PAIRS) {  // a and b hold two pairs each
        if (turned) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float u = a[2 * i], v = a[2 * i + 1], y = b[2 * i], z = b[2 * i + 1];
            a[2 * i] = fmaf(u, cs[i], -(v * sn[i]));
            a[2 * i + 1] = fmaf(v, cs[i], u * sn[i]);
            b[2 * i] = fmaf(y, cs[2 + i], -(z * sn[2 + i]));
            b[2 * i + 1] = fmaf(z, cs[2 + i], y * sn[2 + i]);
          }
        }
      } else if (turned) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float u = a[i], v = b[i];
          a[i] = fmaf(u, cs[i], -(v * sn[i]));
          b[i] = fmaf(v, cs[i], u * sn[i]);
        }
      }
      void* y = is_q ? g.q_out : g.k_out;
      const int64_t to = row * (is_q ? g.q_out_stride : g.k_out_stride) + (int64_t)hh * D;
      store4<YT>(y, to + at_a, a[0], a[1], a[2], a[3]);
      store4<YT>(y, to + at_b, b[0], b[1], b[2], b[3]);
    }
  }
}

hipError_t launch_qk_norm_rope(const RopeArgs& g, bool pairs, int xt, int yt, hipStream_t st) {
  const int L = g.D <= 64 ? 8 : g.D <= 128 ? 16 : 32, HP = 64 / L;
  const int per = (g.Hq + g.Hkv + HP - 1) / HP;
  const int64_t groups = ((int64_t)g.rows + 3) / 4;
  // few rows: their heads are shared out among workgroups
  const int64_t want = 4 * (int64_t)device_cus();
  const int split = (int)(groups >= want ? 1 : groups * per <= want ? per : (want + groups - 1) / groups);
  const dim3 grid((unsigned)groups, split), block(256);
#define MD_ROPE(L_, P_, X_, Y_) hipLaunchKernelGGL((k_qk_norm_rope<L_, P_, X_, Y_>), grid, block, 0, st, g)
#define MD_ROPE_T(L_, P_)                                   \
  do {                                                      \
    if (xt == XF32) {                                       \
      if (yt == XF32) MD_ROPE(L_, P_, XF32, XF32);          \
      else MD_ROPE(L_, P_, XF32, XBF16);                    \
    } else {                                                \
      if (yt == XF32) MD_ROPE(L_, P_, XBF16, XF32);         \
      else MD_ROPE(L_, P_, XBF16, XBF16);                   \
    }                                                       \
  } while (0)
#define MD_ROPE_L(L_)             \
  do {                            \
    if (pairs) MD_ROPE_T(L_, true); \
    else MD_ROPE_T(L_, false);    \
  } while (0)
  if (L == 8) MD_ROPE_L(8);
  else if (L == 16) MD_ROPE_L(16);
  else MD_ROPE_L(32);
#undef MD_ROPE_L
#undef MD_ROPE_T
#undef MD_ROPE
  return hipGetLastError();
}

}  // namespace md

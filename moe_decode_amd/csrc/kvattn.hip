// kvattn.hip -- attention of a batch of ragged query runs over the paged 8-bit
// cache.
//
//   o = softmax(scale * q k^T + mask) v,   k = ks[page, head] K,  v = vs[page, head] V
//
// Both products run on the int8 matrix cores with the cache's codes as they
// lie in memory.  The other operand is split into balanced base-256 digits: a
// query row (one token, one head) as integers of 2^-23 of its largest
// magnitude (three digits; two for bf16 outputs: 2^-15), a softmax weight
// p in [0, 1] as integers of 2^-23 (2^-15).  Every digit's sum is exact in
// int32, so what is rounded is q, p, the joins of the digits and the softmax's
// fp32 arithmetic.
//
// Operand layout.  Keys enter as the A operand (rows = tokens), queries as B
// (columns = (query, head) pairs that share the key head), so the scores come
// out with a column's tokens in one lane: lane l holds column l % 16 and the
// rows 4 g + r, g = l / 16.  Row m of key tile j is token
// 16 (m / 4) + 4 j + m % 4 of the 64, which makes lane group g's sixteen scores
// the tokens 16 g .. 16 g + 15 -- exactly the 16 bytes of the contraction that
// the same lane feeds as the B operand of the second product, whose A operand
// is 16 consecutive tokens of a channel of the transposed values.  The weights
// never leave their lane: no LDS, no lane exchange but the row maximum's.
#include <hip/hip_runtime.h>

#include "common.hpp"
#include "i8.hpp"
#include "kernels.hpp"
#include "rows.hpp"
#include "kv.hpp"

namespace md {

constexpr int kTile = 64;  // tokens per step
constexpr int kWaves = 4;
constexpr float kLog2e = 1.4426950408889634f;

template <int ND>
struct Digits;
// q: |n| <= top, n + bias in bytes, digit = byte ^ 0x80; rows are scaled to
// qtop, since the fp32 factor and product may come out up to one integer
// higher, and one past top would wrap every digit.  p: 0 <= n <= top,
// top + pbias = 2^(8 ND - 1) - 1, so that one fma with 2^23 + pbias leaves the
// biased digits in the low bytes of the sum's bit pattern (the highest digit
// unbiased, 0..127).
template <>
struct Digits<3> {
  static constexpr float top = 8355711.0f, qtop = 8355704.0f;
  static constexpr int bias = 0x808080, pbias = 0x8080;
};
template <>
struct Digits<2> {
  static constexpr float top = 32639.0f, qtop = 32638.0f;
  static constexpr int bias = 0x8080, pbias = 0x80;
};

// Four integers' bytes k: dword of byte k of a, b, c, d.
MD_DEV uint32_t bytes4(uint32_t a, uint32_t b, uint32_t c, uint32_t d, int k) {
  const uint32_t sel = 0x0C0C0400u + 0x0101u * k;  // [a.k, b.k, 0, 0]
  const uint32_t lo = __builtin_amdgcn_perm(b, a, sel), hi = __builtin_amdgcn_perm(d, c, sel);
  return lo | hi << 16;
}

template <int ND>
MD_DEV float join(const i32x4 (&a)[ND], int r) {
  const int low = a[1][r] * 256 + a[0][r];
  if constexpr (ND == 2) return (float)low;
  else return fmaf((float)a[2][r], 65536.0f, (float)low);
}

template <int D, int ND>
__global__ __launch_bounds__(64 * kWaves, D == 256 ? 1 : 2) void k_kv_attn(KvAttn a) {
  constexpr int KS = D / 64, DT = D / 16;
  __shared__ __attribute__((aligned(16))) float s_acc[kWaves][16][D + 4];
  __shared__ float s_m[kWaves][16], s_l[kWaves][16];
  const KvCache& c = a.c;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, g = lane >> 4;
  const int split = blockIdx.x % a.splits, rest = blockIdx.x / a.splits;
  const int h = rest % c.Hkv, ct = rest / c.Hkv, s = blockIdx.y;
  const Seq q = seq_of(a.b, s, c.page);
  const int cols = q.nq * a.G;
  if (ct * 16 >= cols) return;
  const Span sp = span_of(a, q, ct * 16, min(ct * 16 + 16, cols));
  const int per = a.chunk, active = max(1, (sp.t1 - sp.t0 + per - 1) / per);
  if (split >= active) return;
  const int t_begin = sp.t0 + split * per, t_end = min(t_begin + per, sp.t1);

  // this lane's column: query t, head hq; past the last one the last one again
  const int cc = min(ct * 16 + col, cols - 1), qt = cc / a.G, hq = h * a.G + (cc - qt * a.G);
  const int64_t row = (int64_t)q.row0 + qt;
  const int pos = q.len - q.nq + qt;
  const int hi = a.causal ? pos : q.len - 1;                     // last position it sees
  const int lo = a.window ? max(pos - a.window + 1, 0) : 0;      // first

  // its digits
  i32x4 qd[ND][KS];
  float qs, poison = q.bad ? __uint_as_float(0x7FC00000u) : 0.0f;
  {
    float v[KS][16];
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float w[8];
        const int64_t at = row * a.q_stride + (int64_t)hq * D + 64 * k + 16 * g + 8 * e;
        if (a.xt == XF32) load8<XF32>(a.q, at, w);
        else load8<XBF16>(a.q, at, w);
#pragma unroll
        for (int m = 0; m < 8; ++m) {
          v[k][8 * e + m] = w[m];
          top = max(top, __float_as_uint(w[m]) & 0x7FFFFFFFu);
        }
      }
    float t = __uint_as_float(top);
    if (top >= 0x7F800000u) poison = __uint_as_float(0x7FC00000u), t = 0.0f;
    t = fmaxf(t, xor_lanes<16>(t));
    t = fmaxf(t, xor_lanes<32>(t));
    poison += xor_lanes<16>(poison);
    poison += xor_lanes<32>(poison);
    const float up = t >= 0x1p-100f ? Digits<ND>::qtop / t : 0.0f;
    qs = t * (1.0f / Digits<ND>::qtop);
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t n[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const float f = poison == poison ? v[k][4 * w + m] * up : 0.0f;
          n[m] = (uint32_t)(__float2int_rn(f) + Digits<ND>::bias);
        }
#pragma unroll
        for (int d = 0; d < ND; ++d) qd[d][k][w] = (int)(bytes4(n[0], n[1], n[2], n[3], d) ^ 0x80808080u);
      }
  }
  const float qscale = qs * a.scale * kLog2e;

  float m = -INFINITY, l = poison;
  float acc[DT][4];
#pragma unroll
  for (int i = 0; i < DT; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[i][r] = 0.0f;

  const int pshift = a.pshift;
  const int ktok = 16 * (col >> 2) + (col & 3);  // token of this lane's A row in key tile 0
  int id = t_begin + wave < t_end ? q.table[(t_begin + wave) * kTile >> pshift] : 0;
  for (int t = t_begin + wave; t < t_end; t += kWaves) {
    const int base = t * kTile, sub = base & ((1 << pshift) - 1);
    const int page = __builtin_amdgcn_readfirstlane(id);
    if (t + kWaves < t_end) id = q.table[(t + kWaves) * kTile >> pshift];
    if ((unsigned)page >= (unsigned)c.n_pages) {  // a page that is none: the rows that see it are NaN
      if (lo <= base + kTile - 1 && hi >= base) l = __uint_as_float(0x7FC00000u);
      continue;
    }
    const int64_t ph = (int64_t)page * c.Hkv + h;
    const int8_t* kp = c.k + (ph << pshift) * D + (int64_t)sub * D;
    const int8_t* vp = c.v + (ph << pshift) * D + sub;
    float ks = c.k_scale[ph], vs = c.v_scale[ph];
    i32x4 kf[4][KS], vf[DT];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int k = 0; k < KS; ++k)
        kf[j][k] = *reinterpret_cast<const i32x4*>(kp + (ktok + 4 * j) * D + 64 * k + 16 * g);
#pragma unroll
    for (int i = 0; i < DT; ++i)
      vf[i] = *reinterpret_cast<const i32x4*>(vp + ((int64_t)(16 * i + col) << pshift) + 16 * g);
    float off = 0.0f;  // NaN where a scale is not finite
    if (!(ks < INFINITY) || !(vs < INFINITY)) {
      off = __uint_as_float(0x7FC00000u);
      ks = vs = 0.0f;
    }
    float x[16];
    const float f = qscale * ks;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      i32x4 d[ND];
#pragma unroll
      for (int e = 0; e < ND; ++e) {
        d[e] = i32x4{0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < KS; ++k)
          d[e] = __builtin_amdgcn_mfma_i32_16x16x64_i8(kf[j][k], qd[e][k], d[e], 0, 0, 0);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) x[4 * j + r] = join(d, r) * f;
    }
    const int first = base + 16 * g;
    if (base + kTile - 1 > sp.full_hi || base < sp.full_lo) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (first + i > hi || first + i < lo) x[i] = -INFINITY;
    }
    float top = x[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) top = fmaxf(top, x[i]);
    if (top > -INFINITY) l += off;
    top = fmaxf(top, xor_lanes<16>(top));
    top = fmaxf(top, xor_lanes<32>(top));
    const float m1 = fmaxf(m, top), ref = m1 > -INFINITY ? m1 : 0.0f;
    const float alpha = __builtin_amdgcn_exp2f(m - ref);
    m = m1;
    uint32_t n[16];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float p = __builtin_amdgcn_exp2f(x[i] - ref);
      sum += p;
      n[i] = __float_as_uint(fmaf(p, Digits<ND>::top, 8388608.0f + (float)Digits<ND>::pbias));
    }
    l = fmaf(l, alpha, sum);
    i32x4 pd[ND];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < ND; ++e)
        pd[e][j] = (int)(bytes4(n[4 * j], n[4 * j + 1], n[4 * j + 2], n[4 * j + 3], e) ^
                         (e < ND - 1 ? 0x80808080u : 0u));
    const float vf32 = vs * (1.0f / Digits<ND>::top);
#pragma unroll
    for (int i = 0; i < DT; ++i) {
      i32x4 d[ND];
#pragma unroll
      for (int e = 0; e < ND; ++e)
        d[e] = __builtin_amdgcn_mfma_i32_16x16x64_i8(vf[i], pd[e], i32x4{0, 0, 0, 0}, 0, 0, 0);
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[i][r] = fmaf(join(d, r), vf32, acc[i][r] * alpha);
    }
  }
  l += xor_lanes<16>(l);
  l += xor_lanes<32>(l);

  // the waves' shares meet in LDS
#pragma unroll
  for (int i = 0; i < DT; ++i)
    *reinterpret_cast<float4*>(&s_acc[wave][col][16 * i + 4 * g]) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
  if (g == 0) {
    s_m[wave][col] = m;
    s_l[wave][col] = l;
  }
  __syncthreads();
  const int oc = threadIdx.x >> 4, part = threadIdx.x & 15;
  if (ct * 16 + oc >= cols) return;
  const int ot = (ct * 16 + oc) / a.G, oh = h * a.G + (ct * 16 + oc - ot * a.G);
  float mm = -INFINITY, w[kWaves], ll = 0.0f;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) mm = fmaxf(mm, s_m[i][oc]);
  const float ref = mm > -INFINITY ? mm : 0.0f;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    w[i] = __builtin_amdgcn_exp2f(s_m[i][oc] - ref);
    ll += w[i] > 0.0f || !(s_l[i][oc] == s_l[i][oc]) ? s_l[i][oc] * (w[i] > 0.0f ? w[i] : 1.0f) : 0.0f;
  }
  const int64_t orow = (int64_t)q.row0 + ot;
  const bool direct = active == 1;
  const float inv = direct ? (ll == 0.0f ? 0.0f : 1.0f / ll) : 1.0f;
  const int64_t slot = (orow * (a.G * c.Hkv) + oh) * a.splits + split;
#pragma unroll
  for (int i = 0; i < DT / 4; ++i) {
    const int d = 4 * part + 64 * i;
    float o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < kWaves; ++k)
#pragma unroll
      for (int r = 0; r < 4; ++r) o[r] = fmaf(w[k], s_acc[k][oc][d + r], o[r]);
    if (direct) store_out4(a, orow, oh, D, d, o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
    else *reinterpret_cast<float4*>(a.part + slot * D + d) = make_float4(o[0], o[1], o[2], o[3]);
  }
  if (!direct && part == 0) {
    a.part_m[2 * slot] = mm;
    a.part_m[2 * slot + 1] = ll;
  }
}

// The splits of a row: D / 4 lanes per (row, head), 1024 / D heads a workgroup.
__global__ __launch_bounds__(256) void k_kv_join(KvAttn a, int D) {
  const int s = blockIdx.z, head = blockIdx.y * (1024 / D) + (int)threadIdx.x / (D / 4), d = 4 * ((int)threadIdx.x % (D / 4));
  const Seq q = seq_of(a.b, s, a.c.page);
  if ((int)blockIdx.x >= q.nq || head >= a.G * a.c.Hkv) return;
  const int64_t row = (int64_t)q.row0 + blockIdx.x, slot0 = (row * (a.G * a.c.Hkv) + head) * a.splits;
  const int cols = q.nq * a.G, ct = ((int)blockIdx.x * a.G + head % a.G) / 16;
  const Span sp = span_of(a, q, ct * 16, min(ct * 16 + 16, cols));
  const int active = (sp.t1 - sp.t0 + a.chunk - 1) / a.chunk;
  if (active <= 1) return;
  float m = -INFINITY;
  for (int i = 0; i < active; ++i) m = fmaxf(m, a.part_m[2 * (slot0 + i)]);
  const float ref = m > -INFINITY ? m : 0.0f;
  float l = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int i = 0; i < active; ++i) {
    const float w = __builtin_amdgcn_exp2f(a.part_m[2 * (slot0 + i)] - ref), li = a.part_m[2 * (slot0 + i) + 1];
    l += li == li ? w * li : li;
    const float4 p = *reinterpret_cast<const float4*>(a.part + (slot0 + i) * D + d);
    o[0] = fmaf(w, p.x, o[0]);
    o[1] = fmaf(w, p.y, o[1]);
    o[2] = fmaf(w, p.z, o[2]);
    o[3] = fmaf(w, p.w, o[3]);
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  store_out4(a, row, head, D, d, o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
}

KvPlan kv_attn_plan(const KvCache& c, const KvBatch& b, int G, int window, int causal) {
  // enough workgroups to fill the chip several times over, of at least one
  // tile a wave; a split is a fixed number of tiles, so that in a ragged batch
  // every workgroup has the same work
  int64_t most = b.max_kv;
  if (causal && window && (int64_t)window + b.max_q < most) most = (int64_t)window + b.max_q;
  const int64_t tiles = (most + kTile - 1) / kTile + 1;
  const int64_t base = (int64_t)b.S * c.Hkv * (((int64_t)b.max_q * G + 15) / 16);
  int64_t chunk = (tiles * base + 1023) / 1024;
  if (chunk < kWaves) chunk = kWaves;
  KvPlan p;
  p.chunk = (int)(chunk < tiles ? chunk : tiles);
  p.splits = (int)((tiles + p.chunk - 1) / p.chunk);
  return p;
}

hipError_t launch_kv_attn(const KvAttn& a, int D, int yt, hipStream_t st) {
  const int64_t cts = ((int64_t)a.b.max_q * a.G + 15) / 16;
  const dim3 grid((unsigned)(a.splits * cts * a.c.Hkv), a.b.S), block(64 * kWaves);
#define MD_ATT(D_, N_) hipLaunchKernelGGL((k_kv_attn<D_, N_>), grid, block, 0, st, a)
  if (yt == XF32) {
    if (D == 64) MD_ATT(64, 3);
    else if (D == 128) MD_ATT(128, 3);
    else MD_ATT(256, 3);
  } else {
    if (D == 64) MD_ATT(64, 2);
    else if (D == 128) MD_ATT(128, 2);
    else MD_ATT(256, 2);
  }
#undef MD_ATT
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  hipLaunchKernelGGL(k_kv_join, dim3(a.b.max_q, (a.G * a.c.Hkv * D + 1023) / 1024, a.b.S), dim3(256), 0, st, a, D);
  return hipGetLastError();
}

}  // namespace md

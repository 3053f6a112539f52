// kvattn.hip -- attention of a batch of ragged query runs over the paged 8-bit
// cache.
//
//   o = softmax(scale * q k^T + mask) v,   k = ks[page, head] K,  v = vs[page, head] V
//
// Two forms, by the number of (query, head) columns that share a key head: for
// many of them see k_kv_attn_rows; for few, both products run on the int8 matrix
// cores with the cache's codes as they lie in memory.  The other operand is split
// into balanced base-256 digits: a query row (one token, one head) as integers of
// 2^-23 of its largest magnitude (three digits; two for bf16 outputs: 2^-15), a
// softmax weight as integers of 2^-23 of the largest one among its tile of 64
// tokens.  Every digit's sum is exact in int32, so what is rounded is q, p, the
// joins of the digits and the softmax's fp32 arithmetic.
//
// The weights' reference is the tile's own maximum, brought to the running one by
// a factor in fp32, and they have three digits whatever the output's type: the
// integers are steps of one size, so a weight far below the reference loses its
// bits, and where one key holds most of a row's weight (the first token, often)
// the rest of it is a long tail of such weights.  A tail of 2047 tokens beside a
// key of 0.97 of the weight, bf16 out: 0.2% off the definition (the output's
// rounding); 5% against the running maximum with two digits, one of 8191 24%.
//
// Masked calls (M: a tree of drafts, or a window with first positions that stay
// visible) take the same two forms; they differ in which tiles a column sees (kv.hpp:
// the first ones, then those of the window) and in how a cut tile's scores are
// masked: sixteen bits a lane, made of the row's borders and its words of the tree.
// They round their operands as plain calls do, for bf16 outputs more than for fp32
// ones: a query to two digits, or queries and weights to one f16.  That moves some
// outputs to a neighbouring bf16 value (2.5% of them, 9.6%) and their distance from
// the definition, which the output's own rounding makes, from 1.658e-3 of the
// outputs' size to 1.659e-3 and 1.671e-3 (rms; windows of 4096 and 1024 positions).
//
// Operand layout.  Keys enter as the A operand (rows = tokens), queries as B
// (columns = (query, head) pairs that share the key head), so the scores come
// out with a column's tokens in one lane: lane l holds column l % 16 and the
// rows 4 g + r, g = l / 16.  Of 64 tokens, rows 4 g .. 4 g + 3 of every key tile
// are some of 16 g .. 16 g + 15 (which: at the loads), so lane group g's sixteen
// scores are those tokens' -- exactly the 16 bytes of the contraction that
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
// higher, and one past top would wrap every digit.  p (kWeightDigits): 0 <= n <= top,
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
  static constexpr float qtop = 32638.0f;
  static constexpr int bias = 0x8080;
};
constexpr int kWeightDigits = 3;

// Byte k of four integers, as one dword, for every digit k < ND.
template <int ND>
MD_DEV void bytes4(uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t (&out)[ND]) {
  const uint32_t ab = __builtin_amdgcn_perm(b, a, 0x05010400u), cd = __builtin_amdgcn_perm(d, c, 0x05010400u);
  out[0] = __builtin_amdgcn_perm(cd, ab, 0x05040100u);  // a.0 b.0 c.0 d.0
  out[1] = __builtin_amdgcn_perm(cd, ab, 0x07060302u);
  if constexpr (ND == 3) {
    const uint32_t ab2 = __builtin_amdgcn_perm(b, a, 0x0C0C0602u), cd2 = __builtin_amdgcn_perm(d, c, 0x06020C0Cu);
    out[2] = ab2 | cd2;
  }
}

template <int ND>
MD_DEV float join(const i32x4 (&a)[ND], int r) {
  const int low = a[1][r] * 256 + a[0][r];
  if constexpr (ND == 2) return (float)low;
  else return fmaf((float)a[2][r], 65536.0f, (float)low);
}

template <int AUX>
MD_DEV i32x4 load16(rsrc_t r, int off, int soff) {
  const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(r, off, soff, AUX);
  return i32x4{(int)v[0], (int)v[1], (int)v[2], (int)v[3]};
}

// Inside a wave-uniform branch around cheap work: without it the compiler may
// turn the branch into selects that every tile pays for.
MD_DEV void keep_branch() { asm volatile(""); }

MD_DEV float nan_f() { return __uint_as_float(0x7FC00000u); }

// A column's query digits (the lane's 16 channels of each 64) and its state.
// The sign of the score scale goes into the digits, so that a tile's factor is
// never negative and the raw integer scores can be compared before they are
// scaled.
template <int D, int ND, bool M>
struct Column {
  i32x4 qd[ND][D / 64];
  float qscale, m, l;
  int hi, lo;  // the positions it sees
  Seen seen;   // M: instead of them
};
template <int D, int ND, bool M>
MD_DEV void column_init(Column<D, ND, M>& o, const KvAttn& a, const Seq& q, int h, int c, int cols, int g) {
  const int cc = min(c, cols - 1), qt = cc / a.G, hq = h * a.G + (cc - qt * a.G);  // past the last one: that one again
  const int pos = q.len - q.nq + qt;
  if constexpr (M) {
    o.seen = seen_of(a, q, qt);
  } else {
    o.hi = a.causal ? pos : q.len - 1;
    o.lo = a.window ? max(pos - a.window + 1, 0) : 0;
  }
  float v[D / 64][16], poison = q.bad ? nan_f() : 0.0f;
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < D / 64; ++k)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float w[8];
      const int64_t at = ((int64_t)q.row0 + qt) * a.q_stride + (int64_t)hq * D + 64 * k + 16 * g + 8 * e;
      if (a.xt == XF32) load8<XF32>(a.q, at, w);
      else load8<XBF16>(a.q, at, w);
#pragma unroll
      for (int m = 0; m < 8; ++m) {
        v[k][8 * e + m] = w[m];
        top = max(top, __float_as_uint(w[m]) & 0x7FFFFFFFu);
      }
    }
  float t = __uint_as_float(top);
  if (top >= 0x7F800000u) poison = nan_f(), t = 0.0f;
  t = fmaxf(t, xor_lanes<16>(t));
  t = fmaxf(t, xor_lanes<32>(t));
  poison += xor_lanes<16>(poison);
  poison += xor_lanes<32>(poison);
  const float up = t >= 0x1p-100f ? copysignf(Digits<ND>::qtop / t, a.scale) : 0.0f;
  o.qscale = t * (1.0f / Digits<ND>::qtop) * fabsf(a.scale) * kLog2e;
  o.m = -INFINITY;
  o.l = poison;
#pragma unroll
  for (int k = 0; k < D / 64; ++k)
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint32_t n[4], d[ND];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const float f = poison == poison ? v[k][4 * w + m] * up : 0.0f;
        n[m] = (uint32_t)(__float2int_rn(f) + Digits<ND>::bias);
      }
      bytes4<ND>(n[0], n[1], n[2], n[3], d);
#pragma unroll
      for (int e = 0; e < ND; ++e) o.qd[e][k][w] = (int)(d[e] ^ 0x80808080u);
    }
}

// A page's scales for a head.  One that the append does not write (negative,
// not finite, past 2^126) makes the rows that see the page NaN: off is added to their sums.
struct Scales {
  float ks, vs, off;
};
MD_DEV Scales scales_of(float ks, float vs) {
  const bool good = ks >= 0.0f && ks < 0x1p126f && vs >= 0.0f && vs < 0x1p126f;
  return Scales{good ? ks : 0.0f, good ? vs : 0.0f, good ? 0.0f : nan_f()};
}

// One tile's raw scores masked (where it is cut), the running maximum moved:
// returns alpha for what has been summed so far, beta for what the tile's weights
// give, and ref, the tile's own maximum, which they are relative to.
template <int D, int ND, bool M>
MD_DEV float advance(Column<D, ND, M>& o, const KvAttn& a, const Seq& q, float (&x)[16], float f, float off, bool cut,
                     int first, float& ref, float& beta) {
  if (cut) {
    keep_branch();
    if constexpr (M) {
      const uint32_t vis = seen16(a, q, o.seen, first);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (!(vis >> i & 1u)) x[i] = -INFINITY;
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (first + i > o.hi || first + i < o.lo) x[i] = -INFINITY;
    }
  }
  float raw = x[0];
#pragma unroll
  for (int i = 1; i < 16; ++i) raw = fmaxf(raw, x[i]);
  if (raw > -INFINITY) o.l += off;
  float top = raw * f;
  top = fmaxf(top, xor_lanes<16>(top));
  top = fmaxf(top, xor_lanes<32>(top));
  if (top == INFINITY) o.l = nan_f();
  ref = top > -INFINITY ? top : 0.0f;  // a tile that the column does not see: weights of 0
  const float m1 = fmaxf(o.m, top), run = m1 > -INFINITY ? m1 : 0.0f;
  const float alpha = __builtin_amdgcn_exp2f(o.m - run);
  beta = __builtin_amdgcn_exp2f(top - run);
  o.m = m1;
  return alpha;
}

// Sixteen raw scores to softmax weights and their digits, and the weights' sum.
// The fused product and subtraction may leave the largest one just above 0, so the
// weight is clamped to 1 (a digit past the top would wrap).
MD_DEV float weights(const float (&x)[16], float f, float ref, i32x4 (&pd)[kWeightDigits]) {
  using P = Digits<kWeightDigits>;
  float sum = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t n[4], d[kWeightDigits];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float p = __builtin_amdgcn_fmed3f(__builtin_amdgcn_exp2f(fmaf(x[4 * j + r], f, -ref)), 0.0f, 1.0f);
      sum += p;
      n[r] = __float_as_uint(fmaf(p, P::top, 8388608.0f + (float)P::pbias));
    }
    bytes4<kWeightDigits>(n[0], n[1], n[2], n[3], d);
#pragma unroll
    for (int e = 0; e < kWeightDigits; ++e) pd[e][j] = (int)(e < kWeightDigits - 1 ? d[e] ^ 0x80808080u : d[e]);
  }
  return sum;
}

// Few columns (decode): four waves take turns at the tiles of one column tile
// of 16 and meet in LDS.  Bound by the read of the cache: keys and values go
// from HBM straight into the matrix cores' operand registers, the next tile's
// keys while this one's weights are formed and summed, its values while the
// next one's scores are.
//
// A segment is the tiles of one sequence, key head and column tile.  Where
// segments are long (a.pieces > 0) the tiles of all of them, in order, are dealt
// out in equal runs to as many workgroups as run at once: a ragged batch
// leaves nobody waiting, whatever its lengths, which only the device knows.  A
// segment that one workgroup covers is written out, of the others each
// workgroup keeps at most its first and its last one's share in the workspace,
// and the one where a segment begins notes how many shares there are for
// k_kv_join_pieces.  Measured, with the join: 32 sequences of up to 8190 tokens,
// 64 heads on 8 of 128 channels, 65 us (289 MB, 4.4 TB/s; fixed shares of max_kv
// 76), two of up to 131071 on pages of 128 tokens 81 us (402 MB, 5.0 TB/s; 85).
// A form that only loaded took 5% less: it waits for memory.  Half, one and a
// half times and twice as many workgroups, when it took 67 and 83: 75, 77, 73
// and 81, 94, 89 us.

// Sequences, at most, that a workgroup sums up (8 bytes of LDS each).  In a larger
// batch every segment stays whole (one of 32768 tokens among 1024 sequences, 8
// heads on 1 of 64: 34 us; among 1025: 137).
constexpr int kMaxDealt = 1024;

// The tiles that any column of a sequence sees, one at least where it has rows:
// somebody has to write their zeros.
template <bool M>
MD_DEV int tiles_of(const KvAttn& a, const Seq& q, int cols, Span& s) {
  s = span_of<M>(a, q, 0, cols);
  return max(s.head + s.t1 - s.t0, 1);
}

template <int D, int ND>
struct FewLds {
  float acc[kWaves][16][D + 4];
  float m[kWaves][16], l[kWaves][16];
};

// Tiles [t_begin, t_end) of head h's column tile ct; M: numbered with the
// `head` first ones in front and `skip` left out behind them.  slot < 0: they
// are all that it sees, and the outputs are written; else the sums go to that
// slot.
template <int D, int ND, bool M>
MD_DEV void few_columns(const KvAttn& a, const Seq& q, int h, int ct, int cols, const Span& sp, int t_begin, int t_end,
                        int head, int skip, int slot, FewLds<D, ND>& lds) {
  constexpr int DT = D / 16;
  auto& s_acc = lds.acc;
  auto& s_m = lds.m;
  auto& s_l = lds.l;
  const KvCache& c = a.c;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, g = lane >> 4;
  const int pshift = a.pshift;
  // Rows of 128 bytes and more are loaded eight lanes a row, a whole line each:
  // lane (m, g) of load (i, k) takes token 16 (m / 4) + 2 i + (m / 2) % 2,
  // chunk 8 k + 4 (m % 2) + g.  As an A operand its even rows hold a token's
  // first 64 channels and its odd rows the next 64, so it is multiplied by both
  // halves of the query and every result uses every other row of each product
  // (the matrix cores have room; half-line loads cost 13% of the read rate).
  constexpr bool kWide = D > 64;
  constexpr int KI = kWide ? 8 : 4, KK = kWide ? D / 128 : 1;
  const int koff = kWide ? (16 * (col >> 2) + ((col >> 1) & 1)) * D + 64 * (col & 1) + 16 * g
                         : (16 * (col >> 2) + (col & 3)) * D + 16 * g;
  const int voff = (col << pshift) + 16 * g;
  i32x4 kf[KI][KK], vf[DT];
  auto tile_of = [&](int t) { return M && t >= head ? t + skip : t; };
  // a page that is none reads page 0 and counts as one with scale NaN
  auto page_at = [&](int t) { return t < t_end ? q.table[tile_of(t) * kTile >> pshift] : 0; };
  // buffer loads: past the last tile the resources are empty, and the same
  // loads read zeros without memory traffic
  auto load_k = [&](int t, int page) {
    const int sub = (tile_of(t) * kTile) & ((1 << pshift) - 1);
    const rsrc_t r = make_res(c.k + ((((int64_t)page * c.Hkv + h) << pshift) + sub) * D, t < t_end ? kTile * D : 0);
#pragma unroll
    for (int i = 0; i < KI; ++i)
#pragma unroll
      for (int k = 0; k < KK; ++k) kf[i][k] = load16<kAuxStream>(r, koff + (kWide ? 2 : 4) * i * D + 128 * k, 0);
  };
  auto load_v = [&](int t, int page) {
    const int sub = (tile_of(t) * kTile) & ((1 << pshift) - 1);
    const rsrc_t r = make_res(c.v + (((int64_t)page * c.Hkv + h) << pshift) * D + sub, t < t_end ? (D << pshift) - sub : 0);
#pragma unroll
    for (int i = 0; i < DT; ++i) vf[i] = load16<0>(r, voff, (16 * i) << pshift);
  };
  // the first tile is on its way while the queries are rounded
  int t = t_begin + wave;
  int id = __builtin_amdgcn_readfirstlane(page_at(t)), next = page_at(t + kWaves);
  bool good = (unsigned)id < (unsigned)c.n_pages;
  int page = good ? id : 0;
  load_k(t, page);
  load_v(t, page);
  float ks = c.k_scale[(int64_t)page * c.Hkv + h], vs = c.v_scale[(int64_t)page * c.Hkv + h];
  Column<D, ND, M> o;
  column_init<D, ND, M>(o, a, q, h, ct * 16 + col, cols, g);
  float acc[DT][4];
#pragma unroll
  for (int i = 0; i < DT; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[i][r] = 0.0f;
  if (t < t_end) {
    for (; t < t_end; t += kWaves) {
      const Scales sc = scales_of(good ? ks : -1.0f, vs);
      id = __builtin_amdgcn_readfirstlane(next);
      good = (unsigned)id < (unsigned)c.n_pages;
      page = good ? id : 0;
      next = page_at(t + 2 * kWaves);
      float x[16];
#pragma unroll
      for (int i = 0; i < KI; ++i) {
        i32x4 d[ND];
        if constexpr (kWide) {
#pragma unroll
          for (int e = 0; e < ND; ++e) {
            i32x4 d0{0, 0, 0, 0}, d1{0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < KK; ++k) {
              d0 = __builtin_amdgcn_mfma_i32_16x16x64_i8(kf[i][k], o.qd[e][2 * k], d0, 0, 0, 0);
              d1 = __builtin_amdgcn_mfma_i32_16x16x64_i8(kf[i][k], o.qd[e][2 * k + 1], d1, 0, 0, 0);
            }
            d[e] = i32x4{d0[0] + d1[1], d0[2] + d1[3], 0, 0};
          }
          x[2 * i] = join<ND>(d, 0);
          x[2 * i + 1] = join<ND>(d, 1);
        } else {
#pragma unroll
          for (int e = 0; e < ND; ++e)
            d[e] = __builtin_amdgcn_mfma_i32_16x16x64_i8(kf[i][0], o.qd[e][0], i32x4{0, 0, 0, 0}, 0, 0, 0);
#pragma unroll
          for (int r = 0; r < 4; ++r) x[4 * i + r] = join<ND>(d, r);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      load_k(t + kWaves, page);
      ks = c.k_scale[(int64_t)page * c.Hkv + h];
      vs = c.v_scale[(int64_t)page * c.Hkv + h];
      const float f = fmaxf(o.qscale * sc.ks, 1e-37f);
      float ref, beta;
      const int base = tile_of(t) * kTile;
      const float alpha = advance<D, ND, M>(o, a, q, x, f, sc.off, base + kTile - 1 > sp.full_hi || base < sp.full_lo,
                                            base + 16 * g, ref, beta);
      i32x4 pd[kWeightDigits];
      o.l = fmaf(beta, weights(x, f, ref, pd), o.l * alpha);
      const float fv = sc.vs * (1.0f / Digits<kWeightDigits>::top) * beta;
#pragma unroll
      for (int i = 0; i < DT; ++i) {
        i32x4 d[kWeightDigits];
#pragma unroll
        for (int e = 0; e < kWeightDigits; ++e)
          d[e] = __builtin_amdgcn_mfma_i32_16x16x64_i8(vf[i], pd[e], i32x4{0, 0, 0, 0}, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][r] = fmaf(join<kWeightDigits>(d, r), fv, acc[i][r] * alpha);
        if (i & 1) __builtin_amdgcn_sched_barrier(0);
      }
      load_v(t + kWaves, page);
    }
  }
  o.l += xor_lanes<16>(o.l);
  o.l += xor_lanes<32>(o.l);

  // the waves' shares meet in LDS
#pragma unroll
  for (int i = 0; i < DT; ++i)
    *reinterpret_cast<float4*>(&s_acc[wave][col][16 * i + 4 * g]) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
  if (g == 0) {
    s_m[wave][col] = o.m;
    s_l[wave][col] = o.l;
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
    ll = fmaf(w[i], s_l[i][oc], ll);  // 0 * NaN stays NaN
  }
  const int64_t orow = (int64_t)q.row0 + ot;
  const float inv = slot < 0 ? (ll == 0.0f ? 0.0f : 1.0f / ll) : 1.0f;
  const int64_t at = (int64_t)slot * 16 + oc;
#pragma unroll
  for (int i = 0; i < DT / 4; ++i) {
    const int d = 4 * part + 64 * i;
    float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < kWaves; ++k)
#pragma unroll
      for (int r = 0; r < 4; ++r) y[r] = fmaf(w[k], s_acc[k][oc][d + r], y[r]);
    if (slot < 0) store_out4(a, orow, oh, D, d, y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
    else *reinterpret_cast<float4*>(a.part + at * D + d) = make_float4(y[0], y[1], y[2], y[3]);
  }
  if (slot >= 0 && part == 0) reinterpret_cast<float2*>(a.part_m)[at] = make_float2(mm, ll);
}

template <int D, int ND, bool M>
__global__ __launch_bounds__(64 * kWaves, D == 256 ? 1 : 2) void k_kv_attn(KvAttn a) {
  __shared__ __attribute__((aligned(16))) FewLds<D, ND> lds;
  __shared__ int64_t first[kMaxDealt + 1], waves[kWaves];
  const int Hkv = a.c.Hkv;
  const int tid = threadIdx.x;
  int s = blockIdx.y, plain_seg = blockIdx.x;  // without a deal: one segment a workgroup
  int64_t u = 0, end = 1, total = 0, runs = 0;
  int run = 0;
  if (a.pieces) {
    // tiles before each sequence; a thread takes `per` neighbouring ones
    const int per = (a.b.S + 255) >> 8;
    int64_t sum = 0;
#pragma unroll 1
    for (int i = 0; i < per; ++i) {
      const int e = tid * per + i;
      int64_t n = 0;
      if (e < a.b.S) {
        const Seq q = seq_of(a.b, e, a.c.page);
        Span all;
        if (q.nq) n = (int64_t)((q.nq * a.G + 15) / 16) * Hkv * tiles_of<M>(a, q, q.nq * a.G, all);
        first[e] = sum;
      }
      sum += n;
    }
    int64_t upto = sum;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int64_t v = __shfl_up(upto, o, 64);
      if ((tid & 63) >= o) upto += v;
    }
    if ((tid & 63) == 63) waves[tid >> 6] = upto;
    __syncthreads();
    int64_t before = upto - sum;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      if (w < tid >> 6) before += waves[w];
      total += waves[w];
    }
    for (int e = tid * per; e < min(tid * per + per, a.b.S); ++e) first[e] += before;
    if (tid == 0) first[a.b.S] = total;
    __syncthreads();
    // runs of four tiles at least: one a wave
    runs = max(min((int64_t)a.pieces, total / kWaves), (int64_t)(total > 0));
    // Runs that follow each other go to workgroups of one die: the column tiles of a
    // sequence and key head read the same cache, through one L2 (9 x up to 12 drafts on
    // up to 5000 tokens, 16 heads on 2 of 256: 44.5 -> 42 us; one column tile: no change).
    run = blockIdx.x;
    if (run < runs) {
      const int die = run & 7, each = (int)(runs >> 3);
      run = die * each + min(die, (int)(runs & 7)) + (run >> 3);
    }
    if (tid == 0) a.shares[run] = make_int4(0, 0, 0, 0);
    if (run >= runs) return;
    u = run * total / runs;
    end = (run + 1) * total / runs;
    int lo = 0, hi = a.b.S;  // the sequence of tile u: first[lo] <= u < first[lo + 1]
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (first[mid] <= u) lo = mid;
      else hi = mid;
    }
    s = lo;
  }
  for (bool again = false; u < end; again = true) {
    s = __builtin_amdgcn_readfirstlane(s);
    const Seq q = seq_of(a.b, s, a.c.page);
    const int cols = q.nq * a.G, cts = (cols + 15) / 16;
    int seg = plain_seg, from = 0;
    Span all{};
    const int n = cols ? tiles_of<M>(a, q, cols, all) : 0;
    int to = n;
    if (a.pieces) {
      const int64_t in = u - first[s];
      seg = __builtin_amdgcn_readfirstlane((int)(in / n));
      from = __builtin_amdgcn_readfirstlane((int)(in - (int64_t)seg * n));
      to = __builtin_amdgcn_readfirstlane((int)min((int64_t)n, from + (end - u)));
    } else if (seg >= cts * Hkv) {
      return;
    }
    const int h = __builtin_amdgcn_readfirstlane(seg / cts), ct = seg - h * cts;
    const Span sp = span_of<M>(a, q, ct * 16, min(ct * 16 + 16, cols));
    // the first one's share of a workgroup goes to its slot 0, the last one's to 1
    const int slot = from == 0 && to == n ? -1 : 2 * run + (again ? 1 : 0);
    if (again) __syncthreads();  // the LDS of the one before
    // (said to be the same in all lanes, or every load would ask each of them)
    int lo = max(all.t0 + from, sp.t0), hi = min(all.t0 + to, sp.t1), skip = 0;
    if constexpr (M) {
      // of the sequence's tiles in order those that this column tile sees
      skip = all.t0 - all.head;
      lo = from < all.head || sp.head > all.t0 ? from : max(from, sp.t0 - skip);
      hi = min(to, sp.t1 - skip);
    }
    few_columns<D, ND, M>(a, q, h, ct, cols, sp, __builtin_amdgcn_readfirstlane(lo),
                          __builtin_amdgcn_readfirstlane(hi), __builtin_amdgcn_readfirstlane(all.head),
                          __builtin_amdgcn_readfirstlane(skip), slot, lds);
    if (!a.pieces) return;
    if (from == 0 && to < n && tid == 0) {
      const int64_t last = ((first[s] + (int64_t)(seg + 1) * n) * runs - 1) / total;  // the run with its last tile
      a.shares[run] = make_int4((int)(last - run) + 1, s, seg, slot);
    }
    u += to - from;
    while (u < end && u >= first[s + 1]) ++s;  // u < end <= total: there is one that holds it
  }
}

// Many columns (prompts): a workgroup's four waves own 32 columns each and walk
// the same tiles of 64 tokens, staged in LDS; a byte of the cache is read from
// L2 once for 128 columns.  Here the arithmetic around the products counts, so
// they run on the f16 matrix cores, which accumulate in fp32 and need no joins:
// the codes are exact in f16 (converted once per workgroup on their way to
// LDS), a query row is scaled by a power of two to below 2^14 and rounded to
// f16, and so is a weight p times a unit times vs / R, R the power of two at or
// below the largest value scale met so far.  NS = 2 (fp32 outputs) takes a second
// f16 for what the first one leaves, 22 bits together, and the unit 2^14, which
// keeps both parts of weights down to 2^-18 whole; plain calls of 128 channels do not
// fit the registers (22 spilled).  NS = 1: a row's reference
// follows its maximum only where that has grown by 2^7, so p stays below 2^7 and
// the unit is 2^7 (a weight below 2^-21 loses bits, 2^-32 at most); without that
// some column's maximum moves in most tiles and the sums are rescaled there
// (4096 new of 5003 tokens: 160 us, 156).  Per score that leaves half a
// maximum, one fma, one exp2 (a quarter of the rate), the sum and half a
// conversion on the vector ALU.
//
// Measured: 4096 new of 5003 tokens, 16 heads on 4 of 128 channels, bf16 out,
// 149 us (99 GFlop, 0.66 Pflop/s; the int8 form's digits and joins 296).  Every
// wave reads all of a tile's 32 KB from LDS, at 64 bytes a clock and compute
// unit half of that time and twice what the products take; the softmax's vector
// work (a third of the waves' time) stands between the two products, and two waves
// a SIMD overlap these only in part.  Measured
// and dropped, when it took 157: the next tile's first product beside this one's
// softmax (187 to 196, registers), one wave a SIMD (307), wave priorities (162 to
// 164).
//
// 32 x 32 tiles: score row 8 a + 4 hh + b of a 32-token block is its token
// 16 hh + 4 a + b, so lane half hh holds tokens 16 hh .. 16 hh + 15 and feeds
// them, eight consecutive ones a step, as the second product's B operand.
// LDS chunks of 16 bytes are permuted by their row so that the rows a fragment
// read touches fall into different banks.
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// Four codes as f16: 1024 + 128 + code has the bit pattern 0x6400 | (code ^ 0x80).
MD_DEV uint2 codes_f16(uint32_t w) {
  const uint32_t u = w ^ 0x80808080u;
  const f16x2 bias = {(_Float16)-1152.0f, (_Float16)-1152.0f};
  const uint32_t lo = __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u), hi = __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u);
  return make_uint2(__builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, lo) + bias),
                    __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, hi) + bias));
}

constexpr int kRowCols = 128;  // columns of a workgroup

// Tiles of a split of the sequence q.  Plain calls: what the host's bounds gave.
// Masked ones: all column tiles' tiles, by the lengths on the device, over the
// workgroups that run at once (a.deal; one more would wait for all of them), four at
// least and as many as leave a.splits of them enough (2 x 61 drafts on 65535 and 27963 tokens, 32 heads on 8 of 128:
// 263 us with splits of the longest one's, 228).  Every thread of the workgroup calls it; there are at most 256
// sequences where a.splits > 1.
template <bool M>
MD_DEV int split_tiles(const KvAttn& a, const Seq& q) {
  if (!M || a.splits == 1) return a.chunk;
  __shared__ int64_t s_sum[kWaves];
  // tiles, and in the upper bits segments: one more split each, where tiles do not come out even
  int64_t sum = 0;
  Span all;
  if ((int)threadIdx.x < a.b.S) {
    const Seq r = seq_of(a.b, threadIdx.x, a.c.page);
    const int cts = (r.nq * a.G + a.tile - 1) / a.tile;
    if (r.nq) sum = (int64_t)tiles_of<true>(a, r, r.nq * a.G, all) * cts + ((int64_t)cts << 40);
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o, 64);
  if ((threadIdx.x & 63) == 0) s_sum[threadIdx.x >> 6] = sum;
  __syncthreads();
  sum = (s_sum[0] + s_sum[1]) + (s_sum[2] + s_sum[3]);
  const int n = q.nq ? tiles_of<true>(a, q, q.nq * a.G, all) : 1;
  const int64_t total = (sum & ((1ll << 40) - 1)) * a.c.Hkv, groups = max(a.deal - (sum >> 40) * a.c.Hkv, (int64_t)a.deal / 4);
  const int64_t per = max((total + groups - 1) / groups, (int64_t)a.chunk);
  return __builtin_amdgcn_readfirstlane((int)max(per, (int64_t)((n + a.splits - 1) / a.splits)));
}

// Schedules a block of N LDS reads that feed NS matrix instructions each with
// four reads in flight; left to itself the compiler waits for every read right
// after it (4096 new of 5003 tokens, 128 channels: 152 -> 149 us, 2048 of 2048 of
// 4 sequences, 64 channels: 67 -> 62).
template <int N, int NS, int GROUP>
MD_DEV void paced() {
  constexpr int kAhead = 4;
  __builtin_amdgcn_sched_group_barrier(0x100, kAhead, GROUP);
#pragma unroll
  for (int i = 0; i < N - kAhead; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, NS, GROUP);
    __builtin_amdgcn_sched_group_barrier(0x100, 1, GROUP);
  }
  __builtin_amdgcn_sched_group_barrier(0x008, kAhead * NS, GROUP);
}

template <int D, int NS, bool M>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void k_kv_attn_rows(KvAttn a) {
  constexpr int KS = D / 16, DT = D / 32;
  // blocks of 32 tokens of a softmax step: a masked call with two parts of each
  // weight and 128 channels or more takes them one by one, which spares registers:
  // reloads of spilled ones wait for the next tile's loads too (2 x 61 drafts on up
  // to 65535 tokens, 32 heads on 8 of 128: 317 us with 27 spilled, 263 with none)
  constexpr int NB = M && NS == 2 && D > 64 ? 1 : 2;
  constexpr float kLag = NS == 1 ? 7.0f : 0.0f, kUnit = NS == 1 ? 128.0f : 16384.0f;
  constexpr int L = kTile * D / 16 / 256;  // 16-byte chunks of codes per thread, keys or values
  __shared__ __attribute__((aligned(16))) _Float16 s_k[2][kTile * D], s_v[2][kTile * D];
  const KvCache& c = a.c;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 31, hh = lane >> 5;
  // M: many of the splits may have nothing to do (split_tiles); those that have follow
  // each other, since workgroups are spread over the dies by their number
  const int heads = (int)(gridDim.x / a.splits);
  const int split = M ? blockIdx.x / heads : blockIdx.x % a.splits, rest = M ? blockIdx.x % heads : blockIdx.x / a.splits;
  const int h = rest % c.Hkv, s = blockIdx.y;
  const Seq q = seq_of(a.b, s, c.page);
  const int cols = q.nq * a.G;
  const int ct = column_tile(a, rest / c.Hkv, (int)(gridDim.x / (a.splits * c.Hkv)));
  const int per = split_tiles<M>(a, q);
  if (ct * kRowCols >= cols) return;
  const Span sp = span_of<M>(a, q, ct * kRowCols, min(ct * kRowCols + kRowCols, cols));
  const int active = max(1, (sp.head + sp.t1 - sp.t0 + per - 1) / per);
  if (split >= active) return;
  if (M && a.splits > 1 && split == 0 && h == 0 && tid == 0)  // for the join
    reinterpret_cast<int*>(a.shares)[s * (heads / c.Hkv) + ct] = active;
  // M: tiles numbered with the `head` first ones in front
  const int skip = sp.t0 - sp.head;
  const int t_begin = M ? split * per : sp.t0 + split * per, t_end = min(t_begin + per, M ? sp.t1 - skip : sp.t1);
  auto tile_of = [&](int t) { return M && t >= sp.head ? t + skip : t; };
  const int c0 = ct * kRowCols + wave * 32;
  const bool any = c0 < cols;  // a wave past the last column only helps with the loads
  const Span mine = span_of<M>(a, q, any ? c0 : 0, any ? min(c0 + 32, cols) : 1);

  const int pshift = a.pshift;
  u32x4 kr[L], vr[L];
  float ks_n, vs_n;
  auto page_at = [&](int t) { return t < t_end ? q.table[tile_of(t) * kTile >> pshift] : 0; };
  int next = page_at(t_begin);  // the page of the tile that is loaded next, read a tile ahead
  auto load = [&](int t) {      // tile t's codes and scales; a page that is none is page 0 with a scale that is none
    const int id = __builtin_amdgcn_readfirstlane(next);
    next = page_at(t + 1);
    const bool good = (unsigned)id < (unsigned)c.n_pages;
    const int page = good ? id : 0, sub = (tile_of(t) * kTile) & ((1 << pshift) - 1);
    const int64_t ph = (int64_t)page * c.Hkv + h;
    ks_n = good ? c.k_scale[ph] : -1.0f;
    vs_n = c.v_scale[ph];
    const int8_t *kp = c.k + ((ph << pshift) + sub) * D, *vp = c.v + (ph << pshift) * D + sub;
#pragma unroll
    for (int n = 0; n < L; ++n) {
      const int ch = n * 256 + tid;
      kr[n] = *reinterpret_cast<const u32x4*>(kp + 16 * ch);
      vr[n] = *reinterpret_cast<const u32x4*>(vp + ((ch >> 2) << pshift) + 16 * (ch & 3));
    }
  };
  // sixteen lanes of a fragment read hit sixteen chunks of a 256-byte line: its
  // tokens differ in bits 0, 1, 2 and 4, its channels in bits 0..3
  auto kslot = [](int tok, int chunk) {
    const int up = ((tok >> 4) & 1) | ((tok >> 2) & 1) << 1;
    return tok * D + 8 * (chunk ^ (D == 64 ? ((tok >> 1) & 1) | up << 1 : (tok & 3) | up << 2));
  };
  auto vslot = [](int d, int chunk) { return d * kTile + 8 * (chunk ^ ((d >> 1) & 7)); };
  auto stage = [&](int buf) {
#pragma unroll
    for (int n = 0; n < L; ++n) {
      const int ch = n * 256 + tid;
      const int tok = ch / (D / 16), kc = 2 * (ch % (D / 16)), d = ch >> 2, vc = 2 * (ch & 3);
      u32x4 w[2];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const uint2 f = codes_f16(kr[n][m]);
        w[m >> 1][2 * (m & 1)] = f.x;
        w[m >> 1][2 * (m & 1) + 1] = f.y;
      }
#pragma unroll
      for (int m = 0; m < 2; ++m) *reinterpret_cast<u32x4*>(&s_k[buf][kslot(tok, kc + m)]) = w[m];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const uint2 f = codes_f16(vr[n][m]);
        w[m >> 1][2 * (m & 1)] = f.x;
        w[m >> 1][2 * (m & 1) + 1] = f.y;
      }
#pragma unroll
      for (int m = 0; m < 2; ++m) *reinterpret_cast<u32x4*>(&s_v[buf][vslot(d, vc + m)]) = w[m];
    }
  };
  if (t_begin < t_end) load(t_begin);

  // this lane's column
  const int cc = min(c0 + col, cols - 1), qt = cc / a.G, hq = h * a.G + (cc - qt * a.G);
  const int pos = q.len - q.nq + qt;
  const int hi = a.causal ? pos : q.len - 1, lo = a.window ? max(pos - a.window + 1, 0) : 0;
  Seen seen{};
  if constexpr (M) seen = seen_of(a, q, qt);
  f16x8 qf[NS][KS];
  float m = -INFINITY, l = q.bad ? nan_f() : 0.0f, qscale;
  {
    const int64_t at = ((int64_t)q.row0 + qt) * a.q_stride + (int64_t)hq * D + 8 * hh;
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      float w[8];
      if (a.xt == XF32) load8<XF32>(a.q, at + 16 * k, w);
      else load8<XBF16>(a.q, at + 16 * k, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(w[e]) & 0x7FFFFFFFu);
    }
    top = max(top, __float_as_uint(xor_lanes<32>(__uint_as_float(top))));
    if (top >= 0x7F800000u) l = nan_f(), top = 0;
    const int ex = (int)(top >> 23) - 127;  // below -100: as a row of zeros
    const float up = ex >= -100 ? copysignf(__uint_as_float((uint32_t)(127 + 13 - ex) << 23), a.scale) : 0.0f;
    qscale = ex >= -100 ? __uint_as_float((uint32_t)(127 - 13 + ex) << 23) * fabsf(a.scale) * kLog2e : 0.0f;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      float w[8];
      if (a.xt == XF32) load8<XF32>(a.q, at + 16 * k, w);
      else load8<XBF16>(a.q, at + 16 * k, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float f = l == l ? w[e] * up : 0.0f;
        qf[0][k][e] = (_Float16)f;
        if constexpr (NS == 2) qf[1][k][e] = (_Float16)(f - (float)qf[0][k][e]);
      }
    }
  }
  f32x16 acc[DT];
#pragma unroll
  for (int n = 0; n < DT; ++n)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[n][i] = 0.0f;
  int ex_r = 1;  // acc is in steps of R / kUnit, R = 2^(ex_r - 127)

  Scales sc{};
  if (t_begin < t_end) {
    stage(0);
    sc = scales_of(ks_n, vs_n);
    load(t_begin + 1);
  }
  __syncthreads();
  int buf = 0;
  for (int t = t_begin; t < t_end; ++t, buf ^= 1) {
    const int here = tile_of(t);
    if (any && here < mine.t1 && (here >= mine.t0 || (M && here < mine.head))) {
#pragma unroll 1
      for (int b0 = 0; b0 < 2; b0 += NB) {
        f32x16 x[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int i = 0; i < 16; ++i) x[b][i] = 0.0f;
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const int tok = 32 * (b0 + b) + 16 * ((col >> 2) & 1) + 4 * (col >> 3) + (col & 3);
            const f16x8 kf = *reinterpret_cast<const f16x8*>(&s_k[buf][kslot(tok, 2 * k + hh)]);
#pragma unroll
            for (int e = 0; e < NS; ++e) x[b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf, qf[e][k], x[b], 0, 0, 0);
          }
        paced<NB * KS, NS, 0>();
        const int base = here * kTile, first = base + 32 * b0 + 16 * hh;
        if (base + kTile - 1 > mine.full_hi || base < mine.full_lo) {
          keep_branch();
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            if constexpr (M) {
              const uint32_t vis = seen16(a, q, seen, first + 32 * b);
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (!(vis >> i & 1u)) x[b][i] = -INFINITY;
            } else {
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (first + 32 * b + i > hi || first + 32 * b + i < lo) x[b][i] = -INFINITY;
            }
          }
        }
        const float f = fmaxf(qscale * sc.ks, 1e-37f);
        float raw = x[0][0];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int i = 0; i < 16; ++i) raw = fmaxf(raw, x[b][i]);
        if (raw > -INFINITY) l += sc.off;
        raw = fmaxf(raw, xor_lanes<32>(raw)) * f;
        if (raw == INFINITY) l = nan_f();
        const float m1 = raw > m + kLag ? raw : m, ref = m1 > -INFINITY ? m1 : 0.0f;
        const float alpha = __builtin_amdgcn_exp2f(m - ref);
        m = m1;
        // R is a power of two, so both factors are exact
        const int e1 = max(ex_r, (int)(__float_as_uint(sc.vs) >> 23));
        const float down = __uint_as_float((uint32_t)max(127 + ex_r - e1, 0) << 23);
        const float w = sc.vs * __uint_as_float((uint32_t)(254 - e1) << 23) * kUnit;
        ex_r = e1;
        f16x8 pf[NS][2 * NB];
        float sum = 0.0f;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float p = __builtin_amdgcn_exp2f(fmaf(x[b][i], f, -ref));
            sum += p;
            float pw = p * w;
            // both parts from one rounded product: fused into the first conversion and not into the second, a
            // tie could round two ways and leave a weight 2^-11 off
            if constexpr (NS == 2) asm volatile("" : "+v"(pw));
            pf[0][2 * b + (i >> 3)][i & 7] = (_Float16)pw;
            if constexpr (NS == 2) pf[1][2 * b + (i >> 3)][i & 7] = (_Float16)(pw - (float)pf[0][2 * b + (i >> 3)][i & 7]);
          }
        l = fmaf(l, alpha, sum);
        const float scale = alpha * down;
        if (__builtin_amdgcn_ballot_w64(scale != 1.0f)) {
          keep_branch();
#pragma unroll
          for (int n = 0; n < DT; ++n)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[n][i] *= scale;
        }
#pragma unroll
        for (int n = 0; n < DT; ++n) {
          const int d = 32 * n + col;
#pragma unroll
          for (int k = 0; k < 2 * NB; ++k) {
            // block k / 2, step k % 2: tokens 32 (k / 2) + 16 hh + 8 (k % 2) ..
            const f16x8 vf = *reinterpret_cast<const f16x8*>(&s_v[buf][vslot(d, 4 * (b0 + (k >> 1)) + 2 * hh + (k & 1))]);
#pragma unroll
            for (int e = 0; e < NS; ++e) acc[n] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf, pf[e][k], acc[n], 0, 0, 0);
          }
        }
        paced<2 * NB * DT, NS, 1>();
      }
    }
    if (t + 1 < t_end) {
      stage(buf ^ 1);
      sc = scales_of(ks_n, vs_n);
      load(t + 2);
    }
    __syncthreads();
  }
  l += xor_lanes<32>(l);
  if (c0 + col >= cols) return;
  const int64_t orow = (int64_t)q.row0 + qt;
  const float unit = __uint_as_float((uint32_t)ex_r << 23) * (1.0f / kUnit);
  if (active == 1) {
    const float inv = l == 0.0f ? 0.0f : unit / l;
#pragma unroll
    for (int n = 0; n < DT; ++n)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        store_out4(a, orow, hq, D, 32 * n + 2 * i + 4 * hh, acc[n][i] * inv, acc[n][i + 1] * inv, acc[n][i + 2] * inv,
                   acc[n][i + 3] * inv);
  } else {
    const int64_t slot = (orow * (a.G * c.Hkv) + hq) * a.splits + split;
#pragma unroll
    for (int n = 0; n < DT; ++n)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<float4*>(a.part + slot * D + 32 * n + 2 * i + 4 * hh) =
            make_float4(acc[n][i] * unit, acc[n][i + 1] * unit, acc[n][i + 2] * unit, acc[n][i + 3] * unit);
    if (hh == 0) {
      a.part_m[2 * slot] = m;
      a.part_m[2 * slot + 1] = l;
    }
  }
}

// The splits of a row and head, one workgroup each: D / 4 lanes for the
// channels, the other lanes share the splits out and meet in LDS.
template <int D>
__global__ __launch_bounds__(256) void k_kv_join(KvAttn a) {
  constexpr int L = D / 4, P = 256 / L;
  __shared__ float s_l[P];
  __shared__ __attribute__((aligned(16))) float s_o[P][D];
  const int s = blockIdx.z, head = blockIdx.y, part = threadIdx.x / L, d = 4 * ((int)threadIdx.x % L);
  const Seq q = seq_of(a.b, s, a.c.page);
  if ((int)blockIdx.x >= q.nq) return;
  const int64_t row = (int64_t)q.row0 + blockIdx.x, slot0 = (row * (a.G * a.c.Hkv) + head) * a.splits;
  const int cols = q.nq * a.G, ct = ((int)blockIdx.x * a.G + head % a.G) / a.tile;
  int active;
  if (a.masked) {
    active = reinterpret_cast<const int*>(a.shares)[s * ((gridDim.x * a.G + a.tile - 1) / a.tile) + ct];
  } else {
    const Span sp = span_of<false>(a, q, ct * a.tile, min(ct * a.tile + a.tile, cols));
    active = (sp.t1 - sp.t0 + a.chunk - 1) / a.chunk;
  }
  if (active <= 1) return;
  const float2* ml = reinterpret_cast<const float2*>(a.part_m) + slot0;
  float m = -INFINITY;
  for (int i = threadIdx.x & 63; i < active; i += 64) m = fmaxf(m, ml[i].x);
  m = group_max<64>(m);
  const float ref = m > -INFINITY ? m : 0.0f;
  float l = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int i = part; i < active; i += P) {
    const float2 x = ml[i];
    const float w = __builtin_amdgcn_exp2f(x.x - ref);
    const float4 p = *reinterpret_cast<const float4*>(a.part + (slot0 + i) * D + d);
    l = fmaf(w, x.y, l);
    o[0] = fmaf(w, p.x, o[0]);
    o[1] = fmaf(w, p.y, o[1]);
    o[2] = fmaf(w, p.z, o[2]);
    o[3] = fmaf(w, p.w, o[3]);
  }
  *reinterpret_cast<float4*>(&s_o[part][d]) = make_float4(o[0], o[1], o[2], o[3]);
  if (d == 0) s_l[part] = l;
  __syncthreads();
  if (part) return;
  for (int i = 1; i < P; ++i) {
    l += s_l[i];
#pragma unroll
    for (int r = 0; r < 4; ++r) o[r] += s_o[i][d + r];
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  store_out4(a, row, head, D, d, o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
}

// The shares of a segment that several workgroups had: one workgroup for each
// workgroup where one may begin and each of its columns.
template <int D>
__global__ __launch_bounds__(256) void k_kv_join_pieces(KvAttn a) {
  constexpr int L = D / 4, P = 256 / L;
  __shared__ float s_l[P];
  __shared__ __attribute__((aligned(16))) float s_o[P][D];
  const int4 sh = a.shares[blockIdx.x];  // count, sequence, segment, first slot
  if (sh.x <= 1) return;
  const Seq q = seq_of(a.b, sh.y, a.c.page);
  const int cols = q.nq * a.G, cts = (cols + 15) / 16, h = sh.z / cts, c = (sh.z - h * cts) * 16 + (int)blockIdx.y;
  if (c >= cols) return;
  const int part = threadIdx.x / L, d = 4 * ((int)threadIdx.x % L);
  auto at = [&](int i) { return (int64_t)(i ? 2 * ((int)blockIdx.x + i) : sh.w) * 16 + blockIdx.y; };
  const float2* ml = reinterpret_cast<const float2*>(a.part_m);
  float m = -INFINITY;
  for (int i = threadIdx.x & 63; i < sh.x; i += 64) m = fmaxf(m, ml[at(i)].x);
  m = group_max<64>(m);
  const float ref = m > -INFINITY ? m : 0.0f;
  float l = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int i = part; i < sh.x; i += P) {
    const float2 x = ml[at(i)];
    const float w = __builtin_amdgcn_exp2f(x.x - ref);
    const float4 p = *reinterpret_cast<const float4*>(a.part + at(i) * D + d);
    l = fmaf(w, x.y, l);
    o[0] = fmaf(w, p.x, o[0]);
    o[1] = fmaf(w, p.y, o[1]);
    o[2] = fmaf(w, p.z, o[2]);
    o[3] = fmaf(w, p.w, o[3]);
  }
  *reinterpret_cast<float4*>(&s_o[part][d]) = make_float4(o[0], o[1], o[2], o[3]);
  if (d == 0) s_l[part] = l;
  __syncthreads();
  if (part) return;
  for (int i = 1; i < P; ++i) {
    l += s_l[i];
#pragma unroll
    for (int r = 0; r < 4; ++r) o[r] += s_o[i][d + r];
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const int qt = c / a.G;
  store_out4(a, (int64_t)q.row0 + qt, h * a.G + (c - qt * a.G), D, d, o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
}

KvPlan kv_attn_plan(const KvCache& c, const KvBatch& b, int G, int window, int sinks, int causal, int yt, bool masked) {
  int64_t most = b.max_kv;
  if (causal && window && (int64_t)window + b.max_q < most) most = (int64_t)window + b.max_q;
  int64_t tiles = (most + kTile - 1) / kTile + 1;
  if (sinks) {  // and those of the first positions, before the window's
    const int64_t all = ((int64_t)b.max_kv + kTile - 1) / kTile + 1;
    tiles += (sinks + kTile - 1) / kTile;
    if (tiles > all) tiles = all;
  }
  KvPlan p{};
  // More than four column tiles: the form that shares its loads among 128
  // columns (80 columns, 16 sequences of 4000: 41 us, 51 in the other one; 64:
  // 41 both).  fp32 outputs of 256 channels leave it one wave a SIMD, so there
  // it is kept for columns by the hundreds (us here and in the other one: 240
  // columns, 4 sequences of 1000: 42 and 23; 600, 4 of 8000: 176 and 170; 1000,
  // one of 30000: 182 and 250; 8192, one of 4096: 214 and 223; over trees 96
  // columns, 9 of 5000: 77 and 57; 240: 42 and 22; 600: 154 and 161; 1000: 197 and 250).
  const int64_t cols = (int64_t)b.max_q * G;
  p.tile = cols > (c.D == 256 && yt == XF32 ? 768 : 64) ? kRowCols : 16;
  p.splits = 1;
  p.chunk = (int)tiles;
  if (p.tile == 16) {
    // A segment each where they are short, or middling and enough of them: the
    // deal and its join cost some 8 us (64 channels x 2, us without and with:
    // 16 new in 1000 tokens of 4 sequences 12 and 20, 1 in 2000 of 64: 21 and 33,
    // 1 in 2000 of one: 16 and 12, 1 in 4000 of 64: 33 and 41, of one: 26 and 17).
    // Else as many workgroups as run at once (registers: one, two or four on a
    // compute unit).
    const int64_t segments = (int64_t)b.S * c.Hkv * ((cols + 15) / 16);
    const bool whole = tiles <= 17 || (tiles <= 33 && segments >= 16) || (tiles <= 65 && segments >= device_cus());
    if (!whole && b.S <= kMaxDealt) p.pieces = device_cus() * (c.D == 64 ? 4 : c.D == 128 ? 2 : 1);
    return p;
  }
  // where the columns alone give most compute units a workgroup, sequences stay
  // whole (8 of 256 new in 2048 tokens, 16 heads on 4 of 128: 63 us, in two
  // parts 91; 2048 new in 4096: 123, 152); else two workgroups a unit, a split a
  // fixed number of tiles (1024 new in 8192: 126 us; one a unit 146)
  const int64_t base = (int64_t)b.S * c.Hkv * (((int64_t)b.max_q * G + p.tile - 1) / p.tile);
  if (4 * base >= 3 * (int64_t)device_cus()) return p;
  const int64_t want = 2 * device_cus();
  int64_t chunk = (tiles * base + want - 1) / want;
  if (chunk < 4) chunk = 4;
  p.chunk = (int)(chunk < tiles ? chunk : tiles);
  p.splits = (int)((tiles + p.chunk - 1) / p.chunk);
  if (masked && p.splits > 1) {  // split_tiles deals by the lengths: room for twice as many of the longest sequence
    const int64_t most = (tiles + 3) / 4;
    p.splits = (int)(2 * p.splits < most ? 2 * p.splits : most);
    p.chunk = 4;
    p.notes = b.S * (int)((cols + p.tile - 1) / p.tile);
  }
  return p;
}

hipError_t launch_kv_attn(const KvAttn& a0, int D, int yt, hipStream_t st) {
  KvAttn a = a0;
  const int64_t cts = ((int64_t)a.b.max_q * a.G + a.tile - 1) / a.tile;
  const dim3 grid = a.pieces ? dim3(a.pieces) : dim3((unsigned)(a.splits * cts * a.c.Hkv), a.b.S), block(64 * kWaves);
  const int64_t groups = (int64_t)grid.x * grid.y;
  a.deal = 2 * device_cus();
  a.snake = groups > device_cus() && groups <= 2 * device_cus();
#define MD_ATT_M(D_, N_, M_)                                                               \
  do {                                                                                     \
    if (a.tile == 16) hipLaunchKernelGGL((k_kv_attn<D_, N_, M_>), grid, block, 0, st, a);  \
    else hipLaunchKernelGGL((k_kv_attn_rows<D_, N_ - 1, M_>), grid, block, 0, st, a);      \
  } while (0)
#define MD_ATT(D_, N_)                   \
  do {                                   \
    if (a.masked) MD_ATT_M(D_, N_, true); \
    else MD_ATT_M(D_, N_, false);        \
  } while (0)
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
#undef MD_ATT_M
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || (a.splits == 1 && !a.pieces)) return e;
#define MD_JOIN(D_)                                                                                                   \
  do {                                                                                                                \
    if (a.pieces) hipLaunchKernelGGL((k_kv_join_pieces<D_>), dim3(a.pieces, 16), dim3(256), 0, st, a);                \
    else hipLaunchKernelGGL((k_kv_join<D_>), dim3(a.b.max_q, a.G * a.c.Hkv, a.b.S), dim3(256), 0, st, a);             \
  } while (0)
  if (D == 64) MD_JOIN(64);
  else if (D == 128) MD_JOIN(128);
  else MD_JOIN(256);
#undef MD_JOIN
  return hipGetLastError();
}

}  // namespace md

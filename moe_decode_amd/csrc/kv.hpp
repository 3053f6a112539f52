// kv.hpp -- device helpers of the paged cache's kernels.
#pragma once

#include "i8.hpp"
#include "kernels.hpp"

namespace md {

// A sequence's lengths and pages as the device arrays state them.  One whose
// statements do not hold together is bad: its cache is neither read nor
// written, and attention gives NaN for its rows.
struct Seq {
  int row0, nq, len;
  const int* table;
  bool bad;
};
MD_DEV Seq seq_of(const KvBatch& b, int s, int page) {
  Seq q;
  const int a = b.q_start[s], e = b.q_start[s + 1];
  q.len = b.kv_len[s];
  q.table = b.table + (int64_t)s * b.table_stride;
  q.row0 = a;
  q.nq = e - a;
  q.bad = q.len < 0 || q.len > b.max_kv || (int64_t)q.len > (int64_t)b.table_stride * page;
  if (a < 0 || e < a || e > b.rows) {  // its rows cannot be told: none of them is touched
    q.nq = 0;
    q.bad = true;
  } else if (q.nq > b.max_q) {         // more than the grid covers: the first max_q of them
    q.nq = b.max_q;
    q.bad = true;
  }
  if (q.bad) q.len = 0;
  return q;
}

// The tiles of 64 positions [t0, t1) that the columns [c0, c1) see (column
// c is query c / G), and the positions full_lo .. full_hi that all of them see.
// M (masked): they also see positions in the tiles [0, head), head <= t0: the
// first ones, which stay visible.
struct Span {
  int t0, t1, full_lo, full_hi, head;
};
template <bool M>
MD_DEV Span span_of(const KvAttn& a, const Seq& q, int c0, int c1) {
  Span s;
  s.head = 0;
  if (M && a.tree) {
    // before the run: all, or window less the run's tokens that a row sees, which
    // may be none or the whole run; in it: what the row's bits say
    const int base = q.len - q.nq;
    s.full_hi = base - 1;
    s.t0 = 0;
    s.full_lo = 0;
    if (a.window) {
      s.t0 = max(base - a.window, 0) >> 6;
      s.full_lo = max(min(base, base - a.window + q.nq), 0);
    }
    s.t1 = max((q.len + 63) >> 6, s.t0);
    s.head = min((a.sinks + 63) >> 6, s.t0);
    return s;
  }
  if (!a.causal) {
    s.full_lo = 0;
    s.full_hi = q.len - 1;
    s.t0 = 0;
    s.t1 = (q.len + 63) >> 6;
    return s;
  }
  const int p0 = q.len - q.nq + c0 / a.G, p1 = q.len - q.nq + (c1 - 1) / a.G;  // first and last query's position
  s.full_hi = p0;
  s.t0 = 0;
  s.full_lo = 0;
  if (a.window) {
    s.t0 = max(p0 - a.window + 1, 0) >> 6;
    s.full_lo = max(p1 - a.window + 1, 0);
  }
  s.t1 = max((p1 >> 6) + 1, s.t0);
  if (M) s.head = min((a.sinks + 63) >> 6, s.t0);
  return s;
}

// Bits lo .. hi - 1 of sixteen.
MD_DEV uint32_t bits16(int lo, int hi) {
  lo = min(max(lo, 0), 16);
  hi = min(max(hi, 0), 16);
  return ((1u << hi) - 1u) & ~((1u << lo) - 1u);
}

// Where a row of a masked call starts and ends to see positions by their
// number, and its bits of the run (null: no tree).
struct Seen {
  int lo, hi;
  const uint64_t* bits;
};
MD_DEV Seen seen_of(const KvAttn& a, const Seq& q, int qt) {
  Seen s;
  const int base = q.len - q.nq;
  s.bits = a.tree ? a.tree + ((int64_t)q.row0 + qt) * a.words : nullptr;
  s.hi = a.tree ? base - 1 : base + qt;
  s.lo = 0;
  if (a.window) {
    int left = a.window;
    if (a.tree) {
      for (int w = 0; w << 6 < q.nq; ++w) {
        const int n = q.nq - (w << 6);  // the run's tokens of this word
        left -= __popcll(n < 64 ? s.bits[w] & ((1ull << n) - 1ull) : s.bits[w]);
      }
    }
    s.lo = max(s.hi + 1 - max(left, 0), 0);
  }
  return s;
}
// Which of the positions first .. first + 15 it sees.
MD_DEV uint32_t seen16(const KvAttn& a, const Seq& q, const Seen& s, int first) {
  uint32_t m = bits16(s.lo - first, s.hi + 1 - first);
  if (a.window) m |= bits16(0, min(s.hi + 1, a.sinks) - first);
  if (s.bits) {
    const int at = first - (q.len - q.nq);  // the run's token at `first`
    if (at > -16 && at < q.nq) {
      uint64_t b;
      if (at < 0) {
        b = s.bits[0] << -at;
      } else {
        const int w = at >> 6, r = at & 63;
        b = s.bits[w] >> r;
        if (r > 48 && w + 1 < a.words) b |= s.bits[w + 1] << (64 - r);
      }
      m |= (uint32_t)b & bits16(-at, q.nq - at);
    }
  }
  return m;
}

// The column tile of a workgroup, the b-th of n: where the mask is causal the
// last columns see the most, so the heaviest tiles start first; when all run
// at once, two on a compute unit, the second half goes the other way round and
// each unit gets a heavy and a light one (4096 new of 5003 tokens, 16 heads on 4
// of 128 channels: 165 us against 166 heaviest first throughout and 187 in the
// heads' order, on a kernel that takes 149 now).
MD_DEV int column_tile(const KvAttn& a, int b, int n) {
  if (!a.causal) return b;
  const int half = (n + 1) / 2;
  return a.snake && b >= half ? b - half : n - 1 - b;
}

// Four neighbouring outputs of a row's head.
MD_DEV void store_out4(const KvAttn& a, int64_t row, int head, int D, int d, float x, float y, float z, float w) {
  const int64_t at = row * a.out_stride + (int64_t)head * D + d;
  if (a.yt == 0) *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = make_float4(x, y, z, w);
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
        make_uint2(to_bf16(x) | (uint32_t)to_bf16(y) << 16, to_bf16(z) | (uint32_t)to_bf16(w) << 16);
}

}  // namespace md

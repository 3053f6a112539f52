// logprob.hip -- log probabilities of given tokens, entropy and the largest
// alternatives of rows of logits.
//
//   z = scale x,  log p = z - log sum exp z,  entropy = log sum exp z - sum z exp z / sum exp z
//
// Bound by the one read of the logits.  A workgroup takes a segment of a row, some
// steps of N values a thread in registers, the next step's on their way; a thread
// keeps its maximum and its sums of exp and z exp relative to it.  It leaves the
// segment's, and its `top` largest values as 64-bit keys: the order of fp32 in the
// high word, the complement of the id in the low one, so that keys are all
// different, an integer comparison is the order, and equal logits go to the lower
// id.  A row of one segment is finished there, else by a second kernel, a wave for
// each row.
//
// The largest: of each wave's 64 lanes the maxima of the first step are sorted; at
// least `top` values reach the `top`-th of them, and the highest of the four waves'
// bounds lets little more than `top` values pass into LDS.  Later steps use the
// same bound until many have passed; then the list is ranked (each key counts the
// larger ones), cut to `top`, and the bound is its last.  A step that would
// overfill it (equal or ascending logits) has its winners taken one at a time.
//
// Measured: 4096 rows of 32000 fp32 logits without alternatives 88 us (524 MB, 6.0
// TB/s); 288 rows of 131071 bf16 with the 8 largest 32 us and 4.6 for the join (75
// MB: the vector ALU is busy for 21 of them, a chain of steps with a barrier waits for
// the rest; a step a workgroup, bounds and sums joined for each, 44 and 10).  There,
// with the join: three or twelve workgroups a compute unit instead of six 39 and 38 us
// against 37, steps of 16 values a thread 41, 80 registers (six workgroups a compute
// unit at once) 45.  One row of 131071 fp32 with the 5 largest 9.3 us (the join's keys
// ranked without a bound 37).
#include <hip/hip_runtime.h>

#include "common.hpp"
#include "i8.hpp"
#include "kernels.hpp"
#include "rows.hpp"

namespace md {

typedef unsigned long long Key;

// fp32 in the order of unsigned integers; a NaN below -inf (-0 is +0).
MD_DEV uint32_t order_of(float x) { return x == x ? order_key32(x) : 1u; }
MD_DEV Key key_of(float x, int id) { return (Key)order_of(x) << 32 | (uint32_t)~id; }

// The n-th largest (n in 1..64) of the wave's values, one a lane.
template <int OFF>
MD_DEV Key other(Key k) {
  const float lo = xor_lanes<OFF>(__uint_as_float((uint32_t)k)), hi = xor_lanes<OFF>(__uint_as_float((uint32_t)(k >> 32)));
  return (Key)__float_as_uint(hi) << 32 | __float_as_uint(lo);
}
template <int OFF>
MD_DEV float other(float v) { return xor_lanes<OFF>(v); }
template <int SIZE, int OFF, typename V>
MD_DEV V sort_step(V v) {
  const int lane = threadIdx.x & 63;
  const V o = other<OFF>(v);
  const bool up = ((lane & SIZE) == 0) == ((lane & OFF) == 0);  // this lane keeps the larger one
  v = (v > o) == up ? v : o;
  if constexpr (OFF > 1) return sort_step<SIZE, OFF / 2>(v);
  else return v;
}
template <int SIZE = 2, typename V>
MD_DEV V wave_nth(V v, int n) {
  v = sort_step<SIZE, SIZE / 2>(v);
  if constexpr (SIZE < 64) return wave_nth<2 * SIZE>(v, n);
  else return __shfl(v, n - 1, 64);
}

// The larger of the wave's keys, in every lane.
template <int OFF = 32>
MD_DEV Key wave_max_key(Key k) {
  const Key o = other<OFF>(k);
  k = o > k ? o : k;
  if constexpr (OFF > 1) return wave_max_key<OFF / 2>(k);
  else return k;
}

// What the second kernel reads of a segment.
struct Part {
  float m, s, sx, pad;
};

struct Sums {
  float m;
  double s, sx;  // sum exp(z - z_m), sum (z - z_m) exp(z - z_m)
};

MD_DEV float nan_f32() { return __uint_as_float(0x7FC00000u); }

template <int XT>
MD_DEV float logit(const LogpArgs& g, int64_t row, int id) {
  const int64_t at = row * g.stride + id;
  if constexpr (XT == XF32) return static_cast<const float*>(g.logits)[at];
  else return __uint_as_float((uint32_t)static_cast<const uint16_t*>(g.logits)[at] << 16);
}

// One wave: where fewer than top logits are above -inf, the row's -inf ones follow
// in order, then its NaNs.
template <int XT>
MD_DEV void fill(const LogpArgs& g, int64_t row, int have, Key* top) {
  const int lane = threadIdx.x & 63;
  for (int pass = 0; pass < 2 && have < g.top; ++pass)
    for (int i = 0; i < g.vocab && have < g.top; i += 512) {
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = i + 64 * j + lane < g.vocab ? logit<XT>(g, row, i + 64 * j + lane) : 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool it = pass ? x[j] != x[j] : x[j] == -INFINITY;
        const uint64_t all = __builtin_amdgcn_ballot_w64(it);
        const int at = have + __popcll(all & ((1ull << lane) - 1ull));
        if (it && at < g.top) top[at] = key_of(x[j], i + 64 * j + lane);
        have += __popcll(all);
      }
    }
}

// A row's outputs from its sums: thread t of n does every n-th.
template <int XT>
MD_DEV void finish(const LogpArgs& g, int64_t row, const Sums& r, const Key* keys, int t, int n) {
  const bool ok = r.s > 0.0 && r.m < INFINITY;  // false for NaN too
  const double log_s = ok ? log(r.s) : 0.0;
  const double scale = (double)g.scale;
  if (t == 0 && g.entropy) g.entropy[row] = ok ? (float)(log_s - r.sx / r.s) : nan_f32();
  for (int i = t; i < g.n_tokens; i += n) {
    const int id = g.tokens[row * g.n_tokens + i];
    float lp = nan_f32();
    if (ok && (unsigned)id < (unsigned)g.vocab) lp = (float)(((double)logit<XT>(g, row, id) - (double)r.m) * scale - log_s);
    g.logprobs[row * g.n_tokens + i] = lp;
  }
  for (int i = t; i < g.top; i += n) {
    const Key k = keys[i];
    const uint32_t o = (uint32_t)(k >> 32);
    g.top_ids[row * g.top + i] = (int)~(uint32_t)k;
    g.top_logprobs[row * g.top + i] = ok ? (float)(((double)key_logit(o) - (double)r.m) * scale - log_s) : nan_f32();
  }
}

// The top largest of the cnt keys in LDS, in descending order, to out.
MD_DEV void rank_keys(const Key* list, int cnt, int top, Key* out, int t, int n) {
  for (int i = t; i < cnt; i += n) {
    const Key k = list[i];
    int r = 0, j = 0;
    for (; j + 8 <= cnt; j += 8) {
#pragma unroll
      for (int u = 0; u < 8; ++u) r += list[j + u] > k;
    }
    for (; j < cnt; ++j) r += list[j] > k;
    if (r < top) out[r] = k;
  }
}

// The next fp32 value (of +inf: none, a NaN, which nothing reaches).
MD_DEV float above(float x) {
  const uint32_t u = __float_as_uint(x);
  return __uint_as_float(x == 0.0f ? 1u : u >> 31 ? u - 1u : u + 1u);
}

constexpr int kPass = 512;                       // keys that a list holds
constexpr float kLowest = -3.4028234663852886e38f;

template <int XT, int N, int NW, bool TOP>  // N values a thread and step, NW waves
__global__ __launch_bounds__(64 * NW) void k_logprob(LogpArgs g) {
  constexpr int V = XT == XF32 ? 4 : 8, J = N / V, B = 64 * NW;
  __shared__ float s_m[NW], s_s[NW], s_sx[NW], s_tau[NW];
  __shared__ int s_bad[NW], s_cnt;
  __shared__ Key s_best[NW], s_top[kMaxTop], s_list[kPass];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t row = blockIdx.y + (int64_t)gridDim.y * blockIdx.z;
  if (row >= g.rows) return;
  // the row's first value may lie anywhere: loads go by the 16 bytes that hold
  // it, and what lies before it or past its end is left out
  const int es = XT == XF32 ? 4 : 2;
  const char* base = static_cast<const char*>(g.logits) + row * g.stride * es;
  const int shift = (int)(reinterpret_cast<uintptr_t>(base) & 15) / es;
  const char* from = base - shift * es;
  const int last = g.vocab + shift;  // values [shift, last) of `from` are the row's
  const int c_end = min((blockIdx.x + 1) * g.steps * (B * N), (last + B * N - 1) / (B * N) * (B * N));
  // buffer loads: past the row's last 16 bytes they read zeros and touch no memory
  const rsrc_t res = make_res(from, (last * es + 15) & ~15);
  u32x4 w[J];
  int c0 = blockIdx.x * g.steps * (B * N);
  auto load = [&](int at) {
#pragma unroll
    for (int j = 0; j < J; ++j) w[j] = __builtin_amdgcn_raw_buffer_load_b128(res, (j * B + tid) * 16, at * es, 0);
  };
  if (c0 < c_end) load(c0);
  if (tid == 0) s_cnt = 0;
  // y = z log2 e, relative to the thread's maximum m, the lowest finite value at
  // first; exp2(-300) is 0 in fp32, so that -inf adds nothing
  const float c = g.scale * 1.4426950408889634f;
  float m = kLowest, s = 0.0f, sx = 0.0f, tau = -INFINITY;
  int cnt = 0;
  bool bad = false;
  for (; c0 < c_end; c0 += B * N) {
    float v[N];
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if constexpr (XT == XF32) v[j * V + e] = __uint_as_float(w[j][e]);
        else v[j * V + e] = __uint_as_float(e & 1 ? w[j][e >> 1] & 0xFFFF0000u : w[j][e >> 1] << 16);
      }
    if (c0 + B * N < c_end) load(c0 + B * N);
    auto id_of = [&](int n) { return c0 + (n / V * B + tid) * V + n % V - shift; };  // value n's, if it is the row's
    if (c0 < shift || c0 + B * N > last) {
#pragma unroll
      for (int n = 0; n < N; ++n)
        if ((unsigned)id_of(n) >= (unsigned)g.vocab) v[n] = -INFINITY;
    }
    float mine = -INFINITY;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      mine = fmaxf(mine, v[n]);
      bad |= v[n] != v[n];
    }
    const float m1 = fmaxf(m, mine), d = fmaxf((m - m1) * c, -300.0f), f = __builtin_amdgcn_exp2f(d);
    m = m1;
    float ps = 0.0f, px = 0.0f;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const float y = fmaxf((v[n] - m) * c, -300.0f);
      const float e = __builtin_amdgcn_exp2f(y);
      ps += e;
      px = fmaf(y, e, px);
    }
    sx = fmaf(f, fmaf(d, s, sx), px);
    s = fmaf(f, s, ps);
    if constexpr (TOP) {
      const bool first = !(tau > -INFINITY);
      if (first) {  // the same in all threads
        const float nth = wave_nth(mine, g.top);
        __syncthreads();  // s_tau of a step before
        if (lane == 0) s_tau[wave] = nth;
        __syncthreads();
        tau = s_tau[0];
#pragma unroll
        for (int i = 1; i < NW; ++i) tau = fmaxf(tau, s_tau[i]);
      }
      // without a bound: all but -inf; behind a bound's step only larger ones (the lower ids are there)
      const float pass = first ? fmaxf(tau, kLowest) : above(tau);
      if (__builtin_amdgcn_ballot_w64(mine >= pass)) {
#pragma unroll
        for (int n = 0; n < N; ++n)
          if (v[n] >= pass) {
            const int at = atomicAdd(&s_cnt, 1);
            if (at < kPass) s_list[at] = key_of(v[n], id_of(n));
          }
      }
      __syncthreads();
      const int had = cnt;
      cnt = s_cnt;
      __syncthreads();  // all have read it
      if (cnt > kPass) {
        // too many: this step's winners one at a time, in place of what it added
        Key below = ~(Key)0;
        cnt = had;
        for (int j = 0; j < g.top; ++j) {
          Key best = 0;
#pragma unroll 1
          for (int n = 0; n < N; ++n) {  // (values read anew: they need not stay in registers for this)
            const int id = id_of(n);
            const float x = (unsigned)id < (unsigned)g.vocab ? logit<XT>(g, row, id) : -INFINITY;
            const Key k = x >= pass ? key_of(x, id) : 0;
            if (k < below && k > best) best = k;
          }
          best = wave_max_key(best);
          __syncthreads();
          if (lane == 0) s_best[wave] = best;
          __syncthreads();
#pragma unroll
          for (int i = 0; i < NW; ++i) best = s_best[i] > best ? s_best[i] : best;
          if (tid == 0) s_list[cnt] = best;
          ++cnt;
          below = best;
        }
        if (tid == 0) s_cnt = cnt;
        __syncthreads();
      }
      if (cnt > kPass / 2) {  // cut to the largest: a step adds up to kMaxTop where it overfills the list
        rank_keys(s_list, cnt, g.top, s_top, tid, B);
        __syncthreads();
        if (tid < g.top) s_list[tid] = s_top[tid];
        if (tid == 0) s_cnt = g.top;
        cnt = g.top;
        tau = key_logit((uint32_t)(s_top[g.top - 1] >> 32));
        __syncthreads();
      }
    }
  }
  float all = group_max<64>(m);
  const bool wave_bad = __builtin_amdgcn_ballot_w64(bad) != 0;
  if (lane == 0) s_m[wave] = all, s_bad[wave] = wave_bad;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NW; ++i) all = fmaxf(all, s_m[i]), bad |= s_bad[i] != 0;
  const float d = fmaxf((m - all) * c, -300.0f), f = __builtin_amdgcn_exp2f(d);
  sx = group_sum<64>(f * fmaf(d, s, sx));
  s = group_sum<64>(f * s);
  if (lane == 0) s_s[wave] = s, s_sx[wave] = sx;
  Key* out = g.segs == 1 ? s_top : reinterpret_cast<Key*>(g.keys) + (row * g.segs + blockIdx.x) * g.top;
  if constexpr (TOP) {
    __syncthreads();  // s_top of a cut before
    for (int i = cnt + tid; i < g.top; i += B) out[i] = 0;
    rank_keys(s_list, cnt, g.top, out, tid, B);
  }
  __syncthreads();
  Sums r{all, 0.0, 0.0};
#pragma unroll
  for (int i = 0; i < NW; ++i) r.s += s_s[i], r.sx += s_sx[i];
  r.sx *= 0.6931471805599453;
  if (bad) r.s = __longlong_as_double(0x7FF8000000000000ll);
  if (g.segs > 1) {
    if (tid == 0) reinterpret_cast<Part*>(g.part)[row * g.segs + blockIdx.x] = Part{all, (float)r.s, (float)r.sx, 0.0f};
    return;
  }
  if (TOP && cnt < g.top) {
    if (wave == 0) fill<XT>(g, row, cnt, s_top);
    __syncthreads();
  }
  finish<XT>(g, row, r, s_top, tid, B);
}

// A row's segments: one wave.  Up to 64 keys are ranked among all; of more the
// largest are bounded first, as in the segment: a lane's keys in steps of 64, at
// most kMaxJoin of them.  Keys of 0 are none.
template <int XT>
__global__ __launch_bounds__(64) void k_logprob_join(LogpArgs g) {
  __shared__ Key s_list[kMaxTop * kMaxJoin], s_top[kMaxTop];
  __shared__ int s_cnt;
  const int lane = threadIdx.x;
  const int64_t row = blockIdx.x;
  const Part* p = reinterpret_cast<const Part*>(g.part) + row * g.segs;
  const Key* k = reinterpret_cast<const Key*>(g.keys) + row * g.segs * g.top;
  const int n = g.segs * g.top;
  Part q[2];  // up to 128 segments
#pragma unroll
  for (int i = 0; i < 2; ++i) q[i] = lane + 64 * i < g.segs ? p[lane + 64 * i] : Part{kLowest, 0.0f, 0.0f, 0.0f};
  Key key[kPass / 64];  // the keys, up to kPass of them
#pragma unroll
  for (int i = 0; i < kPass / 64; ++i) key[i] = n <= kPass && lane + 64 * i < n ? k[lane + 64 * i] : 0;
  if (lane == 0) s_cnt = 0;
  const float m = group_max<64>(fmaxf(q[0].m, q[1].m));
  double s = 0.0, sx = 0.0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (64 * i >= g.segs) break;
    // (a segment of nothing but -inf: its sums are 0, and its maximum the lowest finite value)
    const double d = ((double)q[i].m - (double)m) * (double)g.scale, w = exp(d);
    s += w * q[i].s;
    sx += w * ((double)q[i].sx + d * q[i].s);
  }
  const Sums r{m, wave_total(s), wave_total(sx)};
  __syncthreads();
  Key best = 0;
  if (n <= kPass) {
#pragma unroll
    for (int i = 0; i < kPass / 64; ++i) best = key[i] > best ? key[i] : best;
  } else {
    for (int i = lane; i < n; i += 64) best = k[i] > best ? k[i] : best;
  }
  Key tau = 1;
  if (n > 64) {
    const Key nth = wave_nth(best, g.top);
    if (nth > tau) tau = nth;
  }
  auto pass = [&](Key x) {
    if (x >= tau) s_list[atomicAdd(&s_cnt, 1)] = x;
  };
  if (n <= kPass) {
#pragma unroll
    for (int i = 0; i < kPass / 64; ++i) pass(key[i]);
  } else {
    for (int i = lane; i < n; i += 64) pass(k[i]);
  }
  __syncthreads();
  const int have = s_cnt;
  rank_keys(s_list, have, g.top, s_top, lane, 64);
  __syncthreads();
  if (have < g.top) {
    fill<XT>(g, row, have, s_top);
    __syncthreads();
  }
  finish<XT>(g, row, r, s_top, lane, 64);
}

// Values a thread and step: 32, or 8 where that leaves compute units without work or
// where one step of 8 holds a row (us, 32 and 8, without alternatives and with the 8
// largest: 4096 rows of 100 bf16 16.0 and 10.2, 31.0 and 18.8, of 2000 fp32 16.8 and
// 11.1, 32.2 and 20.3; 600 rows alike in both); segments of a row: enough for some
// workgroups on every compute unit.
LogpPlan logprob_plan(int64_t rows, int vocab) {
  LogpPlan p{};
  const int64_t cus = device_cus();
  auto steps_of = [&](int n) { return (vocab + 7 + 256 * n - 1) / (256 * n); };  // a row may begin up to 7 values past 16 bytes
  p.values = rows * steps_of(32) >= 2 * cus && steps_of(8) > 1 ? 32 : 8;
  const int total = steps_of(p.values);
  int64_t segs = (kSegGroups * cus + rows - 1) / rows;
  if (segs > total) segs = total;
  if (segs > kMaxSegs) segs = kMaxSegs;
  p.steps = (int)((total + segs - 1) / segs);
  p.segs = (total + p.steps - 1) / p.steps;
  p.waves = 4;
  // A row that one step of sixteen waves holds, at least half full, and a compute unit
  // for each row: no second kernel.  us, in one and in two, the 5 largest of fp32, one
  // row of 32000 in a graph 9.4 and 9.2, from the host 11.6 and 14.3; 64 rows 10.3 and
  // 11.2, 256 rows 13.7 and 16.0; one of 4000 9.6 and 8.3, of 65000 (two steps) 13.5
  // and 9.0.
  constexpr int wide = 1024 * 32;
  if (rows <= cus && vocab > wide / 2 && vocab + 7 <= wide) p = LogpPlan{32, 16, 1, 1};
  return p;
}

hipError_t launch_logprob(const LogpArgs& g, int xt, const LogpPlan& p, hipStream_t st) {
  const unsigned y = g.rows < 32768 ? (unsigned)g.rows : 32768u, z = (unsigned)((g.rows + y - 1) / y);
  const dim3 grid(g.segs, y, z), block(64 * p.waves);
#define MD_LOGP(X_, N_, W_)                                                                    \
  do {                                                                                         \
    if (g.top) hipLaunchKernelGGL((k_logprob<X_, N_, W_, true>), grid, block, 0, st, g);       \
    else hipLaunchKernelGGL((k_logprob<X_, N_, W_, false>), grid, block, 0, st, g);            \
  } while (0)
  if (xt == XF32) {
    if (p.waves == 16) MD_LOGP(XF32, 32, 16);
    else if (p.values == 32) MD_LOGP(XF32, 32, 4);
    else MD_LOGP(XF32, 8, 4);
  } else {
    if (p.waves == 16) MD_LOGP(XBF16, 32, 16);
    else if (p.values == 32) MD_LOGP(XBF16, 32, 4);
    else MD_LOGP(XBF16, 8, 4);
  }
#undef MD_LOGP
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || g.segs == 1) return e;
  if (xt == XF32) hipLaunchKernelGGL((k_logprob_join<XF32>), dim3((unsigned)g.rows), dim3(64), 0, st, g);
  else hipLaunchKernelGGL((k_logprob_join<XBF16>), dim3((unsigned)g.rows), dim3(64), 0, st, g);
  return hipGetLastError();
}

}  // namespace md

// logprob.hip -- log probabilities of given tokens, entropy and the largest
// alternatives of rows of logits.
//
//   z = scale x,  log p = z - log sum exp z,  entropy = log sum exp z - sum z exp z / sum exp z
//
// Bound by the one read of the logits.  A workgroup takes a chunk of a row into
// registers, 32 values a thread (8 where there are few chunks), and leaves for
// it the maximum, the sums of exp and z exp relative to it, and the chunk's
// `top` largest values as 64-bit keys: the order of fp32 in the high word, the
// complement of the id in the low one, so that keys are all different, an
// integer comparison is the order, and equal logits go to the lower id.  A row
// of one chunk is finished there, else by a second kernel, a wave for each row.
//
// The largest of a wave's values: its 64 lanes' own maxima are sorted, and the
// `top`-th of them is a bound that at least `top` values reach.  Only values of
// those `top` lanes can (the keys differ), so at most top values a lane, and
// usually little more than top, pass into LDS, where each counts the larger
// ones: its rank.
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

// The n-th largest (n in 1..64) of the wave's keys, one a lane.
MD_DEV Key wave_nth(Key k, int n) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int size = 2; size <= 64; size <<= 1)
#pragma unroll
    for (int off = size >> 1; off; off >>= 1) {
      const Key o = __shfl_xor(k, off, 64);
      const bool up = ((lane & size) == 0) == ((lane & off) == 0);  // this lane keeps the larger one
      k = (k > o) == up ? k : o;
    }
  return __shfl(k, n - 1, 64);
}

// What the second kernel reads of a chunk.
struct Part {
  float m, s, sx, pad;
};

struct Sums {
  float m;
  double s, sx;  // sum exp(z - z_m), sum (z - z_m) exp(z - z_m)
};

MD_DEV float nan_f32() { return __uint_as_float(0x7FC00000u); }

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
    if (ok && (unsigned)id < (unsigned)g.vocab) {
      const int64_t at = row * g.stride + id;
      float x;
      if constexpr (XT == XF32) x = static_cast<const float*>(g.logits)[at];
      else x = __uint_as_float((uint32_t)static_cast<const uint16_t*>(g.logits)[at] << 16);
      lp = (float)(((double)x - (double)r.m) * scale - log_s);
    }
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
    int r = 0;
    for (int j = 0; j < cnt; ++j) r += list[j] > k;
    if (r < top) out[r] = k;
  }
}

template <int XT, int N>  // N values a thread
__global__ __launch_bounds__(256) void k_logprob(LogpArgs g) {
  constexpr int V = XT == XF32 ? 4 : 8, J = N / V;
  __shared__ float s_m[4], s_s[4], s_sx[4];
  __shared__ int s_bad[4], s_cnt;
  __shared__ Key s_tau[4], s_top[kMaxTop];
  __shared__ Key s_list[4 * kMaxTop * N];
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
  const int c0 = blockIdx.x * 256 * N;
  float v[N];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int i = c0 + (j * 256 + tid) * V;
    u32x4 w{0, 0, 0, 0};
    if (i < last) w = *reinterpret_cast<const u32x4*>(from + (int64_t)i * es);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      float x;
      if constexpr (XT == XF32) x = __uint_as_float(w[e]);
      else x = __uint_as_float(e & 1 ? w[e >> 1] & 0xFFFF0000u : w[e >> 1] << 16);
      v[j * V + e] = i + e >= shift && i + e < last ? x : -INFINITY;
    }
  }
  float m = -INFINITY;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    m = fmaxf(m, v[i]);
    bad |= v[i] != v[i];
  }
  m = group_max<64>(m);
  if (lane == 0) s_m[wave] = m;
  const bool wave_bad = __builtin_amdgcn_ballot_w64(bad) != 0;
  if (lane == 0) s_bad[wave] = wave_bad;
  if (tid == 0) s_cnt = 0;
  __syncthreads();
  m = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
  bad = s_bad[0] | s_bad[1] | s_bad[2] | s_bad[3];
  const float ref = m > -INFINITY ? m : 0.0f;
  float s = 0.0f, sx = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float z = fmaxf((v[i] - ref) * g.scale, -200.0f);  // exp(-200) is 0 here: -inf adds nothing
    const float e = __builtin_amdgcn_exp2f(z * 1.4426950408889634f);
    s += e;
    sx = fmaf(z, e, sx);
  }
  s = group_sum<64>(s);
  sx = group_sum<64>(sx);
  if (lane == 0) s_s[wave] = s, s_sx[wave] = sx;
  if (g.top) {
    Key best = 0;
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int i = c0 + (j * 256 + tid) * V + e;
        const Key k = i >= shift && i < last ? key_of(v[j * V + e], i - shift) : 0;
        best = k > best ? k : best;
      }
    const Key nth = wave_nth(best, g.top);
    if (lane == 0) s_tau[wave] = nth;
    __syncthreads();
    // the best of the four bounds; a wave with fewer values than top has bound 0
    Key tau = 1;
#pragma unroll
    for (int w = 0; w < 4; ++w) tau = s_tau[w] > tau ? s_tau[w] : tau;
    if (__builtin_amdgcn_ballot_w64(best >= tau)) {
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const int i = c0 + (j * 256 + tid) * V + e;
          const Key k = i >= shift && i < last ? key_of(v[j * V + e], i - shift) : 0;
          if (k >= tau) s_list[atomicAdd(&s_cnt, 1)] = k;
        }
    }
  }
  __syncthreads();
  Sums r{m, 0.0, 0.0};
#pragma unroll
  for (int w = 0; w < 4; ++w) r.s += s_s[w], r.sx += s_sx[w];
  if (bad) r.s = __longlong_as_double(0x7FF8000000000000ll);
  const int cnt = g.top ? s_cnt : 0;
  if (g.chunks == 1) {
    if (g.top) rank_keys(s_list, cnt, g.top, s_top, tid, 256);
    __syncthreads();
    finish<XT>(g, row, r, s_top, tid, 256);
    return;
  }
  const int64_t at = row * g.chunks + blockIdx.x;
  if (tid == 0) reinterpret_cast<Part*>(g.part)[at] = Part{m, (float)r.s, (float)r.sx, 0.0f};
  if (g.top) {
    Key* out = reinterpret_cast<Key*>(g.keys) + at * g.top;
    for (int i = cnt + tid; i < g.top; i += 256) out[i] = 0;  // a last chunk of fewer values
    rank_keys(s_list, cnt, g.top, out, tid, 256);
  }
}

// A row's chunks: one wave.  Its keys as in the chunk, a lane's in steps of 64.
template <int XT>
__global__ __launch_bounds__(64) void k_logprob_join(LogpArgs g) {
  __shared__ Key s_list[kMaxTop * kMaxJoin], s_top[kMaxTop];
  __shared__ int s_cnt;
  const int lane = threadIdx.x;
  const int64_t row = blockIdx.x;
  const Part* p = reinterpret_cast<const Part*>(g.part) + row * g.chunks;
  float m = -INFINITY;
  for (int i = lane; i < g.chunks; i += 64) m = fmaxf(m, p[i].m);
  m = group_max<64>(m);
  const double ref = m > -INFINITY ? (double)m : 0.0;
  double s = 0.0, sx = 0.0;
  for (int i = lane; i < g.chunks; i += 64) {
    const Part q = p[i];
    if (q.m == -INFINITY && q.s == 0.0f) continue;  // nothing there (a NaN among its values: s is NaN)
    const double d = ((double)q.m - ref) * (double)g.scale, w = exp(d);
    s += w * q.s;
    sx += w * ((double)q.sx + d * q.s);
  }
  const Sums r{m, wave_sum_f64(s), wave_sum_f64(sx)};
  if (g.top) {
    const Key* k = reinterpret_cast<const Key*>(g.keys) + row * g.chunks * g.top;
    const int n = g.chunks * g.top;
    Key best = 0;
    for (int i = lane; i < n; i += 64) best = k[i] > best ? k[i] : best;
    if (lane == 0) s_cnt = 0;
    const Key nth = wave_nth(best, g.top), tau = nth > 1 ? nth : 1;
    __syncthreads();
    for (int i = lane; i < n; i += 64)
      if (k[i] >= tau) s_list[atomicAdd(&s_cnt, 1)] = k[i];
    __syncthreads();
    rank_keys(s_list, s_cnt, g.top, s_top, lane, 64);
    __syncthreads();
  }
  finish<XT>(g, row, r, s_top, lane, 64);
}

// Values a thread: 32, or 8 where that leaves compute units without work.
int logprob_values(int64_t rows, int vocab) {
  return rows * ((vocab + 8191) / 8192) >= 2 * (int64_t)device_cus() || vocab > kMaxChunks * 2048 - 8 ? 32 : 8;
}
int logprob_chunks(int64_t rows, int vocab) {
  const int per = 256 * logprob_values(rows, vocab);
  return (vocab + 7 + per - 1) / per;  // a row may begin up to 7 values past 16 bytes
}

hipError_t launch_logprob(const LogpArgs& g, int xt, int values, hipStream_t st) {
  const unsigned y = g.rows < 32768 ? (unsigned)g.rows : 32768u, z = (unsigned)((g.rows + y - 1) / y);
  const dim3 grid(g.chunks, y, z), block(256);
  if (xt == XF32) {
    if (values == 32) hipLaunchKernelGGL((k_logprob<XF32, 32>), grid, block, 0, st, g);
    else hipLaunchKernelGGL((k_logprob<XF32, 8>), grid, block, 0, st, g);
  } else {
    if (values == 32) hipLaunchKernelGGL((k_logprob<XBF16, 32>), grid, block, 0, st, g);
    else hipLaunchKernelGGL((k_logprob<XBF16, 8>), grid, block, 0, st, g);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || g.chunks == 1) return e;
  if (xt == XF32) hipLaunchKernelGGL((k_logprob_join<XF32>), dim3((unsigned)g.rows), dim3(64), 0, st, g);
  else hipLaunchKernelGGL((k_logprob_join<XBF16>), dim3((unsigned)g.rows), dim3(64), 0, st, g);
  return hipGetLastError();
}

}  // namespace md

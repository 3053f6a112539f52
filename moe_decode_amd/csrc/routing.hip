// routing.hip -- routing to experts for any number of tokens: logits in fp64,
// softmax or sigmoid scores, a bias that only the choice sees, groups, top-k
// and gates.
//
//   l = W_r x (+ b), s = sigmoid(l) or softmax(l), c = s + balance,
//   idx = the k largest c of the kept groups, gates = s[idx] (/ their sum) * scale
//
// Scores that lie next to each other decide, so everything up to a gate is
// fp64 (the logits are rounded to fp32 once, as the layer's own router's are):
// products of two fp32 values are exact there, and the choice is the
// definition's.
#include <hip/hip_runtime.h>

#include "common.hpp"
#include "i8.hpp"
#include "kernels.hpp"
#include "rows.hpp"

namespace md {

typedef double f64x4 __attribute__((ext_vector_type(4)));

// ---- logits ----------------------------------------------------------------

// Few tokens: a workgroup for each expert, its threads share the width; sums
// as partials [t][e] of one slice.
template <int XT>
__global__ __launch_bounds__(256) void k_route_few(const void* __restrict__ x, int T, int H, const float* __restrict__ Wr,
                                                   int E, double* __restrict__ part) {
  __shared__ double s_sum[kRouteFew][4];
  const int e = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  double acc[kRouteFew];
#pragma unroll
  for (int t = 0; t < kRouteFew; ++t) acc[t] = 0.0;
  for (int c = 8 * tid; c < H; c += 2048) {
    float w[8];
    load8<XF32>(Wr, (int64_t)e * H + c, w);
#pragma unroll
    for (int t = 0; t < kRouteFew; ++t) {
      if (t >= T) break;
      float v[8];
      load8<XT>(x, (int64_t)t * H + c, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[t] = fma((double)w[i], (double)v[i], acc[t]);
    }
  }
#pragma unroll
  for (int t = 0; t < kRouteFew; ++t) {
    if (t >= T) break;
    const double v = wave_sum_f64(acc[t]);
    if (lane == 0) s_sum[t][wave] = v;
  }
  __syncthreads();
  if (tid < T) part[(int64_t)tid * E + e] = (s_sum[tid][0] + s_sum[tid][1]) + (s_sum[tid][2] + s_sum[tid][3]);
}

// Many tokens: a product on the fp64 matrix cores, 64 experts x 64 tokens a
// workgroup, a K-slice each; partials [s][t][e].  Operand layout of the
// 16x16x4 product: A[i][k], B[k][j] at lane 16 k + i (j), D[4 v + lane / 16]
// [lane % 16] in element v.
constexpr int kGT = 64, kGK = 32;

template <int XT>
__global__ __launch_bounds__(256) void k_route_gemm(const void* __restrict__ x, int T, int H, const float* __restrict__ Wr,
                                                    int E, int Ks, double* __restrict__ part) {
  __shared__ float sw[kGK][kGT + 1], sx[kGK][kGT + 1];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int e0 = blockIdx.x * kGT, sl = blockIdx.y;
  const int64_t t0 = (int64_t)blockIdx.z * kGT;
  const int li = lane & 15, kq = lane >> 4, er0 = 2 * (wave & 1), tc0 = 2 * (wave >> 1);
  f64x4 acc[2][2];
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int b = 0; b < 2; ++b) acc[a][b] = f64x4{0.0, 0.0, 0.0, 0.0};
  const int row = tid >> 2, c8 = 8 * (tid & 3);  // the thread's eight values of each tile
  float pw[8], px[8];
  auto fetch = [&](int kc) {
#pragma unroll
    for (int i = 0; i < 8; ++i) pw[i] = px[i] = 0.0f;
    if (e0 + row < E) load8<XF32>(Wr, (int64_t)(e0 + row) * H + kc + c8, pw);
    if (t0 + row < T) load8<XT>(x, (t0 + row) * H + kc + c8, px);
  };
  const int kbeg = sl * Ks, kend = min(kbeg + Ks, H);
  fetch(kbeg);
  for (int kc = kbeg; kc < kend; kc += kGK) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      sw[c8 + i][row] = pw[i];
      sx[c8 + i][row] = px[i];
    }
    __syncthreads();
    if (kc + kGK < kend) fetch(kc + kGK);
#pragma unroll
    for (int k4 = 0; k4 < kGK; k4 += 4) {
      double av[2], bv[2];
#pragma unroll
      for (int a = 0; a < 2; ++a) av[a] = (double)sw[k4 + kq][16 * (er0 + a) + li];
#pragma unroll
      for (int b = 0; b < 2; ++b) bv[b] = (double)sx[k4 + kq][16 * (tc0 + b) + li];
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b) acc[a][b] = __builtin_amdgcn_mfma_f64_16x16x4f64(av[a], bv[b], acc[a][b], 0, 0, 0);
    }
    __syncthreads();
  }
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int64_t t = t0 + 16 * (tc0 + b) + li;
      if (t >= T) continue;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int e = e0 + 16 * (er0 + a) + 4 * v + kq;
        if (e < E) part[((int64_t)sl * T + t) * E + e] = acc[a][b][v];
      }
    }
}

// ---- choice ----------------------------------------------------------------

// A double in the order of unsigned integers, above 0 (-0 is +0; no NaN comes here).
MD_DEV uint64_t order64(double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
  return u >> 63 ? ~u : u | 0x8000000000000000ull;
}

// A wave for each token: lane l holds experts l + 64 i.  Groups are valued by
// 64 / groups lanes each (a power of two); the k winners are taken one at a
// time, the larger high word, then the larger low word, then the lower expert.
__global__ __launch_bounds__(256) void k_route_select(RouteArgs g) {
  __shared__ double s_c[4][256];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * 4 + wave;
  if (t >= g.T) return;
  const int E = g.E;
  double l[4], s[4], c[4];
  double m = -INFINITY;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = lane + 64 * i;
    l[i] = -INFINITY;
    if (e < E) {
      double a = 0.0;
      for (int p = 0; p < g.S; ++p) a += g.part[((int64_t)p * g.T + t) * E + e];
      if (g.bias) a += (double)g.bias[e];
      const float f = (float)a;
      if (g.logits) g.logits[t * E + e] = f;
      l[i] = (double)f;
      m = fmax(m, l[i]);
    }
  }
  if (g.sigmoid) {
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = 1.0 / (1.0 + exp(-l[i]));
  } else {
#pragma unroll
    for (int o = 32; o; o >>= 1) m = fmax(m, __shfl_xor(m, o, 64));
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[i] = lane + 64 * i < E ? exp(l[i] - m) : 0.0;
      sum += s[i];
    }
    sum = wave_sum_f64(sum);
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] /= sum;
  }
  uint32_t hi[4], lo[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = lane + 64 * i;
    hi[i] = lo[i] = 0;
    if (e < E) {
      c[i] = g.balance ? s[i] + (double)g.balance[e] : s[i];
      if (c[i] != c[i]) c[i] = -INFINITY;
      const uint64_t k = order64(c[i]);
      hi[i] = (uint32_t)(k >> 32);
      lo[i] = (uint32_t)k;
    }
  }
  if (g.kept < g.groups) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (lane + 64 * i < E) s_c[wave][lane + 64 * i] = c[i];
    __builtin_amdgcn_wave_barrier();
    const int n = E / g.groups, L = g.lanes, grp = lane / L;
    double a = -INFINITY, b = -INFINITY;  // the group's largest two
    if (grp < g.groups)
      for (int j = lane % L; j < n; j += L) {
        const double v = s_c[wave][grp * n + j];
        b = fmax(b, fmin(a, v));
        a = fmax(a, v);
      }
    for (int o = 1; o < L; o <<= 1) {
      const double a1 = __shfl_xor(a, o, 64), b1 = __shfl_xor(b, o, 64);
      b = fmax(fmin(a, a1), fmax(b, b1));
      a = fmax(a, a1);
    }
    const double value = g.best_two ? a + b : a;
    int rank = 0;
    for (int j = 0; j < g.groups; ++j) {
      const double v = __shfl(value, j * L, 64);
      rank += v > value || (v == value && j < grp);
    }
    const uint64_t keep = __builtin_amdgcn_ballot_w64(grp < g.groups && rank < g.kept);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = lane + 64 * i;
      if (e < E && !(keep >> (e / n * L) & 1)) hi[i] = lo[i] = 0;
    }
  }
  int my_e = 0;
  double my_s = 0.0, sum = 0.0;
  for (int j = 0; j < g.k; ++j) {
    const uint32_t h = wave_max_u32(max(max(hi[0], hi[1]), max(hi[2], hi[3])));
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (hi[i] == h) w = max(w, lo[i]);
    w = wave_max_u32(w);
    int won = -1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t at = __builtin_amdgcn_ballot_w64(hi[i] == h && lo[i] == w);
      if (won < 0 && at) {
        const int who = __builtin_ctzll(at);
        won = who + 64 * i;
        const double v = __shfl(s[i], who, 64);
        sum += v;
        if (lane == j) my_s = v, my_e = won;
        if (lane == who) hi[i] = lo[i] = 0;
      }
    }
  }
  if (lane < g.k) {
    if (g.renorm) my_s = sum == 0.0 ? 0.0 : my_s / sum;
    g.idx[t * g.k + lane] = my_e;
    g.gates[t * g.k + lane] = (float)(my_s * (double)g.scale);
  }
}

// K-slices of the product: enough that every compute unit has a workgroup, a
// slice of 256 at least.
RoutePlan route_plan(int64_t T, int H, int E) {
  RoutePlan p{1, H};
  if (T <= kRouteFew) return p;
  const int64_t tiles = ((E + kGT - 1) / kGT) * ((T + kGT - 1) / kGT);
  const int units = H / 256;
  int S = (int)((device_cus() + tiles - 1) / tiles);
  if (S > units) S = units;
  const int per = (units + S - 1) / S;
  p.Ks = 256 * per;
  p.S = (units + per - 1) / per;
  return p;
}

hipError_t launch_route(const RouteArgs& g, const RoutePlan& p, const void* x, int xt, int H, const float* Wr, hipStream_t st) {
  if (g.T <= kRouteFew) {
    if (xt == XF32) hipLaunchKernelGGL((k_route_few<XF32>), dim3(g.E), dim3(256), 0, st, x, g.T, H, Wr, g.E, g.part);
    else hipLaunchKernelGGL((k_route_few<XBF16>), dim3(g.E), dim3(256), 0, st, x, g.T, H, Wr, g.E, g.part);
  } else {
    const dim3 grid((g.E + kGT - 1) / kGT, p.S, (g.T + kGT - 1) / kGT);
    if (xt == XF32) hipLaunchKernelGGL((k_route_gemm<XF32>), grid, dim3(256), 0, st, x, g.T, H, Wr, g.E, p.Ks, g.part);
    else hipLaunchKernelGGL((k_route_gemm<XBF16>), grid, dim3(256), 0, st, x, g.T, H, Wr, g.E, p.Ks, g.part);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_route_select, dim3((g.T + 3) / 4), dim3(256), 0, st, g);
  return hipGetLastError();
}

}  // namespace md

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
// definition's.  Where the fp64 matrix cores would be what a call waits for (73
// Tflop/s in a large product), the logits are formed on the fp16 ones first, with a bound on their
// error, and only the tokens whose choice that bound leaves open are done in fp64.
#include <hip/hip_runtime.h>

#include "common.hpp"
#include "i8.hpp"
#include "kernels.hpp"
#include "rows.hpp"

namespace md {

typedef double f64x4 __attribute__((ext_vector_type(4)));

// ---- logits ----------------------------------------------------------------

// Few tokens: a workgroup for each expert, its threads share the width; sums
// as partials [t][e] of one slice.  One token of 2048 x 128: 2.9 us, a launch.
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

// Many tokens: a product on the fp64 matrix cores, 32 tokens x 32 experts and a
// K-slice a workgroup, its four waves a quarter of the slice each; partials
// [s][t][e].  An instruction takes 64 clocks, so operands come straight from
// memory, 16 bytes a lane and four steps ahead, without LDS or barriers.  A[i][k],
// B[k][j] of the 16x16x4 product: lane 16 k + i (j); D[4 v + lane / 16]
// [lane % 16] in element v.  A lane's four neighbouring columns go to four
// instructions: which column is which k does not matter to a sum.  LIST: of the
// tokens that a list names, as many as its count says; the grid's workgroups share
// out tiles and slices.  Measured: 128 tokens x 6144 x 256 12.7 us (0.4 Gflop; 5.5 at
// the rate of a large product; twice as many slices: a call 22.1 us where this takes
// 18.5), a list of some 100 tokens 15, 8191 tokens 420 (61 Tflop/s).  The layer's own
// chunk router (k_router_mfma) stays beside it: it leaves the activations' bf16 pairs
// for the experts from the tiles that it stages, and layer calls keep its bits.
constexpr int kGT = 32;
constexpr int kAhead = 4;

// Slices of a list's product, as many as give kListGroups workgroups work.
constexpr int kListGroups = 2048;
struct ListPlan {
  int tiles, S, Ks;  // expert and token tiles, slices of the width, width of one
};
__host__ __device__ inline ListPlan list_plan(int n, int E, int H) {
  ListPlan p;
  p.tiles = ((E + kGT - 1) / kGT) * ((n + kGT - 1) / kGT);
  const int units = H / 256, S = kListGroups / (p.tiles > 0 ? p.tiles : 1);
  const int per = S > 1 ? (units + S - 1) / S : units;
  p.Ks = 256 * per;
  p.S = (units + per - 1) / per;
  return p;
}

template <int XT>
struct Four;  // neighbouring values as they lie in memory
template <>
struct Four<XF32> {
  float4 v;
  MD_DEV void load(const void* p, int64_t i) { v = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i); }
  MD_DEV double at(int j) const { return (double)(j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w); }
};
template <>
struct Four<XBF16> {
  uint2 v;
  MD_DEV void load(const void* p, int64_t i) { v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i); }
  MD_DEV double at(int j) const {
    const uint32_t w = j < 2 ? v.x : v.y;
    return (double)__uint_as_float(j & 1 ? w & 0xFFFF0000u : w << 16);
  }
};

template <int XT, bool LIST>
__global__ __launch_bounds__(256) void k_route_gemm(const void* __restrict__ x, int T, int H, const float* __restrict__ Wr,
                                                    int E, int Ks, double* __restrict__ part, const int* __restrict__ count,
                                                    const int* __restrict__ list) {
  __shared__ double s_acc[3][16][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int li = lane & 15, kq = lane >> 4;
  const int ets = (E + kGT - 1) / kGT;
  int n = T, items = 1;
  if constexpr (LIST) {
    n = min(*count, T);
    const ListPlan p = list_plan(n, E, H);
    Ks = p.Ks;
    items = n ? p.tiles * p.S : 0;
  }
  const int tts = (n + kGT - 1) / kGT;
  for (int item = LIST ? blockIdx.x : 0; item < items; item += LIST ? gridDim.x : 1) {
    const int ex = LIST ? item % ets : blockIdx.x, tx = LIST ? item / ets % tts : blockIdx.z;
    const int sl = LIST ? item / (ets * tts) : blockIdx.y;
    const int e0 = ex * kGT, t0 = tx * kGT;
    // of the last, partial slice a wave's quarter is shorter, but whole steps of 64
    const int width = min(Ks, H - sl * Ks) / 4, kbeg = sl * Ks + wave * width, steps = width / 16;
    int64_t xr[2], wr[2];
#pragma unroll
    for (int a = 0; a < 2; ++a) {  // past the last row: that one again, not stored
      const int t = min(t0 + 16 * a + li, n - 1), e = min(e0 + 16 * a + li, E - 1);
      xr[a] = (int64_t)(LIST ? list[t] : t) * H + kbeg + 4 * kq;
      wr[a] = (int64_t)e * H + kbeg + 4 * kq;
    }
    f64x4 acc[2][2];
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int b = 0; b < 2; ++b) acc[a][b] = f64x4{0.0, 0.0, 0.0, 0.0};
    Four<XT> xv[kAhead][2];
    Four<XF32> wv[kAhead][2];
    auto load = [&](int u, int step) {
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        xv[u][a].load(x, xr[a] + 16 * step);
        wv[u][a].load(Wr, wr[a] + 16 * step);
      }
    };
#pragma unroll
    for (int u = 0; u < kAhead; ++u) load(u, u);  // a quarter has four steps at least
    auto mul = [&](int u) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int b = 0; b < 2; ++b)
            acc[a][b] = __builtin_amdgcn_mfma_f64_16x16x4f64(xv[u][a].at(j), wv[u][b].at(j), acc[a][b], 0, 0, 0);
    };
    // steps come in fours; no branch around a load: the waits count loads, and would count on none of these
    for (int st = kAhead; st < steps; st += kAhead) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        mul(u);
        __builtin_amdgcn_sched_barrier(0);
        load(u, st + u);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) mul(u);
    if (wave) {
#pragma unroll
      for (int i = 0; i < 16; ++i) s_acc[wave - 1][i][lane] = acc[i >> 3][(i >> 2) & 1][i & 3];
    }
    __syncthreads();
    if (wave == 0) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const double v = ((acc[i >> 3][(i >> 2) & 1][i & 3] + s_acc[0][i][lane]) + s_acc[1][i][lane]) + s_acc[2][i][lane];
        const int t = t0 + 16 * (i >> 3) + 4 * (i & 3) + kq, e = e0 + 16 * ((i >> 2) & 1) + li;
        if (t < n && e < E) part[((int64_t)sl * n + t) * E + e] = v;
      }
    }
    if constexpr (LIST) __syncthreads();  // the LDS of this one
  }
}

// The fp16 form.  64 columns of a row, scaled by a power of two to a largest value
// in [2^14, 2^15), are two fp16 (11 + 11 bits, the second at most 2^-11 of the first),
// off by at most 2^-23; a bf16 x is one.  A product with a bf16 x is two products,
// with an fp32 x the three that are not below 2^-22 of it.  64 columns are summed in
// fp32, the small parts first, and added in fp64.  With |x|, |w| the norms of the
// rows, a partial sum over some columns is at most |x| |w| of these, and the parts'
// products add up to at most the whole's.  An instruction is taken to be off by at
// most 2^-23 of its sum: there are four of full size in 64 columns, those of the
// small parts add 2^-8; values below fp16's smallest normal one are lost if the
// instruction flushes them, 2^-14 of 2^14 for each of 64 columns on either side, at
// most 2^-24; a slice's sum is rounded to fp32.  In all, in 2^-23 |x| |w|: 4.01, 1 for
// W_r's parts, 0.5 and 0.5; with an fp32 x 1 more for its parts and 2 for the products left out: fast_error.  What
// fp32's own range loses adds 2^-119 (|x| + |w|).  Measured, in the same unit: random
// rows 0.05, without any cancellation 0.16, with sizes over orders of magnitude (few
// products make the sum) 1.45.  Of 8191 random tokens some 100 are left open (sigmoid,
// 8 of 256).
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
constexpr float fast_error(bool f32) { return (f32 ? 9.25f : 6.25f) * 0x1p-23f; }
constexpr int kTT = 64, kFT = 128;  // tokens and experts of a workgroup
constexpr int kFastStep = 64;  // columns

// The power of two that brings values of at most m into [2^14, 2^15), and back.
MD_DEV float scale_to_half(float m, float& back) {
  const uint32_t e = max(__float_as_uint(m) >> 23, 15u);
  back = __uint_as_float((e - 14) << 23);
  return __uint_as_float((268 - e) << 23);
}
MD_DEV uint32_t half_bits(_Float16 v) { return __builtin_bit_cast(uint16_t, v); }
// v in two fp16, rounded to nearest
MD_DEV void split2(float v, uint32_t& a, uint32_t& b) {
  const _Float16 h = (_Float16)v;
  a = half_bits(h);
  b = half_bits((_Float16)(v - (float)h));
}

// The two parts of W_r as the product's operands (rows up to a whole tile are
// zeros): [32 experts][16 columns][part][lane][8], what 64 columns were scaled by
// ([64 columns][expert of whole tiles]), its rows' squared norms over 256 columns
// each, and an empty list.  A wave makes the operands of 64 columns.
__global__ __launch_bounds__(256) void k_route_split(const float* __restrict__ Wr, int E, int H, uint16_t* __restrict__ planes,
                                                     float* __restrict__ scales, float* __restrict__ norms,
                                                     int* __restrict__ count) {
  __shared__ float s_n[4][32];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = blockIdx.x * 32 + (lane & 31), c0 = blockIdx.y * 256 + 64 * wave + 8 * (lane >> 5);
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *count = 0;
  float v[4][8], nn = 0.0f, most = 0.0f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[k][i] = 0.0f;
    if (e < E) load8<XF32>(Wr, (int64_t)e * H + c0 + 16 * k, v[k]);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      most = fmaxf(most, fabsf(v[k][i]));
      nn = fmaf(v[k][i], v[k][i], nn);
    }
  most = fmaxf(most, xor_lanes<32>(most));
  float back;
  const float up = scale_to_half(most, back);
  if (lane < 32) scales[((int64_t)blockIdx.y * 4 + wave) * (gridDim.x * 32) + e] = back;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    u32x4 o[2];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      uint32_t a[2], b[2];
#pragma unroll
      for (int m = 0; m < 2; ++m) split2(v[k][i + m] * up, a[m], b[m]);
      o[0][i / 2] = a[0] | a[1] << 16;
      o[1][i / 2] = b[0] | b[1] << 16;
    }
#pragma unroll
    for (int p = 0; p < 2; ++p)
      *reinterpret_cast<u32x4*>(planes + (((int64_t)blockIdx.x * (H / 16) + blockIdx.y * 16 + 4 * wave + k) * 2 + p) * 512 +
                                8 * lane) = o[p];
  }
  nn += xor_lanes<32>(nn);
  if (lane < 32) s_n[wave][lane] = nn;
  __syncthreads();
  if (threadIdx.x < 32 && e < E)
    norms[(int64_t)blockIdx.y * E + e] = (s_n[0][lane] + s_n[1][lane]) + (s_n[2][lane] + s_n[3][lane]);
}

// 64 tokens x 32 NW experts and a K-slice a workgroup, NW waves of 64 x 32, two on a
// SIMD.  The parts of W_r, in operand order, come straight from L2, a step of 64
// columns ahead; x goes through LDS: two buffers, and the two steps behind them on
// their way in registers.  A step's sums are added in fp64, and the next step's x is
// scaled and written, beside the step's products.  A[i][k], B[k][j] of the 32x32x16
// product: eight k at lane 32 (k / 8) + i (j); D[8 a + 4 (lane / 32) + b][lane % 32]
// in element 4 a + b.  No load stands behind a branch (rows past T read the last
// one, steps past the last one again the last): the compiler's waits count loads,
// and one that may not have been issued makes them wait for those behind it.
// Measured: 8191 tokens x 6144 columns x 256 experts, bf16, 71 us (52 Gflop of
// parts; the matrix cores are busy for 21 us of them, the vector ALU for 33), fp32
// 94.  In three bf16 parts 91 (96 without a scale for 64 columns), loads behind
// branches +8, the sums and x behind the products +4, workgroups of 64 x 128 (x read
// twice) +8; LDS read two parts ahead, and the order of products and the vector ALU's
// work prescribed: the same.  Measured before with three parts and dropped: both
// operands through LDS +8 us, waves of 128 x 32 (half the loads of W_r, one wave a
// SIMD) +26.
template <int XT, int NW>
__global__ __launch_bounds__(64 * NW, 2) void k_route_fast(const void* __restrict__ x, int T, int H,
                                                       const uint16_t* __restrict__ planes,
                                                       const float* __restrict__ scales, int E, int Ks, int S,
                                                       float* __restrict__ part, float* __restrict__ xnorm,
                                                       const float* __restrict__ wnorm, float* __restrict__ most) {
  constexpr int KS = kFastStep, C = KS / 8, XP = XT == XF32 ? 2 : 1;  // columns, chunks of 16 bytes, parts of x
  constexpr int kTile = kTT * KS;                                     // values of a part of x's tile
  __shared__ __attribute__((aligned(16))) uint16_t lds[2 * XP * kTile];
  __shared__ __attribute__((aligned(16))) float s_back[4][kTT];  // what a step's tokens were scaled by
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  constexpr int FT = 32 * NW;
  const int ets = (E + FT - 1) / FT, whole = (E + kFT - 1) / kFT * kFT;
  // workgroups that follow each other go to different dies: those of one die
  // take the same experts and slice, so that its L2 holds these parts of W_r
  const int combo = blockIdx.x % (ets * S), ex = combo % ets, sl = combo / ets;
  const int t0 = blockIdx.x / (ets * S) * kTT, e0 = ex * FT;
  const int kbeg = sl * Ks, kend = min(kbeg + Ks, H);
  const int l31 = lane & 31, hh = lane >> 5;
  // sixteen lanes of a fragment read hit sixteen chunks of 256 bytes: two rows of 128
  auto slot = [](int row, int chunk) { return row * KS + 8 * (chunk ^ ((row >> 1) & 7)); };
  // staging: NW threads a row, C / NW chunks of 16 bytes
  constexpr int CH = C / NW;
  const int row = tid / NW, ch0 = tid % NW * CH;
  float xreg[2][XT == XF32 ? CH : 1][8];
  u32x4 xraw[2][XT == XF32 ? 1 : CH];
  float xx = 0.0f;
  const bool norms = ex == 0;
  const bool has_t = t0 + row < T;
  const int64_t row_at = (int64_t)min(t0 + row, T - 1) * H + 8 * ch0;
  auto fetch = [&](int kc, int s) {
    const int64_t at = row_at + min(kc, kend - KS);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if constexpr (XT == XF32) load8<XF32>(x, at + 8 * c, xreg[s][c]);
      else xraw[s][c] = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(x) + at + 8 * c);
    }
  };
  // a step's columns of x into LDS: what they are scaled by, and two values a thread at a time
  float up = 0.0f;
  auto put_scale = [&](int s, float* to) {
    float m = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if constexpr (XT == XF32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(xreg[s][c][i]));
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          m = fmaxf(fmaxf(m, fabsf(__uint_as_float(xraw[s][c][i] << 16))), fabsf(__uint_as_float(xraw[s][c][i])));
      }
    }
    m = fmaxf(m, xor_lanes<1>(m));
    m = fmaxf(m, xor_lanes<2>(m));
    if constexpr (NW == 8) m = fmaxf(m, xor_lanes<4>(m));
    float back;
    up = scale_to_half(m, back);
    to[row] = back;  // (a row's lanes, one value: no branch, behind which the compiler would move the sums)
  };
  u32x4 o[XP];
  auto put = [&](int s, int g, uint16_t* b) {
    const int c = g / 4, i = g % 4;
    float u, v;
    if constexpr (XT == XF32) {
      u = xreg[s][c][2 * i], v = xreg[s][c][2 * i + 1];
      uint32_t p[2], q[2];
      split2(u * up, p[0], q[0]);
      split2(v * up, p[1], q[1]);
      o[0][i] = p[0] | p[1] << 16;
      o[XP - 1][i] = q[0] | q[1] << 16;
    } else {  // exact, down to fp16's smallest normal value
      u = __uint_as_float(xraw[s][c][i] << 16), v = __uint_as_float(xraw[s][c][i] & 0xFFFF0000u);
      o[0][i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(u * up, v * up));
    }
    if (norms) xx = fmaf(u, u, fmaf(v, v, xx));
    if (i == 3) {
#pragma unroll
      for (int q = 0; q < XP; ++q) *reinterpret_cast<u32x4*>(b + q * kTile + slot(row, ch0 + c)) = o[q];
    }
  };
  // the wave's operands of W_r, a step's, and what its columns were scaled by
  f16x8 w[KS / 16][2];
  float wback;
  const int e = e0 + 32 * wave + l31;
  const uint16_t* wp = planes + ((int64_t)(NW * ex + wave) * (H / 16) + kbeg / 16) * 1024 + 8 * lane;
  const float* sp = scales + (int64_t)(kbeg / 64) * whole + e;
  auto load_w = [&](int k, int p) { w[k][p] = *reinterpret_cast<const f16x8*>(wp + k * 1024 + p * 512); };
  double acc[2][16];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[t][i] = 0.0;
  if (blockIdx.x == 0) {  // what every token's bound needs: the largest row's squared norm
    float n = 0.0f;  // E is up to 256
    if (tid < E) {
#pragma unroll 16
      for (int c = 0; c < H / 256; ++c) n += wnorm[(int64_t)c * E + tid];
    }
    n = group_max<64>(n);
    if (lane == 0 && wave < 4) s_back[0][wave] = n;
    __syncthreads();
    if (tid == 0) *most = fmaxf(fmaxf(s_back[0][0], s_back[0][1]), fmaxf(s_back[0][2], s_back[0][3]));
    __syncthreads();
  }
  f32x16 d[2][2];  // of two steps: the sums of the one before are added beside the products of this one
  double sw = 0.0;  // what its columns of W_r were scaled by
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int i = 0; i < 16; ++i) d[1][t][i] = 0.0f;
  if (tid < kTT) s_back[3][tid] = 0.0f;
  auto add = [&](int h, int g, const f32x4& sx) {
    const int t = g / 4, a = g % 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[t][4 * a + i] = fma((double)(d[h][t][4 * a + i] * sx[i]), sw, acc[t][4 * a + i]);
  };
  auto scaled = [&](int st, int g) {
    return *reinterpret_cast<const f32x4*>(s_back[st & 3] + 32 * (g / 4) + 8 * (g % 4) + 4 * hh);
  };
  // step st, in LDS h; the next one comes from registers 1 - h
  auto step = [&](int h, int st, bool more) {
    const uint16_t* b = lds + h * XP * kTile;
    uint16_t* nb = lds + (1 - h) * XP * kTile;
    f16x8 v[2][2], v1[2][2];
    auto read = [&](int g) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const uint16_t* at = b + slot(32 * t + l31, 2 * (g % 4) + hh);
        v[g & 1][t] = *reinterpret_cast<const f16x8*>(at);
        if (XP == 2 && g < 4) v1[g & 1][t] = *reinterpret_cast<const f16x8*>(at + kTile);
      }
    };
    const double sw_next = (double)wback;
    if (more) wp += KS * 64, sp += whole;
    wback = *sp;
    f32x4 sx[2];
    read(0);
    sx[0] = scaled(st + 3, 0);
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) d[h][t][i] = 0.0f;
    const float so_far = xx;
    // eight parts, in this order: the loads of W_r behind the products that use their registers up
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      const int k = g % 4, p = g < 4 ? 1 : 0;  // the small products first
      __builtin_amdgcn_sched_barrier(0);
      if (g < 7) {
        read(g + 1);
        sx[(g + 1) & 1] = scaled(st + 3, g + 1);
      }
      if (g == 0) put_scale(1 - h, s_back[(st + 1) & 3]);
      if (XP == 2 && g < 4) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
          d[h][t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v1[g & 1][t], w[k][0], d[h][t], 0, 0, 0);
      }
#pragma unroll
      for (int t = 0; t < 2; ++t)
        d[h][t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v[g & 1][t], w[k][p], d[h][t], 0, 0, 0);
      add(1 - h, g, sx[g & 1]);
      if (CH == 2 || g % 2) put(1 - h, CH == 2 ? g : g / 2, nb);
      __builtin_amdgcn_sched_barrier(0);
      load_w(k, p);
    }
    xx = more ? xx : so_far;
    sw = sw_next;
  };
  fetch(kbeg, 0);
  fetch(kbeg + KS, 1);
  wback = *sp;
#pragma unroll
  for (int p = 1; p >= 0; --p)
#pragma unroll
    for (int k = 0; k < KS / 16; ++k) load_w(k, p);
  put_scale(0, s_back[0]);
#pragma unroll
  for (int g = 0; g < 4 * CH; ++g) put(0, g, lds);
  __syncthreads();
  for (int kc = kbeg, st = 0; kc < kend; kc += 2 * KS, st += 2) {  // a slice is a multiple of 256 columns
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      fetch(kc + (h + 2) * KS, h);
      __builtin_amdgcn_sched_barrier(0);
      step(h, st + h, kc + (h + 1) * KS < kend);
      __syncthreads();
    }
  }
#pragma unroll
  for (int g = 0; g < 8; ++g) add(1, g, scaled((kend - kbeg) / KS + 3, g));
  if (e < E) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int tok = t0 + 32 * t + 8 * (i >> 2) + 4 * hh + (i & 3);
        if (tok < T) part[((int64_t)sl * T + tok) * E + e] = (float)acc[t][i];
      }
  }
  if (norms) {
    xx += xor_lanes<1>(xx);
    xx += xor_lanes<2>(xx);
    if constexpr (NW == 8) xx += xor_lanes<4>(xx);
    if (tid % NW == 0 && has_t) xnorm[(int64_t)sl * T + t0 + row] = xx;
  }
}

// ---- choice ----------------------------------------------------------------

// A double in the order of unsigned integers, above 0 (-0 is +0; no NaN comes here).
MD_DEV uint64_t order64(double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
  return u >> 63 ? ~u : u | 0x8000000000000000ull;
}

// How a token's logits come.
//   kExact   partials of g.S slices, for every token; everything is fp64
//   kBounded the fp16 form's: scores and order in fp32, and a token whose choice
//            the bound on both leaves open is put on the list; the winners' scores
//            are formed again in fp64 for the gates
//   kListed  the list's tokens, as kExact
enum Logits { kExact, kBounded, kListed };

// A wave for each token: lane l holds experts l + 64 i.  Groups are valued by
// 64 / groups lanes each (a power of two); the k winners are taken one at a
// time: the larger key (its high word, then its low one), then the lower expert.
// What the winners bring with them waits in LDS until all are known (carried through
// the rounds by selects and lane reads 22 us where this takes 16.5).
// Measured: one token of 128 experts 4.1 us (a chain of loads, fp64 exp and k
// rounds), 128 of 256 5.8, 8191 of 256 in fp32 16.1 (bound by the vector ALU's issue);
// with loads behind branches, each waited for by itself, 5.2, 7.2 and 16.5.
template <bool B>
struct RouteLds {  // of each expert
  using F = std::conditional_t<B, float, double>;  // scores
  F c[256], s[256];    // s: B: what c may be off by
  double l[B ? 256 : 1];
};
template <Logits FROM>
MD_DEV void route_choose(const RouteArgs& g, RouteLds<FROM == kBounded>& lds, int64_t t, int64_t at, int64_t n, int S) {
  constexpr bool B = FROM == kBounded;
  using F = typename RouteLds<B>::F;
  const int lane = threadIdx.x;
  const int E = g.E;
  // (loaded first: they are on their way with the partials; past the last expert that one again, its
  // values unused: no branch around a load)
  int at_e[4];
  float bias[4] = {0, 0, 0, 0}, bal[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) at_e[i] = min(lane + 64 * i, E - 1);
  if (g.bias) {
#pragma unroll
    for (int i = 0; i < 4; ++i) bias[i] = g.bias[at_e[i]];
  }
  if (g.balance) {
#pragma unroll
    for (int i = 0; i < 4; ++i) bal[i] = g.balance[at_e[i]];
  }
  double l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) l[i] = 0.0;
  using P = std::conditional_t<B, float, double>;
  auto rows = [&](int p) { return reinterpret_cast<const P*>(g.part) + ((int64_t)p * n + at) * E; };
  // the slices in order, some on their way at a time
  constexpr int U = B ? 2 : 8;
  if (S == 1) {
    const P* r = rows(0);
#pragma unroll
    for (int i = 0; i < 4; ++i) l[i] = (double)r[at_e[i]];
  } else {
    for (int p = 0; p < S; p += U) {
      P v[4][U];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const P* r = rows(min(p + j, S - 1));
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i][j] = r[at_e[i]];
      }
#pragma unroll
      for (int j = 0; j < U; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) l[i] += p + j < S ? (double)v[i][j] : 0.0;
    }
  }
  float f[4], m = -INFINITY, far = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = lane + 64 * i;
    f[i] = -INFINITY;
    if (e < E) {
      if (g.bias) l[i] += (double)bias[i];
      f[i] = (float)l[i];
      if (!B && g.logits) g.logits[t * E + e] = f[i];
      far = fmaxf(far, fabsf(f[i]));
      m = fmaxf(m, f[i]);
    }
    if constexpr (!B) l[i] = (double)f[i];
  }
  F s[4], c[4], top_s = 0;  // top_s: softmax's largest score
  if (g.sigmoid) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (B) s[i] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-f[i] * 1.44269504f));
      else s[i] = 1.0 / (1.0 + exp(-l[i]));
    }
  } else {
    m = group_max<64>(m);
    F sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (B) s[i] = __builtin_amdgcn_exp2f((f[i] - m) * 1.44269504f);
      else s[i] = exp(l[i] - (double)m);
      if (lane + 64 * i >= E) s[i] = 0;
      sum += s[i];
    }
    if constexpr (B) sum = group_sum<64>(sum);
    else sum = wave_total(sum);
    top_s = F(1) / sum;
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = B ? s[i] * top_s : s[i] / sum;
  }
  // kBounded: a logit is off by at most off (the definition's rounding to fp32 and
  // the one here included) and an expert's c by delta: a sigmoid by its slope
  // s (1 - s) times off (1.03: the slope around it) and its own roundings, 2^-23 of
  // s below 1 in the quotient, less in the others; a softmax's terms by the factor
  // exp(2 off), 14 2^-24 of s in exp, sum and quotient, and what exp's argument is
  // rounded by, s log(top_s / s) 2^-23; the sums with the balance and here by 2^-24
  // of c each (of its own c: an expert closed by -1e9 leaves the others' bounds alone)
  float off = 0.0f, most = 0.0f, edge = 0.0f, delta[4];  // most: of a group's experts, less what follows their c
  bool open = false;
  auto size = [](float v) { return fabsf(v) < INFINITY ? fabsf(v) : 0.0f; };  // an infinity is exact
  if constexpr (B) {
    float xn = 0.0f;
    for (int p = 0; p < S; ++p) xn += g.xnorm[(int64_t)p * g.T + t];
    far = group_max<64>(far);
    const float nx = sqrtf(xn) * 1.001f, nw = sqrtf(g.most[0]) * 1.001f;  // their own sums' rounding
    off = fast_error(g.f32) * nx * nw + 0x1p-119f * (nx + nw) + 0x1p-22f * far;
    // past this a gate might be off by more than a step of bf16 (4.1 off), or off is no number.  W_r of N(0, 0.05)
    // and x of N(0, 1) stay below it at the largest width
    open = !(off < 0x1p-10f);
    edge = g.sigmoid ? 0x1p-21f : 0x1p-24f * top_s + 1e-14f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      delta[i] = edge + (g.sigmoid ? 1.03f * off * s[i] * (1.0f - s[i]) : s[i] * (2.1f * off + 0x1.2p-20f));
    most = edge + (g.sigmoid ? 0.26f * off : top_s * (2.1f * off + 0x1.2p-20f));
  }
  uint32_t hi[4], lo[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = lane + 64 * i;
    hi[i] = lo[i] = 0;
    if (e < E) {
      c[i] = g.balance ? s[i] + (F)bal[i] : s[i];
      if (c[i] != c[i]) c[i] = -INFINITY;
      if constexpr (B) delta[i] += 0x1p-23f * size(c[i]);
      if constexpr (B) {
        hi[i] = order_key32(c[i]);
      } else {
        const uint64_t k = order64(c[i]);
        hi[i] = (uint32_t)(k >> 32);
        lo[i] = (uint32_t)k;
      }
      lds.c[e] = c[i];
      lds.s[e] = B ? delta[i] : s[i];
      if constexpr (B) lds.l[e] = l[i];
    }
  }
  __builtin_amdgcn_wave_barrier();
  if (g.kept < g.groups) {
    const int per = g.per, L = 1 << g.lane_bits, grp = lane >> g.lane_bits;
    auto larger = [](F p, F q) { return p > q ? p : q; };  // no NaN here
    auto smaller = [](F p, F q) { return p > q ? q : p; };
    F a = -INFINITY, b = -INFINITY;  // the group's largest two
    if (grp < g.groups)
      for (int j = lane & (L - 1); j < per; j += L) {
        const F v = lds.c[grp * per + j];
        b = larger(b, smaller(a, v));
        a = larger(a, v);
      }
    for (int o = 1; o < L; o <<= 1) {
      const F a1 = __shfl_xor(a, o, 64), b1 = __shfl_xor(b, o, 64);
      b = larger(smaller(a, a1), larger(b, b1));
      a = larger(a, a1);
    }
    F value = g.best_two ? a + b : a;
    if (value != value) value = -INFINITY;
    int rank = 0;
    for (int j = 0; j < g.groups; ++j) {
      const F v = lane_of(value, j * L);
      rank += v > value || (v == value && j < grp);
    }
    const uint64_t keep = __builtin_amdgcn_ballot_w64(grp < g.groups && rank < g.kept);
    if constexpr (B) {
      // The least that a kept group may be worth, and the most that another may.  An expert's bounds rise
      // with its c, so those of the largest ones bound the group: 2^-24 of each in its own sum, of their sum
      // and of the one here, twice that allowed
      const float margin = g.best_two ? 2.0f * most + 0x1p-21f * (size(a) + size(b)) : most + 0x1p-21f * size(a);
      const bool in = grp < g.groups;
      const float least = -group_max<64>(in && rank < g.kept ? margin - value : -INFINITY);
      const float best = group_max<64>(in && rank >= g.kept ? value + margin : -INFINITY);
      open |= !(least > best);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = lane + 64 * i;
      if (e < E && !(keep >> ((e * g.per_inv >> 16) << g.lane_bits) & 1)) hi[i] = lo[i] = 0;
    }
  }
  int my_e = 0;
  uint32_t behind = 0;  // behind the last winner: what the others may reach at most
  for (int j = 0; j < g.k + (B ? 1 : 0); ++j) {
    if (B && j == g.k) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (hi[i]) hi[i] = order_key32(c[i] + delta[i]);
    }
    const uint32_t h = wave_max_u32(max(max(hi[0], hi[1]), max(hi[2], hi[3])));
    if (B && j == g.k) {
      behind = h;
      break;
    }
    uint64_t has[4];
    int n_has = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      has[i] = __builtin_amdgcn_ballot_w64(hi[i] == h);
      n_has += __popcll(has[i]);
    }
    if (!B && n_has > 1) {  // the same high word twice: the low one decides
      uint32_t w = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (hi[i] == h) w = max(w, lo[i]);
      w = wave_max_u32(w);
#pragma unroll
      for (int i = 0; i < 4; ++i) has[i] = __builtin_amdgcn_ballot_w64(hi[i] == h && lo[i] == w);
    }
    int who = 0, slot = 0;
#pragma unroll
    for (int i = 3; i >= 0; --i)
      if (has[i]) who = __builtin_ctzll(has[i]), slot = i;
    if (lane == j) my_e = who + 64 * slot;
    if (lane == who) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (slot == i) hi[i] = lo[i] = 0;
    }
  }
  const F my_s = lds.s[my_e];
  if constexpr (B) {
    const float my_c = lds.c[my_e], c0 = __shfl_up(my_c, 1, 64), d0 = __shfl_up(my_s, 1, 64);
    open |= __builtin_amdgcn_ballot_w64(lane > 0 && lane < g.k && !(c0 - my_c > d0 + my_s)) != 0;
    // (0: k experts are all that may be chosen)
    open |= behind && !(lane_of(my_c, g.k - 1) - lane_of(my_s, g.k - 1) > key_logit(behind));
    if (open) {
      if (lane == 0) g.list[atomicAdd(g.count, 1)] = (int)t;  // the order does not matter: each token stands for itself
      return;
    }
  }
  double gate = (double)my_s;
  if constexpr (B) {
    const double my_l = lds.l[my_e];
    gate = g.sigmoid ? 1.0 / (1.0 + exp(-my_l)) : exp(my_l - (double)m) * (double)top_s;
  }
  if (g.renorm) {
    double sum = 0.0;
    for (int j = 0; j < g.k; ++j) sum += lane_of(gate, j);
    gate = sum == 0.0 ? 0.0 : gate / sum;
  }
  if (lane < g.k) {
    g.idx[t * g.k + lane] = my_e;
    g.gates[t * g.k + lane] = (float)(gate * (double)g.scale);
  }
}

template <Logits FROM>
__global__ __launch_bounds__(64) void k_route_select(RouteArgs g) {
  __shared__ RouteLds<FROM == kBounded> lds;
  if constexpr (FROM == kListed) {
    const int n = min(*g.count, g.T), S = list_plan(n, g.E, g.H).S;
    for (int at = blockIdx.x; at < n; at += gridDim.x) {
      route_choose<FROM>(g, lds, g.list[at], at, n, S);
      __syncthreads();  // the LDS of the one before
    }
  } else {
    route_choose<FROM>(g, lds, blockIdx.x, blockIdx.x, g.T, g.S);
  }
}

// Whether the fp16 form pays: both forms' times in us, linear in Gflop (whole tiles
// of experts in the fp16 form), as measured over 128 to 16384 tokens.  us, fp16
// form and fp64: 6144 x 256, bf16, 512 tokens 69 and 41, 1024 60 and 72, 8192 113
// and 439; fp32 1024 63 and 72, 8192 140 and 436; 2048 x 128, fp32, 4096 52 and 53,
// 8192 61 and 93; 4096 x 64, bf16, 4096 49 and 54, 8192 61 and 93.
static bool route_fast(int64_t T, int H, int E, int xt) {
  const double g = 2e-9 * T * H * E, whole = 2e-9 * T * H * ((E + kFT - 1) / kFT * kFT);
  return 18.0 + 16.2 * g > (xt == XF32 ? 48.0 + 3.6 * whole : 46.0 + 2.6 * whole);
}

// K-slices of the product: enough that every compute unit has a workgroup (of 128 x
// 128 as it counts here, whether one of 64 x 256 or two of 64 x 128), a slice of 256
// at least.
RoutePlan route_plan(int64_t T, int H, int E, int xt, bool fast) {
  RoutePlan p{};
  p.Ks = H;
  p.S = 1;
  p.fast = fast && T > kRouteFew && route_fast(T, H, E, xt);
  if (T > kRouteFew) {
    constexpr int step = 256;
    const int tile = p.fast ? kFT : kGT;
    const int64_t tiles = (int64_t)((E + tile - 1) / tile) * ((T + tile - 1) / tile);
    const int units = (H + step - 1) / step;
    int S = (int)((device_cus() + tiles - 1) / tiles);
    if (S > units) S = units;
    const int per = (units + S - 1) / S;
    p.Ks = step * per;
    p.S = (units + per - 1) / per;
  }
  auto take = [&](size_t bytes) {
    const size_t o = p.bytes;
    p.bytes += (bytes + 255) & ~size_t(255);
    return o;
  };
  size_t rows = (size_t)T * p.S;
  if (p.fast) {
    const size_t ets = (E + kFT - 1) / kFT, small = (E + kGT - 1) / kGT;
    p.planes = take(4 * ets * kFT * H);
    p.scales = take(4 * ets * kFT * (H / 64));
    p.wnorm = take(4 * (size_t)E * (H / 256));
    p.most = take(4);
    p.xnorm = take(4 * rows);
    p.count = take(4);
    p.list = take(4 * (size_t)T);
    // fp32 sums; over them the list's slices: kListGroups workgroups of a tile each, or one slice
    rows = std::max((rows + 1) / 2, std::max((size_t)T, (size_t)kListGroups / small * kGT));
  }
  p.part = take(8 * rows * E);
  return p;
}

template <int XT>
static hipError_t launch_fast(const RouteArgs& g, const RoutePlan& p, const void* x, int H, const float* Wr, uint16_t* planes,
                              float* scales, hipStream_t st) {
  const int ets = (g.E + kFT - 1) / kFT;
  hipLaunchKernelGGL(k_route_split, dim3(ets * kFT / 32, H / 256), dim3(256), 0, st, Wr, g.E, H, planes, scales, g.wnorm,
                     g.count);
  const int tiles = p.S * ((g.T + kTT - 1) / kTT);
  float* part = reinterpret_cast<float*>(g.part);
  if (ets == 2)
    hipLaunchKernelGGL((k_route_fast<XT, 8>), dim3(tiles), dim3(512), 0, st, x, g.T, H, planes, scales, g.E, p.Ks, p.S, part,
                       g.xnorm, g.wnorm, g.most);
  else
    hipLaunchKernelGGL((k_route_fast<XT, 4>), dim3(tiles), dim3(256), 0, st, x, g.T, H, planes, scales, g.E, p.Ks, p.S, part,
                       g.xnorm, g.wnorm, g.most);
  hipLaunchKernelGGL((k_route_select<kBounded>), dim3(g.T), dim3(64), 0, st, g);
  hipLaunchKernelGGL((k_route_gemm<XT, true>), dim3(kListGroups), dim3(256), 0, st, x, g.T, H, Wr, g.E, 0, g.part, g.count,
                     g.list);
  hipLaunchKernelGGL((k_route_select<kListed>), dim3(std::min(g.T, kListGroups)), dim3(64), 0, st, g);
  return hipGetLastError();
}

hipError_t launch_route(const RouteArgs& g0, const RoutePlan& p, const void* x, int xt, const float* Wr, void* ws,
                        hipStream_t st) {
  RouteArgs g = g0;
  char* at = static_cast<char*>(ws);
  const int H = g.H;
  g.part = reinterpret_cast<double*>(at + p.part);
  g.S = p.S;
  if (p.fast) {
    g.wnorm = reinterpret_cast<float*>(at + p.wnorm);
    g.xnorm = reinterpret_cast<float*>(at + p.xnorm);
    g.most = reinterpret_cast<float*>(at + p.most);
    g.count = reinterpret_cast<int*>(at + p.count);
    g.list = reinterpret_cast<int*>(at + p.list);
    uint16_t* planes = reinterpret_cast<uint16_t*>(at + p.planes);
    float* scales = reinterpret_cast<float*>(at + p.scales);
    g.f32 = xt == XF32;
    return xt == XF32 ? launch_fast<XF32>(g, p, x, H, Wr, planes, scales, st)
                      : launch_fast<XBF16>(g, p, x, H, Wr, planes, scales, st);
  }
  if (g.T <= kRouteFew) {
    if (xt == XF32) hipLaunchKernelGGL((k_route_few<XF32>), dim3(g.E), dim3(256), 0, st, x, g.T, H, Wr, g.E, g.part);
    else hipLaunchKernelGGL((k_route_few<XBF16>), dim3(g.E), dim3(256), 0, st, x, g.T, H, Wr, g.E, g.part);
  } else {
    const dim3 grid((g.E + kGT - 1) / kGT, p.S, (g.T + kGT - 1) / kGT), block(256);
    if (xt == XF32)
      hipLaunchKernelGGL((k_route_gemm<XF32, false>), grid, block, 0, st, x, g.T, H, Wr, g.E, p.Ks, g.part, nullptr, nullptr);
    else
      hipLaunchKernelGGL((k_route_gemm<XBF16, false>), grid, block, 0, st, x, g.T, H, Wr, g.E, p.Ks, g.part, nullptr, nullptr);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((k_route_select<kExact>), dim3(g.T), dim3(64), 0, st, g);
  return hipGetLastError();
}

}  // namespace md

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
// definition's.  Where the fp64 matrix cores would be what a call waits for (78
// Tflop/s), the logits are formed on the bf16 ones first, with a bound on their
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
// out tiles and slices.  Measured: 128 tokens x 6144 x 256 13.5 us (0.4 Gflop; 5.5 at
// the rate of a large product, twice as many slices 17 with the choice 4 slower), a
// list of some 100 tokens 14, 8191 tokens 420 (61 Tflop/s).
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
    for (int st = 0; st < steps; st += kAhead) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int b = 0; b < 2; ++b)
              acc[a][b] = __builtin_amdgcn_mfma_f64_16x16x4f64(xv[u][a].at(j), wv[u][b].at(j), acc[a][b], 0, 0, 0);
        if (st + kAhead < steps) load(u, st + kAhead + u);
      }
    }
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

// The bf16 form.  An fp32 value is the sum of three bf16 (8 + 8 + 8 bits, each
// part at most 2^-9 of the one before), so a product with a bf16 x is three
// products, with an fp32 x the six that are not below 2^-26 of it.  The first
// parts' product is summed in fp32 over 64 columns, the others, which are small,
// over kRest, and these sums are added in fp64.  With |x|, |w| the norms of the
// rows, a partial sum over some columns is at most |x| |w| of these, and the parts'
// products add up to at most the whole's.  An instruction is taken to be off by at
// most 2^-23 of its sum: there are four of full size in 64 columns, and at most 320
// below 2^-8 (1 + 2^-4) of it in kRest.  In all 2^-23 (4 + 1.33) |x| |w|, and 2^-26
// for the products left out: kFastError.  What lies below bf16's smallest normal
// adds 2^-119 (|x| + |w|).  Measured, random rows, rows without any cancellation,
// growing, falling: at most 0.13 2^-23 |x| |w|.  Of 8191 tokens some 100 are left
// open (sigmoid, 8 of 256).
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
constexpr double kFastError = 5.5 * 0x1p-23;
constexpr int kRest = 1024;
constexpr int kTT = 64, kFT = 128;  // tokens and experts of a workgroup
template <int XT> constexpr int kFastStep = XT == XF32 ? 32 : 64;

MD_DEV void split3(float v, uint16_t& a, uint16_t& b, uint16_t& c) {
  a = to_bf16(v);
  v -= __uint_as_float((uint32_t)a << 16);
  b = to_bf16(v);
  c = to_bf16(v - __uint_as_float((uint32_t)b << 16));
}

// The three parts of W_r as the product's operands (rows up to a whole tile are
// zeros): [32 experts][16 columns][part][lane][8], its rows' squared norms over
// 256 columns each, and an empty list.  A wave makes the operands of 64 columns.
__global__ __launch_bounds__(256) void k_route_split(const float* __restrict__ Wr, int E, int H, uint16_t* __restrict__ planes,
                                                     float* __restrict__ norms, int* __restrict__ count) {
  __shared__ float s_n[4][32];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = blockIdx.x * 32 + (lane & 31), c0 = blockIdx.y * 256 + 64 * wave + 8 * (lane >> 5);
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *count = 0;
  float v[4][8], nn = 0.0f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[k][i] = 0.0f;
    if (e < E) load8<XF32>(Wr, (int64_t)e * H + c0 + 16 * k, v[k]);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    u32x4 o[3];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      uint16_t a[2], b[2], d[2];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        split3(v[k][i + m], a[m], b[m], d[m]);
        nn = fmaf(v[k][i + m], v[k][i + m], nn);
      }
      o[0][i / 2] = a[0] | (uint32_t)a[1] << 16;
      o[1][i / 2] = b[0] | (uint32_t)b[1] << 16;
      o[2][i / 2] = d[0] | (uint32_t)d[1] << 16;
    }
#pragma unroll
    for (int p = 0; p < 3; ++p)
      *reinterpret_cast<u32x4*>(planes + (((int64_t)blockIdx.x * (H / 16) + blockIdx.y * 16 + 4 * wave + k) * 3 + p) * 512 +
                                8 * lane) = o[p];
  }
  nn += xor_lanes<32>(nn);
  if (lane < 32) s_n[wave][lane] = nn;
  __syncthreads();
  if (threadIdx.x < 32 && e < E)
    norms[(int64_t)blockIdx.y * E + e] = (s_n[0][lane] + s_n[1][lane]) + (s_n[2][lane] + s_n[3][lane]);
}

// 64 tokens x 128 experts and a K-slice a workgroup, four waves of 64 x 32, two
// workgroups on a compute unit.  The parts of W_r, in operand order, come straight
// from L2, a step ahead; x goes through LDS: two buffers, and the two steps behind
// them on their way in registers.  A[i][k], B[k][j] of the 32x32x16 product: eight
// k at lane 32 (k / 8) + i (j); D[8 a + 4 (lane / 32) + b][lane % 32] in element
// 4 a + b.
// Measured: 8191 tokens x 6144 columns x 256 experts, bf16, 96 us (77 Gflop of
// parts, 0.8 Pflop/s; the matrix cores are busy for 38 us of them).  With a third
// of W_r's loads 76 us, with every load from the caches 78, without the products 75,
// without the sums in fp64 88: mostly the 16 bytes a lane and product that the parts
// of W_r take through L1, beside the products, not hidden behind them.  Measured and
// dropped: both operands through LDS 104 us, workgroups of 128 x 128 the same as
// this, waves of 128 x 32 (half the loads of W_r, one wave a SIMD) 122.
template <int XT>
__global__ __launch_bounds__(256, 2) void k_route_fast(const void* __restrict__ x, int T, int H,
                                                       const uint16_t* __restrict__ planes, int E, int Ks, int S,
                                                       double* __restrict__ part, float* __restrict__ xnorm,
                                                       const float* __restrict__ wnorm, const float* __restrict__ balance,
                                                       float* __restrict__ most) {
  constexpr int KS = kFastStep<XT>, C = KS / 8, XP = XT == XF32 ? 3 : 1;  // columns, chunks of 16 bytes, parts of x
  constexpr int kTile = kTT * KS;                                         // values of a part of x's tile
  __shared__ __attribute__((aligned(16))) uint16_t lds[2 * XP * kTile];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ets = (E + kFT - 1) / kFT;
  // workgroups that follow each other go to different dies: those of one die
  // take the same experts and slice, so that its L2 holds these parts of W_r
  const int combo = blockIdx.x % (ets * S), ex = combo % ets, sl = combo / ets;
  const int t0 = blockIdx.x / (ets * S) * kTT, e0 = ex * kFT;
  const int kbeg = sl * Ks, kend = min(kbeg + Ks, H);
  const int l31 = lane & 31, hh = lane >> 5;
  // sixteen lanes of a fragment read hit sixteen chunks of 256 bytes: two rows of 128, or four of 64
  auto slot = [](int row, int chunk) { return row * KS + 8 * (chunk ^ (C == 8 ? (row >> 1) & 7 : (row >> 2) & 3)); };
  // staging: four threads a row, C / 4 chunks of 16 bytes
  constexpr int CH = C / 4;
  const int row = tid >> 2, ch0 = (tid & 3) * CH;
  float xreg[2][XT == XF32 ? 8 * CH : 1];
  u32x4 xraw[2][XT == XF32 ? 1 : CH];
  float xx = 0.0f;
  const bool norms = ex == 0;
  const bool has_t = t0 + row < T;
  auto fetch = [&](int kc, int s) {
    const int64_t at = (int64_t)(t0 + row) * H + kc + 8 * ch0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if constexpr (XT == XF32) {
        float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (has_t) load8<XF32>(x, at + 8 * c, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) xreg[s][8 * c + i] = v[i];
      } else {
        xraw[s][c] = u32x4{0, 0, 0, 0};
        if (has_t) xraw[s][c] = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(x) + at + 8 * c);
      }
    }
  };
  auto put = [&](int buf, int s) {
    uint16_t* b = lds + buf * XP * kTile;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if constexpr (XT == XF32) {
        u32x4 o[3];
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          uint16_t p[3][2];
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const float v = xreg[s][8 * c + i + m];
            split3(v, p[0][m], p[1][m], p[2][m]);
            if (norms) xx = fmaf(v, v, xx);
          }
#pragma unroll
          for (int q = 0; q < 3; ++q) o[q][i / 2] = p[q][0] | (uint32_t)p[q][1] << 16;
        }
#pragma unroll
        for (int q = 0; q < 3; ++q) *reinterpret_cast<u32x4*>(b + q * kTile + slot(row, ch0 + c)) = o[q];
      } else {
        *reinterpret_cast<u32x4*>(b + slot(row, ch0 + c)) = xraw[s][c];
        if (norms) {
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const float u = __uint_as_float(xraw[s][c][m] << 16), v = __uint_as_float(xraw[s][c][m] & 0xFFFF0000u);
            xx = fmaf(u, u, fmaf(v, v, xx));
          }
        }
      }
    }
  };
  // the wave's operands of W_r, a step's
  bf16x8 w[KS / 16][3];
  const uint16_t* wp = planes + ((int64_t)(4 * ex + wave) * (H / 16) + kbeg / 16) * 1536 + 8 * lane;
  auto load_w = [&](int k) {
#pragma unroll
    for (int p = 0; p < 3; ++p) w[k][p] = *reinterpret_cast<const bf16x8*>(wp + k * 1536 + p * 512);
  };
  double acc[2][16];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[t][i] = 0.0;
  if (blockIdx.x == 0 && wave == 0) {  // what every token's bound needs: the largest squared norm and finite balance
    float wn_max = 0.0f, bal = 0.0f;
    for (int e = lane; e < E; e += 64) {
      float n = 0.0f;
#pragma unroll 8
      for (int c = 0; c < H / 256; ++c) n += wnorm[(int64_t)c * E + e];
      wn_max = fmaxf(wn_max, n);
      if (balance && balance[e] > -INFINITY) bal = fmaxf(bal, fabsf(balance[e]));
    }
    wn_max = group_max<64>(wn_max);
    bal = group_max<64>(bal);
    if (lane == 0) most[0] = wn_max, most[1] = bal;
  }
  f32x16 d[2], r[2];  // the first parts' product, and the others
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int i = 0; i < 16; ++i) r[t][i] = 0.0f;
  // first, last: of 64 columns; flush: of kRest; more: a step follows
  auto step = [&](int buf, bool first, bool last, bool flush, bool more) {
    constexpr int K = KS / 16;
    const uint16_t* b = lds + buf * XP * kTile;
    bf16x8 v[2][2][XP];
    auto read = [&](int k) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int p = 0; p < XP; ++p)
          v[k & 1][t][p] = *reinterpret_cast<const bf16x8*>(b + p * kTile + slot(32 * t + l31, 2 * k + hh));
    };
    if (first) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) d[t][i] = 0.0f;
    }
    wp += K * 1536;
    read(0);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (k + 1 < K) read(k + 1);
#pragma unroll
      for (int o = 2; o >= 0; --o)
#pragma unroll
        for (int p = 0; p < XP; ++p) {
          const int q = o - p;
          if (q < 0) continue;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            f32x16& to = o ? r[t] : d[t];
            to = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v[k & 1][t][p], w[k][q], to, 0, 0, 0);
          }
        }
      if (more) load_w(k);
    }
    if (last) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[t][i] += (double)d[t][i];
    }
    if (flush) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          acc[t][i] += (double)r[t][i];
          r[t][i] = 0.0f;
        }
    }
  };
#pragma unroll
  for (int k = 0; k < KS / 16; ++k) load_w(k);
  fetch(kbeg, 0);
  if (kbeg + KS < kend) fetch(kbeg + KS, 1);
  put(0, 0);
  __syncthreads();
  for (int kc = kbeg; kc < kend; kc += 2 * KS) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // step kc / KS + h is in LDS h, the next one in registers 1 - h
      const int at = kc + h * KS;
      if (at >= kend) break;
      if (at + 2 * KS < kend) fetch(at + 2 * KS, h);
      step(h, KS == 64 || h == 0, KS == 64 || h == 1, h == 1 && (at + KS - kbeg) % kRest == 0, at + KS < kend);
      if (at + KS < kend) put(1 - h, 1 - h);
      __syncthreads();
    }
  }
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[t][i] += (double)r[t][i];
  const int e = e0 + 32 * wave + l31;
  if (e < E) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int tok = t0 + 32 * t + 8 * (i >> 2) + 4 * hh + (i & 3);
        if (tok < T) part[((int64_t)sl * T + tok) * E + e] = acc[t][i];
      }
  }
  if (norms) {
    xx += xor_lanes<1>(xx);
    xx += xor_lanes<2>(xx);
    if ((tid & 3) == 0 && has_t) xnorm[(int64_t)sl * T + t0 + row] = xx;
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
//   kBounded the bf16 form's: scores and order in fp32, and a token whose choice
//            the bound on both leaves open is put on the list; the winners' scores
//            are formed again in fp64 for the gates
//   kListed  the list's tokens, as kExact
enum Logits { kExact, kBounded, kListed };

// A wave for each token: lane l holds experts l + 64 i.  Groups are valued by
// 64 / groups lanes each (a power of two); the k winners are taken one at a
// time: the larger key (its high word, then its low one), then the lower expert.
// Measured: one token of 128 experts 5.2 us (a chain of loads, fp64 exp and k
// rounds), 128 of 256 7.6, 8191 of 256 in fp32 21 (bound by the vector ALU's issue;
// in fp64 28).
template <Logits FROM>
__global__ __launch_bounds__(64) void k_route_select(RouteArgs g) {
  constexpr bool B = FROM == kBounded;
  using F = std::conditional_t<B, float, double>;  // scores
  __shared__ F s_c[256];
  const int lane = threadIdx.x;
  const int E = g.E;
  int64_t t = blockIdx.x, at = t, n = g.T;
  int S = g.S;
  if constexpr (FROM == kListed) {
    n = min(*g.count, g.T);
    if (t >= n) return;
    S = list_plan((int)n, E, g.H).S;
    t = g.list[t];
  }
  // (loaded first: they are on their way with the partials)
  float bias[4], bal[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    bias[i] = g.bias && lane + 64 * i < E ? g.bias[lane + 64 * i] : 0.0f;
    bal[i] = g.balance && lane + 64 * i < E ? g.balance[lane + 64 * i] : 0.0f;
  }
  double l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) l[i] = 0.0;
  // the slices in order, some on their way at a time
  constexpr int U = B ? 2 : 8;
  for (int p = 0; p < S; p += U) {
    double v[4][U];
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i][j] = p + j < S && lane + 64 * i < E ? g.part[((int64_t)(p + j) * n + at) * E + lane + 64 * i] : 0.0;
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) l[i] += v[i][j];
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
  // rounded by, s log(top_s / s) 2^-23; the sums with the balance and here once more
  float off = 0.0f, most = 0.0f, delta[4];  // most: of a group's experts
  bool open = false;
  if constexpr (B) {
    float xn = 0.0f;
    for (int p = 0; p < S; ++p) xn += g.xnorm[(int64_t)p * g.T + t];
    far = group_max<64>(far);
    const float nx = sqrtf(xn) * 1.001f, nw = sqrtf(g.most[0]) * 1.001f;  // their own sums' rounding
    off = (float)kFastError * nx * nw + 0x1p-119f * (nx + nw) + 0x1p-22f * far;
    open = !(off < 0.01f);  // past where the slopes hold, or no number
    const float edge = g.sigmoid ? 0x1p-21f * (1.0f + g.most[1]) : 0x1p-24f * top_s + 0x1p-23f * g.most[1] + 1e-14f;
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
      if constexpr (B) {
        hi[i] = order_key32(c[i]);
      } else {
        const uint64_t k = order64(c[i]);
        hi[i] = (uint32_t)(k >> 32);
        lo[i] = (uint32_t)k;
      }
    }
  }
  if (g.kept < g.groups) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (lane + 64 * i < E) s_c[lane + 64 * i] = c[i];
    __builtin_amdgcn_wave_barrier();
    const int per = E / g.groups, L = g.lanes, grp = lane / L;
    auto larger = [](F p, F q) { return p > q ? p : q; };  // no NaN here
    auto smaller = [](F p, F q) { return p > q ? q : p; };
    F a = -INFINITY, b = -INFINITY;  // the group's largest two
    if (grp < g.groups)
      for (int j = lane % L; j < per; j += L) {
        const F v = s_c[grp * per + j];
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
      const uint64_t last = __builtin_amdgcn_ballot_w64(grp < g.groups && rank == g.kept - 1);
      const uint64_t next = __builtin_amdgcn_ballot_w64(grp < g.groups && rank == g.kept);
      const float gap = lane_of(value, __builtin_ctzll(last)) - lane_of(value, __builtin_ctzll(next));
      open |= !(gap > most * (g.best_two ? 4.0f : 2.0f));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = lane + 64 * i;
      if (e < E && !(keep >> (e / per * L) & 1)) hi[i] = lo[i] = 0;
    }
  }
  int my_e = 0;
  F my_s = 0, last_c = 0, last_d = 0;
  double my_l = 0.0;
  for (int j = 0; j < g.k + (B ? 1 : 0); ++j) {
    if (B && j == g.k) {  // behind the last winner: what the others may reach at most
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (hi[i]) hi[i] = order_key32(c[i] + delta[i]);
    }
    const uint32_t h = wave_max_u32(max(max(hi[0], hi[1]), max(hi[2], hi[3])));
    if (B && h == 0) break;  // k experts are all that may be chosen
    if (B && j == g.k) {
      open |= !(last_c - last_d > key_logit(h));
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
    F v = s[0], cc = c[0], dd = B ? delta[0] : 0;
    double lv = l[0];
#pragma unroll
    for (int i = 1; i < 4; ++i)
      if (slot == i) v = s[i], cc = c[i], lv = l[i], dd = B ? delta[i] : 0;
    v = lane_of(v, who);
    if constexpr (B) {
      cc = lane_of(cc, who);
      dd = lane_of(dd, who);
      if (j) open |= !(last_c - cc > last_d + dd);
      last_c = cc;
      last_d = dd;
      lv = lane_of(lv, who);
    }
    if (lane == j) my_s = v, my_e = who + 64 * slot, my_l = lv;
    if (lane == who) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (slot == i) hi[i] = lo[i] = 0;
    }
  }
  if constexpr (B) {
    if (open) {
      if (lane == 0) g.list[atomicAdd(g.count, 1)] = (int)t;  // the order does not matter: each token stands for itself
      return;
    }
  }
  double gate = (double)my_s;
  if constexpr (B) gate = g.sigmoid ? 1.0 / (1.0 + exp(-my_l)) : exp(my_l - (double)m) * (double)top_s;
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

// Whether the bf16 form pays: both forms' times in us, linear in Gflop (whole tiles
// of experts in the bf16 form), as measured over 128 to 16384 tokens.  us, bf16
// form and fp64: 6144 x 256, bf16, 512 tokens 57 and 41, 1024 59 and 72, 8192 158
// and 439; fp32 1024 86 and 72, 2048 101 and 120, 8192 257 and 435; 2048 x 128, fp32,
// 4096 76 and 53, 8192 84 and 93; 4096 x 64, bf16, 4096 52 and 54, 8192 66 and 93.
static bool route_fast(int64_t T, int H, int E, int xt) {
  const double g = 2e-9 * T * H * E, whole = 2e-9 * T * H * ((E + kFT - 1) / kFT * kFT);
  return 18.0 + 16.2 * g > (xt == XF32 ? 55.0 + 7.5 * whole : 40.0 + 4.3 * whole);
}

// K-slices of the product: enough that every compute unit has a workgroup, a
// slice of 256 at least (the bf16 form: of 1024).
RoutePlan route_plan(int64_t T, int H, int E, int xt, bool fast) {
  RoutePlan p{};
  p.Ks = H;
  p.S = 1;
  p.fast = fast && T > kRouteFew && route_fast(T, H, E, xt);
  if (T > kRouteFew) {
    const int tile = p.fast ? kFT : kGT, step = p.fast ? 1024 : 256;
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
    p.planes = take(6 * ets * kFT * H);
    p.wnorm = take(4 * (size_t)E * (H / 256));
    p.most = take(8);
    p.xnorm = take(4 * rows);
    p.count = take(4);
    p.list = take(4 * (size_t)T);
    // the list's slices: kListGroups workgroups of a tile each, or one slice
    const size_t listed = (size_t)kListGroups / small * kGT;
    if (rows < listed) rows = listed;
  }
  p.part = take(8 * rows * E);
  return p;
}

template <int XT>
static hipError_t launch_fast(const RouteArgs& g, const RoutePlan& p, const void* x, int H, const float* Wr, uint16_t* planes,
                              hipStream_t st) {
  const int ets = (g.E + kFT - 1) / kFT;
  hipLaunchKernelGGL(k_route_split, dim3(ets * kFT / 32, H / 256), dim3(256), 0, st, Wr, g.E, H, planes, g.wnorm, g.count);
  hipLaunchKernelGGL((k_route_fast<XT>), dim3(ets * p.S * ((g.T + kTT - 1) / kTT)), dim3(256), 0, st, x, g.T, H, planes,
                     g.E, p.Ks, p.S, g.part, g.xnorm, g.wnorm, g.balance, g.most);
  hipLaunchKernelGGL((k_route_select<kBounded>), dim3(g.T), dim3(64), 0, st, g);
  hipLaunchKernelGGL((k_route_gemm<XT, true>), dim3(kListGroups), dim3(256), 0, st, x, g.T, H, Wr, g.E, 0, g.part, g.count,
                     g.list);
  hipLaunchKernelGGL((k_route_select<kListed>), dim3(g.T), dim3(64), 0, st, g);
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
    return xt == XF32 ? launch_fast<XF32>(g, p, x, H, Wr, planes, st) : launch_fast<XBF16>(g, p, x, H, Wr, planes, st);
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

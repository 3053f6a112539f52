// i8gemm.hip -- the product in 8-bit integers with a scale for each token and
// output channel.
//
//   s_t  = max_c |x_tc| / 127                 (fp32, correctly rounded)
//   q_tc = rint(x_tc / s_t)  in -127..127     (ties to even)
//   y_tn = s_t * w_n * sum_c q_tc W_nc (+ b_n)
//
// The sum is exact in int32 (|q W| <= 127 * 128, at most 16384 terms: under
// 2^28), so any order and any split of it gives the same bits; the only
// roundings are the codes, the int-to-fp32 conversion, the two scale products,
// the bias add and the store.
#include <hip/hip_runtime.h>

#include "common.hpp"
#include "i8.hpp"
#include "kernels.hpp"
#include "rows.hpp"

namespace md {

// ---- codes ---------------------------------------------------------------

// A row's scale from its largest magnitude's bits.  One that holds an infinity
// or a NaN gets the scale NaN and codes 0, so its products are NaN and no other
// row's are.
struct RowScale {
  float s;
  Step step;
};
MD_DEV RowScale row_scale_of(uint32_t top) {
  const float amax = __uint_as_float(top), s = top >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : amax / 127.0f;
  return RowScale{s, step_of(s, amax)};
}

// One row per group of WPR waves (WPR 1: four rows a workgroup), the whole row
// in registers between the maximum and the codes: x is read once.  Bound by
// the read of x (8191 x 6144 bf16: 28 us, 5.4 TB/s read and written together).
template <int XT, int WPR, int STEPS>
__global__ __launch_bounds__(256) void k_i8_quantize(const void* __restrict__ x, int T, int K,
                                                     int8_t* __restrict__ codes, float* __restrict__ scales) {
  __shared__ uint32_t red[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int row = WPR == 1 ? (int)blockIdx.x * 4 + wave : (int)blockIdx.x;
  if (WPR == 1 && row >= T) return;
  const int at = 8 * (WPR == 1 ? lane : (int)threadIdx.x);
  constexpr int kStep = 8 * 64 * WPR;
  const int64_t base = (int64_t)row * K;
  float v[STEPS][8];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int c = at + i * kStep;
    if (c < K) {
      load8<XT>(x, base + c, v[i]);
    } else {
#pragma unroll
      for (int m = 0; m < 8; ++m) v[i][m] = 0.0f;
    }
  }
#pragma unroll
  for (int i = 0; i < STEPS; ++i)
#pragma unroll
    for (int m = 0; m < 8; ++m) top = max(top, __float_as_uint(v[i][m]) & 0x7FFFFFFFu);
  top = wave_max_u32(top);
  if constexpr (WPR > 1) {
    if (lane == 0) red[wave] = top;
    __syncthreads();
    top = max(max(red[0], red[1]), max(red[2], red[3]));
  }
  const RowScale s = row_scale_of(top);
  if (at == 0) scales[row] = s.s;
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int c = at + i * kStep;
    if (c < K) *reinterpret_cast<uint2*>(codes + base + c) = codes8(v[i], s.step);
  }
}

hipError_t launch_i8_quantize(const void* x, int xt, int T, int K, int8_t* codes, float* scales, hipStream_t st) {
#define MD_Q(X_, W_, S_)                                                                                            \
  hipLaunchKernelGGL((k_i8_quantize<X_, W_, S_>), dim3(W_ == 1 ? (T + 3) / 4 : T), dim3(256), 0, st, x, T, K, codes, \
                     scales)
#define MD_QS(X_)                          \
  do {                                     \
    if (K <= 512) MD_Q(X_, 1, 1);          \
    else if (K <= 2048) MD_Q(X_, 1, 4);    \
    else if (K <= 6144) MD_Q(X_, 4, 3);    \
    else MD_Q(X_, 4, 8);                   \
  } while (0)
  if (xt == XF32) MD_QS(XF32);
  else MD_QS(XBF16);
#undef MD_QS
#undef MD_Q
  return hipGetLastError();
}

// ---- products ------------------------------------------------------------

constexpr int kOwnTokens = 8;      // up to these each workgroup may form the codes itself
constexpr int kOwnSteps = 4;       // ... of rows of up to 512 times this, one wave a row
constexpr int kFewTokens = 32;     // up to these: k_i8_few
constexpr int kSplitTokens = 512;  // up to these the sum may be split

// Four consecutive outputs of one token; the ones past N are left alone.
template <int YT>
MD_DEV void put4(void* y, int64_t row, int N, int n, const i32x4& a, float xs, const float* ws, const float* bias) {
  float f[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int c = min(n + r, N - 1);
    f[r] = (float)a[r] * ws[c] * xs;
    if (bias) f[r] += bias[c];
  }
  const int64_t o = row * N + n;
  if (YT == XF32) {
    float* p = static_cast<float*>(y) + o;
    if (n + 3 < N && (N & 3) == 0) *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    else
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (n + r < N) p[r] = f[r];
  } else {
    uint16_t* p = static_cast<uint16_t*>(y) + o;
    if (n + 3 < N && (N & 3) == 0) {
      *reinterpret_cast<uint2*>(p) = make_uint2(to_bf16(f[0]) | (uint32_t)to_bf16(f[1]) << 16,
                                                to_bf16(f[2]) | (uint32_t)to_bf16(f[3]) << 16);
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (n + r < N) p[r] = to_bf16(f[r]);
    }
  }
}

// Few tokens: a workgroup owns 16 output channels and NT tiles of 16 tokens,
// its waves split the sum and meet in LDS.  Weights go from HBM straight into
// the matrix cores' operand registers (lane l: row l % 16, 16 bytes at
// 64 step + 16 (l / 16)), codes of x from the L2.
// Reads W once (6144 x 6144, 37.7 MB from HBM, us a call: 4 tokens 11.1, with the
// quantizer's launch 14.6; 32 tokens 21.9 and 25.8): 3.4 TB/s at 4 tokens, half of
// what a plain read reaches.
// OWN: x itself comes in, and every workgroup rounds all of it to codes in its
// LDS while its first weights are on their way: one launch less, which is half
// of a small call (i8_own_codes).
enum Own { kNoOwn, kOwnRow, kOwnRows };
template <int YT, int NT, Own OWN, int XT>
__global__ __launch_bounds__(1024) void k_i8_few(const int8_t* __restrict__ W, const float* __restrict__ ws, int N,
                                                 int K, const void* __restrict__ x, const float* __restrict__ xs_in,
                                                 int T, const float* __restrict__ bias, void* __restrict__ y) {
  extern __shared__ __attribute__((aligned(16))) int8_t few_lds[];  // shares of the sum; OWN: then T rows of codes
  __shared__ uint32_t red[16];                                      // OWN: the waves' maxima, or the rows' scales
  int* part = reinterpret_cast<int*>(few_lds);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, nw = blockDim.x >> 6;
  const int n0 = blockIdx.x * 16, r = lane & 15, g = lane >> 4;
  const int8_t* wp = W + (int64_t)min(n0 + r, N - 1) * K + 16 * g;
  i32x4 a[4], acc[NT];
  // wave w takes the 256-byte pieces w, w + nw, ...
  auto weights = [&](int k) {
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const i32x4*>(wp + k + 64 * i);
  };
  if (wave * 256 < K) weights(wave * 256);
  const int8_t* xp[NT];
  float own = 0.0f;  // OWN: the scale of this lane's token
  if constexpr (OWN == kOwnRow) {
    int8_t* codes = few_lds + nw * 1024;
    uint32_t top = 0;
    for (int c = 8 * tid; c < K; c += 8 * (int)blockDim.x) {
      float v[8];
      load8<XT>(x, c, v);
#pragma unroll
      for (int m = 0; m < 8; ++m) top = max(top, __float_as_uint(v[m]) & 0x7FFFFFFFu);
    }
    top = wave_max_u32(top);
    if (lane == 0) red[wave] = top;
    __syncthreads();
    for (int w = 0; w < nw; ++w) top = max(top, red[w]);
    const RowScale s = row_scale_of(top);
    own = s.s;
    for (int c = 8 * tid; c < K; c += 8 * (int)blockDim.x) {
      float v[8];
      load8<XT>(x, c, v);
      *reinterpret_cast<uint2*>(codes + c) = codes8(v, s.step);
    }
    __syncthreads();
    xp[0] = codes + 16 * g;
  } else if constexpr (OWN == kOwnRows) {
    int8_t* codes = few_lds + nw * 1024;  // rows K + 16 bytes apart: the sixteen of a fragment in different banks
    for (int t = wave; t < T; t += nw) {
      float v[kOwnSteps][8];
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < kOwnSteps; ++i) {
        const int c = 8 * lane + 512 * i;
        if (c < K) {
          load8<XT>(x, (int64_t)t * K + c, v[i]);
#pragma unroll
          for (int m = 0; m < 8; ++m) top = max(top, __float_as_uint(v[i][m]) & 0x7FFFFFFFu);
        }
      }
      const RowScale s = row_scale_of(wave_max_u32(top));
      if (lane == 0) red[t] = __float_as_uint(s.s);
#pragma unroll
      for (int i = 0; i < kOwnSteps; ++i) {
        const int c = 8 * lane + 512 * i;
        if (c < K) *reinterpret_cast<uint2*>(codes + t * (K + 16) + c) = codes8(v[i], s.step);
      }
    }
    __syncthreads();
    own = __uint_as_float(red[min(r, T - 1)]);
    xp[0] = codes + min(r, T - 1) * (K + 16) + 16 * g;
  } else {
#pragma unroll
    for (int t = 0; t < NT; ++t) xp[t] = static_cast<const int8_t*>(x) + (int64_t)min(t * 16 + r, T - 1) * K + 16 * g;
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = i32x4{0, 0, 0, 0};
  for (int k = wave * 256; k < K;) {
    i32x4 b[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) b[t][i] = *reinterpret_cast<const i32x4*>(xp[t] + k + 64 * i);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[i], b[t][i], acc[t], 0, 0, 0);
    k += nw * 256;
    if (k < K) weights(k);
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) *reinterpret_cast<i32x4*>(part + ((wave * NT + t) * 64 + lane) * 4) = acc[t];
  __syncthreads();
  for (int t = wave; t < NT; t += nw) {
    i32x4 sum{0, 0, 0, 0};
    for (int w = 0; w < nw; ++w) sum += *reinterpret_cast<const i32x4*>(part + ((w * NT + t) * 64 + lane) * 4);
    const int tok = t * 16 + r, n = n0 + 4 * g;
    if (tok < T && n < N) put4<YT>(y, tok, N, n, sum, OWN != kNoOwn ? own : xs_in[tok], ws, bias);
  }
}

// Many tokens: BN channels x BT tokens per workgroup of WN x WT waves, 128
// bytes of the sum per step, ST steps' tiles in LDS, filled ST - 1 steps ahead
// by direct loads.  Chunk p (16 bytes) of tile row r holds chunk p ^ (r & 7) of
// the row, so the rows that a fragment read touches spread over the banks (no
// conflicts counted).  Every stage is a variable of its own and the loop is
// unrolled over them: the compiler waits for all direct loads in flight before
// an LDS read that might touch what they fill, and can only tell variables
// apart (404 -> 326 us for 8191 tokens, 5632 channels, 6144 terms with the
// quantizer, which was 35 of them then and is 28 now: 320).  The large tile is bound by LDS reads, which deliver 64
// bytes a clock here: 24 of 1 KB per wave and step against 64 products of 16
// clocks, 1.95 Pop/s of 2.35 that a large library product reaches.  Measured
// and dropped: fragments read half a step ahead (332), 64-byte steps in four
// stages (342), four waves of 128 x 128 outputs (spills: 683), the weights
// straight from L1 into registers (451 to 488).
constexpr int kBK = 128;

// All but the N youngest of this wave's loads have landed, its LDS reads are
// done (the next load may overwrite what they read), and all waves are here.
template <int N>
MD_DEV void landed() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070 | (N & 15) | (N >> 4) << 14);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// part: one of gridDim.y equal shares of the sum, as int32 [share][T][N]; else y.
template <int YT, int BN, int BT, int WN, int WT, int ST, bool PART>
__global__ __launch_bounds__(64 * WN * WT) void k_i8_tile(const int8_t* __restrict__ W, const float* __restrict__ ws,
                                                          int N, int K, const int8_t* __restrict__ xq,
                                                          const float* __restrict__ xs, int T,
                                                          const float* __restrict__ bias, void* __restrict__ y,
                                                          int tn, int tt) {
  constexpr int NW = WN * WT, RN = BN / WN / 16, RT = BT / WT / 16;
  constexpr int LW = BN * kBK / 1024 / NW, LX = BT * kBK / 1024 / NW;  // 1 KB loads per wave and step
  static_assert(LW * NW * 1024 == BN * kBK && LX * NW * 1024 == BT * kBK, "tile");
  __shared__ __attribute__((aligned(16))) int8_t w0[BN * kBK], w1[BN * kBK], w2[ST > 2 ? BN * kBK : 16], w3[ST > 2 ? BN * kBK : 16];
  __shared__ __attribute__((aligned(16))) int8_t x0[BT * kBK], x1[BT * kBK], x2[ST > 2 ? BT * kBK : 16], x3[ST > 2 ? BT * kBK : 16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // workgroups go round the 8 dies: give each die a run of neighbouring tiles
  const int total = tn * tt, per = (total + 7) >> 3;
  const int id = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
  if (id >= total || (int)(blockIdx.x >> 3) >= per) return;
  constexpr int kGroup = 4;
  const int band = id / (kGroup * tn), in = id % (kGroup * tn), rows = min(kGroup, tt - band * kGroup);
  const int t0 = (band * kGroup + in % rows) * BT, n0 = (in / rows) * BN;
  const int share = PART ? K / (int)gridDim.y : K, k0 = PART ? (int)blockIdx.y * share : 0;

  const int lr = lane >> 3, lc = (lane & 7) ^ lr;  // row and chunk of a load's 8 rows
  const int8_t* wsrc[LW];
  const int8_t* xsrc[LX];
#pragma unroll
  for (int i = 0; i < LW; ++i) wsrc[i] = W + (int64_t)min(n0 + (wave * LW + i) * 8 + lr, N - 1) * K + k0 + 16 * lc;
#pragma unroll
  for (int i = 0; i < LX; ++i) xsrc[i] = xq + (int64_t)min(t0 + (wave * LX + i) * 8 + lr, T - 1) * K + k0 + 16 * lc;
  const int steps = share / kBK;
  // past the last step that one again: the number in flight stays the same
  auto load = [&](int8_t* sw, int8_t* sx, int step) {
    const int k = min(step, steps - 1) * kBK;
#pragma unroll
    for (int i = 0; i < LW; ++i)
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(wsrc[i] + k),
                                       (__attribute__((address_space(3))) void*)(sw + (wave * LW + i) * 1024), 16, 0, 0);
#pragma unroll
    for (int i = 0; i < LX; ++i)
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(xsrc[i] + k),
                                       (__attribute__((address_space(3))) void*)(sx + (wave * LX + i) * 1024), 16, 0, 0);
  };
  const int wn = wave % WN, wt = wave / WN, r = lane & 15, g = lane >> 4;
  i32x4 acc[RN][RT];
#pragma unroll
  for (int i = 0; i < RN; ++i)
#pragma unroll
    for (int j = 0; j < RT; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  auto multiply = [&](const int8_t* sw, const int8_t* sx) {
    const int8_t* bw = sw + (wn * RN * 16 + r) * kBK;
    const int8_t* bx = sx + (wt * RT * 16 + r) * kBK;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int o = ((4 * h + g) ^ (r & 7)) * 16;
      i32x4 a[RN], b[RT];
#pragma unroll
      for (int i = 0; i < RN; ++i) a[i] = *reinterpret_cast<const i32x4*>(bw + i * 16 * kBK + o);
#pragma unroll
      for (int j = 0; j < RT; ++j) b[j] = *reinterpret_cast<const i32x4*>(bx + j * 16 * kBK + o);
#pragma unroll
      for (int i = 0; i < RN; ++i)
#pragma unroll
        for (int j = 0; j < RT; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[i], b[j], acc[i][j], 0, 0, 0);
    }
  };
  load(w0, x0, 0);
  if constexpr (ST == 4) {
    load(w1, x1, 1);
    load(w2, x2, 2);
  }
  constexpr int kFly = (ST - 2) * (LW + LX);
  for (int s = 0;;) {
#define MD_STEP(W_, X_, NW_, NX_)  \
  landed<kFly>();                  \
  load(NW_, NX_, s + ST - 1);      \
  __builtin_amdgcn_sched_barrier(0); \
  multiply(W_, X_);                \
  if (++s == steps) break;
    if constexpr (ST == 2) {
      MD_STEP(w0, x0, w1, x1)
      MD_STEP(w1, x1, w0, x0)
    } else {
      MD_STEP(w0, x0, w3, x3)
      MD_STEP(w1, x1, w0, x0)
      MD_STEP(w2, x2, w1, x1)
      MD_STEP(w3, x3, w2, x2)
    }
#undef MD_STEP
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);  // no load into this workgroup's LDS outlives it
#pragma unroll
  for (int j = 0; j < RT; ++j) {
    const int tok = t0 + (wt * RT + j) * 16 + r;
    if (tok >= T) continue;
    const float sc = PART ? 0.0f : xs[tok];
#pragma unroll
    for (int i = 0; i < RN; ++i) {
      const int n = n0 + (wn * RN + i) * 16 + 4 * g;
      if (n >= N) continue;
      if constexpr (PART) {  // rows of N rounded up to 4
        const int64_t np = (N + 3) & ~3;
        *reinterpret_cast<i32x4*>(static_cast<int*>(y) + ((int64_t)blockIdx.y * T + tok) * np + n) = acc[i][j];
      } else {
        put4<YT>(y, tok, N, n, acc[i][j], sc, ws, bias);
      }
    }
  }
}

// The shares of four outputs a thread, added and scaled.
template <int YT>
__global__ __launch_bounds__(256) void k_i8_join(const int* __restrict__ part, int S, int T, int N,
                                                 const float* __restrict__ ws, const float* __restrict__ xs,
                                                 const float* __restrict__ bias, void* __restrict__ y) {
  const int n = 4 * (blockIdx.x * 256 + threadIdx.x), t = blockIdx.y;
  const int64_t np = (N + 3) & ~3;
  if (n >= N) return;
  i32x4 a{0, 0, 0, 0};
  for (int s = 0; s < S; ++s) a += *reinterpret_cast<const i32x4*>(part + ((int64_t)s * T + t) * np + n);
  put4<YT>(y, t, N, n, a, xs[t], ws, bias);
}

// How many shares of the sum make enough workgroups where the outputs alone do
// not: whole steps each, four at least, and together at most one workgroup a
// compute unit (128 tokens, 6144 channels, 6144 terms: two shares 25 us, four
// with up to 512 workgroups 28.6; without shares, on 64 x 64 tiles, 38).
int i8_shares(int N, int K, int T) {
  if (T <= kFewTokens || T > kSplitTokens) return 1;
  const int64_t tiles = (int64_t)((N + 63) / 64) * ((T + 127) / 128);
  int best = 1;
  for (int s = 2; s <= 16 && tiles * s <= 256; ++s)
    if (K % (s * kBK) == 0 && K / (s * kBK) >= 4) best = s;
  return best;
}

static int few_waves(int K) { return K <= 1024 ? 4 : K <= 4096 ? 8 : 16; }

// One token (256 channels of 2048 terms: 7.9 -> 4.7 us), or a few of rows that a
// wave holds, where all workgroups together do not round too much (bf16 in, us
// with the quantizer's launch and without: 2 x 256 x 256 5.5 and 3.7, 4 x 2048 x
// 1024 6.8 and 5.1, 8 x 6144 x 2048 11.0 and 10.3; but 8 x 16384 x 2048 14.4 and
// 18.7, 12 x 2048 x 1024 7.4 and 8.2).
bool i8_own_codes(int N, int K, int T) {
  return T == 1 || (T <= kOwnTokens && K <= 512 * kOwnSteps && (int64_t)N * T * K <= 1 << 27);
}

hipError_t launch_i8_own(const int8_t* W, const float* ws, int N, int K, const void* x, int xt, int T,
                         const float* bias, void* y, int yt, hipStream_t st) {
  const int nw = few_waves(K);
  const dim3 grid((N + 15) / 16), block(64 * nw);
  const size_t lds = (size_t)nw * 1024 + (T == 1 ? (size_t)K : (size_t)T * (K + 16));
#define MD_OWNS(Y_, X_, O_)                                                                                       \
  hipLaunchKernelGGL((k_i8_few<Y_, 1, O_, X_>), grid, block, lds, st, W, ws, N, K, x, (const float*)nullptr, T, bias, y)
#define MD_OWN(Y_, X_)                    \
  do {                                    \
    if (T == 1) MD_OWNS(Y_, X_, kOwnRow); \
    else MD_OWNS(Y_, X_, kOwnRows);       \
  } while (0)
  if (yt == XF32) {
    if (xt == XF32) MD_OWN(XF32, XF32);
    else MD_OWN(XF32, XBF16);
  } else {
    if (xt == XF32) MD_OWN(XBF16, XF32);
    else MD_OWN(XBF16, XBF16);
  }
#undef MD_OWN
#undef MD_OWNS
  return hipGetLastError();
}

template <int YT>
static hipError_t matmul(const int8_t* W, const float* ws, int N, int K, const int8_t* xq, const float* xs, int T,
                         const float* bias, void* y, int shares, int* part, hipStream_t st) {
  if (T <= kFewTokens) {
    const int nw = few_waves(K);
    const dim3 grid((N + 15) / 16), block(64 * nw);
    if (T <= 16)
      hipLaunchKernelGGL((k_i8_few<YT, 1, kNoOwn, XF32>), grid, block, (size_t)nw * 1024, st, W, ws, N, K, xq, xs, T, bias, y);
    else
      hipLaunchKernelGGL((k_i8_few<YT, 2, kNoOwn, XF32>), grid, block, (size_t)nw * 2048, st, W, ws, N, K, xq, xs, T, bias, y);
    return hipGetLastError();
  }
  auto tiles = [&](int bn, int bt) { return (int64_t)((N + bn - 1) / bn) * ((T + bt - 1) / bt); };
#define MD_TILE(BN_, BT_, WN_, WT_, ST_, P_, Y_, S_)                                                                  \
  do {                                                                                                              \
    const int tn = (N + BN_ - 1) / BN_, tt = (T + BT_ - 1) / BT_;                                                   \
    hipLaunchKernelGGL((k_i8_tile<YT, BN_, BT_, WN_, WT_, ST_, P_>),                                                \
                       dim3((unsigned)((((int64_t)tn * tt + 7) >> 3) << 3), S_), dim3(64 * WN_ * WT_), 0, st, W, ws, \
                       N, K, xq, xs, T, bias, Y_, tn, tt);                                                          \
  } while (0)
  if (shares > 1) {
    MD_TILE(64, 128, 2, 2, 4, true, part, shares);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_i8_join<YT>), dim3((N + 1023) / 1024, T), dim3(256), 0, st, part, shares, T, N, ws, xs, bias,
                       y);
  } else if (tiles(256, 256) >= 192) {  // large tiles where they fill the chip: 2048 tokens, 6144 x 6144, 139 -> 113 us
                                       // against the next size; below 192 of them slower (1024 tokens: 77 against 100)
    MD_TILE(256, 256, 4, 2, 2, false, y, 1);
  } else if (tiles(128, 128) >= 256) {  // 384 tokens, 6144 x 2048: 27.9 on 144 of these, 25.6 on the small ones
    MD_TILE(128, 128, 2, 2, 2, false, y, 1);
  } else {
    MD_TILE(64, 64, 2, 2, 4, false, y, 1);
  }
#undef MD_TILE
  return hipGetLastError();
}

// part: i8_shares() * T * (N rounded up to 4) int32, or null (no split: the same
// bits from fewer workgroups).
hipError_t launch_i8_matmul(const int8_t* W, const float* ws, int N, int K, const int8_t* xq, const float* xs, int T,
                            const float* bias, void* y, int yt, int* part, hipStream_t st) {
  const int shares = part ? i8_shares(N, K, T) : 1;
  return yt == XF32 ? matmul<XF32>(W, ws, N, K, xq, xs, T, bias, y, shares, part, st)
                    : matmul<XBF16>(W, ws, N, K, xq, xs, T, bias, y, shares, part, st);
}

}  // namespace md

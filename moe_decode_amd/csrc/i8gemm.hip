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

// One row per group of WPR waves (WPR 1: four rows a workgroup), the whole row
// in registers between the maximum and the codes: x is read once.  Bound by
// the read of x.  A row that holds an infinity or a NaN gets the scale NaN and
// codes 0, so its products are NaN and no other row's are.
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
  const float amax = __uint_as_float(top);
  const bool bad = top >= 0x7F800000u;
  const float s = bad ? __uint_as_float(0x7FC00000u) : amax / 127.0f;
  if (at == 0) scales[row] = s;
  const float up = amax < kTiny ? kTinyUp : 1.0f;
  const bool none = bad || !(s > 0.0f);
  const float ss = none ? 1.0f : s * up, inv = 1.0f / ss;
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int c = at + i * kStep;
    if (c >= K) continue;
    uint32_t w[2] = {0, 0};
    if (!none) {
#pragma unroll
      for (int m = 0; m < 8; ++m) w[m >> 2] |= (uint32_t)(code_of(v[i][m] * up, ss, inv) & 255) << (8 * (m & 3));
    }
    *reinterpret_cast<uint2*>(codes + base + c) = make_uint2(w[0], w[1]);
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
template <int YT, int NT>
__global__ __launch_bounds__(1024) void k_i8_few(const int8_t* __restrict__ W, const float* __restrict__ ws, int N,
                                                 int K, const int8_t* __restrict__ xq, const float* __restrict__ xs,
                                                 int T, const float* __restrict__ bias, void* __restrict__ y) {
  extern __shared__ int part[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, nw = blockDim.x >> 6;
  const int n0 = blockIdx.x * 16, r = lane & 15, g = lane >> 4;
  const int8_t* wp = W + (int64_t)min(n0 + r, N - 1) * K + 16 * g;
  const int8_t* xp[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) xp[t] = xq + (int64_t)min(t * 16 + r, T - 1) * K + 16 * g;
  i32x4 acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = i32x4{0, 0, 0, 0};
  // wave w takes the 256-byte pieces w, w + nw, ...
  for (int k = wave * 256; k < K; k += nw * 256) {
    i32x4 a[4], b[NT][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const i32x4*>(wp + k + 64 * i);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) b[t][i] = *reinterpret_cast<const i32x4*>(xp[t] + k + 64 * i);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[i], b[t][i], acc[t], 0, 0, 0);
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) *reinterpret_cast<i32x4*>(part + ((wave * NT + t) * 64 + lane) * 4) = acc[t];
  __syncthreads();
  for (int t = wave; t < NT; t += nw) {
    i32x4 sum{0, 0, 0, 0};
    for (int w = 0; w < nw; ++w) sum += *reinterpret_cast<const i32x4*>(part + ((w * NT + t) * 64 + lane) * 4);
    const int tok = t * 16 + r, n = n0 + 4 * g;
    if (tok < T && n < N) put4<YT>(y, tok, N, n, sum, xs[tok], ws, bias);
  }
}

// Many tokens: BN channels x BT tokens per workgroup of WN x WT waves, 128
// bytes of the sum per step, double-buffered in LDS.  Chunk p (16 bytes) of
// tile row r holds chunk p ^ (r & 7) of the row, so the 16 rows that a fragment
// read touches spread over the banks.
constexpr int kBK = 128;

template <int YT, int BN, int BT, int WN, int WT>
__global__ __launch_bounds__(64 * WN * WT) void k_i8_tile(const int8_t* __restrict__ W, const float* __restrict__ ws,
                                                          int N, int K, const int8_t* __restrict__ xq,
                                                          const float* __restrict__ xs, int T,
                                                          const float* __restrict__ bias, void* __restrict__ y,
                                                          int tn, int tt) {
  constexpr int NW = WN * WT, RN = BN / WN / 16, RT = BT / WT / 16;
  constexpr int LW = BN * kBK / 1024 / NW, LX = BT * kBK / 1024 / NW;  // 1 KB loads per wave and step
  static_assert(LW * NW * 1024 == BN * kBK && LX * NW * 1024 == BT * kBK, "tile");
  __shared__ __attribute__((aligned(16))) int8_t sw[2][BN * kBK];
  __shared__ __attribute__((aligned(16))) int8_t sx[2][BT * kBK];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // workgroups go round the 8 dies: give each die a run of neighbouring tiles
  const int total = tn * tt, per = (total + 7) >> 3;
  const int id = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
  if (id >= total || (int)(blockIdx.x >> 3) >= per) return;
  constexpr int kGroup = 4;
  const int band = id / (kGroup * tn), in = id % (kGroup * tn), rows = min(kGroup, tt - band * kGroup);
  const int t0 = (band * kGroup + in % rows) * BT, n0 = (in / rows) * BN;

  const int lr = lane >> 3, lc = (lane & 7) ^ lr;  // row and chunk of a load's 8 rows
  const int8_t* wsrc[LW];
  const int8_t* xsrc[LX];
#pragma unroll
  for (int i = 0; i < LW; ++i) wsrc[i] = W + (int64_t)min(n0 + (wave * LW + i) * 8 + lr, N - 1) * K + 16 * lc;
#pragma unroll
  for (int i = 0; i < LX; ++i) xsrc[i] = xq + (int64_t)min(t0 + (wave * LX + i) * 8 + lr, T - 1) * K + 16 * lc;
  auto load = [&](int buf, int k) {
#pragma unroll
    for (int i = 0; i < LW; ++i)
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(wsrc[i] + k),
                                       (__attribute__((address_space(3))) void*)(&sw[buf][(wave * LW + i) * 1024]), 16,
                                       0, 0);
#pragma unroll
    for (int i = 0; i < LX; ++i)
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(xsrc[i] + k),
                                       (__attribute__((address_space(3))) void*)(&sx[buf][(wave * LX + i) * 1024]), 16,
                                       0, 0);
  };
  const int wn = wave % WN, wt = wave / WN, r = lane & 15, g = lane >> 4;
  i32x4 acc[RN][RT];
#pragma unroll
  for (int i = 0; i < RN; ++i)
#pragma unroll
    for (int j = 0; j < RT; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  load(0, 0);
  const int steps = K / kBK;
  for (int s = 0; s < steps; ++s) {
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): this step's tile has landed
    __syncthreads();
    if (s + 1 < steps) load((s + 1) & 1, (s + 1) * kBK);
    const int8_t* bw = &sw[s & 1][(wn * RN * 16 + r) * kBK];
    const int8_t* bx = &sx[s & 1][(wt * RT * 16 + r) * kBK];
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
    __syncthreads();
  }
#pragma unroll
  for (int j = 0; j < RT; ++j) {
    const int tok = t0 + (wt * RT + j) * 16 + r;
    if (tok >= T) continue;
    const float sc = xs[tok];
#pragma unroll
    for (int i = 0; i < RN; ++i) {
      const int n = n0 + (wn * RN + i) * 16 + 4 * g;
      if (n < N) put4<YT>(y, tok, N, n, acc[i][j], sc, ws, bias);
    }
  }
}

template <int YT>
static hipError_t matmul(const int8_t* W, const float* ws, int N, int K, const int8_t* xq, const float* xs, int T,
                         const float* bias, void* y, hipStream_t st) {
  if (T <= 64) {
    const int nw = K <= 1024 ? 4 : K <= 4096 ? 8 : 16;
    const dim3 grid((N + 15) / 16), block(64 * nw);
#define MD_FEW(NT_)                                                                                                  \
  hipLaunchKernelGGL((k_i8_few<YT, NT_>), grid, block, (size_t)nw * NT_ * 1024, st, W, ws, N, K, xq, xs, T, bias, y)
    if (T <= 16) MD_FEW(1);
    else if (T <= 32) MD_FEW(2);
    else MD_FEW(4);
#undef MD_FEW
    return hipGetLastError();
  }
  auto tiles = [&](int b) { return (int64_t)((N + b - 1) / b) * ((T + b - 1) / b); };
#define MD_TILE(B_, WN_, WT_)                                                                                       \
  do {                                                                                                              \
    const int tn = (N + B_ - 1) / B_, tt = (T + B_ - 1) / B_;                                                       \
    hipLaunchKernelGGL((k_i8_tile<YT, B_, B_, WN_, WT_>), dim3((unsigned)((((int64_t)tn * tt + 7) >> 3) << 3)),     \
                       dim3(64 * WN_ * WT_), 0, st, W, ws, N, K, xq, xs, T, bias, y, tn, tt);                       \
  } while (0)
  if (tiles(256) >= 256) MD_TILE(256, 4, 2);
  else if (tiles(128) >= 128) MD_TILE(128, 2, 2);
  else MD_TILE(64, 2, 2);
#undef MD_TILE
  return hipGetLastError();
}

hipError_t launch_i8_matmul(const int8_t* W, const float* ws, int N, int K, const int8_t* xq, const float* xs, int T,
                            const float* bias, void* y, int yt, hipStream_t st) {
  return yt == XF32 ? matmul<XF32>(W, ws, N, K, xq, xs, T, bias, y, st)
                    : matmul<XBF16>(W, ws, N, K, xq, xs, T, bias, y, st);
}

}  // namespace md

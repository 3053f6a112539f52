// kv.hip -- a paged cache of keys and values in 8-bit integers, one scale for
// each page and head: the append into it, its dequantized read and page copies.
//
// Layout (page: tokens per page, a multiple of 64):
//   k       [n_pages][Hkv][page][D]   a token's D codes together
//   v       [n_pages][Hkv][D][page]   a channel's tokens together
//   scales  [n_pages][Hkv]            value = scale * code
// The values are kept transposed because the matrix cores contract over a
// lane's 16 consecutive bytes: keys over channels, values over tokens.
#include <hip/hip_runtime.h>

#include "common.hpp"
#include "i8.hpp"
#include "kernels.hpp"
#include "kv.hpp"
#include "rows.hpp"

namespace md {

// ---- append --------------------------------------------------------------

// rint(q / 2^up), ties to even, for |q| <= 128.
MD_DEV int halved(int q, int up) {
  if (up == 0) return q;
  if (up > 8) return 0;
  return (int)rintf((float)q * __int_as_float((127 - up) << 23));
}

MD_DEV uint32_t halved4(uint32_t w, int up) {
  uint32_t o = 0;
#pragma unroll
  for (int m = 0; m < 4; ++m) o |= (uint32_t)(halved((int8_t)(w >> (8 * m)), up) & 255) << (8 * m);
  return o;
}

// One workgroup per (page that new tokens reach, head, sequence, keys or
// values).  The page's scale: a page whose first token is new takes
// max |new| / 127; one that holds tokens keeps its scale unless max |new| / 127
// is above it, then the scale doubles until it is not, and the held codes are
// halved as often -- by powers of two, so that all raises together cost a held
// code at most one step of the last scale (1/2 + 1/4 + ...).  Only this
// workgroup touches the page's head, so the update needs no atomics.
//
// Bound by the read of the new rows and the write of their codes.  The rows
// stay in registers between the maximum and the codes (64 values a thread at
// most), so they are read once; the values' codes change from token-major to
// channel-major in LDS (20000 bf16 tokens of 8 heads of 128 channels in 2
// sequences: 60 us for 123 MB; read twice and stored byte by byte 90).  A token
// or a few a page: bytes stored as they come (64 sequences, one token each:
// 5.0 us, which is the launch; the other form 6.4).
template <int XT, int NV>  // NV: vectors of 8 values a thread
__global__ __launch_bounds__(1024) void k_kv_append(KvCache c, KvBatch b, const void* __restrict__ kx, int64_t k_stride,
                                                    const void* __restrict__ vx, int64_t v_stride) {
  extern __shared__ __attribute__((aligned(16))) uint32_t s_codes[];  // values: [new token of the page][D] bytes
  __shared__ uint32_t red[16];
  const int h = blockIdx.y % c.Hkv, which = blockIdx.y / c.Hkv, tid = threadIdx.x, D = c.D, P = c.page;
  const int nt = blockDim.x;
  const Seq q = seq_of(b, blockIdx.z, P);
  const int first = max(q.len - q.nq, 0);  // new tokens: positions first .. len - 1
  const int p = first / P + (int)blockIdx.x;
  if (q.bad || q.nq == 0 || (int64_t)p * P >= q.len) return;
  const int id = q.table[p];
  if ((unsigned)id >= (unsigned)c.n_pages) return;
  const int lo = max(first, p * P) - p * P, hi = min(q.len, (p + 1) * P) - p * P;
  const void* x = which ? vx : kx;
  const int64_t stride = which ? v_stride : k_stride;
  // the row of the page's token t is q.row0 + p * P + t - (len - nq)
  const int64_t xrow = (int64_t)q.row0 + (int64_t)p * P - (q.len - q.nq);
  const int n = (hi - lo) * (D / 8), dshift = 31 - __clz(D / 8);  // vectors; at most NV * nt (the launch)
  float v[NV][8];
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < NV; ++e) {
    const int i = tid + e * nt;
    if (i < n) {
      load8<XT>(x, (xrow + lo + (i >> dshift)) * stride + (int64_t)h * D + 8 * (i & (D / 8 - 1)), v[e]);
    } else {
#pragma unroll
      for (int m = 0; m < 8; ++m) v[e][m] = 0.0f;
    }
  }
  float* sp = (which ? c.v_scale : c.k_scale) + (int64_t)id * c.Hkv + h;
  const float was = lo > 0 ? *sp : 0.0f;
#pragma unroll
  for (int e = 0; e < NV; ++e)
#pragma unroll
    for (int m = 0; m < 8; ++m) top = max(top, __float_as_uint(v[e][m]) & 0x7FFFFFFFu);
  top = wave_max_u32(top);
  if ((tid & 63) == 0) red[tid >> 6] = top;
  __syncthreads();
  for (int w = 0; w < nt >> 6; ++w) top = max(top, red[w]);
  // a page that a non-finite value reaches has the scale NaN from then on
  const bool bad = top >= 0x7F800000u || !(was < INFINITY);
  const float need = __uint_as_float(top) / 127.0f;
  float now = need;
  int up = 0;
  if (was > 0.0f) {
    now = was;
    if (need > was) {
      int e0, e1;
      const float f0 = frexpf(was, &e0), f1 = frexpf(need, &e1);
      up = e1 - e0 + (f1 > f0);
      now = ldexpf(was, up);
    }
  }
  if (bad) now = __uint_as_float(0x7FC00000u);
  if (tid == 0) *sp = now;
  const Step step = step_of(now, __uint_as_float(top));
  int8_t* codes = (which ? c.v : c.k) + ((int64_t)id * c.Hkv + h) * (int64_t)P * D;
  if (which == 0 && up > 0) {  // the held tokens 0 .. lo - 1
    for (int i = tid; i < lo * D / 4; i += nt) {
      uint32_t* w = reinterpret_cast<uint32_t*>(codes) + i;
      *w = halved4(*w, up);
    }
  }
  if (NV == 1 && which == 1 && up > 0) {
    for (int i = tid; i < D * ((lo + 3) / 4); i += nt) {
      const int t = 4 * (i >> (dshift + 3));
      uint32_t* w = reinterpret_cast<uint32_t*>(codes + (i & (D - 1)) * P + t);
      const uint32_t old = *w, mine = t + 4 <= lo ? ~0u : (1u << (8 * (lo - t))) - 1;  // the slots from lo on stay
      *w = (halved4(old, up) & mine) | (old & ~mine);
    }
    __syncthreads();
  }
#pragma unroll
  for (int e = 0; e < NV; ++e) {
    const int i = tid + e * nt;
    if (i >= n) break;
    const uint2 w = codes8(v[e], step);
    if (which == 0) {
      *reinterpret_cast<uint2*>(codes + lo * D + 8 * i) = w;
    } else if (NV == 1) {  // a token or a few: byte by byte
      int8_t* to = codes + 8 * (i & (D / 8 - 1)) * P + lo + (i >> dshift);
#pragma unroll
      for (int m = 0; m < 8; ++m) to[m * P] = (int8_t)((m < 4 ? w.x : w.y) >> (8 * (m & 3)));
    } else {
      *reinterpret_cast<uint2*>(s_codes + 2 * i) = w;
    }
  }
  if (NV == 1) return;
  if (which == 0) return;
  __syncthreads();
  // values: a thread makes 16 tokens of four channels from sixteen words of LDS
  const int c0 = (up > 0 ? 0 : lo) / 16, c1 = (hi + 15) / 16;
  const int vshift = 31 - __clz(D / 4);
  for (int i = tid; i < (c1 - c0) * (D / 4); i += nt) {
    const int d = 4 * (i & (D / 4 - 1)), t0 = 16 * (c0 + (i >> vshift));
    uint32_t o[4][4];  // [channel][four tokens]
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t w[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int t = t0 + 4 * k + m;
        w[m] = t >= lo && t < hi ? s_codes[((t - lo) * D + d) >> 2] : 0u;
      }
      const uint32_t ab = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u), cd = __builtin_amdgcn_perm(w[3], w[2], 0x05010400u);
      const uint32_t ef = __builtin_amdgcn_perm(w[1], w[0], 0x07030602u), gh = __builtin_amdgcn_perm(w[3], w[2], 0x07030602u);
      o[0][k] = __builtin_amdgcn_perm(cd, ab, 0x05040100u);
      o[1][k] = __builtin_amdgcn_perm(cd, ab, 0x07060302u);
      o[2][k] = __builtin_amdgcn_perm(gh, ef, 0x05040100u);
      o[3][k] = __builtin_amdgcn_perm(gh, ef, 0x07060302u);
    }
    u32x4 held[4];
    const bool edge = t0 < lo || t0 + 16 > hi;  // held tokens before, slots that no token has reached behind
    if (edge) {
#pragma unroll
      for (int e = 0; e < 4; ++e) held[e] = *reinterpret_cast<const u32x4*>(codes + (d + e) * P + t0);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      u32x4 w{o[e][0], o[e][1], o[e][2], o[e][3]};
      if (edge) {
#pragma unroll
        for (int m = 0; m < 16; ++m) {
          const int t = t0 + m;
          if (t >= lo && t < hi) continue;
          int code = (int8_t)(held[e][m >> 2] >> (8 * (m & 3)));
          if (t < lo) code = halved(code, up);
          w[m >> 2] = (w[m >> 2] & ~(255u << (8 * (m & 3)))) | (uint32_t)(code & 255) << (8 * (m & 3));
        }
      }
      *reinterpret_cast<u32x4*>(codes + (d + e) * P + t0) = w;
    }
  }
}

hipError_t launch_kv_append(const KvCache& c, const KvBatch& b, const void* k, int64_t k_stride, const void* v,
                            int64_t v_stride, int xt, hipStream_t st) {
  const dim3 grid((b.max_q + c.page - 2) / c.page + 1, 2 * c.Hkv, b.S);
  const int tokens = b.max_q < c.page ? b.max_q : c.page;  // of a page, at most
  const int vectors = tokens * c.D / 8;
  // a token or a few: one vector a thread; pages: eight
  const int nv = vectors <= 256 ? 1 : 8, nt = vectors <= 128 * nv ? 128 : (vectors / nv + 63) / 64 * 64;
  const size_t lds = nv == 1 ? 0 : (size_t)tokens * c.D;
#define MD_APP(X_, N_) \
  hipLaunchKernelGGL((k_kv_append<X_, N_>), grid, dim3(nt), lds, st, c, b, k, k_stride, v, v_stride)
  if (xt == XF32) {
    if (nv == 1) MD_APP(XF32, 1);
    else MD_APP(XF32, 8);
  } else {
    if (nv == 1) MD_APP(XBF16, 1);
    else MD_APP(XBF16, 8);
  }
#undef MD_APP
  return hipGetLastError();
}

// ---- read ----------------------------------------------------------------

// Pages as values, both as [n][Hkv][page][D]; a page number outside the cache
// gives NaN.  One workgroup per (page, head, keys or values).
template <int YT>
MD_DEV void store_val(void* y, int64_t i, float f) {
  if constexpr (YT == XF32) static_cast<float*>(y)[i] = f;
  else static_cast<uint16_t*>(y)[i] = to_bf16(f);
}

template <int YT>
__global__ __launch_bounds__(256) void k_kv_read(KvCache c, const int* __restrict__ pages, void* __restrict__ ky,
                                                 void* __restrict__ vy) {
  const int h = blockIdx.y, which = blockIdx.z, tid = threadIdx.x, D = c.D, P = c.page;
  const int id = pages[blockIdx.x];
  const int64_t out = ((int64_t)blockIdx.x * c.Hkv + h) * (int64_t)P * D;
  void* y = which ? vy : ky;
  if ((unsigned)id >= (unsigned)c.n_pages) {
    for (int i = tid; i < P * D; i += 256) store_val<YT>(y, out + i, __uint_as_float(0x7FC00000u));
    return;
  }
  const int64_t at = (int64_t)id * c.Hkv + h;
  const int8_t* codes = (which ? c.v : c.k) + at * P * D;
  const float s = (which ? c.v_scale : c.k_scale)[at];
  if (which == 0) {
    for (int i = tid; i < P * D / 4; i += 256) {
      const uint32_t w = reinterpret_cast<const uint32_t*>(codes)[i];
      float f[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) f[m] = s * (float)(int8_t)(w >> (8 * m));
      if (YT == XF32) reinterpret_cast<float4*>(static_cast<float*>(y) + out)[i] = make_float4(f[0], f[1], f[2], f[3]);
      else
        reinterpret_cast<uint2*>(static_cast<uint16_t*>(y) + out)[i] =
            make_uint2(to_bf16(f[0]) | (uint32_t)to_bf16(f[1]) << 16, to_bf16(f[2]) | (uint32_t)to_bf16(f[3]) << 16);
    }
    return;
  }
  const int vshift = 31 - __clz(D);
  for (int i = tid; i < P / 16 * D; i += 256) {
    const int d = i & (D - 1), t0 = 16 * (i >> vshift);
    const u32x4 w = *reinterpret_cast<const u32x4*>(codes + d * P + t0);
#pragma unroll
    for (int m = 0; m < 16; ++m)
      store_val<YT>(y, out + (int64_t)(t0 + m) * D + d, s * (float)(int8_t)(w[m >> 2] >> (8 * (m & 3))));
  }
}

hipError_t launch_kv_read(const KvCache& c, const int* pages, int n, void* k, void* v, int yt, hipStream_t st) {
  const dim3 grid(n, c.Hkv, 2);
  if (yt == XF32) hipLaunchKernelGGL((k_kv_read<XF32>), grid, dim3(256), 0, st, c, pages, k, v);
  else hipLaunchKernelGGL((k_kv_read<XBF16>), grid, dim3(256), 0, st, c, pages, k, v);
  return hipGetLastError();
}

// ---- page copies ---------------------------------------------------------

// The pairs travel in the kernel's arguments: nothing to allocate, keep or
// upload, so a call can be captured.  One workgroup per 16 KB of a page's
// codes; the caller has checked that no pair reads or writes what another one
// writes.  Bound by memory: 2001 pages of 128 KB in 113 us (4.6 TB/s read and
// written together, a large copy reaches 4.9) with the nontemporal hint on both
// sides, 118 on loads alone, 131 without; 32 KB per workgroup 160.
constexpr int kCopyChunk = 16384;
__global__ __launch_bounds__(256) void k_kv_copy(KvCache c, PagePairs pairs) {
  const int src = pairs.src[blockIdx.x], dst = pairs.dst[blockIdx.x], tid = threadIdx.x;
  const int64_t bytes = (int64_t)c.Hkv * c.page * c.D;
  const int8_t* base = blockIdx.z ? c.v : c.k;
  const u32x4* from = reinterpret_cast<const u32x4*>(base + src * bytes);
  u32x4* to = reinterpret_cast<u32x4*>(const_cast<int8_t*>(base) + dst * bytes);
  const int64_t i0 = (int64_t)blockIdx.y * (kCopyChunk / 16) + tid;
  u32x4 w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i0 + 256 * i < bytes / 16) w[i] = __builtin_nontemporal_load(from + i0 + 256 * i);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i0 + 256 * i < bytes / 16) __builtin_nontemporal_store(w[i], to + i0 + 256 * i);
  if (blockIdx.y == 0) {
    float* s = blockIdx.z ? c.v_scale : c.k_scale;
    for (int h = tid; h < c.Hkv; h += 256) s[(int64_t)dst * c.Hkv + h] = s[(int64_t)src * c.Hkv + h];
  }
}

hipError_t launch_kv_copy(const KvCache& c, const int* src, const int* dst, int n, hipStream_t st) {
  const int chunks = (int)(((int64_t)c.Hkv * c.page * c.D + kCopyChunk - 1) / kCopyChunk);
  for (int at = 0; at < n; at += kPairsPerLaunch) {
    PagePairs p;
    const int m = n - at < kPairsPerLaunch ? n - at : kPairsPerLaunch;
    for (int i = 0; i < m; ++i) {
      p.src[i] = src[at + i];
      p.dst[i] = dst[at + i];
    }
    hipLaunchKernelGGL(k_kv_copy, dim3(m, chunks, 2), dim3(256), 0, st, c, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace md

// kv_abi.cpp -- the C entry points of the 8-bit products and of the paged
// cache: host-side validation (every check runs before anything is enqueued),
// the page bookkeeping, and the launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <functional>

#include "host.hpp"
#include "kernels.hpp"
#include "moe_decode.h"

using md::align256;
using md::aligned16;
using md::aligned4;
using md::fail;
using md::hip_fail;
using md::ok;

namespace {

constexpr int kMaxTokens = 1 << 20;
constexpr int kMaxSeqs = 65535;
constexpr int kMaxHeads = 1024;
constexpr int kMaxKvHeads = 256;
constexpr int kMaxPositions = 1 << 30;  // tiles' borders and windows before position 0 stay in 32 bits
constexpr int kMaxWords = kMaxTokens / 64;
constexpr int kMaxTree = 1024;          // tokens of a run whose masks md_kv_tree makes
constexpr int kMaxGrid = (1 << 24) - 1;  // workgroups of 256 along x: below 2^32 threads

bool valid_xtype(int32_t t) { return t == MD_X_F32 || t == MD_X_BF16; }
int elem(int32_t t) { return t == MD_X_F32 ? 4 : 2; }

md_status check_tokens(int32_t T) {
  if (T < 0) return fail(MD_ERR_SHAPE, "T = %d must not be negative", T);
  if (T > kMaxTokens) return fail(MD_ERR_UNSUPPORTED, "T = %d > %d", T, kMaxTokens);
  return MD_OK;
}

md_status check_width(const char* what, int32_t K) {
  if (K <= 0) return fail(MD_ERR_SHAPE, "%s = %d must be positive", what, K);
  if (K % 256 || K > 16384)
    return fail(MD_ERR_UNSUPPORTED, "%s = %d: supported widths are multiples of 256 up to 16384", what, K);
  return MD_OK;
}

md_status check_i8(const md_qmatrix* W, int32_t T) {
  md_status s = md::check_qmatrix("i8 product", W);
  if (s != MD_OK) return s;
  if (W->type != MD_I8_ROW) return fail(MD_ERR_UNSUPPORTED, "i8 product: type %d, only int8 rows (MD_I8_ROW)", W->type);
  return check_tokens(T);
}

md_status check_device(const char* what, const void* p) {
  if (!p) return fail(MD_ERR_INVALID_ARG, "%s: null pointer", what);
  if (!aligned16(p)) return fail(MD_ERR_ALIGNMENT, "%s: not 16-byte aligned", what);
  return MD_OK;
}

// md_i8_linear's workspace: codes, scales, shares of the sum
size_t codes_bytes(int32_t T, int32_t K) { return align256((size_t)T * K); }
size_t scales_bytes(int32_t T) { return align256(sizeof(float) * (size_t)T); }
size_t shares_bytes(const md_qmatrix* W, int32_t T) {
  const int s = md::i8_shares(W->rows, W->cols, T);
  return s > 1 ? align256(sizeof(int) * (size_t)s * T * ((W->rows + 3) & ~3)) : 0;
}

md_status check_cache(const md_kv_cache* c) {
  if (!c) return fail(MD_ERR_INVALID_ARG, "null cache descriptor");
  if (c->n_pages <= 0 || c->kv_heads <= 0)
    return fail(MD_ERR_SHAPE, "cache: %d pages of %d heads", c->n_pages, c->kv_heads);
  if (c->kv_heads > kMaxKvHeads) return fail(MD_ERR_UNSUPPORTED, "cache: %d key heads > %d", c->kv_heads, kMaxKvHeads);
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return fail(MD_ERR_UNSUPPORTED, "cache: head width %d is none of 64, 128, 256", c->head_dim);
  if (c->page != 64 && c->page != 128 && c->page != 256)
    return fail(MD_ERR_UNSUPPORTED, "cache: %d tokens per page is none of 64, 128, 256", c->page);
  md_status s;
  if ((s = check_device("cache k", c->k)) != MD_OK) return s;
  if ((s = check_device("cache v", c->v)) != MD_OK) return s;
  if ((s = check_device("cache k_scale", c->k_scale)) != MD_OK) return s;
  return check_device("cache v_scale", c->v_scale);
}

// Everything but the pointers, which a batch without rows need not have.
md_status check_batch(const md_kv_cache* c, const md_kv_batch* b) {
  if (!b) return fail(MD_ERR_INVALID_ARG, "null batch descriptor");
  if (b->n_seqs <= 0 || b->rows < 0 || b->max_q <= 0 || b->max_kv <= 0 || b->table_stride <= 0)
    return fail(MD_ERR_SHAPE, "batch: n_seqs %d rows %d max_q %d max_kv %d table_stride %d", b->n_seqs, b->rows,
                b->max_q, b->max_kv, b->table_stride);
  if (b->n_seqs > kMaxSeqs || b->rows > kMaxTokens || b->max_q > kMaxTokens)
    return fail(MD_ERR_UNSUPPORTED, "batch: n_seqs %d (at most %d), rows %d, max_q %d (at most %d)", b->n_seqs, kMaxSeqs,
                b->rows, b->max_q, kMaxTokens);
  if (b->max_kv > kMaxPositions)
    return fail(MD_ERR_UNSUPPORTED, "batch: max_kv %d > %d", b->max_kv, kMaxPositions);
  if ((int64_t)b->table_stride * c->page < b->max_kv)
    return fail(MD_ERR_SHAPE, "batch: %d pages of %d tokens hold no %d tokens", b->table_stride, c->page, b->max_kv);
  return MD_OK;
}

md_status check_batch_ptrs(const md_kv_batch* b) {
  if (!b->q_start || !b->kv_len || !b->table) return fail(MD_ERR_INVALID_ARG, "batch: null pointer");
  if (!aligned4(b->q_start) || !aligned4(b->kv_len) || !aligned4(b->table))
    return fail(MD_ERR_ALIGNMENT, "batch: an array is not 4-byte aligned");
  return MD_OK;
}

md_status check_rows(const char* what, const void* p, int64_t stride, int64_t width, int32_t type) {
  md_status s = check_device(what, p);
  if (s != MD_OK) return s;
  if (stride < width) return fail(MD_ERR_SHAPE, "%s: row stride %lld < %lld", what, (long long)stride, (long long)width);
  if (stride * elem(type) % 16)
    return fail(MD_ERR_ALIGNMENT, "%s: a row stride of %lld values is no multiple of 16 bytes", what, (long long)stride);
  return MD_OK;
}

md::KvCache dev(const md_kv_cache* c) {
  return md::KvCache{c->n_pages, c->page, c->kv_heads, c->head_dim, c->k, c->v, c->k_scale, c->v_scale};
}
md::KvBatch dev(const md_kv_batch* b) {
  return md::KvBatch{b->n_seqs, b->rows, b->max_q, b->max_kv, b->table_stride, b->q_start, b->kv_len, b->table};
}

// Partial sums (one per row or column each) that the attention's workspace
// holds, after its notes on them: maxima and totals, then vectors.
size_t attn_slots(const md::KvPlan& p, const md_kv_batch* b, int32_t q_heads) {
  if (p.pieces) return (size_t)2 * p.pieces * 16;
  return p.splits > 1 ? (size_t)b->rows * q_heads * p.splits : 0;
}

size_t notes_bytes(const md::KvPlan& p) { return p.pieces * sizeof(int4) + p.notes * sizeof(int); }

// A window that reaches past every position is none.
int seen(const md_kv_batch* b, int32_t window) { return window >= b->max_kv ? 0 : window; }

// The attention's checks up to its pointers, and its launch geometry.
md_status attn_plan(const md_kv_cache* c, const md_kv_batch* b, int32_t q_heads, int32_t causal, int32_t window,
                    int32_t sinks, bool masked, int32_t ytype, md::KvPlan* plan, size_t* bytes) {
  md_status s;
  if ((s = check_cache(c)) != MD_OK || (s = check_batch(c, b)) != MD_OK) return s;
  if (q_heads <= 0 || q_heads % c->kv_heads)
    return fail(MD_ERR_SHAPE, "attention: %d query heads on %d key heads", q_heads, c->kv_heads);
  if (q_heads > kMaxHeads) return fail(MD_ERR_UNSUPPORTED, "attention: %d query heads > %d", q_heads, kMaxHeads);
  if (causal != 0 && causal != 1) return fail(MD_ERR_INVALID_ARG, "attention: causal = %d", causal);
  if (window < 0 || (window > 0 && !causal))
    return fail(MD_ERR_INVALID_ARG, "attention: window %d%s", window, causal ? "" : " without causal");
  if (!valid_xtype(ytype)) return fail(MD_ERR_INVALID_ARG, "unknown ytype %d", ytype);
  const int G = q_heads / c->kv_heads;
  *plan = md::kv_attn_plan(dev(c), dev(b), G, seen(b, window), sinks, causal, ytype, masked);
  const int64_t groups = ((int64_t)b->max_q * G + plan->tile - 1) / plan->tile * c->kv_heads * plan->splits;
  if (groups > kMaxGrid) return fail(MD_ERR_UNSUPPORTED, "attention: max_q %d on %d heads", b->max_q, q_heads);
  const size_t slots = attn_slots(*plan, b, q_heads);
  *bytes = slots ? align256(notes_bytes(*plan)) + align256(slots * 2 * sizeof(float)) +
                       align256(slots * c->head_dim * sizeof(float))
                 : 0;
  return MD_OK;
}

// What a mask's call reads: sinks count beside a window only.
int kept(const md_kv_batch* b, const md_kv_mask* m) {
  return seen(b, m->window) ? std::min(m->sinks, b->max_kv) : 0;
}
md_status masked_plan(const md_kv_cache* c, const md_kv_batch* b, int32_t q_heads, const md_kv_mask* m, int32_t ytype,
                      md::KvPlan* plan, size_t* bytes) {
  md_status s;
  if ((s = check_cache(c)) != MD_OK || (s = check_batch(c, b)) != MD_OK) return s;
  if (!m) return fail(MD_ERR_INVALID_ARG, "attention: null mask");
  if (m->sinks < 0) return fail(MD_ERR_INVALID_ARG, "attention: sinks %d", m->sinks);
  if (m->tree) {
    if (m->words > kMaxWords) return fail(MD_ERR_UNSUPPORTED, "attention: a tree of %d words > %d", m->words, kMaxWords);
    if (m->words < 1 || (int64_t)64 * m->words < b->max_q)
      return fail(MD_ERR_SHAPE, "attention: a tree of %d words for runs of %d", m->words, b->max_q);
    if (reinterpret_cast<uintptr_t>(m->tree) & 7u) return fail(MD_ERR_ALIGNMENT, "attention: the tree is not 8-byte aligned");
  }
  if (m->window < 0) return fail(MD_ERR_INVALID_ARG, "attention: window %d", m->window);
  const int sinks = kept(b, m);
  return attn_plan(c, b, q_heads, 1, m->window, sinks, m->tree || sinks, ytype, plan, bytes);
}

// ---- pages -----------------------------------------------------------------

int32_t pages_of(const md_kv_pages* p, int32_t len) { return (int32_t)(((int64_t)len + p->page - 1) / p->page); }

md_status check_pages(const md_kv_pages* p) {
  if (!p || !p->refs || !p->free_pages) return fail(MD_ERR_INVALID_ARG, "pages: null pointer");
  if (p->n_pages <= 0 || p->page <= 0) return fail(MD_ERR_SHAPE, "pages: %d pages of %d tokens", p->n_pages, p->page);
  if (p->n_free < 0 || p->n_free > p->n_pages) return fail(MD_ERR_INVALID_ARG, "pages: n_free %d", p->n_free);
  return MD_OK;
}

// The first n entries of a table: pages that are in use.
md_status check_table(const md_kv_pages* p, const int32_t* table, int32_t n) {
  if (n && !table) return fail(MD_ERR_INVALID_ARG, "pages: null table");
  for (int32_t i = 0; i < n; ++i) {
    if (table[i] < 0 || table[i] >= p->n_pages) return fail(MD_ERR_INVALID_ARG, "pages: entry %d is page %d of %d", i, table[i], p->n_pages);
    if (p->refs[table[i]] <= 0) return fail(MD_ERR_INVALID_ARG, "pages: entry %d is page %d, which is free", i, table[i]);
  }
  return MD_OK;
}

// The free pages are a heap with the lowest number on top.
int32_t take(md_kv_pages* p) {
  std::pop_heap(p->free_pages, p->free_pages + p->n_free, std::greater<int32_t>());
  const int32_t id = p->free_pages[--p->n_free];
  p->refs[id] = 1;
  return id;
}
void give(md_kv_pages* p, int32_t id) {
  p->free_pages[p->n_free++] = id;
  std::push_heap(p->free_pages, p->free_pages + p->n_free, std::greater<int32_t>());
}
void heap_from_refs(md_kv_pages* p) {
  p->n_free = 0;
  for (int32_t i = 0; i < p->n_pages; ++i)
    if (p->refs[i] == 0) p->free_pages[p->n_free++] = i;  // ascending: a heap already
}

}  // namespace

extern "C" {

md_status md_i8_quantize(const void* x, int32_t xtype, int32_t T, int32_t K, int8_t* codes, float* scales,
                         hipStream_t stream) {
  md_status s;
  if (!valid_xtype(xtype)) return fail(MD_ERR_INVALID_ARG, "unknown xtype %d", xtype);
  if ((s = check_tokens(T)) != MD_OK || (s = check_width("K", K)) != MD_OK) return s;
  if (T == 0) return ok();
  if ((s = check_device("x", x)) != MD_OK || (s = check_device("codes", codes)) != MD_OK ||
      (s = check_device("scales", scales)) != MD_OK)
    return s;
  const hipError_t e = md::launch_i8_quantize(x, xtype, T, K, codes, scales, stream);
  return e == hipSuccess ? ok() : hip_fail(e, "quantize launch");
}

md_status md_i8_matmul(const md_qmatrix* W, const int8_t* codes, const float* scales, int32_t T, const float* bias,
                       void* y, int32_t ytype, hipStream_t stream) {
  md_status s;
  if ((s = check_i8(W, T)) != MD_OK) return s;
  if (!valid_xtype(ytype)) return fail(MD_ERR_INVALID_ARG, "unknown ytype %d", ytype);
  if (T == 0) return ok();
  if ((s = check_device("codes", codes)) != MD_OK || (s = check_device("scales", scales)) != MD_OK ||
      (s = check_device("y", y)) != MD_OK || (bias && (s = check_device("bias", bias)) != MD_OK))
    return s;
  const hipError_t e = md::launch_i8_matmul(static_cast<const int8_t*>(W->q), W->row_scale, W->rows, W->cols, codes,
                                            scales, T, bias, y, ytype, nullptr, stream);
  return e == hipSuccess ? ok() : hip_fail(e, "i8 product launch");
}

md_status md_i8_linear_workspace_size(const md_qmatrix* W, int32_t T, size_t* bytes) {
  const md_status s = check_i8(W, T);
  if (s != MD_OK) return s;
  if (!bytes) return fail(MD_ERR_INVALID_ARG, "null size pointer");
  *bytes = T && !md::i8_own_codes(W->rows, W->cols, T) ? codes_bytes(T, W->cols) + scales_bytes(T) + shares_bytes(W, T) : 0;
  return ok();
}

md_status md_i8_linear(const md_qmatrix* W, const void* x, int32_t xtype, int32_t T, const float* bias, void* y,
                       int32_t ytype, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  size_t need = 0;
  md_status s = md_i8_linear_workspace_size(W, T, &need);
  if (s != MD_OK) return s;
  if (!valid_xtype(xtype) || !valid_xtype(ytype)) return fail(MD_ERR_INVALID_ARG, "unknown xtype %d or ytype %d", xtype, ytype);
  if (T == 0) return ok();
  if ((s = check_device("x", x)) != MD_OK || (s = check_device("y", y)) != MD_OK ||
      (bias && (s = check_device("bias", bias)) != MD_OK))
    return s;
  if (md::i8_own_codes(W->rows, W->cols, T)) {
    const hipError_t e = md::launch_i8_own(static_cast<const int8_t*>(W->q), W->row_scale, W->rows, W->cols, x, xtype, T,
                                           bias, y, ytype, stream);
    return e == hipSuccess ? ok() : hip_fail(e, "i8 linear launch");
  }
  if (!workspace || workspace_bytes < need)
    return fail(MD_ERR_WORKSPACE, "workspace: %zu bytes, %zu needed", workspace ? workspace_bytes : 0, need);
  if (!aligned16(workspace)) return fail(MD_ERR_ALIGNMENT, "workspace not 16-byte aligned");
  int8_t* codes = static_cast<int8_t*>(workspace);
  float* scales = reinterpret_cast<float*>(codes + codes_bytes(T, W->cols));
  hipError_t e = md::launch_i8_quantize(x, xtype, T, W->cols, codes, scales, stream);
  if (e != hipSuccess) return hip_fail(e, "quantize launch");
  int* part = shares_bytes(W, T) ? reinterpret_cast<int*>(reinterpret_cast<char*>(scales) + scales_bytes(T)) : nullptr;
  e = md::launch_i8_matmul(static_cast<const int8_t*>(W->q), W->row_scale, W->rows, W->cols, codes, scales, T, bias, y,
                           ytype, part, stream);
  return e == hipSuccess ? ok() : hip_fail(e, "i8 product launch");
}

md_status md_kv_append(const md_kv_cache* c, const md_kv_batch* b, const void* k, int64_t k_stride, const void* v,
                       int64_t v_stride, int32_t xtype, hipStream_t stream) {
  md_status s;
  if ((s = check_cache(c)) != MD_OK || (s = check_batch(c, b)) != MD_OK) return s;
  if (!valid_xtype(xtype)) return fail(MD_ERR_INVALID_ARG, "unknown xtype %d", xtype);
  if (b->rows == 0) return ok();
  const int64_t width = (int64_t)c->kv_heads * c->head_dim;
  if ((s = check_batch_ptrs(b)) != MD_OK || (s = check_rows("k", k, k_stride, width, xtype)) != MD_OK ||
      (s = check_rows("v", v, v_stride, width, xtype)) != MD_OK)
    return s;
  const hipError_t e = md::launch_kv_append(dev(c), dev(b), k, k_stride, v, v_stride, xtype, stream);
  return e == hipSuccess ? ok() : hip_fail(e, "append launch");
}

md_status md_kv_read_pages(const md_kv_cache* c, const int32_t* pages, int32_t n, void* k, void* v, int32_t ytype,
                           hipStream_t stream) {
  md_status s;
  if ((s = check_cache(c)) != MD_OK) return s;
  if (!valid_xtype(ytype)) return fail(MD_ERR_INVALID_ARG, "unknown ytype %d", ytype);
  if (n < 0) return fail(MD_ERR_SHAPE, "n = %d must not be negative", n);
  if (n > kMaxGrid) return fail(MD_ERR_UNSUPPORTED, "n = %d pages > %d", n, kMaxGrid);
  if (n == 0) return ok();
  if (!pages) return fail(MD_ERR_INVALID_ARG, "pages: null pointer");
  if (!aligned4(pages)) return fail(MD_ERR_ALIGNMENT, "pages: not 4-byte aligned");
  if ((s = check_device("k", k)) != MD_OK || (s = check_device("v", v)) != MD_OK) return s;
  const hipError_t e = md::launch_kv_read(dev(c), pages, n, k, v, ytype, stream);
  return e == hipSuccess ? ok() : hip_fail(e, "page read launch");
}

md_status md_kv_copy_pages(const md_kv_cache* c, const int32_t* src, const int32_t* dst, int32_t n,
                           hipStream_t stream) {
  const md_status s = check_cache(c);
  if (s != MD_OK) return s;
  if (n < 0) return fail(MD_ERR_SHAPE, "n = %d must not be negative", n);
  if (n == 0) return ok();
  if (!src || !dst) return fail(MD_ERR_INVALID_ARG, "page pairs: null pointer");
  for (int32_t i = 0; i < n; ++i)
    if (src[i] < 0 || src[i] >= c->n_pages || dst[i] < 0 || dst[i] >= c->n_pages)
      return fail(MD_ERR_INVALID_ARG, "page pair %d: %d -> %d of %d pages", i, src[i], dst[i], c->n_pages);
  // pairs run side by side: a page that is written appears once among all of them
  const size_t words = ((size_t)c->n_pages + 63) / 64;
  uint64_t* written = static_cast<uint64_t*>(std::calloc(words, sizeof(uint64_t)));
  if (!written) return fail(MD_ERR_UNSUPPORTED, "page pairs: no host memory for %d pages", c->n_pages);
  int32_t twice = -1;
  for (int32_t i = 0; i < n && twice < 0; ++i) {
    uint64_t& w = written[dst[i] >> 6];
    const uint64_t bit = uint64_t(1) << (dst[i] & 63);
    if (w & bit) twice = i;
    w |= bit;
  }
  for (int32_t i = 0; i < n && twice < 0; ++i)
    if (written[src[i] >> 6] >> (src[i] & 63) & 1) twice = i;
  std::free(written);
  if (twice >= 0)
    return fail(MD_ERR_INVALID_ARG, "page pair %d (%d -> %d): a page that is written appears in two places", twice,
                src[twice], dst[twice]);
  const hipError_t e = md::launch_kv_copy(dev(c), src, dst, n, stream);
  return e == hipSuccess ? ok() : hip_fail(e, "page copy launch");
}

md_status md_kv_attention_workspace_size(const md_kv_cache* c, const md_kv_batch* b, int32_t q_heads, int32_t causal,
                                         int32_t window, int32_t ytype, size_t* bytes) {
  md::KvPlan plan;
  size_t need = 0;
  const md_status s = attn_plan(c, b, q_heads, causal, window, 0, false, ytype, &plan, &need);
  if (s != MD_OK) return s;
  if (!bytes) return fail(MD_ERR_INVALID_ARG, "null size pointer");
  *bytes = need;
  return ok();
}

md_status md_kv_attention_masked_workspace_size(const md_kv_cache* c, const md_kv_batch* b, int32_t q_heads,
                                                const md_kv_mask* mask, int32_t ytype, size_t* bytes) {
  md::KvPlan plan;
  size_t need = 0;
  const md_status s = masked_plan(c, b, q_heads, mask, ytype, &plan, &need);
  if (s != MD_OK) return s;
  if (!bytes) return fail(MD_ERR_INVALID_ARG, "null size pointer");
  *bytes = need;
  return ok();
}

}  // extern "C"

// The launch of a planned call, its remaining checks in front.
static md_status attend(const md_kv_cache* c, const md_kv_batch* b, const md::KvPlan& plan, size_t need, const void* q,
                        int32_t xtype, int32_t q_heads, int64_t q_stride, float scale, int32_t causal, int32_t window,
                        const md_kv_mask* mask, void* out, int32_t ytype, int64_t out_stride, void* workspace,
                        size_t workspace_bytes, hipStream_t stream) {
  md_status s;
  if (!valid_xtype(xtype)) return fail(MD_ERR_INVALID_ARG, "unknown xtype %d", xtype);
  if (!std::isfinite(scale)) return fail(MD_ERR_INVALID_ARG, "attention: scale %g", scale);
  if (b->rows == 0) return ok();
  const int64_t width = (int64_t)q_heads * c->head_dim;
  if ((s = check_batch_ptrs(b)) != MD_OK || (s = check_rows("q", q, q_stride, width, xtype)) != MD_OK ||
      (s = check_rows("out", out, out_stride, width, ytype)) != MD_OK)
    return s;
  if (q == out) return fail(MD_ERR_INVALID_ARG, "attention: out is q");
  if (need) {
    if (!workspace || workspace_bytes < need)
      return fail(MD_ERR_WORKSPACE, "workspace: %zu bytes, %zu needed", workspace ? workspace_bytes : 0, need);
    if (!aligned16(workspace)) return fail(MD_ERR_ALIGNMENT, "workspace not 16-byte aligned");
  }
  md::KvAttn a{};
  a.c = dev(c);
  a.b = dev(b);
  a.q = q;
  a.out = out;
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.xt = xtype;
  a.yt = ytype;
  a.G = q_heads / c->kv_heads;
  a.causal = causal;
  a.window = seen(b, window);
  a.pshift = c->page == 64 ? 6 : c->page == 128 ? 7 : 8;
  a.scale = scale;
  if (mask) {
    a.sinks = kept(b, mask);
    a.tree = mask->tree;
    a.words = mask->words;
    a.masked = a.tree || a.sinks;  // a window alone is the plain form's
  }
  a.tile = plan.tile;
  a.splits = plan.splits;
  a.chunk = plan.chunk;
  a.pieces = plan.pieces;
  if (need) {
    char* at = static_cast<char*>(workspace);
    a.shares = reinterpret_cast<int4*>(at);
    at += align256(notes_bytes(plan));
    a.part_m = reinterpret_cast<float*>(at);
    at += align256(attn_slots(plan, b, q_heads) * 2 * sizeof(float));
    a.part = reinterpret_cast<float*>(at);
  }
  const hipError_t e = md::launch_kv_attn(a, c->head_dim, ytype, stream);
  return e == hipSuccess ? ok() : hip_fail(e, "attention launch");
}

extern "C" {

md_status md_kv_attention_masked(const md_kv_cache* c, const md_kv_batch* b, const void* q, int32_t xtype,
                                 int32_t q_heads, int64_t q_stride, float scale, const md_kv_mask* mask, void* out,
                                 int32_t ytype, int64_t out_stride, void* workspace, size_t workspace_bytes,
                                 hipStream_t stream) {
  md::KvPlan plan;
  size_t need = 0;
  const md_status s = masked_plan(c, b, q_heads, mask, ytype, &plan, &need);
  if (s != MD_OK) return s;
  return attend(c, b, plan, need, q, xtype, q_heads, q_stride, scale, 1, mask->window, mask, out, ytype, out_stride,
                workspace, workspace_bytes, stream);
}

md_status md_kv_tree(const md_kv_batch* b, const int32_t* parents, uint64_t* masks, int32_t words, int32_t* positions,
                     hipStream_t stream) {
  return md_kv_tree_window(b, parents, 0, 0, masks, words, positions, stream);
}

md_status md_kv_tree_window(const md_kv_batch* b, const int32_t* parents, int32_t window, int32_t sinks, uint64_t* masks,
                            int32_t words, int32_t* positions, hipStream_t stream) {
  if (!b) return fail(MD_ERR_INVALID_ARG, "null batch descriptor");
  if (b->n_seqs <= 0 || b->rows < 0 || b->max_q <= 0)
    return fail(MD_ERR_SHAPE, "batch: n_seqs %d rows %d max_q %d", b->n_seqs, b->rows, b->max_q);
  if (b->n_seqs > kMaxSeqs || b->rows > kMaxTokens || b->max_q > kMaxTree)
    return fail(MD_ERR_UNSUPPORTED, "tree: n_seqs %d (at most %d), rows %d (%d), max_q %d (%d)", b->n_seqs, kMaxSeqs,
                b->rows, kMaxTokens, b->max_q, kMaxTree);
  if (words > kMaxWords) return fail(MD_ERR_UNSUPPORTED, "tree: %d words > %d", words, kMaxWords);
  if (words < 1 || 64 * words < b->max_q) return fail(MD_ERR_SHAPE, "tree: %d words for runs of %d", words, b->max_q);
  if (window < 0 || sinks < 0) return fail(MD_ERR_INVALID_ARG, "tree: window %d, sinks %d", window, sinks);
  if (b->rows == 0) return ok();
  if (!b->q_start || !b->kv_len || !parents || !masks) return fail(MD_ERR_INVALID_ARG, "tree: null pointer");
  if (!aligned4(b->q_start) || !aligned4(b->kv_len) || !aligned4(parents) || (positions && !aligned4(positions)) ||
      (reinterpret_cast<uintptr_t>(masks) & 7u))
    return fail(MD_ERR_ALIGNMENT, "tree: masks not 8-byte aligned, or another array not 4-byte");
  const hipError_t e = md::launch_kv_tree(dev(b), parents, window, sinks, masks, words, positions, stream);
  return e == hipSuccess ? ok() : hip_fail(e, "tree launch");
}

md_status md_kv_attention(const md_kv_cache* c, const md_kv_batch* b, const void* q, int32_t xtype, int32_t q_heads,
                          int64_t q_stride, float scale, int32_t causal, int32_t window, void* out, int32_t ytype,
                          int64_t out_stride, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  md::KvPlan plan;
  size_t need = 0;
  const md_status s = attn_plan(c, b, q_heads, causal, window, 0, false, ytype, &plan, &need);
  if (s != MD_OK) return s;
  return attend(c, b, plan, need, q, xtype, q_heads, q_stride, scale, causal, window, nullptr, out, ytype, out_stride,
                workspace, workspace_bytes, stream);
}

md_status md_kv_pages_reset(md_kv_pages* p) {
  const md_status s = check_pages(p);
  if (s != MD_OK) return s;
  std::fill(p->refs, p->refs + p->n_pages, 0);
  heap_from_refs(p);
  return ok();
}

md_status md_kv_pages_extend(md_kv_pages* p, int32_t* table, int32_t capacity, int32_t len, int32_t new_len,
                             int32_t* copy_src, int32_t* copy_dst, int32_t* n_copy) {
  md_status s = check_pages(p);
  if (s != MD_OK) return s;
  if (!copy_src || !copy_dst || !n_copy) return fail(MD_ERR_INVALID_ARG, "pages: null pointer");
  if (len < 0 || new_len < len) return fail(MD_ERR_SHAPE, "pages: from %d to %d tokens", len, new_len);
  const int32_t have = pages_of(p, len), want = pages_of(p, new_len);
  if (capacity < want) return fail(MD_ERR_SHAPE, "pages: a table of %d entries for %d pages", capacity, want);
  if (want && !table) return fail(MD_ERR_INVALID_ARG, "pages: null table");
  if ((s = check_table(p, table, have)) != MD_OK) return s;
  // the page that len ends in is written next: a shared one is copied first
  const bool copy = new_len > len && len % p->page && p->refs[table[have - 1]] > 1;
  if (want - have + (copy ? 1 : 0) > p->n_free)
    return fail(MD_ERR_UNSUPPORTED, "pages: %d needed, %d free", want - have + (copy ? 1 : 0), p->n_free);
  *n_copy = copy ? 1 : 0;
  if (copy) {
    const int32_t old = table[have - 1];
    copy_src[0] = old;
    copy_dst[0] = table[have - 1] = take(p);
    --p->refs[old];
  }
  for (int32_t i = have; i < want; ++i) table[i] = take(p);
  return ok();
}

md_status md_kv_pages_fork(md_kv_pages* p, const int32_t* table, int32_t len, int32_t* new_table, int32_t capacity) {
  md_status s = check_pages(p);
  if (s != MD_OK) return s;
  if (len < 0) return fail(MD_ERR_SHAPE, "pages: %d tokens", len);
  const int32_t n = pages_of(p, len);
  if (capacity < n) return fail(MD_ERR_SHAPE, "pages: a table of %d entries for %d pages", capacity, n);
  if (n && !new_table) return fail(MD_ERR_INVALID_ARG, "pages: null table");
  if ((s = check_table(p, table, n)) != MD_OK) return s;
  for (int32_t i = 0; i < n; ++i) {
    new_table[i] = table[i];
    ++p->refs[table[i]];
  }
  return ok();
}

md_status md_kv_pages_truncate(md_kv_pages* p, const int32_t* table, int32_t len, int32_t new_len) {
  md_status s = check_pages(p);
  if (s != MD_OK) return s;
  if (new_len < 0 || len < new_len) return fail(MD_ERR_SHAPE, "pages: from %d back to %d tokens", len, new_len);
  const int32_t have = pages_of(p, len), keep = pages_of(p, new_len);
  if ((s = check_table(p, table, have)) != MD_OK) return s;
  for (int32_t i = keep; i < have; ++i)
    if (p->refs[table[i]]-- == 0) {  // named more often than it is held
      for (int32_t j = keep; j <= i; ++j) ++p->refs[table[j]];
      return fail(MD_ERR_INVALID_ARG, "pages: page %d appears more often than it is held", table[i]);
    }
  for (int32_t i = keep; i < have; ++i)
    if (p->refs[table[i]] == 0) {
      give(p, table[i]);
      p->refs[table[i]] = -1;  // given back: once, where the table names it twice
    }
  for (int32_t i = keep; i < have; ++i) p->refs[table[i]] = std::max(p->refs[table[i]], 0);
  return ok();
}

md_status md_kv_pages_compact(md_kv_pages* p, int32_t* tables, int32_t table_stride, const int32_t* lens, int32_t n_seqs,
                              int32_t* copy_src, int32_t* copy_dst, int32_t* n_copy) {
  md_status s = check_pages(p);
  if (s != MD_OK) return s;
  if (!copy_src || !copy_dst || !n_copy) return fail(MD_ERR_INVALID_ARG, "pages: null pointer");
  if (n_seqs < 0 || table_stride <= 0) return fail(MD_ERR_SHAPE, "pages: %d sequences, table_stride %d", n_seqs, table_stride);
  if (n_seqs && (!tables || !lens)) return fail(MD_ERR_INVALID_ARG, "pages: null pointer");
  for (int32_t i = 0; i < n_seqs; ++i) {
    if (lens[i] < 0 || pages_of(p, lens[i]) > table_stride)
      return fail(MD_ERR_SHAPE, "pages: sequence %d has %d tokens in a table of %d entries", i, lens[i], table_stride);
    if ((s = check_table(p, tables + (int64_t)i * table_stride, pages_of(p, lens[i]))) != MD_OK) return s;
  }
  // every holder has to be here, or its table would go stale; the free pages'
  // array serves as the count and is made anew from refs afterwards
  int32_t* count = p->free_pages;
  std::fill(count, count + p->n_pages, 0);
  for (int32_t i = 0; i < n_seqs; ++i)
    for (int32_t j = 0; j < pages_of(p, lens[i]); ++j) ++count[tables[(int64_t)i * table_stride + j]];
  int32_t used = 0;
  for (int32_t i = 0; i < p->n_pages; ++i) {
    if (count[i] != p->refs[i]) {
      const int32_t c = count[i];
      heap_from_refs(p);
      return fail(MD_ERR_INVALID_ARG, "pages: page %d is held %d times and named %d times", i, p->refs[i], c);
    }
    used += p->refs[i] > 0;
  }
  // the used pages behind the first `used` ones fill the free ones before them
  int32_t n = 0, to = 0;
  int32_t* moved = p->free_pages;
  for (int32_t i = used; i < p->n_pages; ++i) {
    if (p->refs[i] == 0) continue;
    while (p->refs[to] != 0) ++to;
    copy_src[n] = i;
    copy_dst[n++] = moved[i] = to;
    p->refs[to] = p->refs[i];
    p->refs[i] = 0;
  }
  for (int32_t i = 0; i < n_seqs; ++i)
    for (int32_t j = 0; j < pages_of(p, lens[i]); ++j) {
      int32_t& e = tables[(int64_t)i * table_stride + j];
      if (e >= used) e = moved[e];
    }
  *n_copy = n;
  heap_from_refs(p);
  return ok();
}

}  // extern "C"

// step_abi.cpp -- the C entry points around the attention and the experts:
// norms and rotation of queries and keys, routing, log probabilities.  Every
// check runs before anything is enqueued.
#include <hip/hip_runtime.h>

#include <cmath>

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
constexpr int kMaxHeads = 1024;
constexpr int kMaxVocab = 1 << 20;
constexpr int kMaxGiven = 64;
constexpr int kMaxE = 256, kMaxK = 8;

bool valid_xtype(int32_t t) { return t == MD_X_F32 || t == MD_X_BF16; }
int elem(int32_t t) { return t == MD_X_F32 ? 4 : 2; }
bool flag(int32_t v) { return v == 0 || v == 1; }

md_status check_rows(const char* what, const void* p, int64_t stride, int64_t width, int32_t type) {
  if (!p) return fail(MD_ERR_INVALID_ARG, "%s: null pointer", what);
  if (!aligned16(p)) return fail(MD_ERR_ALIGNMENT, "%s: not 16-byte aligned", what);
  if (stride < width) return fail(MD_ERR_SHAPE, "%s: row stride %lld < %lld", what, (long long)stride, (long long)width);
  if (stride * elem(type) % 16)
    return fail(MD_ERR_ALIGNMENT, "%s: a row stride of %lld values is no multiple of 16 bytes", what, (long long)stride);
  return MD_OK;
}

md_status check_out(const char* what, const void* x, int64_t x_stride, int32_t xt, const void* y, int64_t y_stride,
                    int64_t width, int32_t yt) {
  md_status s;
  if ((s = check_rows(what, x, x_stride, width, xt)) != MD_OK || (s = check_rows(what, y, y_stride, width, yt)) != MD_OK)
    return s;
  if (x == y && (xt != yt || x_stride != y_stride))
    return fail(MD_ERR_INVALID_ARG, "%s: in place with another type or row stride", what);
  return MD_OK;
}

// Sizes of a routing call.
md_status check_route(int32_t T, int32_t H, int32_t E) {
  if (T < 0 || H <= 0 || E <= 0) return fail(MD_ERR_SHAPE, "routing: T %d H %d E %d", T, H, E);
  if (T > kMaxTokens || E > kMaxE) return fail(MD_ERR_UNSUPPORTED, "routing: T %d (at most %d), E %d (%d)", T, kMaxTokens, E, kMaxE);
  if (H % 256 || H > 16384)
    return fail(MD_ERR_UNSUPPORTED, "H = %d: supported widths are multiples of 256 up to 16384", H);
  return MD_OK;
}
md_status check_routing(const md_routing* r, int32_t E) {
  if (!r) return fail(MD_ERR_INVALID_ARG, "null routing");
  if (r->score != MD_SCORE_SOFTMAX && r->score != MD_SCORE_SIGMOID) return fail(MD_ERR_INVALID_ARG, "unknown score %d", r->score);
  if (!flag(r->best_two) || !flag(r->renorm))
    return fail(MD_ERR_INVALID_ARG, "routing: best_two %d renorm %d", r->best_two, r->renorm);
  if (!std::isfinite(r->scale)) return fail(MD_ERR_INVALID_ARG, "routing: scale %g", r->scale);
  if (r->k <= 0 || r->k > E) return fail(MD_ERR_SHAPE, "routing: k = %d of %d experts", r->k, E);
  if (r->k > kMaxK) return fail(MD_ERR_UNSUPPORTED, "routing: k = %d > %d", r->k, kMaxK);
  if (r->groups <= 0 || E % r->groups || r->groups_kept <= 0 || r->groups_kept > r->groups)
    return fail(MD_ERR_SHAPE, "routing: %d of %d groups of %d experts", r->groups_kept, r->groups, E);
  if (r->groups > 64) return fail(MD_ERR_UNSUPPORTED, "routing: %d groups > 64", r->groups);
  if (r->k > r->groups_kept * (E / r->groups))
    return fail(MD_ERR_SHAPE, "routing: k = %d of %d groups of %d experts", r->k, r->groups_kept, E / r->groups);
  if (r->best_two && E / r->groups < 2) return fail(MD_ERR_SHAPE, "routing: the two best of a group of one");
  if (r->balance && !aligned16(r->balance)) return fail(MD_ERR_ALIGNMENT, "balance not 16-byte aligned");
  return MD_OK;
}

md_status check_logp(int32_t rows, int32_t vocab, int32_t top) {
  if (rows < 0 || vocab <= 0 || top < 0 || top > vocab)
    return fail(MD_ERR_SHAPE, "log probabilities: %d rows of %d, %d largest", rows, vocab, top);
  if (rows > kMaxTokens || vocab > kMaxVocab || top > md::kMaxTop)
    return fail(MD_ERR_UNSUPPORTED, "log probabilities: %d rows (at most %d) of %d (%d), %d largest (%d)", rows, kMaxTokens,
                vocab, kMaxVocab, top, md::kMaxTop);
  return MD_OK;
}
size_t part_bytes(int32_t rows, int segs) { return align256((size_t)rows * segs * 16); }

}  // namespace

extern "C" {

md_status md_qk_norm_rope(const md_rope* r, const int32_t* positions, int32_t rows, const void* q, int32_t q_heads,
                          int64_t q_stride, const void* k, int32_t k_heads, int64_t k_stride, int32_t xtype, void* q_out,
                          int64_t q_out_stride, void* k_out, int64_t k_out_stride, int32_t ytype, hipStream_t stream) {
  if (!r) return fail(MD_ERR_INVALID_ARG, "null rotation descriptor");
  if (!valid_xtype(xtype) || !valid_xtype(ytype)) return fail(MD_ERR_INVALID_ARG, "unknown xtype %d or ytype %d", xtype, ytype);
  if (!flag(r->interleaved)) return fail(MD_ERR_INVALID_ARG, "interleaved = %d", r->interleaved);
  if (!std::isfinite(r->factor) || !std::isfinite(r->eps) || r->eps < 0.0f)
    return fail(MD_ERR_INVALID_ARG, "factor %g, eps %g", r->factor, r->eps);
  if (rows < 0 || q_heads <= 0 || k_heads < 0 || r->head_dim <= 0 || r->rot < 0 || r->rot > r->head_dim)
    return fail(MD_ERR_SHAPE, "rows %d, heads %d and %d of %d, %d turned", rows, q_heads, k_heads, r->head_dim, r->rot);
  if (rows > kMaxTokens || q_heads > kMaxHeads || k_heads > kMaxHeads || r->head_dim > 256 || r->head_dim % 8 || r->rot % 8)
    return fail(MD_ERR_UNSUPPORTED,
                "rows %d (at most %d), heads %d and %d (%d), head width %d and %d turned (multiples of 8 up to 256)", rows,
                kMaxTokens, q_heads, k_heads, kMaxHeads, r->head_dim, r->rot);
  if (rows == 0) return ok();
  const int64_t D = r->head_dim;
  md_status s;
  if ((s = check_out("q", q, q_stride, xtype, q_out, q_out_stride, q_heads * D, ytype)) != MD_OK) return s;
  if (k_heads && (s = check_out("k", k, k_stride, xtype, k_out, k_out_stride, k_heads * D, ytype)) != MD_OK) return s;
  if (r->rot && (!r->inv_freq || !positions)) return fail(MD_ERR_INVALID_ARG, "null inv_freq or positions");
  if (r->rot && (!aligned16(r->inv_freq) || !aligned4(positions)))
    return fail(MD_ERR_ALIGNMENT, "inv_freq not 16-byte aligned, or positions not 4-byte");
  if ((r->q_weight && !aligned16(r->q_weight)) || (r->k_weight && !aligned16(r->k_weight)))
    return fail(MD_ERR_ALIGNMENT, "weights not 16-byte aligned");
  md::RopeArgs g{};
  g.q = q;
  g.k = k;
  g.q_out = q_out;
  g.k_out = k_out;
  g.q_stride = q_stride;
  g.k_stride = k_stride;
  g.q_out_stride = q_out_stride;
  g.k_out_stride = k_out_stride;
  g.q_weight = r->q_weight;
  g.k_weight = r->k_weight;
  g.inv_freq = r->inv_freq;
  g.positions = positions;
  g.rows = rows;
  g.Hq = q_heads;
  g.Hkv = k_heads;
  g.D = r->head_dim;
  g.rot = r->rot;
  g.eps = r->eps;
  g.factor = r->factor;
  const hipError_t e = md::launch_qk_norm_rope(g, r->interleaved != 0, xtype, ytype, stream);
  return e == hipSuccess ? ok() : hip_fail(e, "rotation launch");
}

md_status md_moe_route_workspace_size(int32_t T, int32_t H, int32_t E, size_t* bytes) {
  const md_status s = check_route(T, H, E);
  if (s != MD_OK) return s;
  if (!bytes) return fail(MD_ERR_INVALID_ARG, "null size pointer");
  // enough for either type of x, with the logits or without
  size_t most = 0;
  for (int form = 0; T && form < 3; ++form) {
    const size_t b = md::route_plan(T, H, E, form == 1 ? MD_X_BF16 : MD_X_F32, form < 2).bytes;
    if (b > most) most = b;
  }
  *bytes = most;
  return ok();
}

md_status md_moe_route(const md_routing* r, const void* x, int32_t xtype, int32_t T, int32_t H, const float* W_r,
                       const float* router_bias, int32_t E, int32_t* idx, float* gates, float* logits, void* workspace,
                       size_t workspace_bytes, hipStream_t stream) {
  size_t need = 0;
  md_status s;
  if ((s = md_moe_route_workspace_size(T, H, E, &need)) != MD_OK || (s = check_routing(r, E)) != MD_OK) return s;
  if (!valid_xtype(xtype)) return fail(MD_ERR_INVALID_ARG, "unknown xtype %d", xtype);
  if (T == 0) return ok();
  if (!x || !W_r || !idx || !gates) return fail(MD_ERR_INVALID_ARG, "null x, W_r, idx or gates");
  if (!aligned16(x) || !aligned16(W_r) || !aligned16(idx) || !aligned16(gates) || (router_bias && !aligned16(router_bias)) ||
      (logits && !aligned16(logits)))
    return fail(MD_ERR_ALIGNMENT, "device pointers must be 16-byte aligned");
  if (!workspace || workspace_bytes < need)
    return fail(MD_ERR_WORKSPACE, "workspace: %zu bytes, %zu needed", workspace ? workspace_bytes : 0, need);
  if (!aligned16(workspace)) return fail(MD_ERR_ALIGNMENT, "workspace not 16-byte aligned");
  const md::RoutePlan p = md::route_plan(T, H, E, xtype, !logits);
  md::RouteArgs g{};
  g.T = T;
  g.H = H;
  g.E = E;
  g.k = r->k;
  g.sigmoid = r->score == MD_SCORE_SIGMOID;
  g.groups = r->groups;
  g.kept = r->groups_kept;
  g.lane_bits = 0;
  while (2 * r->groups << g.lane_bits <= 64) ++g.lane_bits;
  g.per = E / r->groups;
  g.per_inv = 65536 / g.per + 1;
  g.best_two = r->best_two;
  g.renorm = r->renorm;
  g.scale = r->scale;
  g.bias = router_bias;
  g.balance = r->balance;
  g.logits = logits;
  g.idx = idx;
  g.gates = gates;
  const hipError_t e = md::launch_route(g, p, x, xtype, W_r, workspace, stream);
  return e == hipSuccess ? ok() : hip_fail(e, "routing launch");
}

// The routed layer's workspace: idx, gates, then what routing and experts need
// one after the other.
static size_t routed_head(const md_moe_layer* L, int32_t T) { return 2 * align256(sizeof(float) * (size_t)T * L->k); }

md_status md_moe_routed_workspace_size(const md_moe_layer* L, int32_t T, size_t* bytes) {
  size_t experts = 0, route = 0;
  md_status s = md_moe_workspace_size(L, T, &experts);
  if (s != MD_OK) return s;
  if ((s = md_moe_route_workspace_size(T, L->H, L->E, &route)) != MD_OK) return s;
  if (!bytes) return fail(MD_ERR_INVALID_ARG, "null size pointer");
  *bytes = routed_head(L, T) + (experts > route ? experts : route);
  return ok();
}

md_status md_moe_layer_forward_routed(const md_moe_layer* L, const md_routing* routing, const float* x, int32_t T, float* y,
                                      int32_t* idx_out, float* gates_out, void* workspace, size_t workspace_bytes,
                                      hipStream_t stream) {
  size_t need = 0;
  md_status s = md_moe_routed_workspace_size(L, T, &need);
  if (s != MD_OK || (s = check_routing(routing, L->E)) != MD_OK) return s;
  if (routing->k != L->k) return fail(MD_ERR_SHAPE, "routing to %d experts, the layer takes %d", routing->k, L->k);
  if (!x || !y) return fail(MD_ERR_INVALID_ARG, "null x or y");
  if (!aligned16(x) || !aligned16(y) || (idx_out && !aligned16(idx_out)) || (gates_out && !aligned16(gates_out)))
    return fail(MD_ERR_ALIGNMENT, "device pointers must be 16-byte aligned");
  if (!workspace || workspace_bytes < need)
    return fail(MD_ERR_WORKSPACE, "workspace: %zu bytes, %zu needed", workspace ? workspace_bytes : 0, need);
  if (!aligned16(workspace)) return fail(MD_ERR_ALIGNMENT, "workspace not 16-byte aligned");
  char* ws = static_cast<char*>(workspace);
  const size_t head = routed_head(L, T);
  int32_t* idx = idx_out ? idx_out : reinterpret_cast<int32_t*>(ws);
  float* gates = gates_out ? gates_out : reinterpret_cast<float*>(ws + head / 2);
  if ((s = md_moe_route(routing, x, MD_X_F32, T, L->H, L->W_r, L->router_bias, L->E, idx, gates, nullptr, ws + head,
                        workspace_bytes - head, stream)) != MD_OK)
    return s;
  return md_moe_experts_forward(L, x, T, idx, gates, y, ws + head, workspace_bytes - head, stream);
}

md_status md_token_logprobs_workspace_size(int32_t rows, int32_t vocab, int32_t top, size_t* bytes) {
  const md_status s = check_logp(rows, vocab, top);
  if (s != MD_OK) return s;
  if (!bytes) return fail(MD_ERR_INVALID_ARG, "null size pointer");
  const int segs = rows ? md::logprob_plan(rows, vocab).segs : 1;
  *bytes = segs > 1 ? part_bytes(rows, segs) + align256((size_t)rows * segs * top * 8) : 0;
  return ok();
}

md_status md_token_logprobs(const void* logits, int32_t xtype, int64_t stride, int32_t rows, int32_t vocab,
                            const int32_t* tokens, int32_t n_tokens, float scale, int32_t top, float* logprobs,
                            float* entropy, int32_t* top_ids, float* top_logprobs, void* workspace,
                            size_t workspace_bytes, hipStream_t stream) {
  size_t need = 0;
  const md_status s = md_token_logprobs_workspace_size(rows, vocab, top, &need);
  if (s != MD_OK) return s;
  if (!valid_xtype(xtype)) return fail(MD_ERR_INVALID_ARG, "unknown xtype %d", xtype);
  if (!(scale > 0.0f && scale <= 0x1p64f)) return fail(MD_ERR_INVALID_ARG, "log probabilities: scale %g", scale);
  if (n_tokens < 0) return fail(MD_ERR_SHAPE, "log probabilities: %d tokens", n_tokens);
  if (n_tokens > kMaxGiven) return fail(MD_ERR_UNSUPPORTED, "log probabilities: %d tokens > %d", n_tokens, kMaxGiven);
  if (stride < vocab) return fail(MD_ERR_SHAPE, "log probabilities: row stride %lld < %d", (long long)stride, vocab);
  if (rows == 0) return ok();
  if (!logits || (n_tokens && (!tokens || !logprobs)) || (top && (!top_ids || !top_logprobs)))
    return fail(MD_ERR_INVALID_ARG, "log probabilities: null pointer");
  if (reinterpret_cast<uintptr_t>(logits) % elem(xtype))
    return fail(MD_ERR_ALIGNMENT, "logits not aligned to their %d bytes", elem(xtype));
  if ((n_tokens && (!aligned4(tokens) || !aligned4(logprobs))) || (top && (!aligned4(top_ids) || !aligned4(top_logprobs))) ||
      !aligned4(entropy))
    return fail(MD_ERR_ALIGNMENT, "log probabilities: an array is not 4-byte aligned");
  if (need) {
    if (!workspace || workspace_bytes < need)
      return fail(MD_ERR_WORKSPACE, "workspace: %zu bytes, %zu needed", workspace ? workspace_bytes : 0, need);
    if (!aligned16(workspace)) return fail(MD_ERR_ALIGNMENT, "workspace not 16-byte aligned");
  }
  md::LogpArgs g{};
  g.logits = logits;
  g.stride = stride;
  g.rows = rows;
  g.vocab = vocab;
  g.n_tokens = n_tokens;
  g.top = top;
  const md::LogpPlan plan = md::logprob_plan(rows, vocab);
  g.segs = plan.segs;
  g.steps = plan.steps;
  g.tokens = tokens;
  g.scale = scale;
  g.logprobs = logprobs;
  g.entropy = entropy;
  g.top_ids = top_ids;
  g.top_logprobs = top_logprobs;
  if (need) {
    g.part = workspace;
    g.keys = static_cast<char*>(workspace) + part_bytes(rows, g.segs);
  }
  const hipError_t e = md::launch_logprob(g, xtype, plan, stream);
  return e == hipSuccess ? ok() : hip_fail(e, "log probabilities launch");
}

}  // extern "C"

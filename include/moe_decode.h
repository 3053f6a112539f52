/* moe_decode.h -- C ABI of libmoe_decode, the gfx950 (MI355X) library for the
 * decode / short-chunk prefill forward of a block-quantized feed-forward or
 * mixture-of-experts layer.
 *
 * The operations follow the pages' statement of the problem:
 *   - a quantized matrix-vector product over Q8_0 / Q4_0 blocks (the Camelid
 *     README, "Engine" and "Supported" sections: Q8_0 weights and Q4_0
 *     "wire GEMVs" checked against a CPU oracle) and over int8 / packed int4
 *     weights with one scale per row (the colibri summary, "model execution
 *     and memory tiers");
 *   - a router with top-k expert selection whose exact ties go to the lower
 *     expert index (the Camelid README, "Experimental lanes");
 *   - the MoE block: router -> top-k routed experts -> gated FFN (GeGLU) per
 *     selected expert -> combine, plus a dense shared-expert branch (the
 *     Camelid README, "Gemma 4": 128 experts, sparse top-8 plus a dense shared
 *     expert; the TurboFieldfare summary, "memory and expert streaming":
 *     router-chosen experts, shared branch computed alongside, prefill in
 *     chunks of at most 128 tokens reusing each expert across rows);
 *   - two more weight codecs: Q4_1 blocks (the Camelid README's bit-exact
 *     q4_1 GEMV) and packed int2 with one scale per row (the colibri summary);
 *   - a host-memory expert tier: the expert set in host RAM, a slot cache of
 *     experts in HBM (the Camelid README's experts-in-RAM lane with a VRAM
 *     expert cache; the TurboFieldfare summary's expert slots);
 *   - the attention block beside it in 8-bit integers: the linear layers with a
 *     scale for each token and output channel (int8 rows, any number of
 *     tokens), a paged cache of keys and values with a scale for each page and
 *     head, the attention that reads it, and the bookkeeping of its pages;
 *   - what a step that checks drafted tokens needs around them: norms and
 *     rotation of queries and keys, attention over a tree of drafts and over a
 *     window with sinks, routing with balance and groups, log probabilities.
 *
 * Conventions (every entry point):
 *   - Pointers marked "device" are HIP device pointers, "host" are host
 *     pointers.  The caller allocates and owns every buffer and the stream; the
 *     library never allocates, frees or synchronizes (one exception, stated
 *     there: md_moe_cached_forward reads the routing back once per call).
 *     Work is enqueued on `stream` (NULL = the null stream) and completes
 *     asynchronously.
 *   - Every argument is validated on the host before anything is enqueued; a
 *     call that returns an error has enqueued nothing and written nothing
 *     (md_moe_cached_forward: nothing after the step that failed).
 *     Unsupported shapes return MD_ERR_UNSUPPORTED: there is no fallback.
 *   - Device data pointers must be 16-byte aligned (MD_ERR_ALIGNMENT).
 *   - md_last_error_detail() returns a thread-local message describing the
 *     last non-OK return on the calling thread.
 *   - Asynchronous faults surface through the HIP runtime on `stream`.
 *   - Results are deterministic: no float atomics; fixed reduction orders.
 *   - Calls that take a workspace may not overlap on the same workspace.
 *
 * Supported shapes: hidden / input widths (cols) are multiples of 256 and at
 * most 16384; rows 1..65536; E <= 256; 1 <= k <= 8; T <= 128 tokens per
 * layer call (longer prompts are split by the caller into chunks of at most
 * 128 tokens); batch <= 8 for md_qgemv; md_i8_*, md_kv_*, md_qk_norm_rope,
 * md_moe_route and md_token_logprobs: see there.
 *
 * Accuracy contract.  Weights are decoded exactly (scale times code) and
 * every contraction y = sum_c w_c x_c is accumulated in fp32 or exactly in
 * integers; the router is accumulated in fp64 and rounded once.  The tolerance
 * the source pages' problem statement sets is
 *     |y - y_exact| <= 1e-4 * S + 1e-6,   S = sum_c |w_c x_c|,
 * and per path the library guarantees:
 *   - md_qgemv (every batch and format), and the FFN / MoE layers' chunks on
 *     block formats (Q8_0, Q4_0, Q4_1: bf16 matrix cores on the exact codes
 *     against activations split into two bf16 halves): the tolerance for
 *     every finite input.
 *   - FFN / MoE layers on the one-token kernels (up to 8 tokens, 16 on small
 *     layers; every format): the activations a 16-byte weight chunk
 *     multiplies -- a group g of 32 consecutive values for Q4_0 / Q4_1 /
 *     packed int4, 16 for Q8_0 / int8, 64 for packed int2 -- are rounded to
 *     integers of 2^-22 of the group's largest magnitude M_g before exact
 *     integer dot products.  Per contraction (gate, up, down, shared expert)
 *         |y - y_exact| <= 2^-22 * A + 2^-19 * S,
 *         A = sum_g M_g * sum_{c in g} |w_c|,
 *     which gives the tolerance whenever A <= 400 * S: a group's largest
 *     activation may exceed the typical magnitude of the activations that
 *     its weights multiply by up to about 400x.  Inputs outside that
 *     precondition (a group holding a value ~1000x the others, with the
 *     weights concentrated on the small ones) can exceed 1e-4 * S; the
 *     seeded workloads sit at A / S <= 15.
 *   - FFN / MoE layers' chunks on the per-row formats (int8, packed int4 /
 *     int2 with one scale per row: int8 matrix cores): each activation row
 *     (a token's x, a pair's h) is rounded to integers of 2^-30 of the row's
 *     largest magnitude M; per contraction
 *         |y - y_exact| <= 2^-30 * M * sum_c |w_c| + 2^-19 * S,
 *     which gives the tolerance whenever M * sum_c |w_c| <= 1e5 * S (the
 *     seeded workloads: <= 80).
 *   A layer's output additionally carries the effect of its gate/up
 *   contractions' error on h, as any fp32 evaluation does.
 */
#ifndef MOE_DECODE_H
#define MOE_DECODE_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MD_ABI_VERSION 1

typedef enum md_status {
    MD_OK = 0,
    MD_ERR_INVALID_ARG = 1,   /* null pointer, bad enum value                 */
    MD_ERR_SHAPE = 2,         /* inconsistent dimensions                      */
    MD_ERR_UNSUPPORTED = 3,   /* valid but outside the supported set          */
    MD_ERR_ALIGNMENT = 4,     /* a device pointer is not 16-byte aligned      */
    MD_ERR_WORKSPACE = 5,     /* workspace missing or too small               */
    MD_ERR_HIP = 6            /* the HIP runtime reported a launch error      */
} md_status;

/* Weight formats.  Canonical layouts (as stored in GGUF-style files; the
 * oracle reads these):
 *   MD_Q8_0   rows of cols/32 blocks of 34 bytes: fp16 d (little-endian) then
 *             32 int8 q;  w = d * q.
 *   MD_Q4_0   rows of cols/32 blocks of 18 bytes: fp16 d then 16 bytes qs;
 *             weight j (0..15) is the low nibble n of qs[j], weight j+16 the
 *             high nibble;  w = d * (n - 8).
 *   MD_I8_ROW rows of cols int8 q; one fp32 scale s per row;  w = s * q.
 *   MD_I4_ROW rows of cols/2 bytes; weight 2j is the low nibble of byte j and
 *             2j+1 the high nibble, two's complement in [-8, 7]; one fp32
 *             scale s per row;  w = s * v.
 *   MD_Q4_1   rows of cols/32 blocks of 20 bytes: fp16 d, fp16 m, then 16
 *             bytes qs in the MD_Q4_0 nibble order, codes n in 0..15 with no
 *             offset;  w = d * n + m  (the Camelid README's bit-exact q4_1
 *             GEMV, "Experimental" rows).
 *   MD_I2_ROW rows of cols/4 bytes; weight 4j+i sits in bits 2i..2i+1 of byte
 *             j, two's complement in [-2, 1]; one fp32 scale s per row;
 *             w = s * v  (the colibri summary's packed int2 per-row format,
 *             "model execution and memory tiers").
 * Device layout (what every compute entry point reads; produced from the
 * canonical layout by md_prepare_layout, same byte count, same row stride):
 *   MD_Q8_0   per row: the cols int8 q of all blocks in order, then the
 *             cols/32 fp16 scales in order.
 *   MD_Q4_0   per row: the 16-byte qs of all blocks in order, then the
 *             cols/32 fp16 scales in order.
 *   MD_Q4_1   per row: the 16-byte qs of all blocks in order, then the
 *             cols/32 (d, m) fp16 pairs in order.
 *   MD_I8_ROW, MD_I4_ROW, MD_I2_ROW: identical to the canonical layout.
 * Every row therefore starts a run of 16-byte quant chunks that a wavefront
 * streams with coalesced 16-byte loads, scales kept out of the way.
 * Every type is taken by every entry point: md_qgemv, the FFN and MoE layers
 * (one-token kernels, grouped GEMMs) and the expert tier. */
typedef enum md_qtype {
  MD_Q8_0 = 1, MD_Q4_0 = 2, MD_I8_ROW = 3, MD_I4_ROW = 4, MD_Q4_1 = 5, MD_I2_ROW = 6
} md_qtype;

typedef enum md_xtype { MD_X_F32 = 0, MD_X_BF16 = 1 } md_xtype;

/* act(a) * u with act = tanh-form GELU (GeGLU) or SiLU (SwiGLU). */
typedef enum md_act { MD_ACT_GELU_TANH = 0, MD_ACT_SILU = 1 } md_act;

/* A quantized matrix (rows = outputs, cols = inputs), device layout. */
typedef struct md_qmatrix {
    int32_t type;              /* md_qtype                                    */
    int32_t rows, cols;
    const void *q;             /* device: rows * md_row_bytes(type, cols)     */
    const float *row_scale;    /* device: rows fp32 (the *_ROW types), else NULL */
} md_qmatrix;

/* A dense gated FFN: y = down( act(gate x) * (up x) ).
 * gate, up: F x H;  down: H x F;  all three of one type. */
typedef struct md_ffn {
    int32_t act;               /* md_act                                      */
    md_qmatrix gate, up, down;
} md_ffn;

/* One MoE layer.  The E experts of each projection are stored expert-major
 * and contiguous: expert e's gate matrix starts at gate_q + e * (F rows of
 * md_row_bytes(type, H)), its scales (the *_ROW types) at gate_scale + e*F;
 * likewise up (F x H) and down (H x F, scales at down_scale + e*H). */
typedef struct md_moe_layer {
    int32_t H, F, E, k;
    int32_t act;               /* md_act                                      */
    int32_t type;              /* md_qtype of the routed experts              */
    const void *gate_q, *up_q, *down_q;                /* device              */
    const float *gate_scale, *up_scale, *down_scale;   /* device or NULL      */
    const float *W_r;          /* device: E x H fp32 router weights           */
    const float *router_bias;  /* device: E fp32, or NULL                     */
    int32_t has_shared;        /* 1: add a dense shared expert (gate 1)       */
    md_ffn shared;             /* its gate/up F_s x H, down H x F_s           */
} md_moe_layer;

int32_t md_abi_version(void);
const char *md_status_string(md_status s);
const char *md_last_error_detail(void);

/* Bytes of one row in either layout (scales of the *_ROW types excluded);
 * -1 if cols is not valid for the type. */
int64_t md_row_bytes(int32_t type, int32_t cols);

/* Convert `count` consecutive matrices (rows x cols each) from the canonical
 * layout at `src` to the device layout at `dst` (both device, same size,
 * must not overlap).  One-time, at weight-load. */
md_status md_prepare_layout(int32_t type, int32_t rows, int32_t cols, int32_t count,
                            const void *src, void *dst, hipStream_t stream);

/* y[b][r] = sum_c w[r][c] * x[b][c] for b < batch (batch 1..8).
 * x: device, batch x cols, fp32 or bf16 (xtype); y: device, batch x rows fp32.
 * Accumulation in fp32.  Needs md_qgemv_workspace_size() bytes of workspace
 * (may be 0, then workspace may be NULL). */
md_status md_qgemv_workspace_size(const md_qmatrix *W /*host*/, int32_t batch, size_t *bytes /*host*/);
md_status md_qgemv(const md_qmatrix *W /*host*/, const void *x, int32_t xtype, int32_t batch, float *y,
                   void *workspace, size_t workspace_bytes, hipStream_t stream);

/* Router for T tokens: logits l[t][e] = sum_c W_r[e][c] x[t][c] (+ bias[e]),
 * accumulated in fp64 and rounded to fp32; idx[t][0..k-1] = the k largest
 * logits in descending order, exact ties broken by the lower expert index
 * (-0 equals +0); gates[t][j] = exp(l_j - l_0) / sum_i exp(l_i - l_0) over
 * the selected k.  idx (int32 T x k), gates (fp32 T x k) and logits (fp32
 * T x E, may be NULL) are device buffers.  Non-finite logits are outside the
 * contract (the selection is then unspecified). */
md_status md_route_workspace_size(int32_t T, int32_t H, int32_t E, int32_t k, size_t *bytes /*host*/);
md_status md_moe_route_topk(const float *x, int32_t T, int32_t H, const float *W_r, const float *bias,
                            int32_t E, int32_t k, int32_t *idx, float *gates, float *logits,
                            void *workspace, size_t workspace_bytes, hipStream_t stream);

/* Dense gated FFN for T tokens (1..128): x, y device T x H fp32. */
md_status md_ffn_workspace_size(const md_ffn *f /*host*/, int32_t T, size_t *bytes /*host*/);
md_status md_ffn_forward(const md_ffn *f /*host*/, const float *x, int32_t T, float *y,
                         void *workspace, size_t workspace_bytes, hipStream_t stream);

/* The MoE layer for T tokens (1..128):
 *   y[t] = sum_{j<k} gates[t][j] * FFN_{idx[t][j]}(x[t])  (+ shared FFN(x[t]))
 * x, y: device T x H fp32.  idx_out (int32 T x k) and gates_out (fp32 T x k)
 * receive the routing when non-NULL.  Only the selected experts' weight bytes
 * are read.  Up to 8 tokens (up to 16 on layers whose whole expert set takes
 * at most 512 MB) every (token, slot) pair runs as its own one-token problem,
 * so an expert that several tokens select is read once per such pair; the
 * layer runs as router, gate/up and down kernels (a shared expert runs inside
 * the routed launches where its shapes are covered, else as its own two
 * launches first).  Longer chunks group the pairs by expert and read each
 * selected expert once per 16-token tile of the tokens that chose it; their
 * shared expert, which needs only x, runs on a second stream of the
 * library's own (one per device, default priority, created at the device's
 * first such call) beside the routing kernels and joins `stream` before the
 * combine, so the call's work still starts after, and ends before, the
 * work around it on `stream` (a graph captured from `stream` takes the side
 * stream's launches in as a branch).  The results are those of the same
 * kernels on `stream` alone, bit for bit.  There is one code path per shape:
 * nothing in the environment selects another. */
md_status md_moe_workspace_size(const md_moe_layer *L /*host*/, int32_t T, size_t *bytes /*host*/);
md_status md_moe_layer_forward(const md_moe_layer *L /*host*/, const float *x, int32_t T, float *y,
                               int32_t *idx_out, float *gates_out,
                               void *workspace, size_t workspace_bytes, hipStream_t stream);

/* md_moe_layer_forward for callers that cannot allocate device memory (code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc): the same kernels and results, with the scratch taken from a
 * 64 MiB array built into the library instead of a caller's workspace.
 * Every GPU the library runs on holds one such array from the library's
 * first use on it until the process ends; its address is looked up once per
 * device, on the first call with that device current.  This call allocates
 * and frees nothing and calls no allocating routine.  All calls on one GPU
 * share its array: calls that overlap on one GPU (other streams, other host
 * threads) race and must be serialized by the caller; the array keeps the
 * last call's contents, and nothing in it needs to start cleared.
 * Everything runs on `stream` (no side stream).
 * Errors: as md_moe_layer_forward; a call whose scratch (the size
 * md_moe_workspace_size reports) exceeds 64 MiB -> MD_ERR_UNSUPPORTED, with
 * nothing enqueued (every layer and token count of the seeded workloads fits:
 * the largest, 128 tokens of a 256-expert layer of hidden size 6144, needs
 * about 62 MiB). */
md_status md_moe_layer_forward_noalloc(const md_moe_layer *L /*host*/, const float *x, int32_t T, float *y,
                                       int32_t *idx_out, float *gates_out, hipStream_t stream);

/* Measurement variant of md_moe_layer_forward: identical work and results,
 * every launch on `stream` (no side stream); additionally records `start` on
 * `stream` just before the launches of stage
 * `stage` and `stop` just after them (HIP events created by the caller), so
 * the elapsed time between the two events is that stage's time on the
 * stream.  A stage the call does not run (the shared expert of a layer
 * without one) records both events back to back; so do the stages that a
 * merged launch covers besides MD_STAGE_GATEUP, which then times the whole
 * merged work (few tokens, a layer with a shared expert on the shapes it
 * covers: the routed+shared gate/up and down launches). */
typedef enum md_stage {
    MD_STAGE_SHARED = 0,      /* dense shared-expert FFN                      */
    MD_STAGE_ROUTER = 1,      /* router logits                                */
    MD_STAGE_SELECT = 2,      /* top-k, gates, expert dispatch                */
    MD_STAGE_GATEUP = 3,      /* selected experts' gate/up + activation       */
    MD_STAGE_DOWN = 4,        /* selected experts' down projection            */
    MD_STAGE_COMBINE = 5      /* gate-weighted combine (+ shared)             */
} md_stage;
md_status md_moe_layer_forward_timed(const md_moe_layer *L /*host*/, const float *x, int32_t T, float *y,
                                     int32_t *idx_out, float *gates_out,
                                     void *workspace, size_t workspace_bytes, hipStream_t stream,
                                     int32_t stage, hipEvent_t start, hipEvent_t stop);

/* Measurement aid: enqueues only the launches of stage `stage` (md_stage) of
 * md_moe_layer_forward with the same arguments, which read the intermediate
 * results that an earlier such call left in `workspace` (and in idx_out /
 * gates_out); the stage's outputs are rewritten with the same values.
 * Relaunching one stage back to back over several workspaces, each left by a
 * different token's call, times that stage's kernels on their real inputs
 * with nothing else in between (HIP events around the whole run give the
 * kernels' average duration, without the dispatch latency that events around
 * one launch add).  The workspace must hold what the earlier call with the
 * same layer, x, T and outputs wrote, untouched since.  Errors: as
 * md_moe_layer_forward; a stage outside 0..5 -> MD_ERR_INVALID_ARG. */
md_status md_moe_layer_stage_relaunch(const md_moe_layer *L /*host*/, const float *x, int32_t T, float *y,
                                      int32_t *idx_out, float *gates_out, void *workspace, size_t workspace_bytes,
                                      hipStream_t stream, int32_t stage);

/* md_moe_layer_forward with a residual: y = residual + layer(x), residual an
 * fp32 [T][H] device buffer (it may be x or y itself).  The residual is added
 * in the layer's last kernel (the down projection or the combine, after the
 * shared expert's output), so layers stack without an extra launch each (the
 * Camelid README, "Gemma 4": resident layer weights and a captured decode
 * graph).  Errors: as md_moe_layer_forward; a null residual ->
 * MD_ERR_INVALID_ARG; not 16-byte aligned -> MD_ERR_ALIGNMENT. */
md_status md_moe_layer_forward_residual(const md_moe_layer *L /*host*/, const float *x, int32_t T,
                                        const float *residual, float *y, int32_t *idx_out, float *gates_out,
                                        void *workspace, size_t workspace_bytes, hipStream_t stream);

/* y = a + b over n fp32 values (device pointers; y may alias a or b): the
 * residual add that joins stacked layers, so a stack of layers (each layer's
 * output added to its input) runs as one sequence of this library's kernels
 * that a caller can capture in a HIP graph and replay without host
 * synchronization (the Camelid README, "Gemma 4": a GPU-resident decode path
 * with resident layer weights and a captured decode graph; "Ornith 1.0 9B": a
 * device-side decode loop, the host synchronizing once per token chunk).
 * Errors: n <= 0 -> MD_ERR_SHAPE; a null pointer -> MD_ERR_INVALID_ARG;
 * pointers not 16-byte aligned -> MD_ERR_ALIGNMENT. */
md_status md_add(const float *a, const float *b, float *y, int64_t n, hipStream_t stream);

/* The experts of a layer for a given routing: y[t] = sum_j gates[t][j] *
 * FFN_{idx[t][j]}(x[t]) -- the layer forward without the router (the
 * TurboFieldfare summary, "memory and expert streaming": the runtime splits
 * the router's choices into cache hits and misses before the experts run).
 * idx, gates: device [T][k] (int32, fp32); a token's k entries must be
 * distinct; entries outside [0, E) are clamped into it.  A shared expert
 * is added as in md_moe_layer_forward.  Needs md_moe_workspace_size(L, T)
 * bytes of workspace.  Errors as md_moe_layer_forward. */
md_status md_moe_experts_forward(const md_moe_layer *L /*host*/, const float *x, int32_t T, const int32_t *idx,
                                 const float *gates, float *y, void *workspace, size_t workspace_bytes,
                                 hipStream_t stream);

/* Host-memory expert tier with an HBM slot cache (the Camelid README,
 * "Supported": experts kept in host RAM with a VRAM-resident expert cache;
 * the TurboFieldfare summary, "memory and expert streaming": a fixed number
 * of expert slots per layer, least-frequently-used replacement with a
 * recency tie-break, the router's choices split into hits and misses; the
 * colibri summary, "model execution and memory tiers": per-layer caches of
 * hot experts).  The whole expert set lives in host memory (pinned, so the
 * copies run asynchronously), S slots of the same layout in HBM.  All arrays
 * of the struct are host memory owned by the caller. */
typedef struct md_expert_cache {
  int32_t E;                 /* experts of the layer                              */
  int32_t S;                 /* HBM slots                                         */
  int32_t *slot_of_expert;   /* [E]: the slot holding expert e, or -1             */
  int32_t *expert_in_slot;   /* [S]: the expert a slot holds, or -1 (empty)       */
  int64_t *uses;             /* [S]: selections of the slot's expert since loaded */
  int64_t *last_use;         /* [S]: the plan step that last selected it          */
  int32_t *slot_idx;         /* [T*k] scratch of md_moe_cached_forward            */
  int64_t step;              /* plan steps so far                                 */
  int64_t hits, misses;      /* distinct-expert hits and misses so far            */
} md_expert_cache;

/* Empties the cache (all slots free, counters zero).  Errors: a null pointer
 * -> MD_ERR_INVALID_ARG; E or S <= 0 -> MD_ERR_SHAPE. */
md_status md_expert_cache_reset(md_expert_cache *c /*host*/);

/* One step of the replacement policy for the n = T*k expert ids in idx
 * (host): every distinct expert already in a slot is a hit (its use count
 * and last use updated); every other one, in order of first appearance,
 * takes an empty slot (lowest index first) or else evicts the slot with the
 * fewest uses, ties to the least recently used, then to the lowest index,
 * among the slots this step has not used.  Writes slot_idx[i] = the slot of
 * idx[i], and the misses as (miss_expert, miss_slot) pairs, *n_miss of them
 * (host arrays of n entries).  Errors: an id outside [0, E) or a null
 * pointer -> MD_ERR_INVALID_ARG; n outside 1..1024 -> MD_ERR_SHAPE; more
 * distinct experts than slots -> MD_ERR_UNSUPPORTED; nothing changes on
 * error. */
md_status md_expert_cache_plan(md_expert_cache *c /*host*/, const int32_t *idx, int32_t n, int32_t *slot_idx,
                               int32_t *miss_expert, int32_t *miss_slot, int32_t *n_miss);

/* Enqueues the copies of the missed experts' gate, up and down matrices (and
 * row scales) from src (E experts, usually pinned host memory) into the
 * slots of dst (a layer descriptor whose E is the slot count, in HBM) on
 * stream.  Errors: src and dst of different H, F, type, act or k ->
 * MD_ERR_SHAPE; an expert or slot out of range or a null pointer ->
 * MD_ERR_INVALID_ARG. */
md_status md_expert_cache_fill(const md_moe_layer *src /*host*/, const md_moe_layer *dst /*host*/,
                               const int32_t *miss_expert, const int32_t *miss_slot, int32_t n_miss,
                               hipStream_t stream);

/* The layer forward with the expert tier: the router and top-k on the GPU
 * (src's W_r / router_bias, device memory), one read-back of the routing
 * (this call synchronizes the stream once), the cache plan, the copies of
 * the misses, then md_moe_experts_forward on the slots with the slot ids.
 * With a copy_stream (and an event copy_done to join it), the misses load on
 * it while dst's shared expert (resident) runs on stream, and the routed
 * experts wait for the copies (the TurboFieldfare summary: misses filled
 * while the shared branch computes); a null copy_stream puts the copies on
 * stream.  idx_out / gates_out (device, nullable) receive the expert ids and
 * gates.  c->slot_idx must hold T*k entries and stay untouched until the
 * next call on the stream (an asynchronous copy reads it).  Workspace:
 * md_moe_cached_workspace_size.  A cache (and its slots) must be used from
 * one compute stream: the call's one synchronisation orders the copies into
 * the slots after the previous calls' reads of them only on that stream.
 * Errors: as md_moe_layer_forward, md_expert_cache_plan and
 * md_expert_cache_fill; a cache whose E / S differ from src->E / dst->E ->
 * MD_ERR_SHAPE; a copy_stream without an event -> MD_ERR_INVALID_ARG.  An
 * error after the plan (a copy or a launch that fails) marks the slots the
 * plan gave to missed experts empty, so their contents are never taken for
 * those experts (nor for the experts they held before). */
md_status md_moe_cached_workspace_size(const md_moe_layer *src /*host*/, const md_moe_layer *dst /*host*/, int32_t T,
                                       size_t *bytes /*host*/);
md_status md_moe_cached_forward(const md_moe_layer *src /*host*/, const md_moe_layer *dst /*host*/,
                                md_expert_cache *c /*host*/, const float *x, int32_t T, float *y, int32_t *idx_out,
                                float *gates_out, void *workspace, size_t workspace_bytes, hipStream_t stream,
                                hipStream_t copy_stream, hipEvent_t copy_done);

/* ---- 8-bit products --------------------------------------------------------
 * The linear layer for any number of tokens on the int8 matrices that md_qgemv
 * reads (MD_I8_ROW), with the activations rounded to 8-bit integers too:
 *     s_t  = max_c |x_tc| / 127               (fp32, correctly rounded)
 *     q_tc = x_tc / s_t to the nearest integer, ties to even (-127..127)
 *     y_tn = s_t * w_n * sum_c q_tc W_nc (+ bias_n),   w_n = row_scale[n].
 * The codes are exactly these (not off by one near a tie); the sum is exact in
 * int32, so the result does not depend on T, on the launch shape or on the
 * other tokens; the conversion, the two scale products and the bias add round
 * to fp32 once each, a bf16 y once more.  A row of zeros gives zeros (plus
 * bias); a row that holds an infinity or a NaN gets the scale NaN, and only its
 * own outputs are NaN.  md_qgemv keeps the activations in fp32 and reads the
 * same weights: it is the more exact one for up to 8 tokens.
 * T: 0..2^20 tokens (0: nothing to do); x, codes, y are dense row-major
 * T x cols, T x cols and T x rows, none overlapping another.  Errors: an
 * unknown xtype / ytype or a null pointer -> MD_ERR_INVALID_ARG; T < 0 or
 * cols <= 0 -> MD_ERR_SHAPE; T > 2^20, a width that is no multiple of 256 or
 * over 16384, a W of another type -> MD_ERR_UNSUPPORTED. */

/* The codes and scales of T rows of K values (xtype: md_xtype). */
md_status md_i8_quantize(const void *x, int32_t xtype, int32_t T, int32_t K, int8_t *codes, float *scales,
                         hipStream_t stream);
/* y from codes and scales; bias: device, W->rows fp32, or NULL; ytype: md_xtype. */
md_status md_i8_matmul(const md_qmatrix *W /*host*/, const int8_t *codes, const float *scales, int32_t T,
                       const float *bias, void *y, int32_t ytype, hipStream_t stream);
/* Both: y = W Q(x) (+ bias), the codes in the workspace (one token and some
 * small calls need none: then the size is 0 and workspace may be NULL). */
md_status md_i8_linear_workspace_size(const md_qmatrix *W /*host*/, int32_t T, size_t *bytes /*host*/);
md_status md_i8_linear(const md_qmatrix *W /*host*/, const void *x, int32_t xtype, int32_t T, const float *bias,
                       void *y, int32_t ytype, void *workspace, size_t workspace_bytes, hipStream_t stream);

/* ---- paged 8-bit cache of keys and values -----------------------------------
 * One layer's cache: n_pages pages of `page` tokens (64, 128 or 256) for
 * kv_heads heads (1..256) of head_dim channels (64, 128 or 256), as 8-bit codes
 * with one fp32 scale for each page and head; a value is scale * code.  The
 * values are held transposed (a channel's tokens together).  All device memory,
 * the caller's; nothing needs to start cleared. */
typedef struct md_kv_cache {
    int32_t n_pages, page, kv_heads, head_dim;
    int8_t *k;                 /* [n_pages][kv_heads][page][head_dim]         */
    int8_t *v;                 /* [n_pages][kv_heads][head_dim][page]         */
    float *k_scale, *v_scale;  /* [n_pages][kv_heads]                         */
} md_kv_cache;

/* A batch of sequences, each with a run of new tokens (any lengths, none
 * included).  Rows q_start[s] .. q_start[s+1]-1 of a call's tensors are
 * sequence s's new tokens; kv_len[s] is its length in the cache, for md_kv_append
 * and causal attention with those tokens counted in, so that token i of n is
 * at position kv_len[s] - n + i.  Its position p lies in page
 * table[s * table_stride + p / page].  Rows behind the last sequence are left
 * as they are.  The arrays are device memory (4-byte aligned) and are read when
 * the kernels run, so a captured graph follows their contents; what the host
 * states bounds them: a sequence with kv_len outside 0..max_kv or past its
 * table, or with more than max_q rows, is bad: the cache is neither read nor
 * written for it, and attention gives NaN for its first max_q rows.  One whose
 * q_start is not ascending within 0..rows is left out altogether.  A page
 * number outside the cache: nothing is written to it, and attention gives NaN
 * for the rows that see one of its positions. */
typedef struct md_kv_batch {
    int32_t n_seqs;            /* 1..65535                                    */
    int32_t rows;              /* rows of the call's tensors, 0..2^20         */
    int32_t max_q, max_kv;     /* bounds of the runs (to 2^20) and of kv_len (to 2^30), >= 1 */
    int32_t table_stride;      /* entries per sequence, * page >= max_kv      */
    const int32_t *q_start;    /* [n_seqs + 1]                                */
    const int32_t *kv_len;     /* [n_seqs]                                    */
    const int32_t *table;      /* [n_seqs][table_stride]                      */
} md_kv_batch;

/* Writes the new tokens' keys and values (rows x kv_heads x head_dim fp32 or
 * bf16, row strides in values, a multiple of 16 bytes) into the cache.  Keys
 * and values alike, for each page and head that new tokens reach:
 *   - where the page's first token is new, scale = max |new| / 127 over the
 *     call's tokens of that page;
 *   - else the scale stays unless max |new| / 127 is above it; then it doubles
 *     until it is not, and the held codes are halved as often, ties to even
 *     (by powers of two, so that all raises together cost a held value at most
 *     one step of the page's scale);
 *   - code = new / scale to the nearest integer, ties to even (-127..127).
 * A token's codes thus depend on which tokens of its page came before or with
 * it, not on the batch around it.  A page and head that an infinity or a NaN
 * reaches has the scale NaN until its first token is written again: the rows
 * that see one of its tokens become NaN, the others do not.  Tokens at negative
 * positions (kv_len below the run's length) are left out.  No page may be
 * written for two sequences in one call: md_kv_pages_extend gives each writer
 * its own.  Errors: as md_kv_attention's. */
md_status md_kv_append(const md_kv_cache *c /*host*/, const md_kv_batch *b /*host*/, const void *k, int64_t k_stride,
                       const void *v, int64_t v_stride, int32_t xtype, hipStream_t stream);

/* out[row] = softmax(scale * q[row] K^T + mask) V for each of q_heads heads (a
 * multiple of kv_heads, at most 1024; head h reads key head h / (q_heads /
 * kv_heads)) over the row's sequence.  causal 1: a row at position p sees
 * positions 0..p, or with window > 0 the last `window` of them (its own
 * included); causal 0: every position below kv_len, whatever the run's length
 * (an encoder's states).  A row that sees nothing gives zeros.  q, out: rows x
 * q_heads x head_dim, fp32 or bf16 (xtype, ytype), row strides in values, a
 * multiple of 16 bytes; out must not overlap q.
 * Accuracy: the cache's codes enter exactly, sums of integers are exact or in
 * fp32, and everything else is fp32.  In the form for few columns a query row (one
 * head) is rounded to integers of its largest magnitude / 8355704 (bf16 out:
 * / 32638), a softmax weight to integers of 1 / 8355711 of the largest weight
 * among its tile (the row's tokens at positions 64 n .. 64 n + 63); the weights'
 * total is taken before that.  The weights' rounding moves an output by at most
 * 4e-6 of the largest magnitude among the values that the row sees, however long
 * the context is.  In the form for many (over 64 columns, max_q * q_heads /
 * kv_heads; fp32 out of 256 channels: over 768) a query's channel and a weight
 * (times its page's value scale) are rounded to 22 bits (bf16 out: 11, and weights
 * below 2^-21 of the row's largest to steps of 2^-31 of it).  A non-finite q makes
 * its own row and head NaN; so does a page whose scale is not in 0..2^126 for the
 * rows that see it.  Scores have to stay within fp32's range: those past it give
 * NaN, or weights of 0.
 * Long sequences are split over workgroups and joined by a second kernel (few
 * columns: all tiles of a batch of up to 1024 sequences are dealt out evenly,
 * following the lengths on the device; in a larger one each sequence's heads have a
 * workgroup each, however long it is); the order of every sum is fixed, so the same
 * batch gives the same bits.
 * Errors: a null pointer, an unknown type, causal not 0 or 1, window < 0 or
 * without causal, a scale that is not finite, out == q -> MD_ERR_INVALID_ARG;
 * sizes that are not positive, a stride below its row, q_heads no multiple of
 * kv_heads, table_stride * page < max_kv -> MD_ERR_SHAPE; sizes outside the
 * sets above -> MD_ERR_UNSUPPORTED; a pointer or row stride off its alignment
 * -> MD_ERR_ALIGNMENT; a workspace below md_kv_attention_workspace_size ->
 * MD_ERR_WORKSPACE. */
md_status md_kv_attention_workspace_size(const md_kv_cache *c /*host*/, const md_kv_batch *b /*host*/, int32_t q_heads,
                                         int32_t causal, int32_t window, int32_t ytype, size_t *bytes /*host*/);
md_status md_kv_attention(const md_kv_cache *c /*host*/, const md_kv_batch *b /*host*/, const void *q, int32_t xtype,
                          int32_t q_heads, int64_t q_stride, float scale, int32_t causal, int32_t window, void *out,
                          int32_t ytype, int64_t out_stride, void *workspace, size_t workspace_bytes,
                          hipStream_t stream);

/* md_kv_attention, causal, with what a row sees set by more than its position (a
 * batch of drafts is checked in one call; a sequence of any length is read in
 * bounded time).
 *   window > 0 with sinks: the last `window` positions up to the row's own and,
 *   of those before them, the first `sinks` of the sequence.  sinks without a
 *   window change nothing: every position up to the row's own is seen.
 *   tree (device, uint64 [rows][words], 64 * words >= max_q): the run's tokens
 *   are the nodes of a tree of drafts.  Row i of a run sees the run's token j
 *   where bit j % 64 of its word j / 64 is set (its own too only then; bits
 *   past the run are not read), and every position before the run; with window
 *   > 0, of a of the run's tokens seen, the last max(window - a, 0) of those
 *   positions, and the first `sinks`.  The window takes no bit away: masks of
 *   paths that may be longer than it come from md_kv_tree_window with the same
 *   window and sinks, and a row then sees what its path gives when its tokens
 *   are decoded one by one.  NULL: no tree (words is not read).
 * A row that sees nothing gives zeros.  Everything else as md_kv_attention with
 * causal 1 (without a window a tree of one chain gives its bits, but for fp32
 * outputs of many columns of 128 channels or more, whose scores are taken in
 * other blocks, and where splits are dealt out by the lengths on the device).
 * Errors: as there; a null mask -> MD_ERR_INVALID_ARG; sinks < 0 ->
 * MD_ERR_INVALID_ARG; words < 1 or 64 * words < max_q -> MD_ERR_SHAPE; a tree
 * off 8 bytes -> MD_ERR_ALIGNMENT; words > 16384 -> MD_ERR_UNSUPPORTED. */
typedef struct md_kv_mask {
    int32_t window;            /* 0: none                                     */
    int32_t sinks;             /* first positions that stay visible           */
    int32_t words;             /* words of a row of tree                      */
    const uint64_t *tree;      /* device [rows][words], or NULL               */
} md_kv_mask;
md_status md_kv_attention_masked_workspace_size(const md_kv_cache *c /*host*/, const md_kv_batch *b /*host*/,
                                                int32_t q_heads, const md_kv_mask *mask /*host*/, int32_t ytype,
                                                size_t *bytes /*host*/);
md_status md_kv_attention_masked(const md_kv_cache *c /*host*/, const md_kv_batch *b /*host*/, const void *q,
                                 int32_t xtype, int32_t q_heads, int64_t q_stride, float scale,
                                 const md_kv_mask *mask /*host*/, void *out, int32_t ytype, int64_t out_stride,
                                 void *workspace, size_t workspace_bytes, hipStream_t stream);

/* The masks of a batch's trees of drafts from their parents: parents (device,
 * int32 [rows]) holds each token's parent, as its number within the sequence's
 * run (below the token's own), or -1 for one that follows the cached tokens
 * directly.  masks (device, uint64 [rows][words]) receives a bit for the token
 * and for each of its ancestors, positions (device, int32 [rows], may be NULL)
 * the place in the text: kv_len - n of the run's n tokens, plus the number of
 * ancestors.  A token whose chain of parents leaves the run, or does not
 * descend, gets no bits and position -1.  Runs of up to 1024 tokens.  Rows
 * behind the last sequence are left as they are, as are those of a sequence
 * whose q_start is not ascending within 0..rows; of one with more than max_q
 * rows the first max_q are written.  Only q_start and kv_len of the batch are
 * read.  Errors: as md_kv_append's for the batch; max_q > 1024 ->
 * MD_ERR_UNSUPPORTED; 64 * words < max_q -> MD_ERR_SHAPE. */
md_status md_kv_tree(const md_kv_batch *b /*host*/, const int32_t *parents, uint64_t *masks, int32_t words,
                     int32_t *positions, hipStream_t stream);

/* md_kv_tree for a sliding window: of a token and its ancestors only the last
 * `window` (0: all of them) have bits, and those whose place in the text is
 * among the first `sinks`.  Beside the same window and sinks in
 * md_kv_attention_masked a row sees, of its path through cache and run, exactly
 * the last `window` tokens up to its own and the first `sinks`.  positions as
 * there.  Errors: as there; a negative window or sinks -> MD_ERR_INVALID_ARG. */
md_status md_kv_tree_window(const md_kv_batch *b /*host*/, const int32_t *parents, int32_t window, int32_t sinks,
                            uint64_t *masks, int32_t words, int32_t *positions, hipStream_t stream);

/* The values that n pages hold (pages: device, n int32): k and v as
 * [n][kv_heads][page][head_dim] in ytype, both with the token before the
 * channel.  Slots that no token has reached give what their codes stand for; a
 * page number outside the cache gives NaN.  n: 0 (nothing to do) .. 2^24 - 1. */
md_status md_kv_read_pages(const md_kv_cache *c /*host*/, const int32_t *pages, int32_t n, void *k, void *v,
                           int32_t ytype, hipStream_t stream);

/* Copies pages, codes and scales: page dst[i] becomes page src[i] for every
 * i < n (src, dst: host arrays, read before the call returns).  The copies run
 * side by side, so a page that is written may appear only once among all src
 * and dst -> MD_ERR_INVALID_ARG, as for a number outside the cache.  One launch
 * for every 448 pairs, the pairs in its arguments: a captured graph keeps
 * them.  n = 0: nothing to do. */
md_status md_kv_copy_pages(const md_kv_cache *c /*host*/, const int32_t *src /*host*/, const int32_t *dst /*host*/,
                           int32_t n, hipStream_t stream);

/* Which pages are in use, and by how many sequences (host state; the layers
 * of a model that share their tables share one).  The caller owns the arrays
 * and keeps each sequence's table (page numbers, ceil(length / page) of them)
 * and length.  Not thread-safe. */
typedef struct md_kv_pages {
    int32_t n_pages, page;
    int32_t *refs;             /* [n_pages]: tables that name the page        */
    int32_t *free_pages;       /* [n_pages]: the free ones, a heap            */
    int32_t n_free;
} md_kv_pages;

/* Every page free. */
md_status md_kv_pages_reset(md_kv_pages *p /*host*/);

/* Makes positions len .. new_len-1 of a sequence writable: new pages for what
 * lies past its last one, lowest number first, and where len ends inside a page
 * that another table names too, a page of its own in that one's place, which
 * the caller fills with md_kv_copy_pages (in every layer) before it appends:
 * copy_src[0] -> copy_dst[0] and *n_copy = 1, else *n_copy = 0.
 * Errors: too few free pages -> MD_ERR_UNSUPPORTED; lengths that shrink or a
 * table too short -> MD_ERR_SHAPE; an entry that names no page in use ->
 * MD_ERR_INVALID_ARG; nothing changes on error (all md_kv_pages_* calls). */
md_status md_kv_pages_extend(md_kv_pages *p /*host*/, int32_t *table /*host*/, int32_t capacity, int32_t len,
                             int32_t new_len, int32_t *copy_src /*host*/, int32_t *copy_dst /*host*/,
                             int32_t *n_copy /*host*/);

/* A second sequence with the first `len` positions of this one: its table
 * names the same pages. */
md_status md_kv_pages_fork(md_kv_pages *p /*host*/, const int32_t *table /*host*/, int32_t len,
                           int32_t *new_table /*host*/, int32_t capacity);

/* Gives up the pages of a sequence past new_len (0: all of them; a draft's
 * rejected tokens: those behind the accepted ones).  A page is free when no
 * table names it any more. */
md_status md_kv_pages_truncate(md_kv_pages *p /*host*/, const int32_t *table /*host*/, int32_t len, int32_t new_len);

/* Moves the used pages to the lowest numbers: the tables (n_seqs rows of
 * table_stride entries, every sequence that holds pages among them) are
 * rewritten, and the caller copies copy_src[i] -> copy_dst[i], i < *n_copy, with
 * md_kv_copy_pages (in every layer) before the next use.  The copy arrays hold
 * n_pages entries.  Errors: a page that the tables do not name as often as it
 * is held -> MD_ERR_INVALID_ARG. */
md_status md_kv_pages_compact(md_kv_pages *p /*host*/, int32_t *tables /*host*/, int32_t table_stride,
                              const int32_t *lens /*host*/, int32_t n_seqs, int32_t *copy_src /*host*/,
                              int32_t *copy_dst /*host*/, int32_t *n_copy /*host*/);

/* ---- around the attention and the experts -------------------------------- */

/* Norms of queries and keys for each head, and their rotation by position, in
 * one pass (before md_kv_append and md_kv_attention).  For each row and head
 *     z = x / sqrt(mean_c x_c^2 + eps) * weight        (no weight: z = x)
 *     y = z, but for the pairs (a, b) of its first `rot` channels:
 *     y_a = f (z_a cos t - z_b sin t),   y_b = f (z_b cos t + z_a sin t),
 *     t = positions[row] * inv_freq[p] of pair p,  f = factor,
 * p pairing channel p with p + rot / 2, or with `interleaved` 2 p with 2 p + 1.
 * x and y are fp32 or bf16 (xtype, ytype); sums and products are fp32, the
 * angle and what is left of it after whole turns fp64, so that far positions
 * keep their accuracy.  head_dim: a multiple of 8 up to 256; rot: a multiple of
 * 8, 0..head_dim.  q: rows x q_heads x head_dim, row strides in values, a
 * multiple of 16 bytes; k likewise, or k_heads 0 (k is not read then).  An
 * output may be its input (same address, type and row stride); otherwise
 * nothing may overlap.  rows: 0..2^20 (0: nothing to do).  An infinity or a NaN
 * reaches the outputs of its own row and head only.  Errors: a null pointer, an
 * unknown type, a factor or eps that is not finite, eps < 0 ->
 * MD_ERR_INVALID_ARG; rows, heads or a head_dim that are not positive, rot outside 0..head_dim,
 * a stride below its row -> MD_ERR_SHAPE; sizes outside the sets, more than
 * 1024 heads of either -> MD_ERR_UNSUPPORTED; a pointer or row stride off 16
 * bytes (positions: 4) -> MD_ERR_ALIGNMENT. */
typedef struct md_rope {
    int32_t head_dim, rot;
    int32_t interleaved;       /* 0: channel p with p + rot / 2; 1: 2 p with 2 p + 1 */
    const float *inv_freq;     /* device [rot / 2]                            */
    float factor;              /* 1 for none                                  */
    float eps;
    const float *q_weight;     /* device [head_dim], or NULL: no norm         */
    const float *k_weight;
} md_rope;
md_status md_qk_norm_rope(const md_rope *r /*host*/, const int32_t *positions, int32_t rows, const void *q,
                          int32_t q_heads, int64_t q_stride, const void *k, int32_t k_heads, int64_t k_stride,
                          int32_t xtype, void *q_out, int64_t q_out_stride, void *k_out, int64_t k_out_stride,
                          int32_t ytype, hipStream_t stream);

/* Routing to experts for any number of tokens (idx and gates as
 * md_moe_experts_forward takes them, 128 tokens a call there):
 *     l_e = sum_c W_r[e][c] x[c] (+ router_bias[e]), in fp64, rounded once to fp32
 *     s_e = 1 / (1 + exp(-l_e)), or exp(l_e) / sum_i exp(l_i)
 *     c_e = s_e + balance_e            (what chooses; balance NULL: s_e)
 * With groups > 1 the E experts are `groups` equal runs; a run's value is its
 * largest c (best_two: the sum of its two largest), and only the experts of the
 * groups_kept runs of the largest values may be chosen.  idx: the k largest c in
 * descending order, gates: their s (not c), with renorm divided by the chosen
 * ones' sum (a sum of 0 gives gates of 0), times scale.  Equal values go to the
 * lower run and expert.  Scores, values and gates are fp64 until a gate is rounded
 * to fp32, so that the choice is the definition's.  Where that pays (from some 2
 * Gflop of products on) a call that asks for no logits forms them on the fp16 matrix
 * cores first, off by at most 6.25 2^-23 |x| |w| (fp32 x: 9.25; the norms of the token
 * and of the longest row of W_r; an instruction there is taken to be off by 2^-23 of
 * its sum), and does in fp64 only the tokens whose choice that leaves open: the
 * choice is the definition's there too, and a gate is off by what its logits' bound
 * allows, relatively by at most 4.1 times it and never by more than 2^-7.9, since a
 * token whose bound passes 2^-10 is done in fp64 (measured: 1e-7).  The same token's
 * gates may differ by that between a long call and a short one; a call that asks for
 * the logits has them all in fp64.
 * x: T x H fp32 or bf16; logits (T x E fp32, may be NULL).  T: 0..2^20 (0: nothing
 * to do); H, E, k as md_moe_route_topk; groups: up to 64.  A NaN is the smallest of
 * all (as -inf is, which closes an expert in balance); idx then still names k
 * different experts of the kept runs.  The workspace's size covers either type of
 * x, with the logits or without.  Errors: null
 * pointers, unknown xtype or score, a flag that is not 0 or 1, a scale that is
 * not finite -> MD_ERR_INVALID_ARG; T < 0, k > E, groups that do not divide E,
 * groups_kept outside 1..groups, fewer experts in them than k, best_two with runs of one
 * expert -> MD_ERR_SHAPE; sizes outside the sets -> MD_ERR_UNSUPPORTED; pointers
 * off 16 bytes -> MD_ERR_ALIGNMENT; the workspace -> MD_ERR_WORKSPACE. */
typedef enum md_score { MD_SCORE_SOFTMAX = 0, MD_SCORE_SIGMOID = 1 } md_score;
typedef struct md_routing {
    int32_t k;
    int32_t score;             /* md_score                                    */
    int32_t groups, groups_kept, best_two;
    int32_t renorm;
    float scale;
    const float *balance;      /* device [E], or NULL                         */
} md_routing;
md_status md_moe_route_workspace_size(int32_t T, int32_t H, int32_t E, size_t *bytes /*host*/);
md_status md_moe_route(const md_routing *r /*host*/, const void *x, int32_t xtype, int32_t T, int32_t H,
                       const float *W_r, const float *router_bias, int32_t E, int32_t *idx, float *gates, float *logits,
                       void *workspace, size_t workspace_bytes, hipStream_t stream);

/* The layer forward with such a routing in place of the layer's own top-k
 * (W_r and router_bias are the layer's; routing->k = L->k): md_moe_route, then
 * md_moe_experts_forward.  T, y, idx_out, gates_out as md_moe_layer_forward. */
md_status md_moe_routed_workspace_size(const md_moe_layer *L /*host*/, int32_t T, size_t *bytes /*host*/);
md_status md_moe_layer_forward_routed(const md_moe_layer *L /*host*/, const md_routing *routing /*host*/, const float *x,
                                      int32_t T, float *y, int32_t *idx_out, float *gates_out, void *workspace,
                                      size_t workspace_bytes, hipStream_t stream);

/* Log probabilities from rows of logits: with z_v = scale * logits[row][v] and
 * Z = sum_v exp(z_v),
 *     logprobs[row][i] = z_t - log Z,  t = tokens[row][i]      (n_tokens of them)
 *     entropy[row]     = log Z - sum_v z_v exp(z_v) / Z
 *     top_ids[row][j], top_logprobs[row][j]: the `top` largest logits in
 *     descending order (equal ones: the lower id first), and z - log Z of each.
 * logits: rows x vocab fp32 or bf16, any row stride (in values) from vocab on;
 * rows may begin at any value (an odd vocabulary).  A logit of -inf has
 * probability 0 and adds nothing to the entropy.  A row with a NaN or +inf, or
 * of -inf alone, has NaN in all its values; top_ids then still are the order's,
 * a NaN taken as the smallest.  A token outside 0..vocab-1 gives NaN.  Sums of a
 * row's parts are fp32, their joins fp64.
 * rows: 0..2^20 (0: nothing to do), vocab: 1..2^20, n_tokens: 0..64, top: 0..32,
 * at most vocab.  tokens, logprobs: [rows][n_tokens], entropy: [rows] or NULL,
 * top_ids, top_logprobs: [rows][top]; those of n_tokens or top 0 are not read.
 * Errors: null pointers, an unknown type, a scale that is not above 0 and up to
 * 2^64 -> MD_ERR_INVALID_ARG; negative sizes, top > vocab, a stride below
 * vocab -> MD_ERR_SHAPE; sizes past the above -> MD_ERR_UNSUPPORTED; logits off
 * their own size, the others off 4 bytes (workspace: 16) -> MD_ERR_ALIGNMENT;
 * the workspace -> MD_ERR_WORKSPACE. */
md_status md_token_logprobs_workspace_size(int32_t rows, int32_t vocab, int32_t top, size_t *bytes /*host*/);
md_status md_token_logprobs(const void *logits, int32_t xtype, int64_t stride, int32_t rows, int32_t vocab,
                            const int32_t *tokens, int32_t n_tokens, float scale, int32_t top, float *logprobs,
                            float *entropy, int32_t *top_ids, float *top_logprobs, void *workspace,
                            size_t workspace_bytes, hipStream_t stream);

/* Measurement aid: reads nbytes of device memory at src once, in address
 * order, with every compute unit busy, and writes nothing unless some lane's
 * xor of the 32-bit words it read equals key (then that lane stores key at
 * sink[0]; for zeroed memory any nonzero key keeps sink untouched).  Timed over a buffer far larger than the caches it gives the HBM
 * read bandwidth this device attains, the practical ceiling of the weight
 * streams above (the Camelid README, "Gemma 4": GPU-resident decode runs at
 * the memory-bandwidth wall).  workgroups: the grid (0 picks 2048; at most
 * one workgroup per 32 KB tile is launched); each workgroup takes its tiles
 * in groups of up to four consecutive ones, every load of a group in flight
 * before any is used.
 * Errors: null pointer -> MD_ERR_INVALID_ARG; nbytes 0 or not a multiple of
 * 16 -> MD_ERR_SHAPE; src not 16-byte aligned -> MD_ERR_ALIGNMENT;
 * workgroups < 0 or > 2^20 -> MD_ERR_INVALID_ARG. */
md_status md_hbm_read_probe(const void *src, size_t nbytes, uint32_t key, uint32_t *sink, int32_t workgroups,
                            hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif

/*
 * moe_decode.h -- C ABI of the decode-time quantized-expert MoE block for
 * AMD Instinct MI355X (gfx950).
 *
 * One decode step of one MoE layer is three calls on one HIP stream:
 *
 *   moe_route_topk   router: top-k experts per token and their weights
 *   moe_expert_plan  cohort plan: slots grouped by expert, distinct experts
 *   moe_decode_step  expert block: fused gate+up, SiLU*up, down projection,
 *                    weighted combine over k per token
 *
 * The pages this follows describe the problem, not an API: a router yields
 * per-token (expert, score) slots and is one named part of the decode cost
 * next to the expert gather and the combine (page "perf(moe): attribute the
 * MoE decode gap at the M = 1 expert gather", Proposed Solution, step 2);
 * routed experts are gathered once per (token, k) slot at M = 1 (same page,
 * Problem / Background); page "perf(moe): batched decode scales 1.55x
 * against 3.25x on dense" proposes a token dimension with a sum over k per
 * token and deduplicating expert ids across the cohort so that each expert
 * plane is read once per step (Proposed Solution), keeps n_tokens a runtime
 * extent that must not re-specialise kernels, asks that unsupported
 * configurations decline rather than fail, and that shapes be validated
 * before dispatch (Implementation Notes).
 *
 * Conventions for every entry point:
 *   - Every array pointer is a DEVICE pointer unless stated otherwise; the
 *     caller owns all memory.  The library allocates nothing and keeps no
 *     per-call state.
 *   - Calls are asynchronous on `hip_stream` (a hipStream_t; NULL = the
 *     default stream).  No call synchronises the host with the device.
 *   - Arguments are validated on the host before anything is enqueued.  A
 *     bad argument returns MOE_ERR_INVALID_ARG, a shape or mode with no
 *     kernel returns MOE_ERR_UNSUPPORTED (the caller falls back), a short
 *     workspace returns MOE_ERR_WORKSPACE; nothing aborts.  A failed launch
 *     returns MOE_ERR_DEVICE.
 *   - Expert ids inside device arrays cannot be checked on the host.  The
 *     kernels never read or write out of bounds on a bad id: the planner
 *     leaves such slots out of every list and the combine writes NaN for
 *     a token that holds one.
 */
#ifndef MOE_DECODE_H
#define MOE_DECODE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MOE_OK = 0,
    MOE_ERR_INVALID_ARG = 1,
    MOE_ERR_UNSUPPORTED = 2,
    MOE_ERR_WORKSPACE = 3,
    MOE_ERR_DEVICE = 4
} moe_status;

/* MOE_DTYPE_F16 is a type of the unquantised products (moe_linear_t), of
 * moe_combine, of the scored router and of the integer products; the quantised layer and
 * the router projection refuse it.  MOE_DTYPE_I8 is a type of x of the integer
 * products (moe_matmul_int, moe_grouped_matmul_int) only. */
typedef enum { MOE_DTYPE_F32 = 0, MOE_DTYPE_BF16 = 1, MOE_DTYPE_F16 = 2, MOE_DTYPE_I8 = 3 } moe_dtype;

/* Storage of the down projection (see moe_layer_t and moe_pack_down). */
typedef enum { MOE_DOWN_ROWS = 0, MOE_DOWN_COLS = 1 } moe_down_layout;

/* Gated activation of the expert MLP (see moe_layer_t). */
typedef enum { MOE_ACT_SWIGLU = 0, MOE_ACT_GEGLU = 1 } moe_activation;

/* Limits enforced by validation. */
#define MOE_MAX_EXPERTS 1024
#define MOE_MAX_TOP_K 16
/* Tokens per call of the expert entry points (one row of combine
 * workgroups per token). */
#define MOE_MAX_TOKENS 65535

/*
 * One MoE layer: stacked expert weights, affine, groups along the input
 * dimension ("4-bit group 64" checkpoints; page "perf(moe): batched decode
 * scales 1.55x against 3.25x on dense", Current Behavior).
 *
 *   w = scale * q + bias,  q in 0 .. 2^bits - 1
 *
 * `bits` (gate and up) and `down_bits` (down) are 4, 6 or 8, `group_size`
 * (all three) 32, 64 or 128: the fused kernel is templated on bits and
 * group size, and 4-bit gate/up with 6-bit down must keep working (same
 * page, Implementation Notes).  A weight matrix is stored as
 * [expert][out][in*bits/32] uint32 words, each row a little-endian bit
 * stream: element c sits in stream bits c*bits .. c*bits+bits-1, stream bit
 * j being bit j % 32 of word j / 32 (at 4 bits: element 8*w+i in nibble i
 * of word w, lowest nibble first).  Scales and biases are fp16 bit
 * patterns, [expert][out][in/group_size].
 *   gate, up : out = dff,    in = hidden
 *   down     : out = hidden, in = dff
 * Each projection picks its kernels by its own width: 4-bit gate and up in
 * groups of 64 run the specialised gate+up kernels (MFMA for large
 * batches), 4-bit down in groups of 64 the specialised down kernels (either
 * down layout); a projection of any other width or group size runs the
 * generic row kernels, and a down projection on them needs MOE_DOWN_ROWS.
 * Every `*_q` pointer must be 16-byte aligned, every scale/bias pointer
 * 4-byte aligned.  The struct itself lives in host memory; the pointers it
 * holds are device pointers.
 *
 * `down_layout` selects how the down projection is stored:
 *   MOE_DOWN_ROWS  as above: down_q [E][hidden][dff/8], scales [E][hidden][dff/64]
 *   MOE_DOWN_COLS  the same bytes regrouped by moe_pack_down so that one
 *                  16-byte chunk (32 consecutive dff inputs) of 64
 *                  consecutive hidden rows is contiguous:
 *                  down_q [E][dff/32][hidden] 16-byte chunks,
 *                  scales and biases [E][dff/64][hidden].
 *                  Needs hidden % 64 == 0 and dff % 128 == 0.
 *
 * `expert_scale` (optional, NULL = none) is one fp32 factor per expert that
 * multiplies the gate and up pre-activations (the expert-scale sidecars of
 * page "perf(moe): attribute ...", Problem / Background).  `clamp_limit`
 * (0 = none) clips gate and up pre-activations to [-L, L] after the sidecar
 * and before SiLU*up (the clamp stage named on the same page).
 *
 * `activation` is MOE_ACT_SWIGLU (h = silu(g) * u) or MOE_ACT_GEGLU
 * (h = gelu(g) * u with the tanh form 0.5 g (1 + tanh(sqrt(2/pi)
 * (g + 0.044715 g^3)))), the GeGLU variant of the fused kernel that page
 * "perf(moe): batched decode scales 1.55x against 3.25x on dense" lists
 * among its kernels (Implementation Notes); the pages give no GELU formula,
 * the tanh form is the one of the gemma checkpoints that kernel serves.
 * `down_scale` (optional, NULL = none) is one fp32 factor per expert that
 * multiplies that expert's down-projection output y before the weighted
 * combine: the second of the "both sidecars" that page "perf(moe):
 * attribute ..." names (Problem / Background), which it does not define
 * further.
 *
 * Field order: the fields through expert_scale are those of the plain
 * 4-bit layer, in that order; the extensions follow, and all-zero
 * extensions mean the plain layer (rows-layout down, no down scale,
 * SwiGLU, down projection as wide as gate and up), so a caller that only
 * knows the plain fields and zero-fills the rest gets the plain layer.
 */
typedef struct {
    int32_t hidden;      /* H, multiple of 64 */
    int32_t dff;         /* expert intermediate size F, multiple of 64 */
    int32_t n_experts;   /* E, 1..MOE_MAX_EXPERTS */
    int32_t top_k;       /* k, 1..min(E, MOE_MAX_TOP_K) */
    int32_t bits;        /* 4, 6 or 8 (gate and up) */
    int32_t group_size;  /* 32, 64 or 128; divides hidden and dff */
    int32_t act_dtype;   /* moe_dtype of x, residual and out (int32, as wide as
                            the enum, so that any value is defined to read) */
    float clamp_limit;   /* >= 0; 0 disables the clamp */
    const uint32_t *gate_q, *up_q;
    const uint16_t *gate_s, *gate_b, *up_s, *up_b;
    const uint32_t *down_q;
    const uint16_t *down_s, *down_b;
    const float *expert_scale; /* [E] or NULL */
    /* extensions; zero = the plain layer */
    int32_t down_layout;       /* moe_down_layout */
    const float *down_scale;   /* [E] or NULL */
    int32_t activation;        /* moe_activation */
    int32_t down_bits;         /* 4, 6 or 8 (down projection); 0 = bits */
} moe_layer_t;

/*
 * Cohort plan of one step (all device arrays, int32, caller-allocated):
 *   counts[E]            slots routed to each expert
 *   offsets[E+1]         exclusive prefix sum of counts
 *   sorted_slots[B*k]    slot ids s = t*k + j grouped by expert, ascending
 *                        expert, ascending slot within an expert
 *   unique_experts[E]    distinct experts in ascending order, -1 after
 *   n_unique[1]          number of distinct experts
 *   work[E][4]           one 16-byte record per distinct expert u, in the
 *                        order of unique_experts: {expert, offsets[expert],
 *                        counts[expert], first slot of that expert}; after
 *                        the last distinct expert {-1, B*k, 0, 0}.  The
 *                        expert kernels read only this record before they
 *                        stream an expert's weights.  16-byte aligned.
 *                        Appended after the five plain arrays; it is
 *                        required (a plan without it is refused with
 *                        MOE_ERR_INVALID_ARG).
 */
typedef struct {
    int32_t *counts, *offsets, *sorted_slots, *unique_experts, *n_unique;
    int32_t *work;
} moe_plan_t;

/*
 * Router.  logits fp32 [n_tokens][n_experts] (finite) -> topk_idx int32
 * [n_tokens][top_k] in descending logit order, ties to the lower expert
 * id, and topk_w fp32 [n_tokens][top_k], the softmax of the kept logits
 * (equal to softmax over all experts, top-k, renormalise).
 * n_tokens == 0 returns MOE_OK without a launch.
 */
moe_status moe_route_topk(const float *logits, int32_t n_tokens, int32_t n_experts,
                          int32_t top_k, int32_t *topk_idx, float *topk_w,
                          void *hip_stream);

/*
 * Cohort planner: a stable counting sort of the n_tokens*top_k slots by
 * expert id and the list of distinct experts, so that each expert's
 * weights are streamed once per step for all the tokens routed to it.
 * Reads topk_idx int32 [n_tokens][top_k]; writes every array of `plan`
 * (a host struct of device pointers).  n_tokens == 0 writes an empty plan.
 */
moe_status moe_expert_plan(const int32_t *topk_idx, int32_t n_tokens, int32_t n_experts,
                           int32_t top_k, const moe_plan_t *plan, void *hip_stream);

/*
 * Router and planner of one step in a single launch (one workgroup, one
 * wave per token) when n_tokens <= 16; larger batches run the two kernels of
 * moe_route_topk and moe_expert_plan.  Same arguments and results as those
 * two calls.
 */
moe_status moe_route_plan(const float *logits, int32_t n_tokens, int32_t n_experts, int32_t top_k,
                          int32_t *topk_idx, float *topk_w, const moe_plan_t *plan,
                          void *hip_stream);

/*
 * Router projection, the step in front of the router: logits[t][e] =
 * sum_h x[t][h] * w_router[e][h] (the pages name the router as one of the
 * per-token decode costs: page "perf(moe): attribute the MoE decode gap at
 * the M = 1 expert gather", Proposed Solution step 2).
 *   x         [n_tokens][hidden], act_dtype (bf16 or fp32), 16-byte aligned
 *   w_router  bf16 bits [n_experts][hidden], 16-byte aligned
 *   logits    fp32 [n_tokens][n_experts], the router's input
 * Products exact, fp32 accumulation in a fixed order (a token's logits do
 * not depend on the rest of the batch).  MOE_ERR_UNSUPPORTED when hidden has
 * no lane geometry (hidden/8 must be a power of two up to 64 times 1..8),
 * n_experts > MOE_MAX_EXPERTS or n_tokens > MOE_MAX_TOKENS; n_tokens == 0
 * launches nothing.  Asynchronous on hip_stream.
 */
moe_status moe_router_logits(const void *x, int32_t n_tokens, int32_t hidden, moe_dtype act_dtype,
                             const uint16_t *w_router, int32_t n_experts, float *logits, void *hip_stream);

/* Bytes of device workspace moe_decode_step needs for up to max_tokens
 * tokens of this layer's shape (0 if the layer is invalid). */
size_t moe_workspace_size(const moe_layer_t *layer, int32_t max_tokens);

/*
 * Expert block of one step.
 *   x         [n_tokens][hidden], act_dtype
 *   topk_idx  int32 [n_tokens][top_k], topk_w fp32 [n_tokens][top_k]
 *   plan      the plan of topk_idx (host struct of device pointers)
 *   out       [n_tokens][hidden] act_dtype; must not alias x
 *   workspace device memory of at least moe_workspace_size(layer, n_tokens)
 *             bytes, 256-byte aligned; its contents need no initialisation
 *
 *   g = Wg[e] x_t, u = Wu[e] x_t   (fp32 accumulation)
 *   g, u *= expert_scale[e]        (if given)
 *   g, u = clip(g, u, -L, L)       (if clamp_limit > 0)
 *   h = silu(g) * u                (gelu(g) * u for MOE_ACT_GEGLU;
 *                                   fp32, never rounded)
 *   y = Wd[e] h                    (fp32)
 *   y *= down_scale[e]             (if given)
 *   o_t = sum_{j<k} topk_w[t][j] * y_{t,j}, in j order, rounded once to
 *         act_dtype (round to nearest even)
 *   out_t = o_t
 *
 * The fp32 partials with one final rounding follow page "perf(moe):
 * batched decode scales 1.55x against 3.25x on dense", Implementation
 * Notes.  Repeated calls are bitwise equal.  Batch invariance: below 16
 * tokens a token's result depends only on that token (bitwise the same
 * whatever else is in the batch).  From 16 tokens up, an expert that holds
 * 3 or more of the batch's tokens runs on the MFMA kernels, and from 128
 * tokens up every expert runs on the MFMA tile kernels; they add the same
 * exact fp32 products in another order, so a token routed to such an
 * expert may differ from its single-token result by fp32 rounding only
 * (relative L2 within 5e-4 of each other, both within the output
 * tolerance of the fp64 definition).  Between 16 and 127 tokens, tokens
 * whose experts all hold fewer than 3 tokens stay bitwise equal.
 */
moe_status moe_decode_step(const moe_layer_t *layer, const void *x, int32_t n_tokens,
                           const int32_t *topk_idx, const float *topk_w, const moe_plan_t *plan,
                           void *out, void *workspace, size_t workspace_bytes, void *hip_stream);

/*
 * moe_decode_step with the residual add of a layer stack fused into the
 * combine's store: out_t = act(residual_t + act(o_t)), i.e. the block's
 * output rounded to act_dtype as moe_decode_step stores it, added to the
 * residual in fp32 and rounded again (the layer stack runs every MoE
 * layer on every decode tick, page "perf(moe):
 * attribute the MoE decode gap at the M = 1 expert gather", Problem /
 * Background).  residual is [n_tokens][hidden] act_dtype or NULL (then
 * exactly moe_decode_step); out must not alias x or residual.
 */
moe_status moe_decode_step_residual(const moe_layer_t *layer, const void *x, int32_t n_tokens,
                                    const int32_t *topk_idx, const float *topk_w,
                                    const moe_plan_t *plan, const void *residual, void *out,
                                    void *workspace, size_t workspace_bytes, void *hip_stream);

/*
 * One layer step from router logits: moe_route_plan, then moe_decode_step,
 * with the same checks and results; topk_idx, topk_w and the plan are
 * outputs here (the plan as moe_route_plan writes it).
 *   logits  fp32 [n_tokens][n_experts], device
 * The pages split a decoded token's MoE time into router, expert GEMV and
 * combine (page "perf(moe): attribute the MoE decode gap at the M = 1
 * expert gather", Proposed Solution); at a few tokens each of those is a
 * short, latency-bound kernel.  So a batch of up to 8 tokens (with at most
 * 256 experts and n_tokens * top_k <= 64) takes two launches
 * instead of three or more: the gate+up workgroups select their own expert
 * from the logits and, with more than one token, deduplicate among
 * themselves so each distinct expert's gate and up rows are streamed once
 * for every token routed to it (one block also writes topk_idx, topk_w and
 * the plan); then one kernel does the down projection and the combine,
 * token by token.  Results are bitwise those of the longer path.
 */
moe_status moe_decode_layer(const moe_layer_t *layer, const float *logits, const void *x,
                            int32_t n_tokens, int32_t *topk_idx, float *topk_w,
                            const moe_plan_t *plan, const void *residual, void *out,
                            void *workspace, size_t workspace_bytes, void *hip_stream);

/*
 * The first half of moe_decode_layer: routes, plans and writes h into the
 * workspace (one launch for up to 8 tokens, else moe_route_plan and the
 * gate+up kernels); moe_expert_down_combine with the same workspace, plan,
 * topk_idx and topk_w is the second half.  Same checks as moe_decode_layer
 * (out and residual aside).
 */
moe_status moe_route_gate_up(const moe_layer_t *layer, const float *logits, const void *x,
                             int32_t n_tokens, int32_t *topk_idx, float *topk_w,
                             const moe_plan_t *plan, void *workspace, size_t workspace_bytes,
                             void *hip_stream);

/*
 * The two halves of moe_decode_step, for callers that instrument or overlap
 * the stages (the pages' fused decode kernel is likewise a gate/up kernel
 * followed by a down kernel: page "perf(moe): batched decode scales 1.55x
 * against 3.25x on dense", Current Behavior).  Same arguments, checks and
 * results as moe_decode_step; enqueue moe_expert_gate_up first, then
 * moe_expert_down_combine with the same workspace, on one stream.
 *   moe_expert_gate_up       writes h = silu(g) * u per slot into the workspace
 *   moe_expert_down_combine  reads h, writes out
 */
moe_status moe_expert_gate_up(const moe_layer_t *layer, const void *x, int32_t n_tokens,
                              const moe_plan_t *plan, void *workspace, size_t workspace_bytes,
                              void *hip_stream);
moe_status moe_expert_down_combine(const moe_layer_t *layer, int32_t n_tokens,
                                   const int32_t *topk_idx, const float *topk_w,
                                   const moe_plan_t *plan, const void *residual, void *out,
                                   void *workspace, size_t workspace_bytes, void *hip_stream);

/*
 * moe_decode_layer for callers that cannot allocate device memory: code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc.  Same arguments, checks and results as moe_decode_layer
 * (bitwise), without the workspace: the h and y intermediates live in a
 * device array of MOE_STATIC_SCRATCH_BYTES that the library reserves per
 * GPU when it is loaded and holds until the process ends.
 *   - MOE_ERR_WORKSPACE when moe_workspace_size(layer, n_tokens) exceeds
 *     MOE_STATIC_SCRATCH_BYTES (8 MiB: up to 93 tokens of the 2048 x 768
 *     top-8 layer).
 *   - hip_stream must belong to the current device (else
 *     MOE_ERR_INVALID_ARG).  The first call on a device looks up the
 *     array's device address; make that call outside graph capture.
 *   - Every call on one GPU shares that GPU's array, which keeps the last
 *     call's contents (nothing in it needs clearing: each step writes h
 *     and y before reading them).  Calls that may overlap on one GPU (other
 *     streams, other host threads) race on it: serialise them.
 * Calls no hipMalloc, hipFree or other allocating routine.
 */
#define MOE_STATIC_SCRATCH_BYTES ((size_t)8 << 20)
moe_status moe_decode_layer_static(const moe_layer_t *layer, const float *logits, const void *x,
                                   int32_t n_tokens, int32_t *topk_idx, float *topk_w,
                                   const moe_plan_t *plan, const void *residual, void *out,
                                   void *hip_stream);

/*
 * Regroup a layer's down projection from MOE_DOWN_ROWS (as stored by the
 * pages' 4-bit checkpoints) to MOE_DOWN_COLS, the layout the decode kernels
 * read fastest: a wave then reads 64 consecutive output rows with one
 * coalesced 1 KiB load per 32 inputs.  A one-time, load-time step; pure byte
 * movement, nothing is re-quantised.  `layer` describes the source
 * (down_layout must be MOE_DOWN_ROWS; 4-bit weights in groups of 64 only,
 * other formats return MOE_ERR_UNSUPPORTED); dst_q (16-byte aligned, E*hidden*dff/2
 * bytes), dst_s and dst_b (E*hidden*dff/64 fp16 each) are device buffers that
 * must not overlap the source.  Asynchronous on hip_stream.
 */
moe_status moe_pack_down(const moe_layer_t *layer, uint32_t *dst_q, uint16_t *dst_s, uint16_t *dst_b,
                         void *hip_stream);

/* Host-only check of a layer descriptor (no device access):
 * MOE_OK, MOE_ERR_INVALID_ARG or MOE_ERR_UNSUPPORTED. */
moe_status moe_layer_check(const moe_layer_t *layer);

/* ------------------------------------------------- unquantised products
 *
 * The layers beside the 4-bit experts: a shared expert or a dense projection
 * kept in bf16 or fp16, experts that are not quantised at all, and a
 * model's small fp32 layers.  moe_matmul is one product with its epilogue,
 * moe_grouped_matmul the same product per expert over a planned batch, and
 * moe_combine the weighted sum over k per token that follows it.  An
 * unquantised expert block is moe_route_plan, two moe_grouped_matmul calls
 * (gated gate+up, then down into fp32 rows) and moe_combine, the same
 * three-part split of router, expert products and combine as the quantised
 * block (page "perf(moe): attribute the MoE decode gap at the M = 1 expert
 * gather", Proposed Solution step 2).
 */

/* f of the epilogue; z is the fp32 sum x.w plus bias.  Factors of z below the smallest
 * normal fp32 value (a SiLU of z < -87.3) may count as zero. */
typedef enum {
    MOE_FN_NONE = 0,
    MOE_FN_RELU = 1,      /* max(z, 0), NaN kept */
    MOE_FN_SILU = 2,      /* z / (1 + exp(-z)) */
    MOE_FN_GELU = 3,      /* z Phi(z), Phi the normal distribution function */
    MOE_FN_GELU_TANH = 4  /* 0.5 z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) */
} moe_fn;

/* How moe_grouped_matmul finds the rows of x and out for the i-th entry of
 * the plan's sorted_slots, slot s = sorted_slots[i]. */
typedef enum {
    MOE_ROWS_TOKEN = 0, /* x row s / top_k (one per token), out row s */
    MOE_ROWS_SLOT = 1,  /* x row s, out row s */
    MOE_ROWS_SORTED = 2 /* x row i, out row i: rows already grouped by expert */
} moe_rows;

/*
 * Weights of a product, in host memory, its pointers device pointers:
 *   w        [n_groups][out_features][in_features], dtype
 *   w_up     NULL, or a second stack of the same layout: the product is
 *            then gated, out = f(z) * z_up
 *   bias     NULL, or [n_groups][out_features], dtype, added to z
 *   bias_up  the same for z_up: given exactly when bias and w_up are
 * Strides are in elements; 0 means packed.  Rows of w (and w_up) lie
 * row_stride apart, matrices group_stride, rows of bias (and bias_up)
 * bias_stride, so gate and up may be the two halves of one stack.
 * clamp_limit (0 = none) clips z and z_up to [-L, L] before f, NaN kept.
 * Pointers and strides need the alignment of one element; when every base
 * address and row is 16-byte aligned and in_features fills whole 16-byte
 * chunks, faster loads are used.  With n_groups 1 group_stride and bias_stride
 * are not used.
 *
 * Any sizes >= 1 are supported up to these limits, past which the calls return
 * MOE_ERR_UNSUPPORTED:
 *   rows of x, w, residual or out of 16 MiB and more (their stride, if given)
 *   a group_stride (packed or given) or bias_stride of more than 2^40 elements
 *   (2^30 - 1) rows or slots
 *   work of more than 2^22 tiles; a tile is at least 64 rows of x by 64 columns of
 *   out, 32 when gated, so a call is supported wherever
 *     ceil(n_rows / 64) * ceil(out_features / 64 or 32) <= 2^22
 *   with floor((n_slots + 63 * min(n_slots, n_groups)) / 64) in the place of
 *   ceil(n_rows / 64) per expert; aligned calls go further, by larger tiles.
 */
typedef struct {
    int32_t in_features, out_features;
    int32_t n_groups;     /* 1 for moe_matmul; experts, 1..MOE_MAX_EXPERTS */
    int32_t dtype;        /* moe_dtype of x, w and bias */
    int32_t out_dtype;    /* moe_dtype of out */
    int32_t fn;           /* moe_fn */
    float clamp_limit;    /* >= 0; 0 = none */
    int32_t reserved;     /* 0 */
    const void *w, *w_up;
    const void *bias, *bias_up;
    int64_t row_stride, group_stride, bias_stride;
} moe_linear_t;

/* Host-only check of a descriptor (no device access). */
moe_status moe_linear_check(const moe_linear_t *linear);

/* Bytes of device workspace the products need for up to max_rows rows (or
 * slots); 0 when none is needed (workspace may then be NULL) or the
 * descriptor is invalid. */
size_t moe_matmul_workspace_size(const moe_linear_t *linear, int32_t max_rows);
size_t moe_grouped_workspace_size(const moe_linear_t *linear, int32_t max_slots);

/*
 * out[r] = residual[r] + f(x[r] w^T + bias)        (f(z) * z_up when gated)
 *   x         [n_rows][in_features], rows x_stride elements apart
 *   residual  NULL, or [n_rows][out_features] of residual_dtype, rows
 *             residual_stride apart
 *   out       [n_rows][out_features], rows out_stride apart
 *   workspace moe_matmul_workspace_size(linear, n_rows) bytes, 256-byte
 *             aligned; contents need no initialisation.  Calls that may
 *             overlap in time need a workspace each.
 * Strides of 0 mean packed rows.  fp32 products and sums throughout (bf16
 * and fp16 products are exact), one rounding to out_dtype at the store.
 * Repeated calls are bitwise equal; which kernel runs, and with it the order
 * of the fp32 sums, depends on the shapes, strides and alignments only.
 * out may be residual itself (same type and stride); it must not overlap
 * anything else.  n_groups must be 1.  n_rows == 0 launches nothing.
 */
moe_status moe_matmul(const moe_linear_t *linear, const void *x, int64_t x_stride, int32_t n_rows,
                      const void *residual, int32_t residual_dtype, int64_t residual_stride, void *out,
                      int64_t out_stride, void *workspace, size_t workspace_bytes, void *hip_stream);

/*
 * The same product for every expert of a planned batch, each over its own
 * rows: for every distinct expert e and every slot the plan lists for it,
 *   out[row] = f(x[row'] w[e]^T + bias[e])
 * with row and row' as `rows` (moe_rows) says.
 *   plan      of n_slots slots over n_groups experts (moe_expert_plan,
 *             moe_route_plan); work and sorted_slots are read
 *             (MOE_ROWS_SORTED: work only)
 *   top_k     slots per token, >= 1; used by MOE_ROWS_TOKEN
 *   x         [n_slots / top_k rounded up] (token) or [n_slots] rows
 *   out       [n_slots] rows
 * Rows that no expert lists (slots the planner left out for a bad expert id)
 * are left as they were.  Each distinct expert's weights are read once per
 * row tile; no host synchronisation: the grid covers the largest number of
 * tiles that n_slots slots can need.  Records or slots outside the plan's
 * range are skipped, so a malformed plan never reads or writes out of bounds.
 * n_slots == 0 launches nothing.  Otherwise as moe_matmul.
 */
moe_status moe_grouped_matmul(const moe_linear_t *linear, const void *x, int64_t x_stride, int32_t n_slots,
                              int32_t top_k, int32_t rows, const moe_plan_t *plan, void *out, int64_t out_stride,
                              void *workspace, size_t workspace_bytes, void *hip_stream);

/*
 * out[t] = residual[t] + sum_{j < top_k} topk_w[t][j] * y[t * top_k + j]
 *   y         [n_tokens * top_k][hidden] of y_dtype, packed (the rows that
 *             moe_grouped_matmul writes by slot)
 *   topk_idx  int32 [n_tokens][top_k]: a token with an id outside
 *             0 .. n_experts-1 becomes NaN and its y rows count for nothing
 *   topk_w    fp32 [n_tokens][top_k]
 *   residual  NULL, or [n_tokens][hidden] of residual_dtype, packed
 *   out       [n_tokens][hidden] of out_dtype, packed; may be residual itself
 *             (same type), must not overlap anything else
 * fp32 sums in j order, the residual added last, one rounding ("f32 partials
 * with a single final rounding", page "perf(moe): batched decode scales 1.55x
 * against 3.25x on dense", Implementation Notes).  Types are any moe_dtype.
 * MOE_ERR_UNSUPPORTED for top_k > MOE_MAX_TOP_K, n_experts > MOE_MAX_EXPERTS,
 * hidden >= 2^22, n_tokens * top_k >= 2^30 and n_tokens * ceil(hidden / 4) > 2^30.
 */
moe_status moe_combine(const void *y, int32_t y_dtype, const int32_t *topk_idx, const float *topk_w,
                       int32_t n_tokens, int32_t hidden, int32_t top_k, int32_t n_experts,
                       const void *residual, int32_t residual_dtype, void *out, int32_t out_dtype,
                       void *hip_stream);

/* ------------------------------------------------------- scored routing
 *
 * The router (page "perf(moe): attribute the MoE decode gap at the M = 1 expert gather",
 * Proposed Solution step 2) of models whose scores are not the softmax of the kept
 * logits: softmax over all experts or sigmoid scores, a bias for balance that
 * only the choice sees, groups of experts of which the best are kept, weights
 * renormalised or not and scaled.
 */
typedef enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 } moe_score;

/* What a group of experts is ranked by: its best c, or the sum of its two best. */
typedef enum { MOE_GROUP_MAX = 0, MOE_GROUP_TOP2 = 1 } moe_group_score;

#define MOE_MAX_GROUPS 64

/*
 * A router, in host memory; bias is a device pointer.  With the logits l of a token:
 *   s = softmax(l) over all experts, or sigmoid(l)
 *   c = s + bias, in 64 bits.  Without a bias experts are in the order of l itself,
 *       in which s rises.  Scores below 1e-300 (a sigmoid of l < -690) may count
 *       as zero, but not for the weights of a renormalised softmax: those are the softmax of
 *       the chosen logits, however far an expert that is not chosen is above them.
 * An expert is masked when its logit is -infinity or the lowest finite value of the logits'
 * type, or its bias is -infinity.  The softmax leaves out experts masked by their logits.
 *   Of n_groups groups of n_experts / n_groups consecutive experts the top_groups best are
 *   kept, by their best unmasked c (l without a bias) or by the sum of their two best
 *   (one where it has one), ties to the lower group, groups without an unmasked expert last.
 *   Of the kept groups' experts the top_k of largest c are chosen, in that order, ties to the
 *   lower expert id, masked ones after all others.
 *   w = s of the chosen, 0 for a masked one; renormalise: divided by their sum (left 0
 *       where that is 0); times scale; rounded once to fp32.
 * A token's ids are -1 and its weights NaN if any unmasked expert's logit is NaN, or
 * +infinity under softmax, or its bias is NaN or +infinity, and under softmax also for such a logit
 * of an expert that only its bias masks, as every score has it in its sum: the planner leaves
 * the token out and the combine makes it NaN.
 */
typedef struct {
    int32_t n_experts;   /* 1..MOE_MAX_EXPERTS */
    int32_t top_k;       /* 1..MOE_MAX_TOP_K, at most the kept groups' experts */
    int32_t score;       /* moe_score */
    int32_t n_groups;    /* 1..MOE_MAX_GROUPS, divides n_experts; 1 = no groups */
    int32_t top_groups;  /* 1..n_groups */
    int32_t group_score; /* moe_group_score */
    int32_t renormalise; /* 0 or 1 */
    float scale;         /* finite, > 0 */
    const float *bias;   /* [n_experts] or NULL */
} moe_router_t;

/* Host-only check of a router (no device access). */
moe_status moe_router_check(const moe_router_t *router);

/*
 * Routes a batch.
 *   logits    [n_tokens][n_experts] of logits_dtype (fp32, bf16 or fp16), rows
 *             logits_stride elements apart (0 = packed)
 *   topk_idx  int32 [n_tokens][top_k], topk_w fp32 [n_tokens][top_k], packed: what
 *             moe_expert_plan, moe_decode_step and moe_combine take
 * Outputs must not overlap one another or the inputs.  A token's result depends on its
 * logits alone.  n_tokens == 0 returns MOE_OK without a launch.
 * MOE_ERR_UNSUPPORTED for 2^26 tokens, 2^30 slots or strides past 2^32 elements and more.
 */
moe_status moe_router_topk(const moe_router_t *router, const void *logits, int32_t logits_dtype,
                           int64_t logits_stride, int32_t n_tokens, int32_t *topk_idx, float *topk_w,
                           void *hip_stream);

/* moe_router_topk, then moe_expert_plan of its choice: one launch for up to 64 tokens of up
 * to 512 experts in up to 16 groups.
 * n_tokens == 0 writes an empty plan. */
moe_status moe_router_plan(const moe_router_t *router, const void *logits, int32_t logits_dtype,
                           int64_t logits_stride, int32_t n_tokens, int32_t *topk_idx, float *topk_w,
                           const moe_plan_t *plan, void *hip_stream);

/* ----------------------------------------------- 8-bit integer products
 *
 * Layers and experts whose weights are 8-bit integers with a scale for each output
 * channel, on activations that are 8-bit integers with a scale for each row: the products
 * of moe_matmul and moe_grouped_matmul on the matrix cores' integer instructions, with the
 * same epilogue, plans and rows.  Activations may be given in fp32, bf16 or fp16; the
 * call then quantises their rows as moe_quantize_rows does.
 */

/*
 * codes[r][c] = x[r][c] * 127 / max |x[r]| rounded to the nearest integer, ties to the even one
 * (of the exact quotient), scales[r] = max |x[r]| / 127 rounded to fp32, so that
 * x ~ codes * scales.  A row of zeros has codes and scale 0; a row that holds an
 * infinity or NaN has codes 0 and scale NaN.
 *   x       [n_rows][n_cols] of dtype (fp32, bf16, fp16), rows x_stride elements apart
 *   codes   int8 [n_rows][n_cols], rows codes_stride apart
 *   scales  fp32 [n_rows]
 * Strides of 0 mean packed rows.  codes and scales must not overlap one another or x.
 * The same call makes weights: a row for each output channel.
 * MOE_ERR_UNSUPPORTED for rows (strides) of 16 MiB and more, or 2^30 rows and more.
 */
moe_status moe_quantize_rows(const void *x, int32_t dtype, int64_t x_stride, int32_t n_rows, int32_t n_cols,
                             int8_t *codes, int64_t codes_stride, float *scales, void *hip_stream);

/*
 * Integer weights of a product, in host memory, its pointers device pointers; as
 * moe_linear_t, with
 *   w          int8 [n_groups][out_features][in_features], w_scale fp32 [n_groups][out_features]
 *   w_up, w_up_scale  both or neither: the gated product's second stack
 *   bias, bias_up     [n_groups][out_features] of bias_dtype (fp32, bf16, fp16)
 * row_tail bytes behind each row's in_features belong to the same buffer and are zero
 * (0 = none are known to be): rows whose in_features and row_tail together fill
 * whole 16-byte chunks, at 16-byte addresses, take the faster loads.  in_features is at most
 * MOE_MAX_I8_INPUTS, for which the sums fit 32 bits whatever the integers; beyond it, and
 * beyond moe_linear_t's other limits, MOE_ERR_UNSUPPORTED.
 */
#define MOE_MAX_I8_INPUTS 131071
typedef struct {
    int32_t in_features, out_features;
    int32_t n_groups;
    int32_t out_dtype;    /* moe_dtype of out: fp32, bf16, fp16 */
    int32_t fn;           /* moe_fn */
    float clamp_limit;    /* >= 0; 0 = none */
    int32_t bias_dtype;
    int32_t row_tail;     /* 0..15 */
    const int8_t *w, *w_up;
    const float *w_scale, *w_up_scale;
    const void *bias, *bias_up;
    int64_t row_stride, group_stride, scale_stride, bias_stride; /* elements; 0 = packed */
} moe_linear_int_t;

/* Host-only check of a descriptor (no device access). */
moe_status moe_linear_int_check(const moe_linear_int_t *linear);

/* Bytes of device workspace for up to max_rows rows, or max_slots slots over at most
 * max_x_rows rows of x, of any type of x; 0 if the descriptor or a number is invalid. */
size_t moe_matmul_int_workspace_size(const moe_linear_int_t *linear, int32_t max_rows);
size_t moe_grouped_int_workspace_size(const moe_linear_int_t *linear, int32_t max_slots, int32_t max_x_rows);

/*
 * out[r] = residual[r] + f(z),  z = x_scale[r] * w_scale * sum_k x[r][k] w[k] + bias
 * (f(z) * z_up when gated).
 *   x         x_dtype MOE_DTYPE_I8: int8 [n_rows][in_features] with x_scale fp32 [n_rows]
 *             x_dtype fp32, bf16 or fp16: quantised within the call; x_scale is NULL
 *   workspace moe_matmul_int_workspace_size(linear, n_rows) bytes, 256-byte aligned; contents
 *             need no initialisation.  Calls that may overlap in time need one each.
 *             x of a floating type asks for all of it, whether the call's kernel writes to it or
 *             not.  x of integers takes less: NULL where K is not split, and without room for
 *             a copy rows that are no whole chunks are read where they are.
 * The integer sum is exact; it and the two scales' product are rounded to fp32 once each, and so is
 * what their product and the bias come to (a fused multiply-add); scales whose product is below
 * 2^-126 lose bits by it, and one past fp32's range is infinite.  What follows is as in moe_matmul;
 * the last product, of f or of the gate, and a residual's sum may be rounded together.  Repeated
 * calls are bitwise equal.
 */
moe_status moe_matmul_int(const moe_linear_int_t *linear, const void *x, int32_t x_dtype, int64_t x_stride,
                         const float *x_scale, int32_t n_rows, const void *residual, int32_t residual_dtype,
                         int64_t residual_stride, void *out, int64_t out_stride, void *workspace,
                         size_t workspace_bytes, void *hip_stream);

/* The same for every expert of a planned batch: moe_grouped_matmul with integer operands.
 * x and x_scale have a row per token or slot, or a sorted row, as `rows` says. */
moe_status moe_grouped_matmul_int(const moe_linear_int_t *linear, const void *x, int32_t x_dtype, int64_t x_stride,
                                 const float *x_scale, int32_t n_slots, int32_t top_k, int32_t rows,
                                 const moe_plan_t *plan, void *out, int64_t out_stride, void *workspace,
                                 size_t workspace_bytes, void *hip_stream);

/* Static description of a status code. */
const char *moe_status_str(moe_status status);

/* ABI version: bumped when a signature or struct changes (8: plain field
 * order of moe_layer_t, moe_decode_step without a residual,
 * moe_decode_step_residual). */
int32_t moe_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MOE_DECODE_H */

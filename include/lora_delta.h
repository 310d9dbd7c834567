/*
 * lora_delta.h -- C ABI of the GB300 (sm_103a) routed multi-tenant LoRA delta.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - All tensors are caller-owned DEVICE memory unless an argument says
 *    "host".  bf16 tensors are row-major with the stated leading dimension.
 *  - Launchers enqueue work on `stream` (a cudaStream_t; NULL is the legacy
 *    default stream): they allocate no device memory and never synchronize
 *    ("Module lora_delta", module invariants).  The one exception is
 *    lora_get_error, which waits on `stream` to read the error word back.
 *    A call whose slots split between the small-segment kernel and the
 *    tensor-core path (lora_delta_fused, lora_delta_segmented) runs the former
 *    on a second stream of the library's, forked from `stream` by an event
 *    and joined back by another: all of the call's work still comes before
 *    anything enqueued on `stream` after it, and inside a stream capture the
 *    fork and the join become part of the captured graph.  That stream and
 *    its two events are created once per device, on the first such call made
 *    outside a capture (a call made during a capture before then runs both
 *    parts on `stream`); calls from several host threads share them, under a
 *    lock.  LORA_FORK=0 in the environment keeps every call on `stream`.
 *  - Return value: LORA_OK (0) or a host-detected LORA_ERR_* status; an error
 *    status means nothing was enqueued.  Nothing is ever thrown.
 *  - Device-detected problems never trap: the offending row / pair is handled
 *    as stated per call and a LORA_DEV_ERR_* bit is OR-ed into the caller's
 *    `err_word` (a device uint32, may be NULL to ignore).  Read it with
 *    lora_get_error.
 *  - Adapter weights, and the tables of their addresses and scales, are read
 *    ahead of the end of the library call before on the stream: they must not
 *    be what that call itself writes (a lora_linear into a pool slot, say).
 *    Other work between the two, such as lora_pool_pack, a copy or a kernel of
 *    the caller's, puts them in order.  Rows, ids and plans need none.
 *  - Alignment: k_in, every slice width, ld_out, offset_start and the pool
 *    rank R must be multiples of 8 elements (16 bytes of bf16), and x / out /
 *    h must be 16-byte aligned; otherwise LORA_ERR_ALIGN.  A pool address in a
 *    device table that is not 16-byte aligned is found on the device: that
 *    slice is skipped and LORA_DEV_ERR_ALIGN is set.
 *  - Limits: 1 <= S <= 8 slices, 8 <= R <= 128, S*R <= 512, max_loras <= 3071
 *    (LORA_ERR_UNSUPPORTED beyond).
 *
 * Pages the calls follow (cited per call below):
 *  [punica]     "vllm/lora/punica_wrapper/punica_base.py": add_shrink,
 *               add_expand, add_lora_linear "Semantics"; prefill_metadata;
 *               add_lora_w13 / add_lora_w2 (in-place MoE deltas).
 *  [sharded]    "vllm.lora.fully_sharded_layers": the float32 shrink buffer
 *               and the shrink-with-scale-1.0 then expand sequence.
 *  [metrale]    "Module lora_delta": LoraPair / LoraRoute layouts, the
 *               padded-rank invariant, apply_lora_bgmv, the scale rule.
 *  [flashinfer] "flashinfer.fused_moe.bgmv_moe_gemm1_lora_delta".
 */
#ifndef LORA_DELTA_H
#define LORA_DELTA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *lora_stream_t; /* == cudaStream_t */

/* host-detected status codes */
#define LORA_OK 0
#define LORA_ERR_ARG 1         /* NULL pointer, negative size, bad flag        */
#define LORA_ERR_SHAPE 2       /* inconsistent sizes                           */
#define LORA_ERR_ALIGN 3       /* a size or pointer breaks the 16-byte rule    */
#define LORA_ERR_CUDA 4        /* a CUDA launch or copy failed                 */
#define LORA_ERR_WORKSPACE 5   /* workspace missing or smaller than required   */
#define LORA_ERR_UNSUPPORTED 6 /* outside the limits stated above              */
#define LORA_ERR_TOO_LARGE 7   /* needs more scratch than the library's fixed
                                  no-allocation buffer holds                   */

/* device-detected bits, OR-ed into *err_word */
#define LORA_DEV_ERR_SLOT 1u    /* seq_slot >= max_loras: the row gets no delta        */
#define LORA_DEV_ERR_EXPERT 2u  /* MoE expert id outside [0, E): pair written as zeros */
#define LORA_DEV_ERR_LORA 4u    /* MoE adapter id >= num_loras: pair written as zeros  */
#define LORA_DEV_ERR_TIMEOUT 8u /* a bounded wait inside a kernel gave up              */
#define LORA_DEV_ERR_ALIGN 16u  /* a table address is not 16-byte aligned: slice skipped */
#define LORA_DEV_ERR_INTERNAL 32u /* a launch invariant of the library failed (a bug)   */
#define LORA_DEV_ERR_SEGMENT 64u  /* segment starts not nondecreasing in [0, n]: clamped  */
#define LORA_DEV_ERR_LENGTH 128u  /* a request's length is negative or past its limits: clamped */
#define LORA_DEV_ERR_PAGE 256u    /* a cache page is missing or outside the cache: skipped  */

/* element types of rows that are not bf16 only */
#define LORA_BF16 0
#define LORA_F16 1

/* Human-readable name of a status code (static string). */
const char *lora_status_string(int status);

/* ABI version of this library (bumped on any signature change). */
int lora_abi_version(void);

/*
 * lora_set_wait_limit_ns -- set the limit, in nanoseconds of the GPU's global
 * timer, after which a bounded wait inside a kernel gives up; returns the
 * previous limit.  None of the pages has this: it is a guard of this
 * library's own kernels.  Every mbarrier wait of the tensor-core kernels is
 * bounded; one that runs out sets LORA_DEV_ERR_TIMEOUT in the call's error
 * word, and its CTA skips its stores, lets its issued MMAs finish, frees its
 * tensor memory and returns, so the context stays usable.  The default is
 * 2 s (2000000000), far above any legitimate wait.  0 makes a wait give up at
 * its first poll that finds the awaited phase incomplete, which lets a test
 * run the time-out path without a fault or a hang.  Process-wide; each
 * launch copies the value current when it is enqueued (a captured CUDA
 * graph keeps the value of its capture).  Thread-safe.
 */
uint64_t lora_set_wait_limit_ns(uint64_t ns);

/*
 * lora_scale -- the adapter scale ([metrale] LoraPair): alpha / r, or
 * alpha / sqrt(r) when use_rslora is nonzero.  Computed on the host; the
 * caller stores it in its scale table.  Applied in the fold (after the
 * expand's rank contraction), never folded into B.  r <= 0 gives 0.
 */
float lora_scale(float alpha, int r, int use_rslora);

/*
 * lora_pool_pack -- pack one PEFT adapter into one padded pool slot
 * ([metrale] module invariants + LoraPair).
 *   a_slot [R, k_in] bf16 (out): rows 0..r-1 = a_r, rows r..R-1 = 0.
 *   b_slot [w, R]    bf16 (out): columns 0..r-1 of each row = b_r, r..R-1 = 0.
 *   a_r    [r, k_in] bf16 (in) : PEFT lora_A, row-major.
 *   b_r    [w, r]    bf16 (in) : PEFT lora_B, row-major.
 * Every element of both slots is written (the zero padding is what lets both
 * stages contract at R).  The caller then stores a_slot / b_slot in its
 * a_table / b_table.  Errors: LORA_ERR_ARG (r < 0, r > R, NULL), ALIGN.
 */
int lora_pool_pack(void *a_slot, void *b_slot, const void *a_r, const void *b_r, int r, int R,
                   int k_in, int w, lora_stream_t stream);

/*
 * Routing tables shared by the linear calls ([metrale] LoraRoute):
 *   a_table, b_table [S * max_loras] uint64 (device): entry j*max_loras + s
 *     is the device address of slot s's A_j [R, k_in] (resp. B_j [w_j, R])
 *     pool region, 0 when slot s does not adapt slice j.
 *   scale_table [max_loras] float (device), or NULL for scale 1.
 *   seq_slot [n] int32 (device): the row's slot; negative = no delta
 *     ([metrale] apply_lora_bgmv); >= max_loras = no delta + LORA_DEV_ERR_SLOT.
 *   widths [S] int32 (HOST): the output slice widths; slice j's columns start
 *     at offset_start + widths[0] + ... + widths[j-1] ([punica] add_expand).
 *
 * Workspace: when n > 1024, or when a workspace is given and n >= 256, the
 * rows are first clustered by slot on the device (a stable counting sort,
 * [punica] prefill_metadata) into a caller-provided scratch buffer of
 * lora_workspace_size(n, S, R, max_loras) bytes, 256-byte aligned; the same
 * buffer holds the fp32 rank intermediate of the tensor-core path that
 * lora_delta_fused takes for slots with many rows.  For n <= 1024 with no
 * workspace each kernel clusters its own rows.
 */
size_t lora_workspace_size(int n, int S, int R, int max_loras);

/*
 * lora_workspace_min_size -- the smallest workspace the linear calls accept
 * for these sizes.  A workspace between this and lora_workspace_size works;
 * the tensor-core path then splits k_in over fewer CTAs.
 */
size_t lora_workspace_min_size(int n, int S, int R, int max_loras);

/*
 * lora_route -- the routing step on its own ([punica] prefill_metadata):
 * a stable clustering of the n rows by slot.
 *   perm      [n] int32 (out): perm[0 .. seg_start[max_loras]) are the rows
 *             with 0 <= slot < max_loras, by ascending slot, then ascending
 *             row index; entries past that are unspecified.
 *   seg_start [max_loras + 2] int32 (out): cluster s is
 *             perm[seg_start[s] .. seg_start[s+1]); the rows with no valid
 *             slot follow, up to seg_start[max_loras + 1] == n.
 * Rows with slot >= max_loras set LORA_DEV_ERR_SLOT.
 */
int lora_route(int32_t *perm, int32_t *seg_start, const int32_t *seq_slot, int n,
               int max_loras, uint32_t *err_word, lora_stream_t stream);

/*
 * lora_route_with_scratch -- lora_route for large batches: the same output
 * (bit for bit), but batches of 2048 rows or more are sorted by many CTAs in
 * chunks of 1024 rows, using a caller-provided scratch buffer of
 * lora_route_scratch_size(n, max_loras) bytes (16-byte aligned; one count per
 * (chunk, slot)).  Errors as lora_route, plus LORA_ERR_WORKSPACE when the
 * scratch is missing or too small.  ([punica] prefill_metadata.)
 */
size_t lora_route_scratch_size(int n, int max_loras);
int lora_route_with_scratch(int32_t *perm, int32_t *seg_start, const int32_t *seq_slot, int n,
                            int max_loras, void *scratch, size_t scratch_bytes,
                            uint32_t *err_word, lora_stream_t stream);

/*
 * lora_shrink -- [punica] add_shrink: for every slice j and routed row i
 *   h[j, i, q] += scale_s * sum_k x[i, k] * A_j,s[q, k],   q < R
 * ("y[i] += (x @ lora_a_stacked[i]) * scale" with A in the [R, k_in] pool
 * layout, so the product is x A^T).  h [S, n, R] float32 (in/out): the
 * [sharded] layers zero it and pass scale 1.0 (scale_table NULL).  Rows with
 * no slot and slices whose a_table entry is 0 are left untouched.
 */
int lora_shrink(float *h, const void *x, int n, int k_in, const int32_t *seq_slot,
                const uint64_t *a_table, const float *scale_table, int S, int R, int max_loras,
                void *workspace, size_t ws_bytes, uint32_t *err_word, lora_stream_t stream);

/*
 * lora_expand -- [punica] add_expand: for every slice j and routed row i
 *   v = scale_s * sum_q h[j, i, q] * B_j,s[c, q]
 *   out[i, off_j + c] = RN_bf16(out + v)   (add_inputs != 0)
 *                     = RN_bf16(v)         (add_inputs == 0)
 * out [n, ld_out] bf16 (in/out).  scale_table NULL means scale 1 (the
 * [punica] expand carries no scale; pass the table to fold it here as
 * [metrale] does).  Rows with no slot and slices whose b_table entry is 0
 * are left untouched bit for bit.  Accumulation is fp32; one rounding to bf16.
 */
int lora_expand(void *out, int64_t ld_out, const float *h, const int32_t *seq_slot,
                const uint64_t *b_table, const float *scale_table, const int32_t *widths, int S,
                int R, int n, int max_loras, int offset_start, int add_inputs, void *workspace,
                size_t ws_bytes, uint32_t *err_word, lora_stream_t stream);

/*
 * lora_expand_gathered -- lora_expand on h as the all-gather of rank-sharded
 * shrinks leaves it ([sharded] _mcp_apply, ColumnParallelLinearWithShardedLoRA
 * and MergedColumnParallelLinearWithShardedLoRA: A sliced along the rank,
 * each of `parts` tensor-parallel ranks shrinks its R / parts rows into an
 * fp32 buffer [S, n, R / parts], and the buffers are all-gathered).  h is
 * [parts][S][n][R / parts] fp32, rank-major: h[p][j][i][q] is rank
 * p * R / parts + q of slice j, row i.  The rest is lora_expand with R the
 * whole rank; each rank calls it with the B rows of its own output columns
 * (b_table, widths) and gets them bit for bit as the unsharded delta does.
 * parts = 1 is lora_expand.  Requires R % parts == 0 (else LORA_ERR_ARG).
 */
int lora_expand_gathered(void *out, int64_t ld_out, const float *h, int parts,
                         const int32_t *seq_slot, const uint64_t *b_table,
                         const float *scale_table, const int32_t *widths, int S, int R, int n,
                         int max_loras, int offset_start, int add_inputs, void *workspace,
                         size_t ws_bytes, uint32_t *err_word, lora_stream_t stream);

/*
 * lora_delta_fused -- the routed delta in one pass ([punica] add_lora_linear,
 * [metrale] apply_lora_bgmv): for every routed row i (s = seq_slot[i]) and
 * slice j whose A and B table entries are both nonzero,
 *   out[i, off_j : off_j + w_j] = RN_bf16(out + scale_s * (x[i] A_j,s^T) B_j,s^T)
 * (RN_bf16(scale_s * ...) when add_inputs == 0).  Both contractions run at
 * the padded rank R, and the rank-R intermediate is fp32.  For slots with
 * few rows it stays on chip; slots with many rows go to the tensor-core path,
 * whose intermediate passes through fp32 planes in the workspace.  x [n, k_in]
 * bf16, out [n, ld_out] bf16.
 */
int lora_delta_fused(void *out, int64_t ld_out, const void *x, int n, int k_in,
                     const int32_t *seq_slot, const uint64_t *a_table, const uint64_t *b_table,
                     const float *scale_table, const int32_t *widths, int S, int R,
                     int max_loras, int offset_start, int add_inputs, void *workspace,
                     size_t ws_bytes, uint32_t *err_word, lora_stream_t stream);

/*
 * lora_delta_segmented -- the delta on rows already grouped by adapter, such
 * as the expert-sorted rows of a grouped MoE GEMM ("expert_apply.rs",
 * apply_expert_lora_sorted / expert_delta_workitems, with the row blocks read
 * from device memory instead of a host copy).  Rows seg_start[s] ..
 * seg_start[s+1] - 1 take adapter s (table entries j * n_segs + s, as in
 * lora_delta_fused with max_loras = n_segs); rows from seg_start[n_segs] on
 * are untouched.  seg_start [n_segs + 1] int32 (device) must start at 0 and
 * be nondecreasing up to at most n; otherwise the starts are clamped into
 * that form (no row outside the batch is read or written) and
 * LORA_DEV_ERR_SEGMENT is set.  Arithmetic, layouts and the other arguments
 * as lora_delta_fused; a workspace of lora_workspace_size(n, S, R, n_segs)
 * bytes is required (no routing sort runs).
 */
int lora_delta_segmented(void *out, int64_t ld_out, const void *x, int n, int k_in,
                         const int32_t *seg_start, int n_segs, const uint64_t *a_table,
                         const uint64_t *b_table, const float *scale_table,
                         const int32_t *widths, int S, int R, int offset_start, int add_inputs,
                         void *workspace, size_t ws_bytes, uint32_t *err_word,
                         lora_stream_t stream);

/*
 * lora_moe_fc1_delta -- [flashinfer] bgmv_moe_gemm1_lora_delta.  For every
 * routed pair (token t, slot j): e = topk_ids[t, j], l = lora_ids[t];
 *   regular (shared_a == 0): w_ptr_a / w_ptr_b are [2, E] int64 tables of
 *     bank base addresses [A_gate, A_up] / [B_gate, B_up];
 *     out[t, j, 0:I]  = RN_bf16(scale * B_gate[l,e] (A_gate[l,e] x[t]))
 *     out[t, j, I:2I] = RN_bf16(scale * B_up[l,e]   (A_up[l,e]   x[t]))
 *   shared  (shared_a != 0): [E] tables, one shared A and a fused
 *     B [2I, rank] (gate rows 0:I, up rows I:2I);
 *     out[t, j, :] = RN_bf16(scale * B_fused[l,e] (A_shared[l,e] x[t]))
 * Adapter l of a bank starts l * stride elements after the bank base; A[l,e]
 * is [rank, H] row-major, B[l,e] is [I, rank] (or [2I, rank]) row-major.
 * out [T, top_k, 2I] bf16 is fully written: pairs with l < 0 are zeros (the
 * page skips them), pairs with l >= num_loras or e outside [0, E) are zeros
 * and set LORA_DEV_ERR_LORA / LORA_DEV_ERR_EXPERT.  The delta stays per
 * (token, slot): no routing weights, no sum over experts.
 * Requires H, I, rank multiples of 8, rank <= 128, E * num_loras <= 3071 and
 * a workspace of lora_moe_workspace_size(T, top_k, E, num_loras, rank,
 * shared_a) bytes.
 */
size_t lora_moe_workspace_size(int T, int top_k, int E, int num_loras, int rank, int shared_a);
int lora_moe_fc1_delta(void *out, const void *x, const int64_t *w_ptr_a, int64_t stride_a,
                       const int64_t *w_ptr_b, int64_t stride_b, int shared_a,
                       const int32_t *topk_ids, const int32_t *lora_ids, int T, int top_k, int E,
                       int H, int I, int rank, int num_loras, float scale, void *workspace,
                       size_t ws_bytes, uint32_t *err_word, lora_stream_t stream);

/*
 * lora_moe_w13_delta -- [punica] add_lora_w13: the gate/up delta of
 * lora_moe_fc1_delta added IN PLACE to y = intermediate_cache1
 * [T, top_k, 2I] bf16 (the expert gate/up GEMM's output, before the
 * activation):
 *   y[t, j, :] = RN_bf16(y[t, j, :] + delta[t, j, :])     (add_inputs != 0)
 *   y[t, j, :] = RN_bf16(delta[t, j, :])                   (add_inputs == 0)
 * with delta and the bank tables, strides and layouts exactly as
 * lora_moe_fc1_delta (regular or shared-A / fused-B mode).  Routing, per pair
 * (t, j): l = lora_ids[t] (the token-to-adapter mapping), e = topk_ids[t, j];
 *   - expert_map [n_global_experts] int32 (device, or NULL = identity):
 *     global expert id -> this rank's local id in [0, E), -1 = the expert
 *     is not on this rank (no delta).  A global id outside the map or a
 *     local id >= E sets LORA_DEV_ERR_EXPERT (no delta);
 *   - adapter_enabled [num_loras] int32 (device, or NULL): an adapter with
 *     entry 0 adds nothing;
 *   - l < 0: no delta; l >= num_loras: no delta + LORA_DEV_ERR_LORA.
 * A pair without a delta is left untouched (y belongs to the caller).
 * Requirements as lora_moe_fc1_delta, with E the local expert count; the
 * workspace is lora_moe_workspace_size(T, top_k, E, num_loras, rank,
 * shared_a) bytes.  Readings: the page gives the signature and docstring
 * only; routing weights are not applied before the activation.
 */
int lora_moe_w13_delta(void *y, const void *x, const int64_t *w_ptr_a, int64_t stride_a,
                       const int64_t *w_ptr_b, int64_t stride_b, int shared_a,
                       const int32_t *topk_ids, const int32_t *lora_ids,
                       const int32_t *expert_map, int n_global_experts,
                       const int32_t *adapter_enabled, int T, int top_k, int E, int H, int I,
                       int rank, int num_loras, float scale, int add_inputs, void *workspace,
                       size_t ws_bytes, uint32_t *err_word, lora_stream_t stream);

/*
 * lora_moe_w2_delta -- [punica] add_lora_w2: the down-projection delta added
 * IN PLACE to y = intermediate_cache3 [T, top_k, H] bf16 (the expert down
 * GEMM's per-pair output, before moe_sum), from x = intermediate_cache2
 * [T * top_k, I] bf16, one activation row per (token, slot) pair p = t *
 * top_k + j:
 *   v[c] = w_p * scale * sum_r B[l,e][c, r] * (A[l,e] x[p])[r]      (fp32)
 *   y[t, j, c] = RN_bf16(y[t, j, c] + v[c])  (add_inputs != 0), else RN_bf16(v[c])
 * w_ptr_a / w_ptr_b: [E] int64 tables of bank base addresses; adapter l of a
 * bank starts l * stride elements after its base; A[l,e] [rank, I] and
 * B[l,e] [H, rank] row-major bf16.  topk_weights [T, top_k] fp32 (device, or
 * NULL: w_p = 1) are the routing weights the down GEMM applied before
 * moe_sum.  Routing (expert_map, adapter_enabled, lora_ids, errors) and the
 * untouched pairs as lora_moe_w13_delta.  Requires H, I, rank multiples of 8,
 * rank <= 128, E * num_loras <= 3071 and a workspace of
 * lora_moe_workspace_size(T, top_k, E, num_loras, rank, 1) bytes (one slice).
 */
int lora_moe_w2_delta(void *y, const void *x, const int64_t *w_ptr_a, int64_t stride_a,
                      const int64_t *w_ptr_b, int64_t stride_b, const int32_t *topk_ids,
                      const int32_t *lora_ids, const int32_t *expert_map, int n_global_experts,
                      const int32_t *adapter_enabled, const float *topk_weights, int T,
                      int top_k, int E, int H, int I, int rank, int num_loras, float scale,
                      int add_inputs, void *workspace, size_t ws_bytes, uint32_t *err_word,
                      lora_stream_t stream);

/*
 * lora_moe_w2_delta_routed -- [punica] add_lora_w2 with the routing that the
 * preceding add_lora_w13 of the same layer handed over ("Reuses routing
 * tensors returned by add_lora_w13"): the same delta as lora_moe_w2_delta,
 * without sorting the pairs again.  `workspace` must be the workspace that a
 * preceding lora_moe_w13_delta call was given, on the same stream, with the
 * same T, top_k, E, num_loras and routing arrays (topk_ids, lora_ids,
 * expert_map, adapter_enabled), and left untouched since: that call wrote the
 * pairs' clustering by (adapter, local expert) at the front of it, and this
 * call reads it.  Every routing decision (no adapter, a switched-off adapter,
 * a non-local expert, a bad id) is taken from there, and its errors were
 * already reported by the w13 call.  x, the banks, topk_weights, y and the
 * arithmetic are as in lora_moe_w2_delta; ws_bytes must be at least
 * lora_moe_workspace_size(T, top_k, E, num_loras, rank, 1).  The workspace is
 * not written before the kernels read the routing, so a following call may
 * reuse it again.
 */
int lora_moe_w2_delta_routed(void *y, const void *x, const int64_t *w_ptr_a, int64_t stride_a,
                             const int64_t *w_ptr_b, int64_t stride_b, const float *topk_weights,
                             int T, int top_k, int E, int H, int I, int rank, int num_loras,
                             float scale, int add_inputs, void *workspace, size_t ws_bytes,
                             uint32_t *err_word, lora_stream_t stream);

/*
 * lora_delta_fused_floor -- a measurement aid, not part of the method (none of
 * the pages has it): moves the bytes that lora_delta_fused moves for a small
 * batch -- every routed slot's A and B (each CTA's share), the slot's x rows
 * and out rows, out written back -- with the same launch plan (grid, thread-
 * block cluster size, shared-memory plan, programmatic dependent launch), but
 * computes nothing: out is written back unchanged.  Timed next to
 * lora_delta_fused on the same inputs, it gives the data-movement floor of a
 * decode step in this launch shape.  Arguments as lora_delta_fused without
 * scale table, add_inputs, workspace and error word; LORA_ERR_UNSUPPORTED
 * unless n <= 1024 and the shape takes the fused small-segment kernel (one k
 * stage per CTA, R a multiple of 16 up to 64, S * R <= 256).
 */
int lora_delta_fused_floor(void *out, int64_t ld_out, const void *x, int n, int k_in,
                           const int32_t *seq_slot, const uint64_t *a_table,
                           const uint64_t *b_table, const int32_t *widths, int S, int R,
                           int max_loras, int offset_start, lora_stream_t stream);

/*
 * lora_delta_fused_noalloc -- lora_delta_fused for callers that cannot
 * allocate device memory.  The pages have no counterpart to this call: it
 * exists for callers whose memory is fixed up front (a budget set at start
 * up, an allocator that refuses allocations after warm-up, a runtime that
 * only lends this library the tensors it already owns) and who therefore
 * cannot provide lora_delta_fused's scratch workspace.
 * Same arguments and results as lora_delta_fused minus the workspace: the
 * scratch comes from a fixed buffer inside the library of
 * lora_noalloc_scratch_bytes() bytes (4 MiB).  The buffer sits in its own
 * CUDA module, which the runtime loads lazily by default: the first call on a
 * device (with that device current) looks the buffer up, and that is when the
 * driver reserves its 4 MiB on the device, which then holds it until the
 * process exits.  Make one warm-up call on every device before the memory
 * budget is fixed and before any stream capture; later calls reserve
 * nothing.  The looked-up address is cached per device and is stale after a
 * cudaDeviceReset.  A call whose smallest workspace
 * (lora_workspace_min_size(n, S, R, max_loras)) exceeds the buffer returns
 * LORA_ERR_TOO_LARGE and enqueues nothing.  Apart from that first reservation
 * the call never allocates (no cudaMalloc, no allocating library routine).
 * All calls share the one buffer: calls that
 * may overlap on the GPU (different streams) race and must be serialized by
 * the caller.  The buffer keeps the last call's contents; nothing in it needs
 * to start at zero.
 */
size_t lora_noalloc_scratch_bytes(void);
int lora_delta_fused_noalloc(void *out, int64_t ld_out, const void *x, int n, int k_in,
                             const int32_t *seq_slot, const uint64_t *a_table,
                             const uint64_t *b_table, const float *scale_table,
                             const int32_t *widths, int S, int R, int max_loras,
                             int offset_start, int add_inputs, uint32_t *err_word,
                             lora_stream_t stream);

/*
 * Serving step around the delta.  A request's keys and values live in pages of
 * `page_size` tokens (a multiple of 16, at most 1024); block_table[b][p] is
 * the page that holds tokens p * page_size .. of request b.  None of the pages
 * has these calls: a step's order is lora_batch_plan once, then in each layer
 * the projections with lora_delta_fused (seq_slot of the plan),
 * lora_kv4_append (slot_map of the plan) and lora_kv4_attention.
 * Limits: at most 4096 requests of at most 2^29 tokens (max_pages * page_size);
 * n_reqs * max_pages below 2^31, and n_reqs * max_pages * (page_size / 16) *
 * kv_heads and n * q_heads / kv_heads below 2^31 for the attention
 * (LORA_ERR_UNSUPPORTED beyond).
 */

/*
 * lora_batch_plan -- the maps of one step from the requests' lengths, and the
 * pages that its new tokens need.  Request b holds ctx_len[b] tokens and adds
 * new_len[b]; its rows follow those of request b - 1.
 *   ctx_len, new_len [n_reqs] int32 (in).
 *   req_slot    [n_reqs] int32 (in) or NULL: the request's adapter slot.
 *   block_table [n_reqs, ld_table] int32 (in/out): entries below
 *               ceil(ctx / page_size) are read; the entries of new pages, up to
 *               ceil((ctx + new) / page_size), are written.
 *   free_pages, free_count (in), free_left (out): a stack of free pages and its
 *               height; page k of all the step's new pages, in request order,
 *               is free_pages[*free_count - 1 - k], and *free_left is the height
 *               left.  free_left may be free_count.  With a free_left and a seq_len
 *               of its own the call changes nothing that it reads, and can be repeated.
 *               All three NULL: the tables hold every page already.
 *               (In place, of these or of the lengths below, the call runs on at
 *               most 8 SMs.)
 *   row_start   [n_reqs + 1] int32 (out): request b's rows are row_start[b] ..
 *               row_start[b + 1] - 1.
 *   seq_len     [n_reqs] int32 (out): ctx + new.  It may be ctx_len itself, which
 *               then holds the next step's lengths; no other output may share
 *               memory with an input (LORA_ERR_ARG).
 *   row_req, position, seq_slot [n_rows] int32, slot_map [n_rows] int64 (out):
 *               the row's request, its token's position, its adapter slot and
 *               its cache slot page * page_size + position % page_size.  Rows
 *               past the last request get -1, 0, -1 and -1 (no delta, not
 *               stored), so a batch may be padded to a fixed n_rows.
 * Handled, with LORA_DEV_ERR_LENGTH: a negative length counts as 0, a length
 * past max_pages * page_size is cut there, and rows past n_rows are cut off
 * (row_start and seq_len count what is left).  With LORA_DEV_ERR_PAGE: a token
 * whose page is missing (an entry < 0, the stack empty) gets slot -1, and the
 * table an entry of -1.  Requires 16-byte aligned row arrays.
 */
int lora_batch_plan(const int32_t *ctx_len, const int32_t *new_len, const int32_t *req_slot,
                    int n_reqs, int n_rows, int page_size, int32_t *block_table, int64_t ld_table,
                    int max_pages, const int32_t *free_pages, const int32_t *free_count,
                    int32_t *free_left, int32_t *row_start, int32_t *seq_len, int32_t *row_req,
                    int32_t *position, int64_t *slot_map, int32_t *seq_slot, uint32_t *err_word,
                    lora_stream_t stream);

/*
 * lora_batch_plan_bounded -- lora_batch_plan with the number of entries of
 * free_pages: a *free_count above free_cap counts as free_cap and one below 0 as
 * 0, with LORA_DEV_ERR_PAGE.  lora_batch_plan takes *free_count as it is, so there
 * the stack must have that many entries.
 */
int lora_batch_plan_bounded(const int32_t *ctx_len, const int32_t *new_len,
                            const int32_t *req_slot, int n_reqs, int n_rows, int page_size,
                            int32_t *block_table, int64_t ld_table, int max_pages,
                            const int32_t *free_pages, int free_cap, const int32_t *free_count,
                            int32_t *free_left, int32_t *row_start, int32_t *seq_len,
                            int32_t *row_req, int32_t *position, int64_t *slot_map,
                            int32_t *seq_slot, uint32_t *err_word, lora_stream_t stream);

/*
 * lora_pages_release -- the pages of finished requests back onto the free
 * stack: for every b with done[b] != 0, the entries >= 0 among its first
 * ceil(seq_len[b] / page_size), in (request, page) order, are stored from
 * free_pages[*free_count] up, become -1 in the table, and are counted in
 * *free_count.  Pages beyond free_cap stay in the table (LORA_DEV_ERR_PAGE); a
 * length outside [0, max_pages * page_size] is clamped (LORA_DEV_ERR_LENGTH).
 */
int lora_pages_release(const int32_t *done, const int32_t *seq_len, int n_reqs, int page_size,
                       int32_t *block_table, int64_t ld_table, int max_pages, int32_t *free_pages,
                       int free_cap, int32_t *free_count, uint32_t *err_word,
                       lora_stream_t stream);

/*
 * The 4-bit cache: [num_pages][kv_heads][page_size / 16] tiles of 16 tokens.
 * head_dim is 64, 128 or 256, in groups of 64.  A (token, head, group) keeps
 * m = f16(min), s = f16((max - min) * (1 / 15)) and codes
 * c = clamp(rint((x - m) * (1 / s)), 0, 15) (0 where s is 0), each step rounded
 * to float32, and stands for s * c + m.  Magnitudes up to 65504 are held (above
 * 65440 the top of a group may read as an infinity in float16 rows, and attention
 * wants magnitudes up to 2^15, since it may round s * c + m to float16); a group with
 * an infinity, a NaN or more keeps NaNs for s and m, and reads as NaN.  The bytes of
 * a tile, W = min(D, 128):
 *   key codes [D / W][16 tokens][4 c][W / 32 words]: nibble i of word w is dim
 *     64 (w / 2) + 16 c + 8 (w % 2) + i of the plane; key pairs [16][D / 64] of f16 (s, m);
 *   value codes [D / W][2 h][8 g][4 c][W / 32 words]: nibble j of the low (high) half of
 *     word w is dim 64 (w / 2) + 8 g + 4 (w % 2) + j of token 8 h + 2 c (+ 1); value pairs.
 * dtype (LORA_BF16 or LORA_F16) is the type of the rows beside it.
 * lora_kv4_page_bytes gives the bytes of one page, all heads (0 for sizes
 * that are not supported).  `pages` must be 16-byte aligned.
 */
size_t lora_kv4_page_bytes(int page_size, int kv_heads, int head_dim);

/*
 * lora_kv4_append -- quantise the rows k, v [n, kv_heads * head_dim] (row
 * strides ld_k, ld_v in elements, multiples of 8) and store row i at slot
 * slot_map[i].  A negative slot is not stored; a slot past the cache is not
 * stored and sets LORA_DEV_ERR_PAGE.  Slots of one call must differ.
 */
int lora_kv4_append(void *pages, int64_t num_pages, int page_size, int kv_heads, int head_dim,
                    int dtype, const void *k, int64_t ld_k, const void *v, int64_t ld_v,
                    const int64_t *slot_map, int n, uint32_t *err_word, lora_stream_t stream);

/*
 * lora_kv4_read -- the values that stored rows stand for, rounded once to the
 * row type: row i of k, v is slot slot_map[i]; a negative slot reads as zeros,
 * one past the cache too, with LORA_DEV_ERR_PAGE.
 */
int lora_kv4_read(const void *pages, int64_t num_pages, int page_size, int kv_heads, int head_dim,
                  int dtype, void *k, int64_t ld_k, void *v, int64_t ld_v, const int64_t *slot_map,
                  int n, uint32_t *err_word, lora_stream_t stream);

/*
 * lora_kv4_attention -- causal attention of a step's rows over the cache.  Row
 * i of request b (row_start[b] <= i < row_start[b + 1]) stands at position
 * P = seq_len[b] - row_start[b + 1] + i and sees the tokens t <= P, with
 * window > 0 only t > P - window:
 *   out[i, h] = sum_t softmax_t(scale * q[i, h] . K[t, h / g]) V[t, h / g],
 *   g = q_heads / kv_heads
 * over the values that the cache stands for.  q, out [n, q_heads * head_dim]
 * with row strides ld_q, ld_out (multiples of 8 elements).  lse [n, q_heads]
 * float32 (out) or NULL: the log of the softmax's denominator.  max_q_len:
 * the most rows of one request, known to the host; a request with more gets
 * zeros and LORA_DEV_ERR_LENGTH.  Tokens in a page outside [0, num_pages) or
 * past the table are not seen (LORA_DEV_ERR_PAGE / LORA_DEV_ERR_LENGTH).  A row
 * that sees nothing, and rows outside every request, get zeros (lse -inf).
 * What the cache holds at tokens that are not seen has no influence.
 * Magnitudes of q are taken up to 2^100; scores of any size are.
 * workspace: lora_kv4_attention_workspace_size() bytes (some 47 MB, for any batch),
 * 256-byte aligned.  Its first lora_kv4_attention_zeroed_bytes() bytes must be
 * zero before its first use and are left zero; calls that may overlap (a graph's
 * replays among them) need workspaces of their own.
 */
size_t lora_kv4_attention_workspace_size(void);
size_t lora_kv4_attention_zeroed_bytes(void);
int lora_kv4_attention(void *out, int64_t ld_out, const void *q, int64_t ld_q, int n, int q_heads,
                       const void *pages, int64_t num_pages, int page_size, int kv_heads,
                       int head_dim, int dtype, const int32_t *block_table, int64_t ld_table,
                       int max_pages, const int32_t *row_start, const int32_t *seq_len, int n_reqs,
                       int max_q_len, float scale, int window, float *lse, void *workspace,
                       size_t ws_bytes, uint32_t *err_word, lora_stream_t stream);

/*
 * The routed-expert layer around the deltas.  A pair p = t * top_k + j sends
 * token t to expert topk_ids[t, j].  A layer's order is lora_moe_dispatch,
 * lora_moe_linear (with the delta that lora_moe_fc1_delta leaves for the sorted
 * rows: T = their number, top_k = 1, topk_ids = row_expert, lora_ids =
 * row_lora), lora_moe_linear again, lora_moe_w2_delta likewise, lora_moe_combine.
 * None of the pages has these calls.  Matrices hold 16-bit values, row-major
 * with row strides ld in elements, multiples of 8 (of one row it does not
 * matter), 16-byte aligned; H, k_in, n_out are multiples of 8 (LORA_ERR_ALIGN).
 * No output, the workspace and the error word among them, may share memory with
 * another argument (LORA_ERR_ARG), but for `out` with `residual` as stated.
 * Columns of one buffer may interleave.
 * Limits: E <= 1024, top_k <= 64, T * top_k < 2^30, n <= 2^30 rows of a product
 * (LORA_ERR_UNSUPPORTED).
 */
#define LORA_MOE_MAX_TOP_K 64

/*
 * lora_moe_dispatch -- the tokens' rows sorted by expert, stable in p, and the
 * plan that leads back.
 *   topk_ids [T, top_k] int32: -1 is no expert (a padded token), silently; an id
 *     outside [0, E) gets no row either, with LORA_DEV_ERR_EXPERT.
 *   expert_map [n_global_experts] int32 or NULL: as in lora_moe_w13_delta, global
 *     expert id -> this rank's id, -1 = not on this rank (no row).
 *   lora_ids [T] int32 or NULL (all -1): the token's adapter.
 *   seg_start [E + 1] int32 (out): expert e's rows are seg_start[e] ..
 *     seg_start[e + 1] - 1; seg_start[0] is 0.
 *   pair_row [T, top_k] int32 (out): the pair's row, -1: none.
 *   row_pair, row_expert, row_lora [T * top_k] int32 (out): the row's pair, expert
 *     and its token's adapter; -1 from row seg_start[E] on.
 *   rows [T * top_k, H] (out): rows[pair_row[t, j]] = x[t]; rows from seg_start[E]
 *     on are left as they were.
 * The gradient for x is lora_moe_combine of the rows' gradients without weights.
 */
int lora_moe_dispatch(void *rows, int64_t ld_rows, int32_t *seg_start, int32_t *row_pair,
                      int32_t *pair_row, int32_t *row_expert, int32_t *row_lora, const void *x,
                      int64_t ld_x, const int32_t *topk_ids, const int32_t *lora_ids,
                      const int32_t *expert_map, int n_global_experts, int T, int top_k, int E,
                      int H, uint32_t *err_word, lora_stream_t stream);

/*
 * lora_moe_combine -- the rows back at their tokens:
 *   out[t] = RN(residual[t] + sum_j weights[t, j] * rows[pair_row[t, j]])
 * over the pairs that have a row (pair_row inside [0, T * top_k)), in float32 and
 * in the order of j.  weights [T, top_k] float32 or NULL (1); residual [T, H] or
 * NULL (0), which may be `out` itself with the same row stride.  A token without a
 * row gets its residual.  dtype: LORA_BF16 or LORA_F16.
 */
int lora_moe_combine(void *out, int64_t ld_out, const void *rows, int64_t ld_rows,
                     const int32_t *pair_row, const float *weights, const void *residual,
                     int64_t ld_residual, int T, int top_k, int H, int dtype,
                     lora_stream_t stream);

/*
 * lora_moe_combine_grad -- the gradient of lora_moe_combine for its rows and
 * weights (that for the residual is grad_out itself):
 *   grad_rows[pair_row[t, j]] = RN(weights[t, j] * grad_out[t])
 *   grad_weights[t, j] = grad_out[t] . rows[pair_row[t, j]]   (float32; 0 without a row)
 * grad_weights [T, top_k] float32 or NULL.  Rows that no pair has are left as
 * they were.
 */
int lora_moe_combine_grad(void *grad_rows, int64_t ld_grad_rows, float *grad_weights,
                          const void *grad_out, int64_t ld_grad_out, const void *rows,
                          int64_t ld_rows, const int32_t *pair_row, const float *weights, int T,
                          int top_k, int H, int dtype, lora_stream_t stream);

/* activations of the products below */
#define LORA_ACT_NONE 0
#define LORA_ACT_RELU 1
#define LORA_ACT_SILU 2
#define LORA_ACT_GELU 3      /* 0.5 z (1 + erf(z / sqrt 2)) */
#define LORA_ACT_GELU_TANH 4 /* 0.5 z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) */

/*
 * lora_linear -- the base layer that a delta belongs to: x [n, k_in] times
 * w [n_out, k_in] transposed, with everything after it in one pass:
 *   z = x w^T + bias + delta                        (float32)
 *   out = RN(act(z) + residual)                     gated == 0: [n, n_out]
 *   out = RN(act(z[:, :I]) * z[:, I:] + residual)   gated == 1: [n, I], I = n_out / 2
 * bias [n_out], delta [n, n_out], residual (as out) or NULL, of x's type; the
 * residual may be `out` itself with the same row stride.  delta is added ahead
 * of the activation, where an adapter's part belongs.  gated == 1 needs n_out a
 * multiple of 16.
 * workspace: lora_linear_workspace_size(n, 1) bytes (0, or some 42 MB at any size),
 * 256-byte aligned, or NULL: with it, tiles may be shared by several SMs along k_in
 * where there are not enough for all.  Its first lora_linear_zeroed_bytes() bytes must be
 * zero before its first use and are left zero, after LORA_DEV_ERR_TIMEOUT too; calls that
 * may overlap (a graph's replays among them) need workspaces of their own.
 */
size_t lora_linear_workspace_size(int n, int groups);
size_t lora_linear_zeroed_bytes(void);
int lora_linear(void *out, int64_t ld_out, const void *x, int64_t ld_x, int n, int k_in,
                const void *w, int64_t ld_w, int n_out, const void *bias, const void *delta,
                int64_t ld_delta, const void *residual, int64_t ld_residual, int activation,
                int gated, int dtype, void *workspace, size_t ws_bytes, uint32_t *err_word,
                lora_stream_t stream);

/*
 * lora_moe_linear -- lora_linear for sorted rows, each expert's with its own
 * weights: rows seg_start[e] .. seg_start[e + 1] - 1 take w + e * stride_w
 * elements (a multiple of ld_w) and bias [E, n_out].  seg_start [E + 1] int32 (device), as
 * lora_moe_dispatch writes it, must be nondecreasing within [0, n]; starts outside
 * are clamped with LORA_DEV_ERR_SEGMENT, and what rows get then is not specified.
 * Rows outside every segment are left as they were, and what x, delta and residual
 * hold there has no influence.  workspace: lora_linear_workspace_size(n, E) bytes, as
 * for lora_linear.
 */
int lora_moe_linear(void *out, int64_t ld_out, const void *rows, int64_t ld_rows, int n, int k_in,
                    const int32_t *seg_start, int E, const void *w, int64_t ld_w,
                    int64_t stride_w, int n_out, const void *bias, const void *delta,
                    int64_t ld_delta, const void *residual, int64_t ld_residual, int activation,
                    int gated, int dtype, void *workspace, size_t ws_bytes, uint32_t *err_word,
                    lora_stream_t stream);

/*
 * lora_get_error -- copy the device error word to *host_out after all work
 * queued on `stream` so far has finished (this call synchronizes `stream`),
 * then clear it on the device when `clear` is nonzero.
 */
int lora_get_error(uint32_t *err_word, uint32_t *host_out, int clear, lora_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LORA_DELTA_H */

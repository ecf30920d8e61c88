/*
 * moe.h -- C ABI of the GB300 (sm_103a) Mixture-of-Experts SwiGLU FFN layer, forward and backward.
 *
 * One GPU, one CUDA stream per call, no host synchronisation on the compute path.  Every entry
 * point takes plain pointers and sizes; the caller owns and allocates every buffer (device
 * memory unless stated otherwise).  The library never allocates device memory.
 *
 * The layer (the pages give the systems around it, not its formulas; see "readings" below):
 *   logits = x W_r (+ b_r)                          [T,E] fp32
 *   p      = softmax(logits) over the E routed experts
 *   idx    = top-k experts by logit, larger first, a tie going to the lower expert index
 *   gates  = p[idx]  (renormalised over the k selected when cfg.renorm != 0)
 *   dispatch: per-expert queues in token order (histogram, exclusive prefix sum, stable
 *             permutation); with a capacity C = ceil(cf*T*k/E) the positions >= C are dropped
 *   expert e: h = silu(x_r W_gate[e]^T) * (x_r W_up[e]^T),  o = h W_down[e]^T
 *   y_t    = sum over kept slots j of gates[t,j] * o_{t,j}  +  sum over shared experts s of o^s_t
 *
 * Sources on the pages:
 *   - "MoEBlaze: Breaking the Memory Wall for Efficient MoE Training on Modern GPUs" (Korean
 *     summary): Methodology item 1 (dispatch queues instead of a dense token-by-expert routing
 *     matrix), item 2 (fused scatter/gather around the expert FFN; activation checkpointing that
 *     keeps a minimum and recomputes the rest in backward), the training-loop figure (fused
 *     expert kernels forward, checkpoint, fused expert kernels backward, gradient reduce) and
 *     Limitations (static top-k routing).
 *   - "Piper: Efficient Large-Scale MoE Training via Resource Modeling and Pipelined Hybrid
 *     Parallelism" (Japanese explainer, "the problem"): the router picks a few experts per
 *     token; loads can be heavily skewed; fine-grained experts give tall-and-skinny GEMMs.
 *   - "DisagMoE" technical summary, section 2.2: dispatch and combine around the expert FFN.
 *
 * Readings where the pages are silent: softmax over all E then top-k; selection by logit with
 * ties to the lower index; slot order = descending logit; capacity drops in token order (t, then
 * slot); dropped slots contribute zero and get zero gate gradient; kept gates are not
 * renormalised after drops; shared experts have weight 1 and sit outside softmax/top-k; SwiGLU
 * without biases.
 *
 * Data types and layouts (all row-major, contiguous):
 *   bf16 values are passed as raw 16-bit patterns (moe_bf16).
 *   x, y, dy, dx          [T, d_model]          bf16
 *   W_r                   [d_model, E]          fp32       b_r [E] fp32 (nullable)
 *   W_gate, W_up          [E+S, d_ff, d_model]  bf16       (out x in, like torch Linear)
 *   W_down                [E+S, d_model, d_ff]  bf16
 *   experts E..E+S-1 are the S shared (always-on) experts.
 *   idx                   [T, k] int32          gates, dgates [T, k] fp32
 *   dW_r                  [d_model, E] fp32     db_r [E] fp32
 *   dW_gate, dW_up, dW_down: same shapes as the weights, bf16, OVERWRITTEN (not accumulated).
 *
 * Expert-ordered ("permuted") rows.  moe_dispatch writes x_perm in a padded, expert-contiguous
 * layout with room for moe_perm_rows() rows:
 *   segment g (routed experts g < E first, then shared experts) starts at row P_g, a multiple of
 *   256; P_0 = 0, P_{g+1} = P_g + roundup(n_g, 256), where n_g = min(counts[g], C) for routed
 *   experts and n_g = T for shared ones.  Rows P_g + n_g .. P_{g+1}-1 are zero padding.
 *   The kept assignment (t, j) of expert e with queue position q sits at row P_e + q; shared
 *   expert s sees token t at row P_{E+s} + t.
 * The exact (unpadded) numbering is reported as well: offsets[e] is the exclusive prefix sum of
 * the kept counts and row_of_slot[t,j] = offsets[e] + q (or -1 when dropped).
 *
 * Kept activations (MoEBlaze, Methodology item 2: selective checkpointing, here with an adjustable
 * granularity).  By default the backward recomputes the SwiGLU pre-activations a = x W_gate^T and
 * b = x W_up^T from x_perm.  With keep_rows > 0, the forward also writes a and b (bf16) of the
 * first keep_rows expert-ordered rows (rounded down to a multiple of 256, at most all rows), and the
 * backward takes them instead of recomputing those rows: 2 * d_ff * 2 bytes kept per row buy
 * 4 * d_model * d_ff FLOP per row.  moe_layer_fwd / moe_layer_bwd keep them in `saved` (which grows
 * by those bytes: moe_workspace_size), so the workspace stays free for other layers between the
 * forward and the backward; moe_expert_ffn_fwd / moe_expert_ffn_bwd keep them in the workspace,
 * which must then reach the matching backward untouched.  moe_keep_rows_for_budget chooses
 * keep_rows from a byte budget (the adaptive granularity of the MoEBlaze summary's future work).
 *
 * Gathered operand loads (MoEBlaze summary, Methodology item 2, first bullet: the dispatch gather
 * fused with the expert feed-forward).  With gather_in_gemm = 1, moe_layer_fwd and moe_layer_bwd
 * write no x_perm or dY_perm: the dispatch builds its tables and the token of every padded row, and
 * the GEMMs that read those rows (gate/up, dh', the recompute, the weight gradients) fetch them from
 * x and dy in token order, four rows per TMA tile::gather4 copy, from four producer warps.  For
 * finite x and dy the results are those of gather_in_gemm = 0 bit for bit (a pad row reads token 0's
 * row instead of zeros, and its zero gate zeroes every gradient term it feeds).  It is the slower
 * choice on GB300: a stage's
 * 32 gather copies take about twice as long as the tensor cores' work on it, where one TMA box of a
 * contiguous x_perm tile keeps up, so the GEMMs that gather run at about half their speed while the
 * separate gather they save costs 0.1 to 0.5 ms per step.  It saves the x_perm and dY_perm traffic
 * (2 (T + N) d bytes each way) for a workload where that matters more than GEMM time.
 *
 * Workspace.  Size it with moe_workspace_size(), zero its header once with moe_workspace_init(),
 * and pass the same workspace to every call of one layer instance.  moe_dispatch leaves the
 * routing tables in it that moe_expert_ffn_fwd/bwd, moe_combine and moe_combine_bwd read; the
 * fused moe_layer_fwd/bwd keep all their intermediates there.  Calls that share a workspace
 * must be ordered on one stream.
 *
 * Errors.  Argument checks are synchronous: a call that returns anything but MOE_OK enqueued no
 * work.  Errors found on the device (an expert id out of range, a bounded wait that ran out)
 * are recorded in the workspace; moe_check_error() synchronises the stream, returns the first
 * such error since the last check, and clears it.  Device waits never spin unboundedly.
 *
 * Requirements: 1 <= k <= E <= 256; 0 <= S <= 8; d_model and d_ff multiples of 64 and <= 16384;
 * 1 <= T <= 1048576 and T*k <= 2^24; every pointer 16-byte aligned; sm_103a device.
 */
#ifndef MOE_GB300_H
#define MOE_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MOE_OK = 0,
    MOE_ERR_INVALID_ARG = 1,   /* a null pointer, a misaligned pointer or a shape out of range */
    MOE_ERR_UNSUPPORTED = 2,   /* a valid shape the library does not handle (or not an sm_103 device) */
    MOE_ERR_WORKSPACE = 3,     /* workspace smaller than moe_workspace_size() */
    MOE_ERR_CUDA = 4,          /* a CUDA runtime/driver call failed */
    MOE_ERR_BAD_INDEX = 5,     /* (device) an expert id outside [0, E): the dispatch that saw it
                                * publishes no rows (see moe_dispatch); or a group's rows out of
                                * range or out of order (see "Grouped products") */
    MOE_ERR_TIMEOUT = 6        /* (device) a bounded wait ran out; outputs of that call are invalid */
} moe_status_t;

typedef struct {
    int32_t T;                 /* tokens */
    int32_t d_model;           /* model width d */
    int32_t d_ff;              /* expert hidden width f */
    int32_t E;                 /* routed experts */
    int32_t k;                 /* experts per token */
    int32_t n_shared;          /* S always-on shared experts */
    int32_t renorm;            /* 1: gates renormalised over the k selected */
    float capacity_factor;     /* cf > 0: capacity ceil(cf*T*k/E) per expert; <= 0: dropless */
    int32_t keep_rows;         /* >= 0: expert-ordered rows whose gate/up pre-activations the forward
                                * keeps for the backward (see "Kept activations"); 0 recomputes all */
    int32_t gather_in_gemm;    /* 0 or 1, moe_layer_fwd / moe_layer_bwd only: 1 gathers the x and dy
                                * rows inside the expert GEMMs' operand loads (TMA tile::gather4 from
                                * token order) instead of copying them to x_perm / dY_perm first;
                                * same results, slower on GB300 (see "Gathered operand loads") */
} moe_config_t;

typedef uint16_t moe_bf16;                 /* raw bf16 bit pattern */
typedef struct CUstream_st* moe_stream_t;  /* a cudaStream_t; NULL is the legacy default stream */

/* Workspace bytes for any call of this configuration, and bytes of the `saved` buffer that
 * moe_layer_fwd fills and moe_layer_bwd reads: idx int32 [T,k], then gates fp32 [T,k], then, when
 * the gates are not renormalised, from the next 256-byte boundary the router logits fp32 [T,E]
 * (bias included: the backward's softmax reads them instead of recomputing x W_r), then, when
 * keep_rows > 0, from the next 256-byte boundary the kept a and b [keep, d_ff] bf16 (keep =
 * keep_rows rounded down to 256, at most moe_perm_rows()).  Host only; touches no device. */
moe_status_t moe_workspace_size(const moe_config_t* cfg, size_t* ws_bytes, size_t* saved_bytes);

/* Where the parts of `saved` after idx and gates sit (the layout above): the logits' byte offset
 * and size (both 0 with renormalised gates, which keep none), and the kept a, b block's offset and
 * size (a first, b right after it; size 0 when keep_rows is 0).  Every pointer is nullable.  Host
 * only; touches no device. */
moe_status_t moe_saved_layout(const moe_config_t* cfg, size_t* logits_off, size_t* logits_bytes, size_t* kept_off,
                              size_t* kept_bytes);

/* Checkpoint granularity from a memory budget (MoEBlaze summary, Limitations and future work:
 * adaptive checkpoint granularity driven by memory pressure at run time; Methodology item 2: keep
 * a minimum and recompute the rest).  *keep_rows receives the largest keep_rows (a multiple of 256,
 * at most moe_perm_rows()) whose kept a and b -- 4 * d_ff bytes per expert-ordered row, the bytes
 * `saved` grows by -- fit in budget_bytes; *kept_bytes (nullable) receives those bytes.  The
 * cfg's own keep_rows is ignored; set it to the result.  Rows kept cost no recompute GEMM work in
 * the backward (4 * d_model * d_ff FLOP each).  Host only; touches no device. */
moe_status_t moe_keep_rows_for_budget(const moe_config_t* cfg, uint64_t budget_bytes, int32_t* keep_rows,
                                      uint64_t* kept_bytes);

/* The same with the budget taken from the current device's free memory at the time of the call
 * (cudaMemGetInfo) less reserve_bytes (0 if free memory is below it): the kept share follows the
 * memory pressure of each step.  MOE_ERR_CUDA if the query fails. */
moe_status_t moe_keep_rows_for_free_memory(const moe_config_t* cfg, uint64_t reserve_bytes, int32_t* keep_rows,
                                           uint64_t* kept_bytes);

/* Rows (capacity) of x_perm / o_perm / dx_perm buffers: each is [rows, d_model] bf16.  Host only. */
moe_status_t moe_perm_rows(const moe_config_t* cfg, int64_t* rows);

/* Zero the workspace header (error word and device counters).  Call once after allocating. */
moe_status_t moe_workspace_init(const moe_config_t* cfg, void* ws, size_t ws_bytes, moe_stream_t stream);

/* Router (Piper explainer, "the problem": a router sends each token to a few experts; MoEBlaze
 * summary, Limitations: a static top-k routing policy): logits, softmax, top-k and gates for every
 * token, by the readings above.  b_r and logits may be NULL.  Writes idx [T,k], gates [T,k], and
 * logits [T,E] when non-NULL.  ws is this configuration's workspace (moe_workspace_size).  For
 * E <= 128 and k <= 8 the logits run on the tensor cores: W_r is split in ws into three bf16 parts
 * whose sum equals it within fp32 rounding, and the products are summed in fp32 over 256-wide
 * slices of d_model (E <= 32: the parts stacked in one MMA and d_model split across CTAs, so that
 * the whole GPU streams x); other shapes use an fp32 tile product with warp-per-token selection. */
moe_status_t moe_route(const moe_config_t* cfg, const moe_bf16* x, const float* W_r, const float* b_r,
                       int32_t* idx, float* gates, float* logits, void* ws, size_t ws_bytes,
                       moe_stream_t stream);

/* Dispatch queues (MoEBlaze, Methodology item 1): per-expert histogram, exclusive prefix sum with
 * a decoupled look-back, stable (token-order) ranks, capacity, and the 16-byte gather of x rows into
 * x_perm (padded layout above; pad rows are zeroed; shared-expert segments hold copies of x).
 * Outputs: counts [E] (raw demand, sums to T*k), offsets [E+1] (exact), row_of_slot [T,k]
 * (exact row or -1), token_of_row [T*k] (entries >= offsets[E] are left untouched),
 * x_perm [moe_perm_rows(), d_model].  Leaves the padded tables in ws for the calls below.
 * An id outside [0,E) anywhere in idx records MOE_ERR_BAD_INDEX (read with moe_check_error) and
 * empties the whole dispatch, since the queue positions of that call cannot be trusted: counts
 * still hold the demand of the valid ids, but every segment is published with no rows (offsets
 * all 0, row_of_slot all -1, token_of_row and x_perm not written), so the calls that follow on
 * this workspace touch no rows.  The next dispatch with valid ids starts afresh. */
moe_status_t moe_dispatch(const moe_config_t* cfg, const int32_t* idx, const moe_bf16* x,
                          int32_t* counts, int32_t* offsets, int32_t* row_of_slot, int32_t* token_of_row,
                          moe_bf16* x_perm, void* ws, size_t ws_bytes, moe_stream_t stream);

/* moe_dispatch for callers that cannot allocate device memory: no workspace argument.  (The
 * pages have no counterpart; this exists for integration.)  Meant for code that runs where
 * cudaMalloc is not available or not allowed: inside a memory arena or pool owned by a host
 * framework that cannot grow at step time, or on a path that must not pay cudaMalloc's implicit
 * synchronisation.  Outputs and their meaning are those of moe_dispatch (counts, offsets,
 * row_of_slot, token_of_row, x_perm with room for moe_perm_rows() rows); the caller still
 * provides every input and output buffer.
 * Scratch: a fixed device array of about 3.6 MB inside the library, which every GPU that loads
 * the library holds until the process exits.  Limits: T*k <= 262144 assignments and
 * moe_perm_rows() <= 393216 rows; larger configurations return MOE_ERR_UNSUPPORTED and enqueue
 * nothing.  The first call on each device looks up the array's device address
 * (cudaGetSymbolAddress, with that device current); make that first call before any stream
 * capture.  (The address is looked up again on every call, so a device reset or a re-created
 * primary context between calls is safe.)  The call allocates nothing: no cudaMalloc, cudaFree or
 * allocating library routine.
 * Every call shares the one array and leaves its contents behind (each call clears what must
 * start at zero), so calls that may overlap on the GPU -- on different streams, or from several
 * host threads -- race and must be serialised by the caller.
 * status: nullable device pointer to one int32 (4-byte aligned).  With no workspace there is no
 * error word for moe_check_error, so the call's device-side outcome lands here, written on the
 * stream after the scan: MOE_OK, MOE_ERR_BAD_INDEX (an id outside [0,E); as in moe_dispatch the
 * whole dispatch is then empty: offsets all 0, row_of_slot all -1, token_of_row and x_perm not
 * written) or MOE_ERR_TIMEOUT (a bounded wait ran out; outputs invalid).  Read it after the
 * stream's work completes.  With status NULL a bad id still empties the dispatch, unreported. */
moe_status_t moe_dispatch_noalloc(const moe_config_t* cfg, const int32_t* idx, const moe_bf16* x,
                                  int32_t* counts, int32_t* offsets, int32_t* row_of_slot,
                                  int32_t* token_of_row, moe_bf16* x_perm, int32_t* status,
                                  moe_stream_t stream);

/* Grouped expert SwiGLU FFN on the rows moe_dispatch laid out in ws: tcgen05/TMEM tiles fed by
 * TMA, a per-expert tile scheduler, SwiGLU fused into the first GEMM's epilogue.
 * o_perm [moe_perm_rows(), d_model] bf16 receives every segment's rows (pad rows are zero). */
moe_status_t moe_expert_ffn_fwd(const moe_config_t* cfg, const moe_bf16* x_perm,
                                const moe_bf16* W_gate, const moe_bf16* W_up, const moe_bf16* W_down,
                                moe_bf16* o_perm, void* ws, size_t ws_bytes, moe_stream_t stream);

/* Weighted combine back to token order (MoEBlaze summary, Methodology item 2: the reverse
 * dispatch after the expert FFN; DisagMoE technical summary, section 2.2: combine), by token owner
 * (no atomics, fixed slot order, fp32 sums, one rounding):
 * y[t] = sum_kept gates[t,j] o_perm[row(t,j)] + sum_s o_perm[P_{E+s}+t].  Reads the row tables
 * moe_dispatch left in ws. */
moe_status_t moe_combine(const moe_config_t* cfg, const moe_bf16* o_perm, const float* gates,
                         moe_bf16* y, void* ws, size_t ws_bytes, moe_stream_t stream);

/* Backward of the expert FFN and of the combine's gate weighting, recomputing the SwiGLU
 * activations from x_perm (MoEBlaze, Methodology item 2: selective checkpointing).
 * Reads dy [T,d] in token order; writes dx_perm [moe_perm_rows(), d_model] (gradient of x_perm,
 * padded layout), dgates [T,k] (dy . o, zero for dropped slots), dW_gate, dW_up, dW_down. */
moe_status_t moe_expert_ffn_bwd(const moe_config_t* cfg, const moe_bf16* x_perm, const moe_bf16* dy,
                                const float* gates,
                                const moe_bf16* W_gate, const moe_bf16* W_up, const moe_bf16* W_down,
                                moe_bf16* dx_perm, float* dgates,
                                moe_bf16* dW_gate, moe_bf16* dW_up, moe_bf16* dW_down,
                                void* ws, size_t ws_bytes, moe_stream_t stream);

/* Router backward with the selection held fixed: recompute logits from x, then
 * dlogits [T,E] fp32 from dgates, dW_r = x^T dlogits, db_r = sum_t dlogits (db_r nullable).
 * Without renorm: dl_e = p_e (dg_{slot(e)} [e selected] - sum_j dg_j g_j); with renorm:
 * dl_{idx_j} = g_j (dg_j - sum_m dg_m g_m) and 0 elsewhere.  b_r nullable. */
moe_status_t moe_router_bwd(const moe_config_t* cfg, const moe_bf16* x, const float* W_r, const float* b_r,
                            const int32_t* idx, const float* gates, const float* dgates,
                            float* dlogits, float* dW_r, float* db_r,
                            void* ws, size_t ws_bytes, moe_stream_t stream);

/* Input gradient, by token owner: dx[t] = sum_kept dx_perm[row(t,j)] + sum_s dx_perm[P_{E+s}+t]
 * + dlogits[t] W_r^T.  dlogits may be NULL (no router term).  Uses the tables of moe_dispatch. */
moe_status_t moe_combine_bwd(const moe_config_t* cfg, const moe_bf16* dx_perm, const float* dlogits,
                             const float* W_r, moe_bf16* dx, void* ws, size_t ws_bytes, moe_stream_t stream);

/* FP8 expert GEMMs, forward (the MoEBlaze summary names mixed-precision and quantised experts as
 * future work; the format is this library's reading).  Format: OCP FP8 E4M3 (max 448, no
 * infinities), one fp32 scale per row.  The steps are exposed one by one (quantise, gate/up, down)
 * and composed by moe_layer_fwd_fp8 below.
 *
 * moe_quantize_rows_e4m3: src [rows, cols] bf16 -> codes [rows, cols] uint8 and scales [rows]
 * fp32, with scale = amax / 448 over the row (1 for an all-zero row) and code = e4m3(v / scale),
 * both in fp32, rounded to nearest even and saturated.  cols a multiple of 16, at most 16384;
 * 16-byte-aligned pointers.  Used for token or x_perm rows, h rows, and the rows (output channels)
 * of W_gate, W_up and W_down.  Argument errors are returned before any work is queued. */
moe_status_t moe_quantize_rows_e4m3(const moe_bf16* src, int64_t rows, int32_t cols, uint8_t* codes,
                                    float* scales, moe_stream_t stream);

/* The gate/up projection and SwiGLU of moe_expert_ffn_fwd with e4m3 operands on the tensor cores
 * (kind::f8f6f4): h = silu(a) * b, a = s_x s_g (q_x . q_g), b = s_x s_u (q_x . q_u), accumulated in
 * fp32.  x8 / x_scale: the quantised x_perm rows [moe_perm_rows(), d_model] / [moe_perm_rows()]
 * (pad rows: zero codes); wg8, wu8 [E+S, d_ff, d_model] codes with wg_scale, wu_scale [E+S, d_ff].
 * Writes h [moe_perm_rows(), d_ff] bf16.  Uses the tables of moe_dispatch in ws. */
moe_status_t moe_gate_up_fp8(const moe_config_t* cfg, const uint8_t* x8, const float* x_scale,
                             const uint8_t* wg8, const float* wg_scale, const uint8_t* wu8,
                             const float* wu_scale, moe_bf16* h, void* ws, size_t ws_bytes,
                             moe_stream_t stream);

/* The down projection with e4m3 operands: o = s_h s_d (q_h . q_d) per row and output channel,
 * accumulated in fp32 and stored bf16.  h8 / h_scale: quantised h rows [moe_perm_rows(), d_ff] /
 * [moe_perm_rows()] (moe_quantize_rows_e4m3 of h); wd8 [E+S, d_model, d_ff] codes with wd_scale
 * [E+S, d_model] (one scale per output channel: the rows of W_down).  Writes o_perm
 * [moe_perm_rows(), d_model] bf16.  Uses the tables of moe_dispatch in ws. */
moe_status_t moe_down_fp8(const moe_config_t* cfg, const uint8_t* h8, const float* h_scale, const uint8_t* wd8,
                          const float* wd_scale, moe_bf16* o_perm, void* ws, size_t ws_bytes,
                          moe_stream_t stream);

/* The whole forward with e4m3 expert GEMMs: route as moe_layer_fwd; quantise the T token rows of
 * x once (a row's codes are the same in every expert it visits); dispatch, gathering those codes
 * and row scales into the padded expert rows; moe_gate_up_fp8 (h kept in bf16); quantise the h
 * rows this step fills; moe_down_fp8; and the combine.  The weights come quantised
 * (moe_quantize_rows_e4m3 of every row of W_gate, W_up and W_down, as above).  The router stays
 * fp32.  Fills `saved` like moe_layer_fwd (idx, gates, logits), so moe_layer_bwd can follow with
 * the bf16 weights.
 * keep_rows must be 0 (MOE_ERR_INVALID_ARG otherwise): the call's scratch uses the workspace
 * buffers that would carry kept activations to the backward. */
moe_status_t moe_layer_fwd_fp8(const moe_config_t* cfg, const moe_bf16* x, const float* W_r, const float* b_r,
                               const uint8_t* wg8, const float* wg_scale, const uint8_t* wu8,
                               const float* wu_scale, const uint8_t* wd8, const float* wd_scale, moe_bf16* y,
                               void* saved, void* ws, size_t ws_bytes, moe_stream_t stream);

/* Per-column e4m3 codes, written transposed, for the FP8 backward's weights (same format as
 * moe_quantize_rows_e4m3: scale = amax / 448 over the column, 1 for an all-zero column; code =
 * e4m3(v / scale) rounded to nearest even and saturated, both in fp32).  For each of G experts the
 * source is [top[g]; bottom[g]], rows_top + rows_bottom rows of `cols` bf16 values (bottom NULL when
 * rows_bottom is 0); codes[g] receives its transpose [cols, rows_top + rows_bottom] and scales[g]
 * one scale per column.  Used as
 *   W_down [G, d, f]                     -> codes [G, f, d], scales [G, f]   (top = W_down)
 *   W_gate, W_up [G, f, d] (stacked)     -> codes [G, d, 2f], scales [G, d]  (top = W_gate, bottom = W_up)
 * rows_top + rows_bottom a multiple of 16, at most 32768; 16-byte-aligned pointers.  The column
 * maxima are gathered in `scales` before it receives the scales.  Argument errors return before
 * any work is queued. */
moe_status_t moe_quantize_cols_e4m3(const moe_bf16* top, const moe_bf16* bottom, int64_t G, int32_t rows_top,
                                    int32_t rows_bottom, int32_t cols, uint8_t* codes, float* scales,
                                    moe_stream_t stream);

/* The whole backward with e4m3 expert GEMMs (the MoEBlaze summary names mixed-precision and
 * quantised experts as future work; the format is this library's reading): as moe_layer_bwd, with
 *   dh' = (s_dy q_dy) (s_wd q_wd)^T     dY rows quantised per row; W_down's columns per d_ff channel
 *                                       (wdt8, wdt_scale from moe_quantize_cols_e4m3 of W_down)
 *   a, b = the forward's e4m3 products, recomputed from the x rows (quantised per row) and the
 *          forward's row codes of W_gate and W_up (wg8, wg_scale, wu8, wu_scale)
 *   dA, dB, Hg from the SwiGLU backward in fp32, held in bf16 (dh' too)
 *   dX = (s_ab q_ab) (s_w q_w)^T        the joined row [dA | dB] quantised per row; column i of
 *                                       W_gate and W_up quantised together per d_model channel
 *                                       (wgut8, wgut_scale from moe_quantize_cols_e4m3 of W_gate over W_up)
 * accumulated in fp32.  The weight gradients stay bf16 products of dA, dB, Hg and the bf16 x and dY
 * rows; the router stays fp32.  `saved` comes from moe_layer_fwd or moe_layer_fwd_fp8 of the same
 * configuration; keep_rows must be 0 (MOE_ERR_INVALID_ARG otherwise). */
moe_status_t moe_layer_bwd_fp8(const moe_config_t* cfg, const moe_bf16* x, const float* W_r, const float* b_r,
                               const uint8_t* wg8, const float* wg_scale, const uint8_t* wu8, const float* wu_scale,
                               const uint8_t* wdt8, const float* wdt_scale, const uint8_t* wgut8,
                               const float* wgut_scale, const void* saved, const moe_bf16* dy, moe_bf16* dx,
                               float* dW_r, float* db_r, moe_bf16* dW_gate, moe_bf16* dW_up, moe_bf16* dW_down,
                               void* ws, size_t ws_bytes, moe_stream_t stream);

/* The whole forward: route, dispatch, expert FFN, combine (MoEBlaze summary, the training-loop
 * figure: fused expert kernels forward, then checkpoint).  Fills `saved` with idx and gates, the
 * router logits (gates not renormalised; T * E fp32, small beside x), and the kept a and b of the
 * first keep_rows expert-ordered rows when keep_rows > 0; every other activation is recomputed in
 * the backward (Methodology item 2). */
moe_status_t moe_layer_fwd(const moe_config_t* cfg, const moe_bf16* x, const float* W_r, const float* b_r,
                           const moe_bf16* W_gate, const moe_bf16* W_up, const moe_bf16* W_down,
                           moe_bf16* y, void* saved, void* ws, size_t ws_bytes, moe_stream_t stream);

/* The whole backward from x, the weights, `saved` and dy (MoEBlaze summary, the training-loop
 * figure: fused expert kernels backward, then gradient reduce): rebuilds the dispatch queues from
 * the saved idx, recomputes the expert activations of the rows not kept (Methodology item 2), takes
 * the router's softmax from the saved logits, and writes dx, dW_r, db_r (nullable) and the expert
 * weight gradients.  `saved` must come from moe_layer_fwd of the same configuration (keep_rows
 * included); a caller that writes idx and gates into it by hand writes the logits too. */
moe_status_t moe_layer_bwd(const moe_config_t* cfg, const moe_bf16* x, const float* W_r, const float* b_r,
                           const moe_bf16* W_gate, const moe_bf16* W_up, const moe_bf16* W_down,
                           const void* saved, const moe_bf16* dy,
                           moe_bf16* dx, float* dW_r, float* db_r,
                           moe_bf16* dW_gate, moe_bf16* dW_up, moe_bf16* dW_down,
                           void* ws, size_t ws_bytes, moe_stream_t stream);

/* Types of the calls below. */
typedef enum { MOE_BF16 = 0, MOE_FP16 = 1, MOE_FP32 = 2 } moe_dtype_t;

/* ---- Expert selection ----------------------------------------------------------------------------
 * The choice of experts from router logits, apart from the product that makes them: for routers other than the
 * layer's softmax and top-k (sigmoid scores, a bias that balances the load, groups of experts, scaled
 * weights), on the logits of moe_route or of the caller's own router.  The layer's other calls take what it
 * gives: moe_dispatch the experts, moe_combine the weights; back through them, moe_select_bwd makes dlogits of
 * the weights' gradients, moe_combine_bwd the input gradient and moe_router_wgrad the router's (the layer's calls have
 * limits of their own: 256 experts, 2^20 tokens).
 *
 * For every token, with logits l [E] and the bias b [E]:
 *   s_e     = softmax(l)_e or sigmoid(l_e)
 *   key_e   = s_e + b_e                                  (the bias enters the keys only)
 *   groups  of E / groups consecutive experts, scored by the sum of their group_top largest keys; the
 *             top_groups best stay (a tie goes to the lower group)
 *   idx     = the k largest keys among the groups that stay, larger first (a tie goes to the lower expert)
 *   w_j     = s[idx_j], with renorm s[idx_j] / sum_m s[idx_m]; times scale
 * The order of experts and groups is that of keys formed, and added up, in 64 bits, whatever the type of the logits and the
 * size of the biases (two that are nearer than 64 bits' own rounding go as they round), and where there is no bias and no
 * sum of two keys, that of the logits, which is the scores' own.  Weights and gradients are computed in 32 bits, and
 * renormalised weights are finite and sum to scale however small the scores.
 *
 * Masks.  A logit of -inf masks its expert, as do a NaN and a bias of -inf or NaN: it counts in no group's
 * score, a group of masked experts only comes last, and it is chosen only where its token has fewer than k others left
 * (then by lower index, after them), so that idx is always k different experts.  A score of -inf is 0, and so are the
 * weight and its gradient, whatever came back for it; a token of nothing else has weights of 0.  A NaN or
 * +inf makes NaN of the weights that a NaN or an infinite softmax enters: all of a token with softmax not
 * renormalised, else those of the slots that hold one, and with renorm of the whole token.
 *
 * The gradient, c = dweights, the selection held (the bias has none), h_j = w_j / scale:
 *   renorm       dl of slot j's expert += w_j (c_j - sum_m c_m h_m), with sigmoid times 1 - s_j
 *   else         sigmoid: += scale c_j s_j (1 - s_j);  softmax: dl_e = scale p_e (c_slot(e) - sum_m c_m p_m)
 * and 0 elsewhere.  A slot whose idx is out of range has no part in it; one expert in several slots gets the sum of their
 * terms, in slot order.
 *
 * Nothing is kept between calls, no workspace is needed, results are the same on every run, and calls on several
 * streams do not disturb each other.  logits and dlogits are 16-byte aligned, the others 4-byte; outputs do not
 * overlap inputs. */
typedef enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 } moe_score_t;

typedef struct {
    int32_t T;                 /* tokens, 0 .. 2^24 */
    int32_t E, k;              /* experts, 1 .. 1024; experts of a token, 1 .. 32, at most those of top_groups groups */
    int32_t score;             /* MOE_SCORE_SOFTMAX or MOE_SCORE_SIGMOID */
    int32_t groups;            /* of experts: 1 .. 64, a divisor of E; 1: none */
    int32_t top_groups;        /* groups that stay, 1 .. groups */
    int32_t group_top;         /* keys summed to a group's score: 1 or 2 */
    int32_t renorm;            /* 1: weights divided by their sum over the k slots */
    float scale;               /* of the weights */
    int32_t dtype;             /* of logits and dlogits: MOE_FP32, MOE_BF16 or MOE_FP16 */
} moe_select_t;

/* logits [T, E], bias [E] fp32 or NULL -> idx [T, k], weights [T, k] fp32. */
moe_status_t moe_select(const moe_select_t* cfg, const void* logits, const float* bias, int32_t* idx, float* weights,
                        moe_stream_t stream);

/* logits [T, E], idx [T, k], dweights [T, k] fp32 -> dlogits [T, E] (dtype), overwritten. */
moe_status_t moe_select_bwd(const moe_select_t* cfg, const void* logits, const int32_t* idx, const float* dweights,
                            void* dlogits, moe_stream_t stream);

/* The router's gradients from dlogits [T, E] fp32: dW_r = x^T dlogits [d_model, E], db_r = the sum of dlogits over
 * the tokens [E] (nullable), both fp32 and overwritten.  The product takes dlogits in bf16, as
 * moe_router_bwd's does; db_r sums them as they are.  Of cfg it uses T, d_model and E; ws is the workspace
 * of this configuration. */
moe_status_t moe_router_wgrad(const moe_config_t* cfg, const moe_bf16* x, const float* dlogits, float* dW_r,
                              float* db_r, void* ws, size_t ws_bytes, moe_stream_t stream);

/* ---- Grouped products --------------------------------------------------------------------------
 * Matrix products over rows grouped by expert, group g having a weight of its own and any number of
 * rows: for an expert FFN other than the layer's SwiGLU one (another activation, a bias, one matrix,
 * adapters), on the layer's dispatched rows (moe_segments) or on rows laid out by the caller.
 *   moe_grouped_mm      y_r  = W[g] x_r                       for every row r of every group g
 *   moe_grouped_mm_dx   dx_r = W[g]^T dy_r
 *   moe_grouped_mm_dw   dW[g] = sum over the group's rows of dy_r x_r^T
 *   moe_grouped_mm_i8   y_r  = s_r (P[g] q_r) t[g]            8-bit integers q, P with their scales s, t
 *   moe_grouped_mm_mxf4 y_r  = P[g] q_r                       4-bit floating point with a scale for 32 values
 *
 * Groups.  row_begin, row_end [groups] int32 on the device: group g is rows row_begin[g] ..
 * row_end[g] - 1.  Groups come in row order and do not overlap (0 <= row_begin[g] <= row_end[g] <=
 * row_begin[g + 1], row_end[groups - 1] <= rows); any of them may be empty, of any length, and start
 * at any row, and rows between groups belong to none.  The offsets [groups + 1] of packed groups serve
 * as both arrays (row_end = offsets + 1).  Rows of no group are not read into any product and their
 * outputs are not written.  Values out of range or out of order record MOE_ERR_BAD_INDEX
 * (moe_check_error) and the call writes nothing.  (A product of no rows writes nothing and looks at no
 * group; moe_grouped_mm_dw looks at them.)  The buffer's rows choose the kernel: few rows a group are
 * fastest in a buffer of their own number.
 *
 * Pointers.  Rows, weights and codes are 16-byte aligned; row_begin, row_end and the scales of 8-bit
 * integers 4-byte aligned, so that they may be parts of larger arrays.
 *
 * Numerics.  Products are exact and summed in fp32 by the tensor cores, and each output is rounded once.
 * At every 16 products the tensor cores drop up to a unit of the sum's last place, towards zero.  So y and
 * dx are off by at most n_in / 16 (n_out / 16) x 2^-23 of the sum of the products' magnitudes before they
 * are rounded: 2^-14 at 8192 columns, 2^-11, half a step of fp16, at 65536 (values of one sign: 4.2e-4 low
 * there, 1.0e-4 at 16384; values of both signs far less).  dW, over any number of rows, is summed 2048
 * rows of a group at a time (2^-16) and the parts are added in fp32 in row order, whatever its type;
 * additions to an fp32 dW (accumulate, and those parts) take subnormal values as zero.  NaN and infinities
 * stay within the rows (moe_grouped_mm, _dx, _i8) or the group (_dw) that hold them.  Results are the same
 * on every run. */
typedef struct {
    int64_t rows;              /* rows of x, y, dx, dy (0 allowed), <= 2^28 */
    int32_t n_in, n_out;       /* widths of x and y: multiples of 8, 8 .. 65536 */
    int32_t groups;            /* 1 .. 1024 */
    int32_t dtype;             /* MOE_BF16 or MOE_FP16: x, y, dx, dy and W (moe_grouped_mm_i8: y) */
    int32_t dw_dtype;          /* type of dW: dtype or MOE_FP32 */
    int32_t accumulate;        /* 1: dW += the gradient (MOE_FP32 only); 0: dW is overwritten, with
                                * zeros for an empty group */
    int64_t in_stride;         /* elements between the rows of x and dx (moe_grouped_mm_i8: of the */
    int64_t out_stride;        /* codes), and of y and dy: multiples of 8 (codes: 16), at least the
                                * width; 0: the width */
} moe_grouped_t;

/* Workspace bytes for any call of this description; its header is zeroed once with
 * moe_grouped_workspace_init.  It must be 256-byte aligned; calls that share it must be ordered on one
 * stream.  moe_check_error reads and clears the errors recorded in it. */
moe_status_t moe_grouped_workspace_size(const moe_grouped_t* cfg, size_t* ws_bytes);
moe_status_t moe_grouped_workspace_init(const moe_grouped_t* cfg, void* ws, size_t ws_bytes, moe_stream_t stream);

/* The groups of the rows that the last moe_dispatch on ws laid out (x_perm, o_perm): row_begin,
 * row_end [E + n_shared], the padded segments P_g and their ends P_g + n_g. */
moe_status_t moe_segments(const moe_config_t* cfg, int32_t* row_begin, int32_t* row_end, void* ws, size_t ws_bytes,
                          moe_stream_t stream);

/* x [rows, n_in], W [groups, n_out, n_in] -> y [rows, n_out]. */
moe_status_t moe_grouped_mm(const moe_grouped_t* cfg, const int32_t* row_begin, const int32_t* row_end, const void* x,
                            const void* W, void* y, void* ws, size_t ws_bytes, moe_stream_t stream);

/* dy [rows, n_out], W [groups, n_out, n_in] -> dx [rows, n_in].  (Also the forward product of weights
 * stored [groups, in, out].) */
moe_status_t moe_grouped_mm_dx(const moe_grouped_t* cfg, const int32_t* row_begin, const int32_t* row_end,
                               const void* dy, const void* W, void* dx, void* ws, size_t ws_bytes,
                               moe_stream_t stream);

/* dy [rows, n_out], x [rows, n_in] -> dW [groups, n_out, n_in]. */
moe_status_t moe_grouped_mm_dw(const moe_grouped_t* cfg, const int32_t* row_begin, const int32_t* row_end,
                               const void* dy, const void* x, void* dW, void* ws, size_t ws_bytes,
                               moe_stream_t stream);

/* Rows of 8-bit integers: src [rows, cols] (dtype MOE_BF16 or MOE_FP16) -> codes [rows, cols] and
 * scales [rows] fp32, scale = amax / 127 over the row (1 where that is zero) and code = v / scale
 * rounded to nearest even, at most 127 in magnitude, all in fp32 with IEEE division.  (A value of half the
 * row's largest lies between the codes 63 and 64; the scale's rounding decides, so another way to divide
 * by 127 may give the other one.)  A NaN or an infinity in a row makes its scale NaN, and so its products.
 * For activations (one scale per token) and for the rows of weights (one per output channel).  cols a
 * multiple of 16, at most 65536. */
moe_status_t moe_quantize_rows_i8(const void* src, int32_t dtype, int64_t rows, int32_t cols, int8_t* codes,
                                  float* scales, moe_stream_t stream);

/* codes [rows, n_in] int8, scales [rows] fp32, Wq [groups, n_out, n_in] int8, W_scale [groups, n_out]
 * fp32 -> y [rows, n_out] (dtype).  n_in a multiple of 16.  One group is a dense product.  The sums of
 * integer products are exact up to 2^24 in magnitude; beyond it they lose what the sums of
 * moe_grouped_mm lose. */
moe_status_t moe_grouped_mm_i8(const moe_grouped_t* cfg, const int32_t* row_begin, const int32_t* row_end,
                               const int8_t* codes, const float* scales, const int8_t* Wq, const float* W_scale,
                               void* y, void* ws, size_t ws_bytes, moe_stream_t stream);

/* Microscaled 4-bit floating point (OCP Microscaling Formats 1.0, MXFP4): every 32 consecutive values of a row share
 * one power of two X, and each is an e2m1 code, 0, 0.5, 1, 1.5, 2, 3, 4 or 6 with a sign, times X.
 *   codes   [rows, cols / 2] bytes, two codes to a byte, the value of the lower index in the low four bits
 *             (magnitude in the low three of them, in the order above; sign in the fourth)
 *   scales  [rows, stride] bytes, the first cols / 32 of a row its X as E8M0: 2^(byte - 127); 255 is NaN.  stride,
 *             from moe_mx_scale_stride, is cols / 32 rounded up to 16
 * For activations and for weights alike (weights [groups, n_out, n_in] are groups * n_out rows).
 *
 * moe_quantize_rows_mxf4: src [rows, cols] (dtype MOE_BF16, MOE_FP16 or MOE_FP32), X = 2^(floor(log2(largest
 * magnitude)) - 2), at least 2^-127 (and that for a block of zeros), code = v / X to the nearest, ties to the even
 * code, at most 6 in magnitude.  A NaN or an infinity makes its block's X NaN, with codes of 0.  Bytes of a row of
 * scales past cols / 32 are set to 0.  cols a multiple of 32, at most 65536; rows at most 2^28; all
 * pointers 16-byte aligned. */
moe_status_t moe_mx_scale_stride(int32_t cols, int32_t* stride);
moe_status_t moe_quantize_rows_mxf4(const void* src, int32_t dtype, int64_t rows, int32_t cols, uint8_t* codes,
                                    uint8_t* scales, moe_stream_t stream);

/* codes [rows, n_in / 2] with scales [rows, stride], Wq [groups, n_out, n_in / 2] with W_scale [groups, n_out,
 * stride] -> y [rows, n_out] (dtype).  n_in and in_stride (in values, of the codes' rows) multiples of 32; the scales'
 * rows are stride bytes apart whatever in_stride is, and their bytes past n_in / 32 are not used.  Rows, weights, codes and
 * scales are 16-byte aligned.  Products with both scales are exact and summed in fp32 by the tensor cores (they
 * lose no more than moe_grouped_mm's sums: at 65536 columns of one sign less than 1e-5 when measured), products
 * below fp32's range may count as 0, and a scale of NaN makes NaN of the outputs of its row or of its weight's
 * output channel.  Few rows of a long contraction are summed in two or four parts, added in their order. */
moe_status_t moe_grouped_mm_mxf4(const moe_grouped_t* cfg, const int32_t* row_begin, const int32_t* row_end,
                                 const uint8_t* codes, const uint8_t* scales, const uint8_t* Wq, const uint8_t* W_scale,
                                 void* y, void* ws, size_t ws_bytes, moe_stream_t stream);

/* Synchronise `stream`, return the first device-side error recorded in ws since the last check
 * (MOE_OK if none) and clear it.  Returns MOE_ERR_CUDA if the stream itself reports an error. */
moe_status_t moe_check_error(void* ws, moe_stream_t stream);

/* Test hook: make dispatch scan block `stall_block` never publish its counts (-1: off), make the
 * first CTA pair of every expert GEMM and grouped product (of few rows: the first block) skip its
 * fill number `stall_fill` of the operand ring -- no
 * loads, no expected bytes, so the MMA's wait for that stage never completes (-1: off) -- and bound
 * every device wait of later calls by `timeout_ns` (0: the default, 2 s).  Used to check that a
 * wait that runs out returns MOE_ERR_TIMEOUT through moe_check_error instead of hanging: the kernel
 * that gives up still waits, with the same bound, for the copies and MMAs it has in flight before
 * it frees its shared memory and TMEM, so the next call runs normally.  Outputs of the stalled call
 * are invalid. */
moe_status_t moe_debug_inject(void* ws, int32_t stall_block, int32_t stall_fill, uint64_t timeout_ns,
                              moe_stream_t stream);

/* Kernel timing.  While enabled, every kernel launch of the library is bracketed by two CUDA
 * events recorded on its launching stream.  moe_profile_enable(on) also clears the totals.
 * moe_profile_read(kernel, ...) waits for the recorded events and returns, for kernel id
 * 0..n-1, its name, summed milliseconds and launch count; MOE_ERR_INVALID_ARG past the last id.
 * Host-side state shared by the whole process; not for concurrent use from several threads. */
moe_status_t moe_profile_enable(int32_t on);
moe_status_t moe_profile_read(int32_t kernel, const char** name, double* total_ms, int32_t* launches);

/* The SM clock a tensor-core GEMM kernel actually ran at: while profiling is enabled, one thread of
 * each of its CTAs adds the SM cycles (clock64) and nanoseconds (globaltimer) from its entry to its
 * exit on the current device; *mhz receives cycles / ns x 1000 over all its CTAs since
 * moe_profile_enable (0 when none ran, and for the grouped products, which take no such readings; same
 * kernel ids as moe_profile_read).  Under the GPU's power cap this is the clock the kernel's work ran
 * at, which nvidia-smi's periodic samples miss.  moe_profile_enable touches the current device for
 * this (MOE_ERR_CUDA if it cannot); moe_profile_sm_clock synchronises with it.  The other kernels
 * record nothing here. */
moe_status_t moe_profile_sm_clock(int32_t kernel, double* mhz);

/* Static text for a status code. */
const char* moe_status_string(moe_status_t status);

#ifdef __cplusplus
}
#endif

#endif /* MOE_GB300_H */

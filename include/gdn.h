/*
 * gdn.h -- C ABI of the Gated DeltaNet state-rebuild library for MI355X (gfx950).
 *
 * What the library computes.  Hybrid LLMs interleave full-attention layers with
 * Gated DeltaNet linear-attention layers whose recurrent state cannot be rolled
 * back to an arbitrary prefix boundary.  Tail-Replay (arXiv 2608.30310, abstract;
 * gist.science technical summary, "Mecanismos Principais") rebuilds each
 * linear-attention layer's state at a matched-prefix boundary by replaying only the
 * most recent r tokens of the prefix, starting from a zero state, through the
 * Gated DeltaNet recurrence.  Full prefill of the whole prefix is the baseline it
 * is compared with (same pages, "Resultados").  Per (sequence, v-head):
 *
 *     S_t = alpha_t (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T,
 *     o_t = scale * S_t^T q_t,        alpha_t = exp(g_t),  g_t <= 0,
 *
 * with S a d_k x d_v matrix.  g = -inf is legal and means alpha = 0.
 *
 * Layouts (row-major, contiguous, packed varlen in "THD" order):
 *     q, k       [T, h_qk, d_k]      in qkv_dtype
 *     v          [T, h_v,  d_v]      in qkv_dtype
 *     g, beta    [T, h_v]            fp32
 *     cu_seqlens [n_seqs + 1]        int32, sequence n owns tokens [cu[n], cu[n+1])
 *     r          [n_seqs]            int32 replay lengths, 0 <= r[n] <= cu[n+1]-cu[n]
 *     S0, S_out  [n_seqs, h_v, d_k, d_v]  fp32
 *     o_out      [T_out, h_v, d_v]   in o_dtype; rows packed per sequence in order
 * v-head h reads q/k head floor(h * h_qk / h_v) (grouped value heads).
 *
 * Pointers are device pointers unless marked (host).  Every call is asynchronous
 * on `stream` (a hipStream_t; NULL = the null stream) except gdn_device_status.
 *
 * Ownership: the caller owns every buffer, including the workspace.  The compute
 * calls never allocate, free or synchronise; they print nothing unless the
 * environment variable GDN_DEBUG is 1 (then a host-side rejection says why on
 * stderr).  Their only global state is a per-device cache of the occupancy query
 * (written once, atomically); calls are re-entrant given distinct workspaces.
 *
 * Errors: problems checkable on the host (null required pointer, bad dims,
 * h_v % h_qk != 0, unsupported d, misaligned pointer, small workspace) return a
 * non-zero gdn_status before anything is enqueued.  A failed launch returns
 * GDN_ERR_LAUNCH.  The device-resident cu_seqlens / r are validated by the kernel
 * itself: on a bad value it sets a bit in the workspace's status word, skips the
 * offending sequences and leaves their outputs unspecified.  The kernels only ever
 * set bits in that word (atomically), never clear it: gdn_device_status reports
 * what the calls since the previous gdn_device_status on that workspace (or since
 * it was zero-filled) recorded, and clears it.  A new workspace must therefore be
 * zero-filled once before its first use.  Non-finite q/k/v/beta or g > 0 are not
 * checked; the result is then undefined and gdn_state_relerr's non-finite count
 * exposes it.
 *
 * Arithmetic: the state is fp32 throughout.  fp32 inputs use fp32 matrix products.
 * bf16 inputs use matrix products with fp16 operands and fp32 accumulation: q and k
 * enter exactly (bf16 values of magnitude in [2^-14, 65504], which L2-normalised q and
 * k are; smaller entries round to fp16 subnormals), the intermediate state and pseudo-
 * values are rounded to fp16 once per product (relative error <= 2^-11).  Their range
 * is checked nowhere: state entries, and v-sized intermediates, must stay below ~10^3
 * in magnitude (the state is scaled by at most 64 internally); beyond that the fp16
 * operands overflow and the outputs turn non-finite (again exposed by the non-finite
 * count).  Gated DeltaNet states with unit keys, beta in [0, 1] and O(1) values stay
 * orders of magnitude inside this.
 */
#ifndef GDN_H
#define GDN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define GDN_ABI_VERSION 3

typedef enum {
    GDN_OK = 0,
    GDN_ERR_NULL = 1,          /* a required pointer is NULL */
    GDN_ERR_SHAPE = 2,         /* negative / inconsistent sizes, h_v % h_qk != 0 */
    GDN_ERR_DTYPE = 3,         /* unknown dtype code */
    GDN_ERR_UNSUPPORTED = 4,   /* valid but not built: d_k or d_v outside {64, 128} */
    GDN_ERR_ALIGN = 5,         /* a pointer is not 16-byte aligned */
    GDN_ERR_WORKSPACE = 6,     /* workspace missing or smaller than gdn_workspace_bytes() */
    GDN_ERR_LAUNCH = 7,        /* the HIP launch failed */
    GDN_ERR_DEVICE_INPUT = 8,  /* device-side cu_seqlens / r invalid (from gdn_device_status) */
    GDN_ERR_HIP = 9,           /* a HIP runtime call failed (gdn_device_status only) */
    GDN_ERR_DEVICE_WAIT = 10,  /* a bounded wait inside a workgroup expired: results invalid
                                  (from gdn_device_status; not expected on working hardware) */
    GDN_ERR_SCRATCH = 11       /* request larger than the static device scratch of an
                                  allocation-free entry point */
} gdn_status;

typedef enum { GDN_F32 = 0, GDN_BF16 = 1 } gdn_dtype;

typedef struct {
    int32_t n_seqs;            /* packed sequences (a stack of independent layers may be packed as sequences) */
    int32_t h_qk, h_v;         /* q/k heads and v heads, h_v % h_qk == 0 */
    int32_t d_k, d_v;          /* head dims, each 64 or 128 */
    int32_t qkv_dtype;         /* gdn_dtype of q, k, v */
    int32_t o_dtype;           /* gdn_dtype of o: qkv_dtype, or GDN_F32 */
    float scale;               /* o_t = scale * S_t^T q_t */
    int64_t total_tokens;      /* T == cu_seqlens[n_seqs] (host copy) */
    int64_t total_out_tokens;  /* rows of o_out: sum r[n] (replay) or T (prefill); a replay
                                  without o_out only needs total_out_tokens <= total_tokens */
} gdn_desc;

/* ABI version of the loaded library (GDN_ABI_VERSION). */
int32_t gdn_abi_version(void);

/* Static description of a status code. */
const char *gdn_status_str(int32_t status);

/* (host) Replay length for a matched prefix of L tokens under budget fraction rho:
 * clamp(ceil(rho * L), 0, L) -- the pages replay the last 5-10 % of the matched
 * prefix (Tail-Replay abstract; technical summary, "Resultados"). */
int32_t gdn_replay_len(int32_t L, double rho);

/* (host) Workspace bytes a call with this descriptor needs: 256 (the status word), plus
 * n_seqs * h_v * 4 rounded up to 256 for gdn_adaptive_replay_len.  Zero-fill a new
 * workspace once before its first use (the status word accumulates bits). */
size_t gdn_workspace_bytes(const gdn_desc *desc);

/* Tail replay: for every sequence n and v-head h, run the recurrence from S = 0 over
 * the last r[n] tokens [cu[n+1]-r[n], cu[n+1]) and write the state after the last
 * token to S_out (the state at the prefix boundary; technical summary,
 * "Reconstrucao de Estado Independente").  o_out (nullable) receives o_t for the
 * replayed tokens, packed per sequence; cu_out (nullable, [n_seqs+1]) receives the
 * output row offsets.  r[n] = 0 gives S = 0 (the pages' Zero-Only baseline) and no
 * o rows; r[n] = L_n gives exactly gdn_prefill with S0 = NULL. */
int32_t gdn_replay(const gdn_desc *desc, const void *q, const void *k, const void *v,
                   const float *g, const float *beta, const int32_t *cu_seqlens,
                   const int32_t *r, float *S_out, void *o_out, int32_t *cu_out,
                   void *workspace, size_t workspace_bytes, void *stream);

/* Full prefill: the recurrence over every whole sequence from S0 (NULL = zero
 * state).  This is the baseline Tail-Replay is measured against: processing the
 * whole matched prefix again (fugumt.com page, English abstract; gist.science
 * technical summary, "Resultados", where replay is compared with full prefill for
 * quality and time to first token).  o_out (nullable) has one row per token, in token
 * order.  With S0 set to a rebuilt state it continues a prefix into its unmatched
 * suffix, the step that produces the first token after a cache hit (same section). */
int32_t gdn_prefill(const gdn_desc *desc, const void *q, const void *k, const void *v,
                    const float *g, const float *beta, const int32_t *cu_seqlens,
                    const float *S0, float *S_out, void *o_out,
                    void *workspace, size_t workspace_bytes, void *stream);

/* Error report: relerr[s] = ||S_a[s] - S_ref[s]||_F / ||S_ref[s]||_F (||S_a[s]||_F when
 * the reference is zero), fp64 accumulation; nonfinite[s] (nullable) counts the
 * non-finite entries of S_a[s].  States are d_k x d_v fp32 blocks.  It measures how
 * far a replayed state is from the full-prefill state at the same boundary: the pages'
 * claim is that a short recent tail approximates that state because the gated updates
 * attenuate older inputs (fugumt.com page, English abstract), and that zeroing the state
 * instead ("Zero-Only", relative error 1 here) degrades quality (technical summary,
 * "Resultados"). */
int32_t gdn_state_relerr(const float *S_a, const float *S_ref, int64_t n_states, int32_t d_k,
                         int32_t d_v, float *relerr_out, int32_t *nonfinite_out, void *stream);

/* Adaptive replay length.  The replayed state differs from the full-prefill state by
 * the older state carried through the window's per-token maps alpha_t (I - beta_t k_t
 * k_t^T), whose product has norm at most prod alpha_t for unit keys and beta in
 * [0, 1]; the gated updates attenuate distant tokens (Tail-Replay, arXiv 2608.30310,
 * abstract; technical summary, "Mecanismos Principais"), while the pages fix r as a
 * 5-10 % budget ("Resultados").  This picks r per sequence from the gates instead:
 *
 *     r_h[n] = the smallest r in [0, min(L_n, r_max)] with sum over the last r tokens
 *              of g[t, h] <= ln(eps)   (i.e. prod alpha <= eps), or min(L_n, r_max);
 *     r_out[n] = clamp(max_h r_h[n], min(r_min, L_n), min(r_max, L_n)),
 *
 * so ||S_full - S_replay||_F <= eps ||S_before||_F in every head whenever r_out[n] is
 * below the cap.  The comparison is exact: each g is rounded to a multiple of 2^-32
 * nats (g >= 0 or NaN counts as 0; g <= -2^20, including -inf, as -2^20) and summed in
 * integers against floor(ln(eps) * 2^32); eps >= 1 gives r_h = 0.
 * desc: n_seqs, h_v and total_tokens are read (the other fields are ignored).
 * g [T, h_v] fp32 and cu_seqlens [n_seqs+1] are device arrays; r_out [n_seqs] (device,
 * int32) can be passed straight to gdn_replay.  The workspace must hold
 * gdn_workspace_bytes(desc) bytes; its status word reports GDN_ERR_DEVICE_INPUT for a
 * bad cu_seqlens (those sequences get r_out = 0).  Host errors: eps <= 0 or NaN,
 * r_min < 0 or r_max < r_min -> GDN_ERR_SHAPE. */
int32_t gdn_adaptive_replay_len(const gdn_desc *desc, const float *g, const int32_t *cu_seqlens,
                                double eps, int32_t r_min, int32_t r_max, int32_t *r_out,
                                void *workspace, size_t workspace_bytes, void *stream);

/* Allocation-free gdn_adaptive_replay_len, for callers that cannot allocate device
 * memory or take a workspace (code under HIP graph capture, tight serving loops,
 * harnesses that forbid allocation).  Same arguments and result as
 * gdn_adaptive_replay_len minus the workspace: its per-head lengths live in the
 * library's own static device scratch, 65536 int32 per GPU (plus a 256-byte status
 * block), held until the process ends; it calls no allocator.  Limit: n_seqs * h_v <=
 * 65536, else GDN_ERR_SCRATCH before anything is enqueued.  All calls on one GPU share
 * that scratch: calls that overlap on one GPU (concurrent streams, threads) race and give
 * undefined r_out; calls ordered on one stream are fine.  A bad device cu_seqlens shows
 * as r_out[n] = 0 for the sequences concerned (there is no status word to read).
 * GDN_ERR_HIP if the scratch's device address cannot be looked up. */
int32_t gdn_adaptive_replay_len_static(const gdn_desc *desc, const float *g,
                                       const int32_t *cu_seqlens, double eps, int32_t r_min,
                                       int32_t r_max, int32_t *r_out, void *stream);

/* Segment-parallel tail replay: gdn_replay's result (up to rounding) in less time when
 * few (sequence, v-head) chains are long, e.g. one layer of one sequence.  The recurrence
 * is affine in the state, so over any stretch of tokens S_end = M S_start + S_local, with
 * S_local the state the stretch builds from zero and M the product of its per-token maps
 * alpha_t (I - beta_t k_t k_t^T) (technical summary, "Mecanismos Principais", for the
 * recurrence; the pages replay one window per layer from a zero state).  Each window is
 * cut into P chunk-aligned segments of ceil(ceil(r/64)/P) chunks (trailing ones may be
 * empty); one launch forms every segment's S_local and M together, a combine chains
 * S_start(p+1) = M_p S_start(p) + S_local(p) from S_start(0) = 0 with fp32 sums (bf16
 * inputs: each fp32 operand as fp16 hi + lo halves, three products, about fp32 accuracy
 * inside the fp16 range the bf16 path already requires) and writes the final state to
 * S_out, and, when o_out is given, a second launch re-runs each segment
 * from its true start for the outputs (layouts as gdn_replay; cu_out likewise).
 * n_segments: P in [1, 64], or 0 for the library's choice, clamp(min(128 / (n_seqs h_v),
 * chunks / 6), 1, 16) with chunks = ceil(total_out_tokens / n_seqs / 64) when
 * total_out_tokens > 0 (segments shorter than ~6 chunks cost more than they save); P = 1
 * runs gdn_replay itself.  Requires d_k == d_v (else GDN_ERR_UNSUPPORTED); n_segments
 * outside [0, 64] -> GDN_ERR_SHAPE.  The
 * workspace must hold gdn_segmented_workspace_bytes(desc, n_segments) bytes (its first
 * 256 are the status word, as for every call); it also carries the segments' states,
 * 3 n_seqs P h_v d_k^2 floats.  Errors in the device cu_seqlens / r are reported through
 * the status word as for gdn_replay.  Compared with gdn_replay: S and o agree to the
 * rounding of the products (fp16 operands for bf16 inputs), not bit for bit. */
size_t gdn_segmented_workspace_bytes(const gdn_desc *desc, int32_t n_segments);
int32_t gdn_replay_segmented(const gdn_desc *desc, const void *q, const void *k, const void *v,
                             const float *g, const float *beta, const int32_t *cu_seqlens,
                             const int32_t *r, float *S_out, void *o_out, int32_t *cu_out,
                             int32_t n_segments, void *workspace, size_t workspace_bytes,
                             void *stream);

/* (host, synchronising) Wait for `stream`, read the status word of `workspace` and
 * clear it.  *status_host: GDN_OK, GDN_ERR_DEVICE_INPUT (a call since the previous
 * read found a bad cu_seqlens / r) or GDN_ERR_DEVICE_WAIT.  Returns GDN_ERR_HIP if the
 * wait, the copy or the clear failed. */
int32_t gdn_device_status(const void *workspace, void *stream, int32_t *status_host);

/* ---------------------------------------------------------------------------------------
 * The rest of a hybrid model's step after a cache hit.  The matched prefix's recurrent states
 * are rebuilt by gdn_replay and its full-attention keys and values are kept exactly; the
 * unmatched suffix is then prefilled from both and tokens follow one by one (technical summary,
 * "Mecanismos Principais" and "Resultados").  Beside gdn_prefill that takes the short causal
 * convolution in front of a recurrent layer, the scan of a state space layer, single-token
 * steps, and for the full-attention layers the norm and rotation of q and k with the append to
 * a paged cache, and attention of the new tokens over that cache.
 *
 * They follow the conventions above: caller-owned buffers, asynchronous on `stream`, host
 * errors before anything is enqueued, device-resident integers checked by the kernels into the
 * workspace's status word.  A workspace starts zero-filled; its first 256 bytes are the status
 * word.  Two calls that may run at the same time (two streams, two graphs) need a workspace
 * each.  Rows of x, y, q, k, v may be columns of a wider buffer: a stride field gives the
 * elements from one token's row to the next, the rows themselves are contiguous and start on
 * 16 bytes.  Outputs must not overlap inputs except where it is said.  Rows behind the last
 * sequence (tokens at or after cu_seqlens[n_seqs]) are left as they were.  Non-finite inputs
 * are not checked: a token's reach the outputs of its own sequence only, but may reach those of
 * the same call's earlier tokens too.  What a cache holds behind a sequence's kv_len is never read.
 *
 * Single-token calls: row i uses state slots[i] of a pool of n_slots states, updated in place;
 * slots NULL: state i.  slots[i] = -1 marks a padded row: neither its state nor its output is
 * touched.  A slot out of range, or equal to an earlier row's, sets the status bit and leaves
 * that row's output and state as they were.
 * --------------------------------------------------------------------------------------- */

/* Short causal convolution, one filter of `width` taps (2, 3 or 4) per channel:
 *     y[t, c] = act(bias[c] + sum_j weight[c, j] x[t - (width - 1) + j, c]),
 * act = SiLU or none.  weight [channels, width] and bias [channels] (nullable) are fp32; x, y and
 * the states [., width - 1, channels] (the last inputs, oldest first) have `dtype`.
 * channels * element size must be a multiple of 16 bytes. */
typedef struct {
    int32_t n_seqs;            /* packed sequences; gdn_conv_step: rows */
    int32_t n_slots;           /* gdn_conv_step: states of the pool */
    int32_t channels, width;
    int32_t dtype;             /* gdn_dtype */
    int32_t silu;              /* 1: SiLU behind the sum, 0: none */
    int64_t total_tokens;      /* rows of x and y; gdn_conv_step: n_seqs */
    int64_t x_stride, y_stride;
} gdn_conv_desc;

/* Prompts: state0 (nullable: zero) [n_seqs, width - 1, channels] are the inputs in front of each
 * sequence, state_out (nullable, may be state0) those behind it. */
int32_t gdn_conv(const gdn_conv_desc *desc, const void *x, const float *weight, const float *bias,
                 const int32_t *cu_seqlens, const void *state0, void *state_out, void *y,
                 void *workspace, size_t workspace_bytes, void *stream);
/* One token per row; state [n_slots, width - 1, channels]. */
int32_t gdn_conv_step(const gdn_conv_desc *desc, const void *x, const float *weight, const float *bias,
                      void *state, const int32_t *slots, void *y, void *workspace,
                      size_t workspace_bytes, void *stream);

/* Selective state space recurrence, per (sequence, head h), group q = floor(h h_qk / h_v):
 *     dt'_t = softplus(dt[t, h] + dt_bias[h])   (softplus = 0: the sum itself, not negative),
 *     S_t = exp(dt'_t A[h]) S_{t-1} + dt'_t B[t, q] x[t, h]^T,   y_t = S_t^T C[t, q] + D[h] x[t, h],
 * S [d_k, d_v] as in gdn_prefill.  x, y [T, h_v, d_v], B, C [T, h_qk, d_k], dt [T, h_v] have
 * `dtype`; A, dt_bias, D [h_v] are fp32 (the last two nullable); states are fp32.  A is finite
 * and not positive, dt finite.  d_k and d_v in {64, 128}. */
typedef struct {
    int32_t n_seqs;            /* packed sequences; gdn_ssm_step: rows */
    int32_t n_slots;           /* gdn_ssm_step: states of the pool */
    int32_t h_qk, h_v;         /* heads of B and C, heads of x: h_v % h_qk == 0 */
    int32_t d_k, d_v;          /* state size, head size */
    int32_t dtype;             /* gdn_dtype */
    int32_t softplus;          /* 1: softplus over dt + dt_bias, 0: the sum itself */
    int64_t total_tokens;      /* rows of x, B, C, dt; gdn_ssm_step: n_seqs */
    int64_t total_out_tokens;  /* rows of y: total_tokens, or sum r[n] with replay lengths */
    int64_t x_stride, b_stride, c_stride, dt_stride, y_stride;   /* dt_stride: any >= h_v;
                                  gdn_ssm_scan: 64 rows span less than 2 GiB */
} gdn_ssm_desc;

/* Bytes of gdn_ssm_scan's workspace: 256, and for few long sequences the states of the segments
 * that they are cut into (0 for a descriptor that is refused). */
size_t gdn_ssm_workspace_bytes(const gdn_ssm_desc *desc);
/* Prompts.  r NULL: whole sequences from S0 (nullable: zero).  r [n_seqs]: the last r[n] tokens of
 * each, as gdn_replay takes them (S0 is then the state in front of the window), y's rows packed
 * per window and cu_out (nullable) [n_seqs + 1] their offsets.  y is nullable; S_out may be S0.
 * bf16: products take bf16 operands with fp32 sums; M (the chunk's C_i . B_j and gates) and S are
 * rounded to bf16 once for their products in y, half a bf16 step of each term, and nothing else is
 * rounded to less than 16 bits, however the batch is cut; S_out is accurate to fp32 (its operands
 * enter in three bf16 terms). */
int32_t gdn_ssm_scan(const gdn_ssm_desc *desc, const void *x, const void *B, const void *C, const void *dt,
                     const float *A, const float *dt_bias, const float *D, const int32_t *cu_seqlens,
                     const int32_t *r, const float *S0, float *S_out, void *y, int32_t *cu_out,
                     void *workspace, size_t workspace_bytes, void *stream);
/* One token per row; S [n_slots, h_v, d_k, d_v]. */
int32_t gdn_ssm_step(const gdn_ssm_desc *desc, const void *x, const void *B, const void *C, const void *dt,
                     const float *A, const float *dt_bias, const float *D, float *S, const int32_t *slots,
                     void *y, void *workspace, size_t workspace_bytes, void *stream);

/* One token of the gated delta rule per row, fp32 arithmetic throughout; layouts and fields as
 * gdn_prefill with n_seqs = total_tokens = total_out_tokens rows, S [n_slots, h_v, d_k, d_v]. */
int32_t gdn_step(const gdn_desc *desc, const void *q, const void *k, const void *v, const float *g,
                 const float *beta, float *S, int32_t n_slots, const int32_t *slots, void *o,
                 void *workspace, size_t workspace_bytes, void *stream);

/* A paged cache and the new tokens that meet it.  k_cache and v_cache hold n_pages pages of
 * page_size tokens; entry e of head h, token j of page p is at p page_stride + j token_stride +
 * h head_stride + e (elements, both caches alike, multiples of 16 bytes).  block_table
 * [n_seqs, max_pages] gives each sequence's pages in order; entries behind its last page are not
 * read.  kv_len [n_seqs] counts a sequence's cached tokens, its new ones among them:
 * token i of L new ones is at position kv_len - L + i. */
typedef struct {
    int32_t n_seqs;
    int32_t h_q, h_kv;         /* query heads, cache heads: h_q % h_kv == 0 */
    int32_t d;                 /* head dim: 64, 128 or 256 */
    int32_t dtype;             /* gdn_dtype of q, k, v, the caches and the outputs */
    int32_t page_size, n_pages, max_pages;
    int32_t max_kv_len;        /* no kv_len is larger (host copy), at most 2^30 */
    int32_t rot_dim;           /* gdn_qk_norm_rope: entries that turn, a multiple of 16, <= d */
    int32_t interleaved;       /* pairs (2 i, 2 i + 1) instead of (i, i + rot_dim / 2) */
    int32_t norm;              /* 1: root-mean-square norm in front of the rotation */
    int32_t max_pos;           /* rows of cos_sin */
    float eps;                 /* of the norm */
    float scale;               /* gdn_paged_attn: of the scores */
    int64_t total_tokens;      /* new tokens: rows of q, k, v and the outputs */
    int64_t q_stride, k_stride, v_stride, o_stride;
    int64_t page_stride, token_stride, head_stride;
} gdn_paged_desc;

/* q_out = rot(q / rms(q) * q_weight), and k likewise and v as it is into the caches at the
 * tokens' positions; rms(x)^2 = mean of x^2 over the head + eps, weights [d] fp32 (NULL: ones).
 * The weights and cos_sin are 16-byte aligned.
 * cos_sin [max_pos, rot_dim] fp32: the rot_dim / 2 cosines, then sines, of a position; pair i
 * turns (a, b) to (a cos - b sin, b cos + a sin).  positions (nullable) [T]: rotate by these
 * instead of the place in the cache.  q_out may be q.  A token without a place in the cache, or a
 * page or position out of range, sets the status bit; nothing is stored for it in the caches (nor
 * in q_out for a bad position).  Tokens of one call have places of their own. */
int32_t gdn_qk_norm_rope(const gdn_paged_desc *desc, const void *q, const void *k, const void *v,
                         const float *q_weight, const float *k_weight, const float *cos_sin,
                         const int32_t *block_table, const int32_t *cu_seqlens, const int32_t *kv_len,
                         const int32_t *positions, void *k_cache, void *v_cache, void *q_out,
                         void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of gdn_paged_attn's workspace: 256, and the parts of rows whose keys are split over
 * workgroups (0 for a descriptor that is refused). */
size_t gdn_paged_workspace_bytes(const gdn_paged_desc *desc);
/* Each new token attends to the cached tokens at its position and before:
 *     o = sum_j softmax_j(scale q . k_j) v_j,  lse = ln sum_j exp(scale q . k_j)  (nullable, [T, h_q] fp32),
 * query head h with cache head floor(h h_kv / h_q).  A token in front of the cache's first one
 * (kv_len < L) sees nothing: o = 0, lse = -inf.  A bad cu_seqlens, kv_len or page sets the status
 * bit; the outputs of those sequences are unspecified.  bf16: products take q, k, v as they are, with
 * fp32 scores, sums and outputs before the final rounding.  Probabilities have 16 bits in batches of up
 * to 32 rows a sequence on average (rows: tokens times query heads on a cache head); in larger ones they
 * are rounded to bf16 once, half a bf16 step of each term p_j v_j. */
int32_t gdn_paged_attn(const gdn_paged_desc *desc, const void *q, const void *k_cache, const void *v_cache,
                       const int32_t *block_table, const int32_t *cu_seqlens, const int32_t *kv_len,
                       void *o, float *lse, void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H */

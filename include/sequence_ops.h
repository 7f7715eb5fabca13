/*
 * sequence_ops.h - C ABI of what a hybrid model's step runs beside its conv and its linear
 * attention: the selective state space scan (packed prompts, single tokens, speculative verify and
 * commit), the norm of q and k heads with their rotation, and the verdict on drafted tokens.
 * Hand-written HIP kernels for AMD Instinct MI355X (gfx950), built as libseqops.so.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - As in conv_verify.h, whose element types and return codes are used here: every data
 *    pointer is a DEVICE pointer, the shape is a host pointer, the caller owns every buffer
 *    (workspaces too), nothing is allocated, copied or synchronized, no pointer is kept, and
 *    the kernels run on `hip_stream` (NULL = the null stream).  Thread-safe and stateless
 *    apart from a thread-local error detail.
 *  - All validation happens on the host before any HIP call; a call that returns an error has
 *    launched nothing and written nothing.  (A call of several launches can fail with
 *    CV_EHIP_BASE - e between them.)
 *  - Strides are in ELEMENTS; the innermost dimension is contiguous.
 *  - Buffers that are written must not overlap any other.
 */
#ifndef SEQUENCE_OPS_H
#define SEQUENCE_OPS_H

#include <stdint.h>

#include "conv_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SEQUENCE_OPS_ABI_VERSION 1

/*
 * The selective state space scan.  For every row (sequence), channel c < d, state n < d_state and
 * token t:
 *
 *   delta    = softplus(dt[t,c] + dt_bias[c])       (softplus = 0: dt[t,c] + dt_bias[c])
 *   h[c,n]   = exp(delta A[c,n]) h[c,n] + delta x[t,c] B[t,n]
 *   y        = sum_n C[t,n] h[c,n] + D[c] x[t,c]
 *   out[t,c] = y z[t,c] / (1 + exp(-z[t,c]))        rounded once to the x dtype; z NULL: y (its
 *                                                   strides are checked all the same: 0 will do)
 *
 *  - Layouts.  With packed rows (prefill) token t of row i is row cu_seqlens[i] + t and the seq
 *    strides are unused:
 *      x, dt, z, out  [n_seq, T, d]        x + i*x_seq_stride + t*x_tok_stride + c
 *      B, C           [n_seq, T, d_state]  likewise; one B and C for all channels
 *      A              [d, d_state] fp32 contiguous, finite
 *      D, dt_bias     [d] fp32, or NULL (0)
 *      state          [n_slots, d, d_state] contiguous below the slot dimension
 *    B and C may be views of one projection's rows, z of another's.
 *  - slot_idx [n_seq] int32 or NULL (row i uses slot i).  A row of slot -1 is padded: nothing of
 *    it is written.  A row whose slot is outside [0, n_slots) or whose token count is outside
 *    [0, T] is skipped in the same way.  Device-side preconditions, not checked: the slots of rows
 *    that write are distinct; cu_seqlens stays inside the token buffers.
 *  - Supported (else CV_ENOTSUP): d a multiple of 8; d_state a multiple of 8, 8..64; (x, state)
 *    types (F32, F32), (BF16, BF16), (BF16, F32); x, dt, z, out, A, D, dt_bias and the state 16-byte
 *    aligned, their strides multiples of 16 bytes; B and C aligned to their elements; prefill: any four
 *    tokens of x, dt, z, B and out, and any 16 of C, within 2 GiB.
 *  - Numerics: delta, decays, states and sums are held in fp32.  A state stored as bf16 is rounded
 *    once, after the last token of the call.  Decays, softplus and the gate's sigmoid count as 0
 *    below 2^-126, fp32's normal range (z or dt + dt_bias under -87).  A token's values that are not
 *    finite change the outputs of their own and of later tokens only (x, dt, z: of their own
 *    channel), which are not finite then and may be NaN where the formula has an infinity.
 */
typedef struct sq_scan_shape {
    int32_t n_seq;        /* rows, >= 0 (0: nothing to do)                                  */
    int32_t T;            /* tokens of every row, 1..32; prefill: the longest prompt, >= 1  */
    int32_t d;            /* channels, >= 1                                                 */
    int32_t d_state;      /* states of a channel                                            */
    int32_t x_dtype;      /* cv_dtype_t of x, dt, z, B, C and out                           */
    int32_t state_dtype;  /* cv_dtype_t of the state pool                                   */
    int32_t n_slots;      /* slots of the pool, >= n_seq when slot_idx is NULL              */
    int32_t softplus;     /* 1: delta = softplus(dt + dt_bias), 0: delta = dt + dt_bias     */
    int64_t x_seq_stride, x_tok_stride;
    int64_t dt_seq_stride, dt_tok_stride;
    int64_t z_seq_stride, z_tok_stride;
    int64_t b_seq_stride, b_tok_stride;
    int64_t c_seq_stride, c_tok_stride;
    int64_t out_seq_stride, out_tok_stride;
    int64_t state_slot_stride;   /* >= d*d_state if n_slots > 1                             */
    int64_t tokens;       /* prefill: tokens of all rows together, or 0 if that is not known;
                             sizes the grid and the workspace, and tells whether the strides
                             of out keep its elements apart (not known: of any two tokens)  */
} sq_scan_shape_t;

/* The tensors of a call; what an entry point does not use is ignored there. */
typedef struct sq_scan_data {
    const void *x, *dt, *z, *B, *C;
    const float *A, *D, *dt_bias;
} sq_scan_data_t;

/*
 * Packed prompts.  Row i holds cu_seqlens[i+1] - cu_seqlens[i] tokens (0..T; other counts:
 * the row is skipped).  It starts from its slot's state, or from zeros where
 * has_initial_state[i] == 0 (NULL: all 1), and its slot is left with the state after its last
 * token (a row of no tokens: with its starting state).  Where shape->tokens is given, rows in
 * order that would hold more than that together may be skipped.
 * workspace: selscan_prefill_workspace(shape) bytes (16-byte aligned; NULL if that is 0), free
 * again once the call's work on the stream is done.
 */
CV_API int selscan_prefill(const sq_scan_shape_t *shape, const sq_scan_data_t *data, void *state,
                           const int32_t *slot_idx, const int32_t *cu_seqlens,
                           const int32_t *has_initial_state, void *out, void *workspace,
                           int64_t workspace_bytes, void *hip_stream);

/* Bytes of selscan_prefill's workspace for a shape (>= 0), or an error code (< 0). */
CV_API int64_t selscan_prefill_workspace(const sq_scan_shape_t *shape);

/* T tokens for each row, one launch: out for all of them, and the state after the last. */
CV_API int selscan_update(const sq_scan_shape_t *shape, const sq_scan_data_t *data, void *state,
                          const int32_t *slot_idx, void *out, void *hip_stream);

/* The same outputs with the state only read: the verify of T draft tokens. */
CV_API int selscan_verify(const sq_scan_shape_t *shape, const sq_scan_data_t *data,
                          const void *state, const int32_t *slot_idx, void *out, void *hip_stream);

/* Folds the first num_tokens[i] (0..T; NULL: T) tokens of row i into its state: the commit of the
 * accepted drafts.  z, C and D, their strides and those of out are ignored; 0 tokens leave the
 * state untouched. */
CV_API int selscan_commit(const sq_scan_shape_t *shape, const sq_scan_data_t *data, void *state,
                          const int32_t *slot_idx, const int32_t *num_tokens, void *hip_stream);

/* How a call of this shape is launched (host only; nothing is launched). */
typedef enum sq_scan_call {
    SQ_SCAN_PREFILL = 0, SQ_SCAN_UPDATE = 1, SQ_SCAN_VERIFY = 2, SQ_SCAN_COMMIT = 3
} sq_scan_call_t;
typedef struct sq_scan_info {
    int64_t workgroups;     /* of the launch that makes the outputs (the states)            */
    int64_t workspace_bytes;
    int32_t threads;        /* of a workgroup                                               */
    int32_t channels;       /* of a workgroup                                               */
    int32_t segment_tokens; /* prompts: tokens of a segment of a cut row; 0: none is cut    */
    int32_t launches;       /* 2 where rows are cut, 0 where there is nothing to do         */
} sq_scan_info_t;
CV_API int selscan_describe(int call, const sq_scan_shape_t *shape, sq_scan_info_t *info);

/*
 * The RMS norm of each head of q and k and the rotation of its first rot channels by the token's
 * position, in one pass.  For every token t and head, with u = x / sqrt(mean(x^2) + eps) * weight
 * (weight NULL: u = x) and angle[i] = positions[t] * inv_freq[i], i < rot / 2:
 *
 *   (out[e], out[f]) = (u[e] cos - u[f] sin, u[f] cos + u[e] sin)
 *       e, f = i, i + rot/2;   interleaved: e, f = 2i, 2i + 1
 *   out[c] = u[c] for c >= rot
 *
 * The product and its remainder modulo a turn are taken in fp64, the rest in fp32, rounded once.
 *   q, k and their outs  [tokens, heads, dim]   q + t*q_tok_stride + h*q_head_stride + c
 *   q_weight, k_weight   [dim] of the x dtype or NULL;   inv_freq [rot/2] fp32
 *   positions            [tokens] int32 or int64, any value
 * k_heads may be 0 (k, k_out and k_weight are not read).  q_out may be q itself, and k_out k (same
 * strides).  Supported (else CV_ENOTSUP): dim a multiple of 16 up to 256, rot a multiple of 16
 * up to dim (0: no rotation, positions and inv_freq are not read); pointers 16-byte aligned
 * (inv_freq and positions: their elements), strides multiples of 16 bytes.
 */
typedef struct sq_rotary_shape {
    int64_t tokens;       /* >= 0 (0: nothing to do)                                        */
    int32_t q_heads;      /* >= 1                                                           */
    int32_t k_heads;      /* >= 0                                                           */
    int32_t dim, rot;
    float eps;            /* >= 0 and finite                                                */
    int32_t x_dtype;      /* cv_dtype_t of q, k, their outs and weights                     */
    int32_t interleaved;
    int32_t wide_positions;   /* 1: int64, 0: int32                                         */
    int64_t q_tok_stride, q_head_stride, k_tok_stride, k_head_stride;
    int64_t q_out_tok_stride, q_out_head_stride, k_out_tok_stride, k_out_head_stride;
} sq_rotary_shape_t;
CV_API int norm_rotary(const sq_rotary_shape_t *shape, const void *q, const void *k,
                       const void *q_weight, const void *k_weight, const void *positions,
                       const float *inv_freq, void *q_out, void *k_out, void *hip_stream);

/*
 * The verdict on drafted tokens, from the target's probabilities and given random numbers.
 *
 * Row i holds T tokens: token 0 is certain (the last one chosen), tokens 1..T-1 are drafts, each
 * drawn to follow its parent (token t - 1, or parent[i,t] in a tree).  target[i,t] are the target's
 * probabilities of what follows token t, draft[i,t] those that draft t + 1 was drawn from (NULL: drafts
 * are certain, as from a greedy draft model or a tree of candidates).  From token 0 on, at the
 * current token c with P = target[i,c]:
 *
 *   its children j = c + 1 (a tree: those with parent c, in their order) are tried in turn:
 *     accepted, and the new current token, if  uniform[i,j-1] * q < P(x_j),
 *       q = draft[i,c](x_j), or without a draft 1 less the P of children tried before
 *     (a child whose token was tried before is not accepted);
 *   if none is accepted, the next token is drawn, and that ends the row:
 *     from max(P - draft[i,c], 0) if a child was tried against a draft,
 *     from P without the tokens of the children tried, if there was no draft,
 *     from P where no child was tried (behind the last draft), or where nothing else is left.
 *
 * The token drawn from weights w is the lowest v with  sum_{u <= v} w(u) > uniform[i,T-1] * sum(w),
 * or the last with w(v) > 0 if rounding leaves none; sums and products are taken in fp64.  Weights that
 * are not positive finite numbers count as 0; if none is left the token is -1.
 *
 *   tokens       [n_seq, T] int32: a draft outside [0, vocab) (a pad) is not tried
 *   parent       [n_seq, T] int32 or NULL (a chain): -1 for token 0, -1..t-1 for others, where -1 is
 *                a token that follows none and is never reached.  A row with another parent is
 *                skipped.  With parent draft must be NULL (else CV_ENOTSUP).
 *   target       [n_seq, T, vocab], draft [n_seq, T-1, vocab] of one dtype
 *   uniform      [n_seq, T] fp32 in [0, 1)
 *   slot_idx     [n_seq] int32 or NULL: a row of a negative slot is padded: nothing of it is written
 * Outputs, int32:
 *   num_tokens   [n_seq] how many tokens to commit: token 0 and the accepted drafts, 1..T.  Of a chain they
 *                are the row's first ones, which selscan_commit and linattn_commit fold; of a tree path
 *                names them, and a commit's inputs are to be gathered along it first
 *   next_token   [n_seq] the token drawn
 *   window_index [n_seq] or NULL: the last accepted token's place in the row (a chain: num_tokens - 1)
 *   path         [n_seq, T] or NULL: the places of the tokens to commit, then -1
 * workspace: accept_drafts_workspace(shape) bytes (16-byte aligned), free again once the call's
 * work on the stream is done.  Supported (else CV_ENOTSUP): T up to 32; data aligned to its
 * elements; vocab up to 2^24.
 */
typedef struct sq_accept_shape {
    int32_t n_seq;        /* rows, >= 0 (0: nothing to do)                                  */
    int32_t T;            /* tokens of a row, 1..32                                         */
    int32_t vocab;        /* >= 1                                                           */
    int32_t p_dtype;      /* cv_dtype_t of target and draft                                 */
    int64_t tokens_stride, parent_stride, uniform_stride, path_stride;   /* of rows         */
    int64_t target_seq_stride, target_tok_stride;
    int64_t draft_seq_stride, draft_tok_stride;
} sq_accept_shape_t;
CV_API int accept_drafts(const sq_accept_shape_t *shape, const int32_t *tokens,
                         const int32_t *parent, const void *target, const void *draft,
                         const float *uniform, const int32_t *slot_idx, int32_t *num_tokens,
                         int32_t *next_token, int32_t *window_index, int32_t *path,
                         void *workspace, int64_t workspace_bytes, void *hip_stream);

/* Bytes of accept_drafts' workspace for a shape (>= 0), or an error code (< 0). */
CV_API int64_t accept_drafts_workspace(const sq_accept_shape_t *shape);

CV_API const char *seqops_strerror(int code);
/* Detail of this thread's last error in this library ("" if none). */
CV_API const char *seqops_last_error(void);
CV_API int seqops_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif

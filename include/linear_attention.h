/*
 * linear_attention.h - C ABI of what a linear-attention layer runs behind its conv: linear
 * attention with a decay for each head (packed prompts, single tokens, speculative verify and
 * commit), the gated head norm and the norm at a block's end.  Hand-written HIP kernels for
 * AMD Instinct MI355X (gfx950), built as liblinattn.so.
 *
 * Recurrence, for every row (sequence), value head h < v_heads and token t, with the q and k
 * head hq = h / (v_heads / q_heads):
 *
 *   S_t      = exp(g[t,h]) * S_{t-1} + k[t,hq] v[t,h]^T         S is [dk, dv]
 *   out[t,h] = scale * S_t^T q[t,hq]                            rounded once to the x dtype
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
 *  - Element layouts (strides in ELEMENTS, innermost dimension contiguous).  With packed rows
 *    (prefill) token t of row i is row cu_seqlens[i] + t and the seq strides are unused:
 *      q, k    [n_seq, T, q_heads, dk]   q + i*q_seq_stride + t*q_tok_stride + hq*q_head_stride
 *      v, out  [n_seq, T, v_heads, dv]   likewise
 *      g       [n_seq, T, v_heads] fp32  g + i*g_seq_stride + t*g_tok_stride + h: the log of
 *              the decay; g_tok_stride 0 (and g_seq_stride 0) is one decay for each head, NULL
 *              is no decay.  -inf empties the state before its token.  Values below -1e6 count
 *              as -1e6 (exp() of either is 0).
 *      state   [n_slots, v_heads, dk, dv] contiguous below the slot dimension
 *    q, k and v may be views of one buffer (the conv's output row q | k | v).
 *  - slot_idx [n_seq] int32 or NULL (row i uses slot i).  A row of slot -1 is padded: nothing
 *    of it is written.  A row whose slot is outside [0, n_slots) or whose token count is
 *    outside [0, T] is skipped in the same way.  Device-side preconditions, not checked: the
 *    slots of rows that write are distinct; cu_seqlens stays inside the token buffers.
 *  - Buffers that are written must not overlap any other.
 *  - Supported (else CV_ENOTSUP): dk and dv multiples of 8, 8..256; (x, state) types (F32,
 *    F32), (BF16, BF16), (BF16, F32); pointers 16-byte aligned (g, index vectors: 4-byte);
 *    the x strides and state_slot_stride multiples of 16 bytes.
 *  - Numerics: log decays are summed in 64 bits, states and sums are held in 32.  A state
 *    stored as bf16 is rounded once, after the last token of the call.  Where q, k, v are
 *    bf16, fp32 factors go through the matrix cores as sums of bf16 parts (two parts where
 *    only out depends on them or the state is bf16: 2^-17; three for an fp32 state: 2^-24).
 *    A token's q, k, v that are not finite change the outputs of their own and of later
 *    tokens only.  An output or state that a non-finite value reaches is non-finite; whether
 *    as inf or NaN is not specified.
 */
#ifndef LINEAR_ATTENTION_H
#define LINEAR_ATTENTION_H

#include <stdint.h>

#include "conv_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LINEAR_ATTENTION_ABI_VERSION 2

typedef struct la_shape {
    int32_t n_seq;        /* rows, >= 0 (0: nothing to do)                                  */
    int32_t T;            /* tokens of every row, 1..32; prefill: the longest prompt, >= 1  */
    int32_t q_heads;      /* heads of q and k, >= 1                                         */
    int32_t v_heads;      /* heads of v, g, out and the state: a multiple of q_heads        */
    int32_t dk, dv;       /* channels of a q/k head and of a v head                         */
    float scale;          /* finite; multiplies out                                         */
    int32_t x_dtype;      /* cv_dtype_t of q, k, v and out                                  */
    int32_t state_dtype;  /* cv_dtype_t of the state pool                                   */
    int32_t n_slots;      /* slots of the pool, >= n_seq when slot_idx is NULL              */
    int64_t q_seq_stride, q_tok_stride, q_head_stride;
    int64_t k_seq_stride, k_tok_stride, k_head_stride;
    int64_t v_seq_stride, v_tok_stride, v_head_stride;
    int64_t out_seq_stride, out_tok_stride, out_head_stride;
    int64_t g_seq_stride, g_tok_stride;
    int64_t state_slot_stride;   /* >= v_heads*dk*dv if n_slots > 1                         */
    int64_t tokens;       /* prefill: tokens of all rows together, or 0 if that is not known;
                             sizes the grid and the workspace, and tells whether the strides
                             of out keep its elements apart (not known: of any two tokens)  */
} la_shape_t;

/*
 * Packed prompts.  Row i holds cu_seqlens[i+1] - cu_seqlens[i] tokens (0..T; other counts:
 * the row is skipped).  It starts from its slot's state, or from zeros where
 * has_initial_state[i] == 0 (NULL: all 1), and its slot is left with the state after its last
 * token (a row of no tokens: with its starting state).  Where shape->tokens is given, rows in
 * order that would hold more than that together may be skipped.
 * workspace: linattn_prefill_workspace(shape) bytes (16-byte aligned; NULL if that is 0), free
 * again once the call's work on the stream is done.
 */
CV_API int linattn_prefill(const la_shape_t *shape, const void *q, const void *k, const void *v,
                           const float *g, void *state, const int32_t *slot_idx,
                           const int32_t *cu_seqlens, const int32_t *has_initial_state, void *out,
                           void *workspace, int64_t workspace_bytes, void *hip_stream);

/* Bytes of linattn_prefill's workspace for a shape (>= 0), or an error code (< 0). */
CV_API int64_t linattn_prefill_workspace(const la_shape_t *shape);

/* T tokens for each row, one launch: out for all of them, and the state after the last. */
CV_API int linattn_update(const la_shape_t *shape, const void *q, const void *k, const void *v,
                          const float *g, void *state, const int32_t *slot_idx, void *out,
                          void *hip_stream);

/* The same outputs with the state only read: the verify of T draft tokens. */
CV_API int linattn_verify(const la_shape_t *shape, const void *q, const void *k, const void *v,
                          const float *g, const void *state, const int32_t *slot_idx, void *out,
                          void *hip_stream);

/* Folds the first num_tokens[i] (0..T; NULL: T) tokens of row i into its state: the commit of
 * the accepted drafts.  The q and out strides and the scale are ignored; 0 tokens leave the
 * state untouched. */
CV_API int linattn_commit(const la_shape_t *shape, const void *k, const void *v, const float *g,
                          void *state, const int32_t *slot_idx, const int32_t *num_tokens,
                          void *hip_stream);

/* How a call of this shape is launched (host only; nothing is launched). */
typedef enum la_call {
    LA_CALL_PREFILL = 0, LA_CALL_UPDATE = 1, LA_CALL_VERIFY = 2, LA_CALL_COMMIT = 3
} la_call_t;
typedef enum la_kernel {
    LA_KERNEL_TOKENS = 0,        /* token by token                                          */
    LA_KERNEL_FEW = 1,           /* up to 32 bf16 tokens in one pass over the state         */
    LA_KERNEL_CHUNKED = 2,       /* bf16 tokens in chunks of 64                             */
    LA_KERNEL_CHUNKED_F32 = 3    /* fp32 tokens in chunks of 32                             */
} la_kernel_t;
typedef struct la_launch_info {
    int64_t workgroups;     /* of the launch that makes the outputs (the states)            */
    int64_t workspace_bytes;
    int32_t kernel;         /* la_kernel_t                                                  */
    int32_t threads;        /* of a workgroup                                               */
    int32_t state_cols;     /* columns of a state in a workgroup                            */
    int32_t segment_tokens; /* prompts: tokens of a segment of a cut row; 0: none is cut    */
    int32_t launches;       /* 3 where rows are cut, 0 where there is nothing to do         */
    int32_t streaming;      /* 1: the states' loads and stores go past the caches           */
} la_launch_info_t;
CV_API int linattn_describe(int call, const la_shape_t *shape, la_launch_info_t *info);

/* Gate activations of norm_gated. */
typedef enum la_act { LA_SILU = 0, LA_SIGMOID = 1 } la_act_t;

/* Rows of heads (norm_gated) or whole rows (norm_residual: heads = 1, head strides unused). */
typedef struct la_norm_shape {
    int64_t rows;         /* >= 0 (0: nothing to do)                                        */
    int32_t heads;        /* >= 1                                                           */
    int32_t dim;          /* channels that share one mean of squares: a multiple of 8, up to
                             2048 (norm_gated) or 16384 (norm_residual)                     */
    float eps;            /* >= 0 and finite                                                */
    float scale;          /* norm_residual: multiplies the block's output; finite           */
    int32_t x_dtype;      /* y, gate, weights, out: CV_F32 or CV_BF16                       */
    int32_t res_dtype;    /* norm_residual: residual stream; CV_F32, or CV_BF16 with BF16 x */
    int32_t activation;   /* norm_gated: la_act_t                                           */
    int32_t gate_first;   /* norm_gated: 1 = norm(y * act(gate)), 0 = norm(y) * act(gate)   */
    int64_t y_row_stride, y_head_stride;
    int64_t gate_row_stride, gate_head_stride;   /* norm_residual: row stride 0 = one gate
                                                    for each channel                        */
    int64_t out_row_stride, out_head_stride;
    int64_t res_row_stride, res_out_row_stride;  /* norm_residual                           */
} la_norm_shape_t;

/*
 * The gated RMS norm of each head, with n(x) = x / sqrt(mean(x^2) + eps) * weight[dim]:
 *   out = n(y) * act(gate), or n(y * act(gate)) with gate_first.
 * gate NULL: no gate.  out may be y itself (same strides).  fp32 inside, rounded once.
 */
CV_API int norm_gated(const la_norm_shape_t *shape, const void *y, const void *gate,
                      const void *weight, void *out, void *hip_stream);

/*
 * The end of a block and the start of the next one:
 *   u = y,  n(y; post_weight) if that is not NULL;   u = u * gate if gate is not NULL
 *   r = residual + scale * u           stored to residual_out, rounded to the res dtype
 *   out = n(r; pre_weight)             from the r before that rounding; NULL out: not wanted
 * residual_out may be residual itself (same strides).
 */
CV_API int norm_residual(const la_norm_shape_t *shape, const void *y, const void *post_weight,
                         const void *gate, const void *residual, void *residual_out,
                         const void *pre_weight, void *out, void *hip_stream);

CV_API const char *linattn_strerror(int code);
/* Detail of this thread's last error in this library ("" if none). */
CV_API const char *linattn_last_error(void);
CV_API int linattn_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif

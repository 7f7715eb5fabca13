// C-ABI entry points of liblinattn.so: host-side validation, launch planning and error
// reporting.  Every check runs before any HIP call.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "api_checks.h"
#include "la_internal.h"
#include "linear_attention.h"

namespace {

struct Need { bool q, out, packed, verify; };

// What every entry point of the recurrence checks; *empty: there is nothing to do.
int check_attn(const la_shape_t *s, const Need &need, int *xb, int *sb, bool *empty) {
    if (!s) return fail(CV_EINVAL, "shape is NULL");
    if (s->n_seq < 0) return fail(CV_EINVAL, "n_seq (%d) is negative", s->n_seq);
    if (s->T < 1) return fail(CV_EINVAL, "T (%d) must be at least 1", s->T);
    if (!need.packed && s->T > 32)
        return fail(CV_ENOTSUP, "T (%d) is over 32: longer rows are prompts (linattn_prefill)", s->T);
    if (s->q_heads < 1 || s->v_heads < 1 || s->v_heads % s->q_heads != 0)
        return fail(CV_EINVAL, "v_heads (%d) must be a multiple of q_heads (%d), both at least 1",
                    s->v_heads, s->q_heads);
    if (s->dk < 1 || s->dv < 1) return fail(CV_EINVAL, "dk (%d) and dv (%d) must be at least 1", s->dk, s->dv);
    if (s->dk % 8 || s->dv % 8 || s->dk > 256 || s->dv > 256)
        return fail(CV_ENOTSUP, "dk (%d) and dv (%d) must be multiples of 8 up to 256", s->dk, s->dv);
    if (need.out && !std::isfinite(s->scale)) return fail(CV_EINVAL, "scale is not finite");
    *xb = dtype_bytes(s->x_dtype);
    *sb = dtype_bytes(s->state_dtype);
    if (!*xb || !*sb) return fail(CV_EINVAL, "unknown element type (x %d, state %d)", s->x_dtype, s->state_dtype);
    if (*xb == 4 && *sb == 2) return fail(CV_ENOTSUP, "fp32 x with a bf16 state");
    if (s->n_slots < 0) return fail(CV_EINVAL, "n_slots (%d) is negative", s->n_slots);

    const struct { const char *name; int64_t stride; bool used; int elem; } strides[] = {
        {"q_seq_stride", s->q_seq_stride, need.q && !need.packed, *xb},
        {"q_tok_stride", s->q_tok_stride, need.q, *xb},
        {"q_head_stride", s->q_head_stride, need.q, *xb},
        {"k_seq_stride", s->k_seq_stride, !need.packed, *xb},
        {"k_tok_stride", s->k_tok_stride, true, *xb},
        {"k_head_stride", s->k_head_stride, true, *xb},
        {"v_seq_stride", s->v_seq_stride, !need.packed, *xb},
        {"v_tok_stride", s->v_tok_stride, true, *xb},
        {"v_head_stride", s->v_head_stride, true, *xb},
        {"out_seq_stride", s->out_seq_stride, need.out && !need.packed, *xb},
        {"out_tok_stride", s->out_tok_stride, need.out, *xb},
        {"out_head_stride", s->out_head_stride, need.out, *xb},
        {"state_slot_stride", s->state_slot_stride, true, *sb},
        {"g_seq_stride", s->g_seq_stride, !need.packed, 0},
        {"g_tok_stride", s->g_tok_stride, true, 0},
    };
    for (const auto &d : strides) {
        if (!d.used) continue;
        if (d.stride < 0) return fail(CV_EINVAL, "%s (%lld) is negative", d.name, (long long)d.stride);
        if (d.elem && d.stride % (16 / d.elem))
            return fail(CV_ENOTSUP, "%s (%lld) is not a multiple of 16 bytes", d.name, (long long)d.stride);
    }
    const int64_t per_slot = (int64_t)s->v_heads * s->dk * s->dv;
    if (s->n_slots > 1 && s->state_slot_stride < per_slot)
        return fail(CV_EINVAL, "state_slot_stride (%lld) is below a slot's %lld elements",
                    (long long)s->state_slot_stride, (long long)per_slot);
    if (need.packed && s->tokens < 0) return fail(CV_EINVAL, "tokens (%lld) is negative", (long long)s->tokens);
    if (need.out) {
        // of packed rows the tokens of all together; where they are not known, what would overlap
        // with any two of them (T bounds a row, and says nothing of their number)
        const int64_t toks = !need.packed ? s->T : s->tokens > 0 ? s->tokens : std::min<int64_t>(2, sat_mul(s->n_seq, s->T));
        Dim d[3] = {{s->v_heads, s->out_head_stride}, {toks, s->out_tok_stride},
                    {need.packed ? 1 : s->n_seq, s->out_seq_stride}};
        if (!apart(s->dv, d, 3)) return fail(CV_EINVAL, "the strides of out make its rows overlap");
    }
    *empty = s->n_seq == 0;
    return CV_OK;
}

// What a call passes over and the 256 MiB Infinity Cache will hardly hold until it is read again (in
// a model, behind every other layer's work).  From about 96 MiB on a state's loads and stores are
// faster past the caches (256 rows of 2 MiB: 165 us for 184; 64 rows in turn with others: 54 for
// 60), below they are not (16 rows: 18 us for 17).
bool past_caches(int64_t bytes) { return bytes > (96 << 20); }

laimpl::AttnArgs attn_args(const la_shape_t *s, const void *q, const void *k, const void *v, const float *g,
                           const void *state, const int32_t *slot_idx, const int32_t *cu,
                           const int32_t *num_tokens, const int32_t *has_init, void *out, bool write_state) {
    laimpl::AttnArgs a{};
    a.q = q; a.k = k; a.v = v; a.g = g; a.state = const_cast<void *>(state); a.out = out;
    a.slot_idx = slot_idx; a.cu_seqlens = cu; a.num_tokens = num_tokens; a.has_init = has_init;
    a.q_seq = s->q_seq_stride; a.q_tok = s->q_tok_stride; a.q_head = s->q_head_stride;
    a.k_seq = s->k_seq_stride; a.k_tok = s->k_tok_stride; a.k_head = s->k_head_stride;
    a.v_seq = s->v_seq_stride; a.v_tok = s->v_tok_stride; a.v_head = s->v_head_stride;
    a.o_seq = s->out_seq_stride; a.o_tok = s->out_tok_stride; a.o_head = s->out_head_stride;
    a.g_seq = s->g_seq_stride; a.g_tok = s->g_tok_stride;
    a.s_slot = s->state_slot_stride;
    a.n_seq = s->n_seq; a.T = s->T; a.v_heads = s->v_heads; a.group = s->v_heads / s->q_heads;
    a.dk = s->dk; a.dv = s->dv; a.n_slots = s->n_slots;
    a.scale = s->scale;
    a.write_state = write_state;
    return a;
}

// Workgroups below which the recurrent kernel takes its narrow tiles: fewer than the chip's
// 256 compute units have of the wide ones to hold two each.
constexpr int64_t kWideBlocks = 512;

// A launch of one kernel over rows, heads and tiles of the state's columns.
struct Plan {
    int kernel;                   // la_kernel_t
    const void *fn;
    int64_t tiles, blocks;
    int cols, threads;
    bool streaming;
};

Plan plan_recurrent(const la_shape_t *s, int xb, int sb) {
    laimpl::RecurrentPlan p = laimpl::pick_recurrent(xb, sb, s->dk, true);
    const int64_t heads = (int64_t)s->n_seq * s->v_heads;
    int64_t tiles = (s->dv + p.cols - 1) / p.cols;
    if (sat_mul(heads, tiles) < kWideBlocks) {
        p = laimpl::pick_recurrent(xb, sb, s->dk, false);
        tiles = (s->dv + p.cols - 1) / p.cols;
    }
    return {LA_KERNEL_TOKENS, p.fn, tiles, sat_mul(heads, tiles), p.cols, p.threads, false};
}

// How packed prompts are cut into workgroups.
//
// Along a row: its tokens are one chain of chunks in one workgroup unless that chain is much
// longer than the share of all chunks that each of the chip's slots would have (two workgroups on
// each of 256 compute units): then rows are cut into segments of about that share, at the price
// of passing over their k and v twice (one prompt of 16384 with 32 heads: 857 us uncut, 194-199 in
// 16 segments; 5 of up to 777 fp32 tokens with 6 heads of 96 x 72: 91 us uncut, 36 in segments of 128).
//
// Across a head (bf16 tokens; fp32 ones go in tiles of 64): tiles of 128 columns, since what a
// chunk reads and the products q.k serve all of a tile; tiles of 64 where the wide ones would leave
// most compute units empty (64 workgroups of 32 chunks: 122 us for 160) or the state's way in and
// out counts, in a few chunks of one generation of workgroups (8 rows of up to 160 tokens, 48
// heads: 21 us for 27).
struct Cut {
    laimpl::ChunkedPlan plan;
    int64_t tiles, segments, places, ws_states, ws_bytes;
    int32_t seg_len;
};
Cut cut_prompts(const la_shape_t *s, int xb, int sb, bool wide) {
    constexpr int64_t kSlots = 512;
    constexpr int64_t kLeast = 4;
    Cut c{};
    c.plan = xb == 4 ? laimpl::pick_chunked_f32(s->dk) : laimpl::pick_chunked(sb, s->dk, wide);
    const int64_t chunk = c.plan.chunk;
    c.tiles = (s->dv + c.plan.cols - 1) / c.plan.cols;
    c.segments = s->n_seq;
    c.seg_len = s->T;
    const int64_t heads = s->v_heads * c.tiles;
    int64_t tokens = sat_mul(s->n_seq, s->T);
    if (s->tokens > 0 && s->tokens < tokens) tokens = s->tokens;
    // (no row holds more than all tokens together, however far T bounds it)
    const int64_t chain = (std::min<int64_t>(s->T, tokens) + chunk - 1) / chunk;
    const int64_t share = std::max(kLeast, sat_mul(tokens / chunk + 1, heads) / kSlots);
    const int64_t segments = tokens / (share * chunk) + s->n_seq;
    const int64_t states = sat_mul(segments, heads);
    // (combine's grid has one workgroup for each 4 KiB of a row's state)
    const int64_t combines = sat_mul(sat_mul(s->n_seq, heads), c.plan.ws_bytes / 16 / c.plan.threads);
    if (chain > share + share / 2 && chain > 2 * kLeast && states <= INT32_MAX && combines <= INT32_MAX) {
        c.seg_len = (int32_t)(share * chunk);
        c.segments = segments;
        // only rows of more than seg_len tokens have places in the workspace
        c.places = tokens / c.seg_len + std::min<int64_t>(s->n_seq, tokens / c.seg_len);
        c.ws_states = c.places * heads;
        c.ws_bytes = sat_add(sat_mul(c.ws_states, c.plan.ws_bytes), (4 * c.ws_states + 15) / 16 * 16);
    }
    const int64_t blocks = sat_mul(c.segments, heads);
    if (wide && (blocks <= 128 || (chain <= 4 && blocks <= kSlots))) return cut_prompts(s, xb, sb, false);
    return c;
}
Cut cut_prompts(const la_shape_t *s, int xb, int sb) { return cut_prompts(s, xb, sb, xb == 2 && s->dv > 64); }

// Whether prompts go in chunks: a chunk lies within 32-bit offsets.  (Tokens 32 MiB and more apart
// go one by one.)
bool in_chunks(const la_shape_t *s) {
    const int64_t far = std::max(std::max(s->q_tok_stride, s->k_tok_stride), std::max(s->v_tok_stride, s->out_tok_stride));
    return far < (1 << 24);
}

int chunked(laimpl::AttnArgs a, const Cut &c, void *workspace, void *stream) {
    a.tiles = (int32_t)c.tiles;
    a.seg_len = c.seg_len;
    a.segments = (int32_t)c.segments;
    a.places = (int32_t)c.places;
    a.ws = workspace;
    a.ws_total = reinterpret_cast<float *>(static_cast<char *>(workspace) + c.ws_states * c.plan.ws_bytes);
    const int64_t blocks = sat_mul(c.segments, a.v_heads * c.tiles);
    if (c.ws_states) {
        int rc = launch(c.plan.first, blocks, c.plan.threads, 0, &a, stream);
        if (rc != CV_OK) return rc;
        int vectors = (int)(c.plan.ws_bytes / 16);
        rc = launch(c.plan.combine, (int64_t)a.n_seq * a.v_heads * c.tiles * (vectors / c.plan.threads), c.plan.threads,
                    0, &a, stream, &vectors);
        if (rc != CV_OK) return rc;
    }
    return launch(c.plan.run, blocks, c.plan.threads, 0, &a, stream);
}

// update, verify and commit
Plan plan_few(const la_shape_t *s, const Need &need, int xb, int sb) {
    const int64_t heads = (int64_t)s->n_seq * s->v_heads;
    // fp32 tokens are one chunk of a prompt from 12 on, 16 without outputs (128 rows of 32 heads, verify
    // of 8: 112 us one by one, 159 as a chunk, of 16: 205 and 162, of 32: 382 and 174; 8 rows of 16: 18
    // and 12).
    if (xb == 4 && s->T >= (need.out ? 12 : 16) && in_chunks(s)) {
        const laimpl::ChunkedPlan p = laimpl::pick_chunked_f32(s->dk);
        const int64_t tiles = (s->dv + p.cols - 1) / p.cols;
        return {LA_KERNEL_CHUNKED_F32, p.run, tiles, sat_mul(heads, tiles), p.cols, p.threads, false};
    }
    // On the matrix cores where tokens are bf16, single ones from 512 workgroups on (256 rows of 32
    // heads: 184 us for 197 by the recurrence); for few workgroups the recurrence starts sooner (one row
    // of 48 heads: 4.4 us for 6.5).  The two meet later than here: 12 rows of 48 heads, 576 workgroups,
    // take 16.9 us for 13.1, 30 rows 36.2 for 35.6.
    const int64_t tiles = (s->dv + 127) / 128;
    if (xb == 4 || (s->T == 1 && sat_mul(heads, tiles) < kWideBlocks)) return plan_recurrent(s, xb, sb);
    return {LA_KERNEL_FEW, laimpl::pick_few(sb, s->dk, s->T, need.out, !need.verify), tiles, sat_mul(heads, tiles), 128, 256,
            past_caches(sat_mul(heads, (int64_t)s->dk * s->dv * sb))};
}

constexpr Need kNeeds[] = {{true, true, true, false}, {true, true, false, false}, {true, true, false, true},
                           {false, false, false, false}};   // by la_call_t

int few_tokens(const la_shape_t *s, const Need &need, const void *q, const void *k, const void *v, const float *g,
               const void *state, const int32_t *slot_idx, const int32_t *num_tokens, void *out, void *stream) {
    g_detail[0] = 0;
    int xb, sb;
    bool empty;
    int rc = check_attn(s, need, &xb, &sb, &empty);
    if (rc != CV_OK || empty) return rc;
    if (!slot_idx && s->n_slots < s->n_seq)
        return fail(CV_EINVAL, "n_slots (%d) is below n_seq (%d) and there is no slot_idx", s->n_slots, s->n_seq);
    const Pointer ps[] = {{"q", q, need.q, 16}, {"k", k, true, 16}, {"v", v, true, 16},
                          {"state", state, true, 16}, {"out", out, need.out, 16}, {"g", g, false, 4},
                          {"slot_idx", slot_idx, false, 4}, {"num_tokens", num_tokens, false, 4}};
    if ((rc = check_pointers(ps)) != CV_OK) return rc;
    laimpl::AttnArgs a = attn_args(s, q, k, v, g, state, slot_idx, nullptr, num_tokens, nullptr, out, !need.verify);
    const Plan p = plan_few(s, need, xb, sb);
    a.tiles = (int32_t)p.tiles;
    a.streaming = p.streaming;
    a.seg_len = s->T;                              // a row is one segment (LA_KERNEL_CHUNKED_F32)
    a.segments = s->n_seq;
    return launch(p.fn, p.blocks, p.threads, 0, &a, stream);
}

int check_norm(const la_norm_shape_t *s, bool residual, int *xb, int *rb) {
    if (!s) return fail(CV_EINVAL, "shape is NULL");
    if (s->rows < 0 || s->heads < 1 || s->dim < 1)
        return fail(CV_EINVAL, "rows (%lld) must be >= 0, heads (%d) and dim (%d) at least 1",
                    (long long)s->rows, s->heads, s->dim);
    if (residual && s->heads != 1) return fail(CV_EINVAL, "heads (%d) must be 1", s->heads);
    const int most = residual ? 16384 : 2048;
    if (s->dim % 8 || s->dim > most)
        return fail(CV_ENOTSUP, "dim (%d) must be a multiple of 8 up to %d", s->dim, most);
    if (!(s->eps >= 0.0f) || !std::isfinite(s->eps)) return fail(CV_EINVAL, "eps must be finite and >= 0");
    if (residual && !std::isfinite(s->scale)) return fail(CV_EINVAL, "scale is not finite");
    if (!residual && s->activation != LA_SILU && s->activation != LA_SIGMOID)
        return fail(CV_EINVAL, "unknown activation %d", s->activation);
    *xb = dtype_bytes(s->x_dtype);
    *rb = residual ? dtype_bytes(s->res_dtype) : *xb;
    if (!*xb || !*rb) return fail(CV_EINVAL, "unknown element type (x %d, residual %d)", s->x_dtype, s->res_dtype);
    if (*xb == 4 && *rb == 2) return fail(CV_ENOTSUP, "fp32 x with a bf16 residual");
    const struct { const char *name; int64_t stride; bool used; int elem; } strides[] = {
        {"y_row_stride", s->y_row_stride, true, *xb}, {"y_head_stride", s->y_head_stride, !residual, *xb},
        {"gate_row_stride", s->gate_row_stride, true, *xb}, {"gate_head_stride", s->gate_head_stride, !residual, *xb},
        {"out_row_stride", s->out_row_stride, true, *xb}, {"out_head_stride", s->out_head_stride, !residual, *xb},
        {"res_row_stride", s->res_row_stride, residual, *rb}, {"res_out_row_stride", s->res_out_row_stride, residual, *rb},
    };
    for (const auto &d : strides) {
        if (!d.used) continue;
        if (d.stride < 0) return fail(CV_EINVAL, "%s (%lld) is negative", d.name, (long long)d.stride);
        if (d.stride % (16 / d.elem))
            return fail(CV_ENOTSUP, "%s (%lld) is not a multiple of 16 bytes", d.name, (long long)d.stride);
    }
    return CV_OK;
}

}  // namespace

extern "C" {

int64_t linattn_prefill_workspace(const la_shape_t *s) {
    g_detail[0] = 0;
    int xb, sb;
    bool empty;
    const int rc = check_attn(s, kNeeds[LA_CALL_PREFILL], &xb, &sb, &empty);
    if (rc != CV_OK || empty || !in_chunks(s)) return rc;
    return cut_prompts(s, xb, sb).ws_bytes;
}

int linattn_prefill(const la_shape_t *s, const void *q, const void *k, const void *v, const float *g, void *state,
                    const int32_t *slot_idx, const int32_t *cu_seqlens, const int32_t *has_initial_state,
                    void *out, void *workspace, int64_t workspace_bytes, void *hip_stream) {
    const int64_t need_ws = linattn_prefill_workspace(s);
    if (need_ws < 0) return (int)need_ws;
    if (s->n_seq == 0) return CV_OK;
    int rc;
    if (!slot_idx && s->n_slots < s->n_seq)
        return fail(CV_EINVAL, "n_slots (%d) is below n_seq (%d) and there is no slot_idx", s->n_slots, s->n_seq);
    if (workspace_bytes < need_ws)
        return fail(CV_EINVAL, "workspace of %lld bytes, %lld are needed", (long long)workspace_bytes, (long long)need_ws);
    const Pointer ps[] = {{"q", q, true, 16}, {"k", k, true, 16}, {"v", v, true, 16}, {"state", state, true, 16},
                          {"out", out, true, 16}, {"cu_seqlens", cu_seqlens, true, 4},
                          {"workspace", workspace, need_ws > 0, 16}, {"g", g, false, 4},
                          {"slot_idx", slot_idx, false, 4}, {"has_initial_state", has_initial_state, false, 4}};
    if ((rc = check_pointers(ps)) != CV_OK) return rc;
    const int xb = dtype_bytes(s->x_dtype), sb = dtype_bytes(s->state_dtype);
    laimpl::AttnArgs a = attn_args(s, q, k, v, g, state, slot_idx, cu_seqlens, nullptr, has_initial_state, out, true);
    if (!in_chunks(s)) {
        const Plan p = plan_recurrent(s, xb, sb);
        a.tiles = (int32_t)p.tiles;
        return launch(p.fn, p.blocks, p.threads, 0, &a, hip_stream);
    }
    return chunked(a, cut_prompts(s, xb, sb), workspace, hip_stream);
}

int linattn_update(const la_shape_t *s, const void *q, const void *k, const void *v, const float *g, void *state,
                   const int32_t *slot_idx, void *out, void *hip_stream) {
    return few_tokens(s, kNeeds[LA_CALL_UPDATE], q, k, v, g, state, slot_idx, nullptr, out, hip_stream);
}

int linattn_verify(const la_shape_t *s, const void *q, const void *k, const void *v, const float *g,
                   const void *state, const int32_t *slot_idx, void *out, void *hip_stream) {
    return few_tokens(s, kNeeds[LA_CALL_VERIFY], q, k, v, g, state, slot_idx, nullptr, out, hip_stream);
}

int linattn_commit(const la_shape_t *s, const void *k, const void *v, const float *g, void *state,
                   const int32_t *slot_idx, const int32_t *num_tokens, void *hip_stream) {
    return few_tokens(s, kNeeds[LA_CALL_COMMIT], nullptr, k, v, g, state, slot_idx, num_tokens, nullptr,
                      hip_stream);
}

int linattn_describe(int call, const la_shape_t *s, la_launch_info_t *info) {
    g_detail[0] = 0;
    if (call < LA_CALL_PREFILL || call > LA_CALL_COMMIT) return fail(CV_EINVAL, "unknown call %d", call);
    if (!info) return fail(CV_EINVAL, "info is NULL");
    int xb, sb;
    bool empty;
    const Need &need = kNeeds[call];
    const int rc = check_attn(s, need, &xb, &sb, &empty);
    if (rc != CV_OK) return rc;
    *info = la_launch_info_t{};
    if (empty) return CV_OK;
    info->launches = 1;
    if (need.packed && in_chunks(s)) {
        const Cut c = cut_prompts(s, xb, sb);
        info->kernel = xb == 4 ? LA_KERNEL_CHUNKED_F32 : LA_KERNEL_CHUNKED;
        info->workgroups = sat_mul(c.segments, s->v_heads * c.tiles);
        info->threads = c.plan.threads;
        info->state_cols = c.plan.cols;
        info->workspace_bytes = c.ws_bytes;
        if (c.ws_states) info->launches = 3, info->segment_tokens = c.seg_len;
        return CV_OK;
    }
    const Plan p = need.packed ? plan_recurrent(s, xb, sb) : plan_few(s, need, xb, sb);
    info->kernel = p.kernel;
    info->workgroups = p.blocks;
    info->threads = p.threads;
    info->state_cols = p.cols;
    info->streaming = p.streaming;
    return CV_OK;
}

int norm_gated(const la_norm_shape_t *s, const void *y, const void *gate, const void *weight, void *out,
               void *hip_stream) {
    g_detail[0] = 0;
    int xb, rb;
    int rc = check_norm(s, false, &xb, &rb);
    if (rc != CV_OK) return rc;
    Dim d[2] = {{s->heads, s->out_head_stride}, {s->rows, s->out_row_stride}};
    if (!apart(s->dim, d, 2)) return fail(CV_EINVAL, "the strides of out make its rows overlap");
    if (s->rows == 0) return CV_OK;
    const Pointer ps[] = {{"y", y, true, 16}, {"gate", gate, false, 16}, {"weight", weight, true, 16}, {"out", out, true, 16}};
    if ((rc = check_pointers(ps)) != CV_OK) return rc;
    laimpl::NormArgs a{};
    a.y = y; a.gate = gate; a.weight = weight; a.out = out;
    a.rows = s->rows; a.heads = s->heads; a.dim = s->dim; a.eps = s->eps;
    a.y_row = s->y_row_stride; a.y_head = s->y_head_stride;
    a.gate_row = s->gate_row_stride; a.gate_head = s->gate_head_stride;
    a.out_row = s->out_row_stride; a.out_head = s->out_head_stride;
    a.sigmoid = s->activation == LA_SIGMOID; a.gate_first = s->gate_first != 0;
    const laimpl::NormPlan p = laimpl::pick_gated(xb, s->dim);
    const int64_t groups = sat_mul(s->rows, s->heads);
    return launch(p.fn, groups / p.per_block + (groups % p.per_block != 0), p.threads, 0, &a, hip_stream);
}

int norm_residual(const la_norm_shape_t *s, const void *y, const void *post_weight, const void *gate,
                  const void *residual, void *residual_out, const void *pre_weight, void *out, void *hip_stream) {
    g_detail[0] = 0;
    int xb, rb;
    int rc = check_norm(s, true, &xb, &rb);
    if (rc != CV_OK) return rc;
    Dim d[1] = {{s->rows, s->out_row_stride}}, e[1] = {{s->rows, s->res_out_row_stride}};
    if (!apart(s->dim, e, 1) || (out && !apart(s->dim, d, 1)))
        return fail(CV_EINVAL, "the strides of residual_out or out make rows overlap");
    if (s->rows == 0) return CV_OK;
    const Pointer ps[] = {{"y", y, true, 16}, {"post_weight", post_weight, false, 16}, {"gate", gate, false, 16},
                          {"residual", residual, true, 16}, {"residual_out", residual_out, true, 16},
                          {"pre_weight", pre_weight, out != nullptr, 16}, {"out", out, false, 16}};
    if ((rc = check_pointers(ps)) != CV_OK) return rc;
    laimpl::NormArgs a{};
    a.y = y; a.gate = gate; a.weight = pre_weight; a.post_weight = post_weight; a.residual = residual;
    a.out = out; a.residual_out = residual_out;
    a.rows = s->rows; a.heads = 1; a.dim = s->dim; a.eps = s->eps; a.scale = s->scale;
    a.y_row = s->y_row_stride; a.gate_row = s->gate_row_stride; a.out_row = s->out_row_stride;
    a.res_row = s->res_row_stride; a.res_out_row = s->res_out_row_stride;
    const laimpl::NormPlan p = laimpl::pick_residual(xb, rb, s->dim);
    return launch(p.fn, s->rows / p.per_block + (s->rows % p.per_block != 0), p.threads, 0, &a, hip_stream);
}

const char *linattn_strerror(int code) {
    if (code == CV_OK) return "success";
    if (code == CV_EINVAL) return "invalid argument";
    if (code == CV_ENOTSUP) return "not supported by the compiled kernels";
    if (code <= CV_EHIP_BASE) return "HIP kernel launch failed";
    return "unknown error";
}

const char *linattn_last_error(void) { return g_detail; }

int linattn_abi_version(void) { return LINEAR_ATTENTION_ABI_VERSION; }

}  // extern "C"

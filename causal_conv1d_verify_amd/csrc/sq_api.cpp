// C-ABI entry points of libseqops.so: host-side validation, launch planning and error reporting.
// Every check runs before any HIP call.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "api_checks.h"
#include "sequence_ops.h"
#include "sq_internal.h"

namespace {

struct Need { bool out, packed, verify; };
constexpr Need kNeeds[] = {{true, true, false}, {true, false, false}, {true, false, true}, {false, false, false}};   // by sq_scan_call_t

struct Stride { const char *name; int64_t stride; bool used; int elem; };   // elem: a multiple of 16 bytes of such elements

int check_strides(const Stride *strides, int n) {
    for (int i = 0; i < n; ++i) {
        const Stride &d = strides[i];
        if (!d.used) continue;
        if (d.stride < 0) return fail(CV_EINVAL, "%s (%lld) is negative", d.name, (long long)d.stride);
        if (d.elem && d.stride % (16 / d.elem))
            return fail(CV_ENOTSUP, "%s (%lld) is not a multiple of 16 bytes", d.name, (long long)d.stride);
    }
    return CV_OK;
}

// The name of a stride over which sq_prompt.hip's 32-bit offsets do not reach: of four tokens, of C a
// stage; NULL if they do.
const char *far_tokens(const sq_scan_shape_t *s, bool out) {
    const int64_t most = INT32_MAX / 4;
    const struct { const char *name; int64_t stride; int tokens; bool used; } strides[] = {
        {"x_tok_stride", s->x_tok_stride, 3, true}, {"dt_tok_stride", s->dt_tok_stride, 3, true},
        {"z_tok_stride", s->z_tok_stride, 3, out}, {"b_tok_stride", s->b_tok_stride, 3, true},
        {"c_tok_stride", s->c_tok_stride, 15, out}, {"out_tok_stride", s->out_tok_stride, 3, out},
    };
    for (const auto &d : strides)
        if (d.used && sat_add(sat_mul(d.tokens, d.stride), std::max(s->d, 64)) > (dtype_bytes(s->x_dtype) == 4 ? most : 2 * most)) return d.name;
    return nullptr;
}

// What every entry point of the scan checks; *empty: there is nothing to do.
int check_scan(const sq_scan_shape_t *s, const Need &need, int *xb, int *sb, bool *empty) {
    if (!s) return fail(CV_EINVAL, "shape is NULL");
    if (s->n_seq < 0) return fail(CV_EINVAL, "n_seq (%d) is negative", s->n_seq);
    if (s->T < 1) return fail(CV_EINVAL, "T (%d) must be at least 1", s->T);
    if (!need.packed && s->T > 32)
        return fail(CV_ENOTSUP, "T (%d) is over 32: longer rows are prompts (selscan_prefill)", s->T);
    if (s->d < 1 || s->d_state < 1) return fail(CV_EINVAL, "d (%d) and d_state (%d) must be at least 1", s->d, s->d_state);
    if (s->d % 8) return fail(CV_ENOTSUP, "d (%d) must be a multiple of 8", s->d);
    if (s->d_state % 8 || s->d_state > 64)
        return fail(CV_ENOTSUP, "d_state (%d) must be a multiple of 8 up to 64", s->d_state);
    if (s->softplus != 0 && s->softplus != 1) return fail(CV_EINVAL, "softplus (%d) must be 0 or 1", s->softplus);
    *xb = dtype_bytes(s->x_dtype);
    *sb = dtype_bytes(s->state_dtype);
    if (!*xb || !*sb) return fail(CV_EINVAL, "unknown element type (x %d, state %d)", s->x_dtype, s->state_dtype);
    if (*xb == 4 && *sb == 2) return fail(CV_ENOTSUP, "fp32 x with a bf16 state");
    if (s->n_slots < 0) return fail(CV_EINVAL, "n_slots (%d) is negative", s->n_slots);
    const bool rows = !need.packed;
    const Stride strides[] = {
        {"x_seq_stride", s->x_seq_stride, rows, *xb}, {"x_tok_stride", s->x_tok_stride, true, *xb},
        {"dt_seq_stride", s->dt_seq_stride, rows, *xb}, {"dt_tok_stride", s->dt_tok_stride, true, *xb},
        {"z_seq_stride", s->z_seq_stride, rows && need.out, *xb}, {"z_tok_stride", s->z_tok_stride, need.out, *xb},
        {"b_seq_stride", s->b_seq_stride, rows, 0}, {"b_tok_stride", s->b_tok_stride, true, 0},
        {"c_seq_stride", s->c_seq_stride, rows && need.out, 0}, {"c_tok_stride", s->c_tok_stride, need.out, 0},
        {"out_seq_stride", s->out_seq_stride, rows && need.out, *xb}, {"out_tok_stride", s->out_tok_stride, need.out, *xb},
        {"state_slot_stride", s->state_slot_stride, true, *sb},
    };
    if (const int rc = check_strides(strides, sizeof strides / sizeof *strides)) return rc;
    const int64_t per_slot = (int64_t)s->d * s->d_state;
    if (s->n_slots > 1 && s->state_slot_stride < per_slot)
        return fail(CV_EINVAL, "state_slot_stride (%lld) is below a slot's %lld elements",
                    (long long)s->state_slot_stride, (long long)per_slot);
    if (need.packed && s->tokens < 0) return fail(CV_EINVAL, "tokens (%lld) is negative", (long long)s->tokens);
    if (need.out) {
        // of packed rows the tokens of all together; where they are not known, what would overlap
        // with any two of them
        const int64_t toks = rows ? s->T : s->tokens > 0 ? s->tokens : std::min<int64_t>(2, sat_mul(s->n_seq, s->T));
        Dim d[2] = {{toks, s->out_tok_stride}, {rows ? s->n_seq : 1, s->out_seq_stride}};
        if (!apart(s->d, d, 2)) return fail(CV_EINVAL, "the strides of out make its rows overlap");
    }
    if (const char *far = need.packed ? far_tokens(s, true) : nullptr)
        return fail(CV_ENOTSUP, "%s: four tokens (of C: 16) span more than 2 GiB", far);
    *empty = s->n_seq == 0;
    return CV_OK;
}

int check_data(const sq_scan_data_t *p, const Need &need, int xb) {
    if (!p) return fail(CV_EINVAL, "data is NULL");
    const Pointer ps[] = {{"x", p->x, true, 16}, {"dt", p->dt, true, 16}, {"z", need.out ? p->z : nullptr, false, 16},
                          {"B", p->B, true, xb}, {"C", need.out ? p->C : nullptr, need.out, xb}, {"A", p->A, true, 16},
                          {"D", need.out ? p->D : nullptr, false, 16}, {"dt_bias", p->dt_bias, false, 16}};
    return check_pointers(ps);
}

sqimpl::ScanArgs scan_args(const sq_scan_shape_t *s, const sq_scan_data_t *p, const Need &need, const void *state,
                           const int32_t *slot_idx, const int32_t *cu, const int32_t *num_tokens,
                           const int32_t *has_init, void *out) {
    sqimpl::ScanArgs a{};
    a.x = p->x; a.dt = p->dt; a.B = p->B; a.A = p->A; a.dt_bias = p->dt_bias;
    if (need.out) a.z = p->z, a.C = p->C, a.D = p->D;
    a.state = const_cast<void *>(state); a.out = out;
    a.slot_idx = slot_idx; a.cu_seqlens = cu; a.num_tokens = num_tokens; a.has_init = has_init;
    a.x_seq = s->x_seq_stride; a.x_tok = s->x_tok_stride;
    a.dt_seq = s->dt_seq_stride; a.dt_tok = s->dt_tok_stride;
    a.z_seq = s->z_seq_stride; a.z_tok = s->z_tok_stride;
    a.b_seq = s->b_seq_stride; a.b_tok = s->b_tok_stride;
    a.c_seq = s->c_seq_stride; a.c_tok = s->c_tok_stride;
    a.o_seq = s->out_seq_stride; a.o_tok = std::max<int64_t>(s->out_tok_stride, s->d);   // less: there is one token
    a.s_slot = s->state_slot_stride;
    a.n_seq = s->n_seq; a.T = s->T; a.d = s->d; a.d_state = s->d_state; a.n_slots = s->n_slots;
    a.softplus = s->softplus;
    a.write_state = !need.verify;
    a.seg_len = s->T;                              // a row is one segment
    a.segments = s->n_seq;
    return a;
}

// How packed prompts are cut into workgroups: a row's tokens are one chain in one workgroup for each
// 64 channels unless few chains leave most of the chip idle; then rows are cut into segments, at the
// price of passing over all but a row's last one twice.
//
// Which: where fewer than 256 workgroups, one for each compute unit, would be busy.  128 take 202 us for
// 2048 tokens of 8192 channels and 125 cut, 256 203 either way; from there on cutting loses (384: 284 us
// and 317 cut, 512: 285 and 401).
//
// How long: eight workgroups for each of 256 compute units (one prompt of 16384 x 4096: 420 us in segments of
// 512 tokens, 456 of 1024, 526 of 2048).  Not under 64 tokens (5 rows of up to 333 tokens, 1048 channels: 29.6
// us in segments of 64, 45 of 128, 28.5 of 32; 4096 tokens of 64 channels: 26.8, 32.5, 31.6), and not so many
// that joining them, which each does with all before it, takes longer than passing over one: the root of the
// chain's stages, and of the state's size (64 channels of 16384 tokens: 46.8 us in segments of 128, 55.6 of 64,
// 57.8 of 256; of 65536: 85.8 of 256, 107 of 128 or 512).
struct Cut {
    sqimpl::PromptPlan plan;
    int64_t tiles, segments, places, ws_bytes;
    int32_t seg_len;
};
Cut cut_prompts(const sq_scan_shape_t *s, int xb, int sb) {
    constexpr int64_t kSlots = 2048, kBusy = 256;  // workgroups: of cut rows, and of uncut ones that are left so
    constexpr int64_t kLeast = 4;                  // stages
    Cut c{};
    c.plan = sqimpl::pick_prompt(xb, sb, s->d_state);
    const int64_t stage = c.plan.stage;
    c.tiles = ((int64_t)s->d + c.plan.channels - 1) / c.plan.channels;
    c.segments = s->n_seq;
    c.seg_len = s->T;
    int64_t tokens = sat_mul(s->n_seq, s->T);
    if (s->tokens > 0 && s->tokens < tokens) tokens = s->tokens;
    const int64_t chain = (std::min<int64_t>(s->T, tokens) + stage - 1) / stage;
    const int64_t work = sat_mul(tokens / stage + 1, c.tiles);
    const int64_t joins = (int64_t)std::sqrt((double)chain * ((s->d_state + 15) / 16)) / 4;
    const int64_t share = std::max(std::max(kLeast, joins), work / kSlots);
    const int64_t segments = tokens / (share * stage) + s->n_seq;
    if (chain > 2 * kLeast && chain > 2 * share && work / chain < kBusy && sat_mul(segments, c.tiles) <= INT32_MAX) {
        c.seg_len = (int32_t)(share * stage);
        c.segments = segments;
        // only rows of more than seg_len tokens have places in the workspace
        c.places = tokens / c.seg_len + std::min<int64_t>(s->n_seq, tokens / c.seg_len);
        c.ws_bytes = sat_mul(sat_mul(c.places, c.tiles), 4 * (c.plan.ws_floats + c.plan.total_floats));
    }
    return c;
}

// Outputs of 8 and more tokens go in groups of four as prompts do, where a token takes fewer
// instructions (16 states; 8 rows of 17: 9.6 us for 12.9, 128 rows of 8: 58.5 for 60.2, of 17: 107 for
// 125, of 32: 156 for 206), with over 32 states of 4 and more (64 rows of 4, 64 states: 32.8 for 36.2, of
// 8: 38.9 for 65).  For fewer the state's way in counts, which that kernel has in pieces of 16
// bytes (128 rows of 4: 45 us for 35; 256 rows of 1: 105 for 47 and more), and its 16 states at least (8
// states, 64 rows of 8: 13 us for 10).  Tokens too far apart for its offsets go the other way too.
sqimpl::ScanPlan plan_few(const sq_scan_shape_t *s, const Need &need, int xb, int sb) {
    if (need.out && s->d_state > 8 && s->T >= (s->d_state > 32 ? 4 : 8) && !far_tokens(s, true)) return sqimpl::pick_groups(xb, sb, s->d_state, s->T);
    return sqimpl::pick_scan(xb, sb, s->d_state, s->T == 1, need.out);
}

int few_tokens(const sq_scan_shape_t *s, const sq_scan_data_t *p, const Need &need, const void *state,
               const int32_t *slot_idx, const int32_t *num_tokens, void *out, void *stream) {
    g_detail[0] = 0;
    int xb, sb;
    bool empty;
    int rc = check_scan(s, need, &xb, &sb, &empty);
    if (rc != CV_OK || empty) return rc;
    if (!slot_idx && s->n_slots < s->n_seq)
        return fail(CV_EINVAL, "n_slots (%d) is below n_seq (%d) and there is no slot_idx", s->n_slots, s->n_seq);
    if ((rc = check_data(p, need, xb)) != CV_OK) return rc;
    const Pointer ps[] = {{"state", state, true, 16}, {"out", out, need.out, 16}, {"slot_idx", slot_idx, false, 4},
                          {"num_tokens", num_tokens, false, 4}};
    if ((rc = check_pointers(ps)) != CV_OK) return rc;
    sqimpl::ScanArgs a = scan_args(s, p, need, state, slot_idx, nullptr, num_tokens, nullptr, out);
    const sqimpl::ScanPlan plan = plan_few(s, need, xb, sb);
    a.tiles = (int32_t)(((int64_t)s->d + plan.channels - 1) / plan.channels);
    return launch(plan.run, sat_mul(s->n_seq, a.tiles), plan.threads, 0, &a, stream);
}

int check_rotary(const sq_rotary_shape_t *s, int *xb) {
    if (!s) return fail(CV_EINVAL, "shape is NULL");
    if (s->tokens < 0 || s->q_heads < 1 || s->k_heads < 0)
        return fail(CV_EINVAL, "tokens (%lld) and k_heads (%d) must be >= 0, q_heads (%d) at least 1",
                    (long long)s->tokens, s->k_heads, s->q_heads);
    if (s->dim < 1 || s->rot < 0 || s->rot > s->dim)
        return fail(CV_EINVAL, "dim (%d) must be at least 1, rot (%d) in 0..dim", s->dim, s->rot);
    if (s->dim % 16 || s->dim > 256 || s->rot % 16)
        return fail(CV_ENOTSUP, "dim (%d) must be a multiple of 16 up to 256, rot (%d) a multiple of 16", s->dim, s->rot);
    if ((int64_t)s->q_heads + s->k_heads > (1 << 20))
        return fail(CV_ENOTSUP, "%lld heads", (long long)s->q_heads + s->k_heads);
    if (!(s->eps >= 0.0f) || !std::isfinite(s->eps)) return fail(CV_EINVAL, "eps must be finite and >= 0");
    *xb = dtype_bytes(s->x_dtype);
    if (!*xb) return fail(CV_EINVAL, "unknown element type (x %d)", s->x_dtype);
    const bool k = s->k_heads > 0;
    const Stride strides[] = {
        {"q_tok_stride", s->q_tok_stride, true, *xb}, {"q_head_stride", s->q_head_stride, true, *xb},
        {"k_tok_stride", s->k_tok_stride, k, *xb}, {"k_head_stride", s->k_head_stride, k, *xb},
        {"q_out_tok_stride", s->q_out_tok_stride, true, *xb}, {"q_out_head_stride", s->q_out_head_stride, true, *xb},
        {"k_out_tok_stride", s->k_out_tok_stride, k, *xb}, {"k_out_head_stride", s->k_out_head_stride, k, *xb},
    };
    if (const int rc = check_strides(strides, sizeof strides / sizeof *strides)) return rc;
    Dim q[2] = {{s->tokens, s->q_out_tok_stride}, {s->q_heads, s->q_out_head_stride}};
    Dim ko[2] = {{s->tokens, s->k_out_tok_stride}, {s->k_heads, s->k_out_head_stride}};
    if (!apart(s->dim, q, 2) || (k && !apart(s->dim, ko, 2)))
        return fail(CV_EINVAL, "the strides of q_out or k_out make heads overlap");
    return CV_OK;
}

int check_accept(const sq_accept_shape_t *s, bool parent, bool draft, bool path, int *pb) {
    if (!s) return fail(CV_EINVAL, "shape is NULL");
    if (s->n_seq < 0 || s->T < 1 || s->vocab < 1)
        return fail(CV_EINVAL, "n_seq (%d) must be >= 0, T (%d) and vocab (%d) at least 1", s->n_seq, s->T, s->vocab);
    if (s->T > 32) return fail(CV_ENOTSUP, "T (%d) is over 32", s->T);
    if (s->vocab > 1 << 24) return fail(CV_ENOTSUP, "vocab (%d) is over 2^24", s->vocab);
    *pb = dtype_bytes(s->p_dtype);
    if (!*pb) return fail(CV_EINVAL, "unknown element type (p %d)", s->p_dtype);
    if (parent && draft) return fail(CV_ENOTSUP, "a tree with a draft's probabilities");
    const Stride strides[] = {
        {"tokens_stride", s->tokens_stride, true, 0}, {"parent_stride", s->parent_stride, parent, 0},
        {"uniform_stride", s->uniform_stride, true, 0}, {"path_stride", s->path_stride, path, 0},
        {"target_seq_stride", s->target_seq_stride, true, 0}, {"target_tok_stride", s->target_tok_stride, true, 0},
        {"draft_seq_stride", s->draft_seq_stride, draft, 0}, {"draft_tok_stride", s->draft_tok_stride, draft, 0},
    };
    if (const int rc = check_strides(strides, sizeof strides / sizeof *strides)) return rc;
    Dim d[1] = {{s->n_seq, s->path_stride}};
    if (path && !apart(s->T, d, 1)) return fail(CV_EINVAL, "path_stride (%lld) makes its rows overlap", (long long)s->path_stride);
    return CV_OK;
}

int64_t accept_parts(const sq_accept_shape_t *s) { return (s->vocab + sqimpl::kPart - 1) / sqimpl::kPart; }
int64_t accept_bytes(const sq_accept_shape_t *s) {
    return (s->n_seq * (accept_parts(s) * 8 + (int64_t)sizeof(sqimpl::Verdict)) + 15) / 16 * 16;
}

}  // namespace

extern "C" {

int64_t selscan_prefill_workspace(const sq_scan_shape_t *s) {
    g_detail[0] = 0;
    int xb, sb;
    bool empty;
    const int rc = check_scan(s, kNeeds[SQ_SCAN_PREFILL], &xb, &sb, &empty);
    if (rc != CV_OK || empty) return rc;
    return cut_prompts(s, xb, sb).ws_bytes;
}

int selscan_prefill(const sq_scan_shape_t *s, const sq_scan_data_t *p, void *state, const int32_t *slot_idx,
                    const int32_t *cu_seqlens, const int32_t *has_initial_state, void *out, void *workspace,
                    int64_t workspace_bytes, void *hip_stream) {
    const int64_t need_ws = selscan_prefill_workspace(s);
    if (need_ws < 0) return (int)need_ws;
    if (s->n_seq == 0) return CV_OK;
    const Need &need = kNeeds[SQ_SCAN_PREFILL];
    const int xb = dtype_bytes(s->x_dtype), sb = dtype_bytes(s->state_dtype);
    int rc;
    if (!slot_idx && s->n_slots < s->n_seq)
        return fail(CV_EINVAL, "n_slots (%d) is below n_seq (%d) and there is no slot_idx", s->n_slots, s->n_seq);
    if (workspace_bytes < need_ws)
        return fail(CV_EINVAL, "workspace of %lld bytes, %lld are needed", (long long)workspace_bytes, (long long)need_ws);
    if ((rc = check_data(p, need, xb)) != CV_OK) return rc;
    const Pointer ps[] = {{"state", state, true, 16}, {"out", out, true, 16}, {"cu_seqlens", cu_seqlens, true, 4},
                          {"workspace", workspace, need_ws > 0, 16}, {"slot_idx", slot_idx, false, 4},
                          {"has_initial_state", has_initial_state, false, 4}};
    if ((rc = check_pointers(ps)) != CV_OK) return rc;
    sqimpl::ScanArgs a = scan_args(s, p, need, state, slot_idx, cu_seqlens, nullptr, has_initial_state, out);
    const Cut c = cut_prompts(s, xb, sb);
    a.tiles = (int32_t)c.tiles;
    a.seg_len = c.seg_len;
    a.segments = (int32_t)c.segments;
    const int64_t blocks = sat_mul(c.segments, c.tiles);
    if (c.ws_bytes) {
        a.places = (int32_t)c.places;
        a.ws = static_cast<float *>(workspace);
        a.ws_total = a.ws + c.places * c.tiles * c.plan.ws_floats;
        if ((rc = launch(c.plan.first, blocks, c.plan.threads, 0, &a, hip_stream)) != CV_OK) return rc;
    }
    return launch(c.plan.run, blocks, c.plan.threads, 0, &a, hip_stream);
}

int selscan_update(const sq_scan_shape_t *s, const sq_scan_data_t *p, void *state, const int32_t *slot_idx, void *out,
                   void *hip_stream) {
    return few_tokens(s, p, kNeeds[SQ_SCAN_UPDATE], state, slot_idx, nullptr, out, hip_stream);
}

int selscan_verify(const sq_scan_shape_t *s, const sq_scan_data_t *p, const void *state, const int32_t *slot_idx,
                   void *out, void *hip_stream) {
    return few_tokens(s, p, kNeeds[SQ_SCAN_VERIFY], state, slot_idx, nullptr, out, hip_stream);
}

int selscan_commit(const sq_scan_shape_t *s, const sq_scan_data_t *p, void *state, const int32_t *slot_idx,
                   const int32_t *num_tokens, void *hip_stream) {
    return few_tokens(s, p, kNeeds[SQ_SCAN_COMMIT], state, slot_idx, num_tokens, nullptr, hip_stream);
}

int selscan_describe(int call, const sq_scan_shape_t *s, sq_scan_info_t *info) {
    g_detail[0] = 0;
    if (call < SQ_SCAN_PREFILL || call > SQ_SCAN_COMMIT) return fail(CV_EINVAL, "unknown call %d", call);
    if (!info) return fail(CV_EINVAL, "info is NULL");
    int xb, sb;
    bool empty;
    const int rc = check_scan(s, kNeeds[call], &xb, &sb, &empty);
    if (rc != CV_OK) return rc;
    *info = sq_scan_info_t{};
    if (empty) return CV_OK;
    const Need &need = kNeeds[call];
    info->launches = 1;
    if (need.packed) {
        const Cut c = cut_prompts(s, xb, sb);
        info->workgroups = sat_mul(c.segments, c.tiles);
        info->threads = c.plan.threads;
        info->channels = c.plan.channels;
        info->workspace_bytes = c.ws_bytes;
        if (c.ws_bytes) info->launches = 2, info->segment_tokens = c.seg_len;
        return CV_OK;
    }
    const sqimpl::ScanPlan p = plan_few(s, need, xb, sb);
    info->workgroups = sat_mul(s->n_seq, ((int64_t)s->d + p.channels - 1) / p.channels);
    info->threads = p.threads;
    info->channels = p.channels;
    return CV_OK;
}

int norm_rotary(const sq_rotary_shape_t *s, const void *q, const void *k, const void *q_weight, const void *k_weight,
                const void *positions, const float *inv_freq, void *q_out, void *k_out, void *hip_stream) {
    g_detail[0] = 0;
    int xb;
    int rc = check_rotary(s, &xb);
    if (rc != CV_OK || s->tokens == 0) return rc;
    const bool has_k = s->k_heads > 0;
    const Pointer ps[] = {{"q", q, true, 16}, {"k", has_k ? k : nullptr, has_k, 16}, {"q_weight", q_weight, false, 16},
                          {"k_weight", has_k ? k_weight : nullptr, false, 16},
                          {"positions", s->rot ? positions : nullptr, s->rot > 0, s->wide_positions ? 8 : 4},
                          {"inv_freq", s->rot ? inv_freq : nullptr, s->rot > 0, 4}, {"q_out", q_out, true, 16},
                          {"k_out", has_k ? k_out : nullptr, has_k, 16}};
    if ((rc = check_pointers(ps)) != CV_OK) return rc;
    sqimpl::RotaryArgs a{};
    a.x[0] = q; a.x[1] = k; a.weight[0] = q_weight; a.weight[1] = k_weight; a.out[0] = q_out; a.out[1] = k_out;
    a.positions = positions; a.inv_freq = inv_freq;
    a.tok[0] = s->q_tok_stride; a.tok[1] = s->k_tok_stride;
    a.head[0] = s->q_head_stride; a.head[1] = s->k_head_stride;
    a.out_tok[0] = s->q_out_tok_stride; a.out_tok[1] = s->k_out_tok_stride;
    a.out_head[0] = s->q_out_head_stride; a.out_head[1] = s->k_out_head_stride;
    a.tokens = s->tokens; a.heads[0] = s->q_heads; a.heads[1] = s->k_heads; a.dim = s->dim; a.rot = s->rot;
    a.eps = s->eps; a.interleaved = s->interleaved != 0; a.wide = s->wide_positions != 0;
    const sqimpl::RotaryPlan p = sqimpl::pick_rotary(xb, s->dim);
    // few tokens: their heads over as many wavefronts as there are sets of them; many: one each, which
    // makes the token's angles once
    const int64_t sets = ((int64_t)s->q_heads + s->k_heads + p.heads - 1) / p.heads;
    a.blocks_per_token = (int32_t)std::max<int64_t>(1, std::min<int64_t>(sets, 2048 / s->tokens));
    const int64_t waves = sat_mul(s->tokens, a.blocks_per_token), per = p.threads / 64;
    return launch(p.fn, waves / per + (waves % per != 0), p.threads, 0, &a, hip_stream);
}

int64_t accept_drafts_workspace(const sq_accept_shape_t *s) {
    g_detail[0] = 0;
    int pb;
    const int rc = check_accept(s, false, false, false, &pb);
    return rc != CV_OK ? rc : accept_bytes(s);
}

int accept_drafts(const sq_accept_shape_t *s, const int32_t *tokens, const int32_t *parent, const void *target,
                  const void *draft, const float *uniform, const int32_t *slot_idx, int32_t *num_tokens,
                  int32_t *next_token, int32_t *window_index, int32_t *path, void *workspace, int64_t workspace_bytes,
                  void *hip_stream) {
    g_detail[0] = 0;
    int pb;
    int rc = check_accept(s, parent, draft, path, &pb);
    if (rc != CV_OK || s->n_seq == 0) return rc;
    if (workspace_bytes < accept_bytes(s))
        return fail(CV_EINVAL, "workspace of %lld bytes, %lld are needed", (long long)workspace_bytes, (long long)accept_bytes(s));
    const Pointer ps[] = {{"tokens", tokens, true, 4}, {"parent", parent, false, 4}, {"target", target, true, pb},
                          {"draft", draft, false, pb}, {"uniform", uniform, true, 4}, {"slot_idx", slot_idx, false, 4},
                          {"num_tokens", num_tokens, true, 4}, {"next_token", next_token, true, 4},
                          {"window_index", window_index, false, 4}, {"path", path, false, 4},
                          {"workspace", workspace, true, 16}};
    if ((rc = check_pointers(ps)) != CV_OK) return rc;
    const sqimpl::AcceptPlan p = sqimpl::pick_accept(pb);
    sqimpl::AcceptArgs a{};
    a.tokens = tokens; a.parent = parent; a.target = target; a.draft = draft; a.uniform = uniform; a.slot_idx = slot_idx;
    a.num = num_tokens; a.next = next_token; a.last = window_index; a.path = path;
    a.tokens_row = s->tokens_stride; a.parent_row = s->parent_stride; a.uniform_row = s->uniform_stride;
    a.path_row = s->path_stride;
    a.target_seq = s->target_seq_stride; a.target_tok = s->target_tok_stride;
    a.draft_seq = s->draft_seq_stride; a.draft_tok = s->draft_tok_stride;
    a.verdicts = static_cast<sqimpl::Verdict *>(workspace);
    a.sums = reinterpret_cast<double *>(a.verdicts + s->n_seq);
    a.n_seq = s->n_seq; a.T = s->T; a.vocab = s->vocab;
    a.parts = (int32_t)accept_parts(s);
    a.chunks = (a.parts + p.parts - 1) / p.parts;
    if ((rc = launch(p.sums, sat_mul(s->n_seq, a.chunks), p.threads, 0, &a, hip_stream)) != CV_OK) return rc;
    return launch(p.pick, s->n_seq, p.threads, 0, &a, hip_stream);
}

const char *seqops_strerror(int code) {
    if (code == CV_OK) return "success";
    if (code == CV_EINVAL) return "invalid argument";
    if (code == CV_ENOTSUP) return "not supported by the compiled kernels";
    if (code <= CV_EHIP_BASE) return "HIP kernel launch failed";
    return "unknown error";
}

const char *seqops_last_error(void) { return g_detail; }

int seqops_abi_version(void) { return SEQUENCE_OPS_ABI_VERSION; }

}  // extern "C"

// The host side of liblinattn.so (la_api.cpp) under AddressSanitizer and UndefinedBehaviorSanitizer,
// with stand-ins for the kernels' pickers and for hipLaunchKernel, which records the launch instead
// of running it.  A fuzz of shapes over the full range of every field: a refused call launches
// nothing, an accepted one launches grids within the hardware limits that are exactly the workgroups
// its plan needs; and the segments of random rows fit the grid and the workspace that a call asks for.
#include <hip/hip_runtime_api.h>

#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <random>
#include <vector>

#include "la_internal.h"
#include "linear_attention.h"

using namespace laimpl;

namespace {
char g_marker[16];
const void *mark(int i) { return &g_marker[i]; }
struct Launch { int code; unsigned grid, block; AttnArgs a; };
std::vector<Launch> g_launches;
long g_mismatches = 0;

void check(bool ok, const char *what, const la_shape_t *s) {
    if (ok) return;
    if (++g_mismatches > 20) return;
    std::printf("MISMATCH %s", what);
    if (s)
        std::printf(" n_seq %d T %d heads %d %d d %d %d types %d %d slots %d tokens %lld", s->n_seq, s->T, s->q_heads,
                    s->v_heads, s->dk, s->dv, s->x_dtype, s->state_dtype, s->n_slots, (long long)s->tokens);
    std::printf("\n");
}
}  // namespace

namespace laimpl {
// the real pickers' tiles
RecurrentPlan pick_recurrent(int, int state_bytes, int dk, bool wide) {
    const int vc = 16 / state_bytes;
    (void)dk;
    return {mark(0), (wide ? 16 : 8) * vc, 256};
}
static ChunkedPlan chunked(int rows, int cols, int chunk, int code) {
    return {mark(code), mark(code + 1), mark(4), cols, 256, chunk, (int64_t)rows * cols * 4};
}
ChunkedPlan pick_chunked(int, int dk, bool wide) { return chunked(dk <= 64 ? 64 : dk <= 128 ? 128 : dk <= 192 ? 192 : 256, wide ? 128 : 64, 64, 2); }
ChunkedPlan pick_chunked_f32(int dk) { return chunked(dk <= 64 ? 64 : dk <= 96 ? 96 : dk <= 128 ? 128 : dk <= 192 ? 192 : 256, 64, 32, 2); }
const void *pick_few(int, int, int, bool, bool) { return mark(1); }
NormPlan pick_gated(int, int dim) { return {mark(5), 256, dim <= 8 ? 256 : 4}; }
NormPlan pick_residual(int, int, int dim) { return {mark(6), dim <= 4096 ? 512 : 1024, dim <= 512 ? 4 : 1}; }
}  // namespace laimpl

extern "C" {
hipError_t hipLaunchKernel(const void *fn, dim3 grid, dim3 block, void **args, size_t, hipStream_t) {
    Launch l{(int)(static_cast<const char *>(fn) - g_marker), grid.x, block.x, {}};
    check(l.code >= 0 && l.code < 7, "kernel", nullptr);
    if (l.code < 5) std::memcpy(&l.a, args[0], sizeof l.a);
    g_launches.push_back(l);
    return hipSuccess;
}
const char *hipGetErrorString(hipError_t) { return "stub"; }
}

namespace {
std::mt19937_64 g_rng(7);
int64_t below(int64_t n) { return (int64_t)(g_rng() % (uint64_t)n); }
template <typename T, size_t N>
T one_of(const T (&v)[N]) { return v[g_rng() % N]; }

int32_t any32() {
    static const int32_t odd[] = {0, 1, -1, 2, 8, 31, 32, 33, 64, 128, 256, 264, INT32_MAX, INT32_MIN, INT32_MAX - 7, 1 << 24};
    return below(4) ? one_of(odd) : (int32_t)g_rng();
}
int64_t any64() {
    static const int64_t odd[] = {0, 8, 16, 64, 128, 1024, -8, INT64_MAX, INT64_MAX - 7, INT64_MIN, 1LL << 31, 1LL << 40, 1LL << 62};
    return below(4) ? one_of(odd) : (int64_t)g_rng();
}
int32_t log_size(int bits) { return (int32_t)((g_rng() & ((1ull << (1 + below(bits))) - 1)) | (below(4) ? 1 : 0)); }

int64_t times(int64_t a, int64_t b) {
    int64_t r;
    return __builtin_mul_overflow(a, b, &r) ? INT64_MAX / 16 * 16 : r;
}

// Sizes that belong together, over the whole range, with a field or two of anything.
la_shape_t shape(bool wild) {
    la_shape_t s{};
    s.q_heads = 1 + log_size(below(8) ? 5 : 24) % (1 << 24);
    s.v_heads = (int32_t)(s.q_heads * (1 + below(4)));
    s.n_seq = log_size(below(4) ? 10 : 31);
    if (below(16) == 0) {                          // as much as the fields hold
        s.q_heads = 1;
        s.v_heads = INT32_MAX - (int32_t)below(9);
        s.n_seq = INT32_MAX - (int32_t)below(9);
    }
    s.T = below(3) ? (int32_t)(1 + below(32)) : log_size(31);
    s.dk = (int32_t)(8 + 8 * below(32));
    s.dv = (int32_t)(8 + 8 * below(32));
    s.scale = 0.1f;
    s.x_dtype = below(2) ? CV_BF16 : CV_F32;
    s.state_dtype = s.x_dtype == CV_F32 || below(2) ? CV_F32 : CV_BF16;
    s.n_slots = below(2) ? s.n_seq : log_size(31);
    s.q_head_stride = s.k_head_stride = s.dk;
    s.v_head_stride = s.out_head_stride = s.dv;
    s.q_tok_stride = s.k_tok_stride = (int64_t)s.q_heads * s.dk;
    s.v_tok_stride = s.out_tok_stride = (int64_t)s.v_heads * s.dv;
    s.q_seq_stride = s.k_seq_stride = times(s.T, s.q_tok_stride);
    s.v_seq_stride = s.out_seq_stride = times(s.T, s.v_tok_stride);
    s.g_tok_stride = s.v_heads;
    s.g_seq_stride = (int64_t)s.T * s.v_heads;
    s.state_slot_stride = (int64_t)s.v_heads * s.dk * s.dv;
    s.tokens = below(3) ? below((int64_t)1 << (1 + below(40))) : 0;
    for (int n = wild ? (int)below(4) : 0; n > 0; --n) {
        int32_t *w[] = {&s.n_seq, &s.T, &s.q_heads, &s.v_heads, &s.dk, &s.dv, &s.x_dtype, &s.state_dtype, &s.n_slots};
        int64_t *x[] = {&s.q_seq_stride, &s.q_tok_stride, &s.q_head_stride, &s.k_seq_stride, &s.k_tok_stride,
                        &s.k_head_stride, &s.v_seq_stride, &s.v_tok_stride, &s.v_head_stride, &s.out_seq_stride,
                        &s.out_tok_stride, &s.out_head_stride, &s.g_seq_stride, &s.g_tok_stride, &s.state_slot_stride,
                        &s.tokens};
        if (below(2)) *w[g_rng() % 9] = any32();
        else *x[g_rng() % 16] = any64();
    }
    return s;
}

typedef __int128 wide;

// The launches of an accepted call against its description.
void accepted(int call, const la_shape_t *s) {
    la_launch_info_t info;
    check(linattn_describe(call, s, &info) == CV_OK, "described", s);
    check((int)g_launches.size() == info.launches, "launches", s);
    if (s->n_seq == 0) return;
    for (const Launch &l : g_launches) {
        const AttnArgs &a = l.a;
        check(l.grid >= 1 && l.grid <= INT32_MAX && l.block == 256, "grid", s);
        const int64_t cols = info.state_cols;
        check((wide)a.tiles * cols >= s->dv && (wide)(a.tiles - 1) * cols < s->dv, "tiles", s);
        const wide rows = info.kernel >= LA_KERNEL_CHUNKED && l.code != 4 ? a.segments : s->n_seq;
        if (l.code != 4) check((wide)l.grid == rows * s->v_heads * a.tiles, "workgroups", s);
        else check((wide)l.grid % ((wide)s->n_seq * s->v_heads * a.tiles) == 0, "workgroups of the sums", s);
    }
    const AttnArgs &a = g_launches.back().a;
    check((int64_t)g_launches.back().grid == info.workgroups, "workgroups described", s);
    if (info.launches == 3) {
        const int code[] = {g_launches[0].code, g_launches[1].code, g_launches[2].code};
        check(code[0] == 3 && code[1] == 4 && code[2] == 2, "order of the launches", s);
        check(a.seg_len == info.segment_tokens && a.seg_len < s->T, "segments", s);
        const wide states = (wide)a.places * s->v_heads * a.tiles;
        const wide ws = (const char *)a.ws_total - (const char *)a.ws;
        const wide each = (wide)(s->dk <= 64 ? 64 : s->x_dtype == CV_F32 && s->dk <= 96 ? 96 : s->dk <= 128 ? 128
                                 : s->dk <= 192 ? 192 : 256) * info.state_cols * 4;
        check(a.places > 0 && ws == states * each && ws + 4 * states <= info.workspace_bytes, "workspace", s);
        // rows of at most T tokens, of all tokens together: what the device counts
        const int64_t most = s->tokens > 0 ? s->tokens : INT64_MAX;
        for (int turn = 0; turn < 3; ++turn) {
            wide left = most, segments = 0, places = 0;
            const int64_t rows = s->n_seq < 4096 ? s->n_seq : 4096;
            for (int64_t i = 0; i < rows; ++i) {
                int64_t n = turn == 0 ? s->T : turn == 1 ? (int64_t)a.seg_len + 1 : below((int64_t)s->T + 1);
                if (n > s->T) n = s->T;
                if ((wide)n > left) n = (int64_t)left;
                left -= n;
                const int64_t own = n == 0 ? 1 : (n + a.seg_len - 1) / a.seg_len;
                segments += own;
                if (own > 1) places += own;
            }
            segments += s->n_seq - rows;
            check(segments <= a.segments && places <= a.places, "rows within the grid and the workspace", s);
        }
    } else if (info.kernel >= LA_KERNEL_CHUNKED) {
        check(a.seg_len == s->T && a.segments == s->n_seq && info.workspace_bytes == 0, "whole rows", s);
    }
}

void norms(long n) {
    alignas(64) static char buffer[64];
    long taken = 0;
    for (long i = 0; i < n; ++i) {
        la_norm_shape_t s{};
        s.rows = below(4) ? log_size(20) : any64();
        s.heads = below(4) ? 1 + log_size(6) : any32();
        s.dim = below(4) ? (int32_t)(8 + 8 * below(300)) : any32();
        s.eps = 1e-6f;
        s.scale = 1.0f;
        s.x_dtype = below(8) ? (int32_t)below(2) : any32();
        s.res_dtype = s.x_dtype;
        s.activation = (int32_t)below(2);
        int64_t *x[] = {&s.y_row_stride, &s.y_head_stride, &s.gate_row_stride, &s.gate_head_stride, &s.out_row_stride,
                        &s.out_head_stride, &s.res_row_stride, &s.res_out_row_stride};
        for (int64_t *p : x) *p = below(8) ? (p == x[1] || p == x[3] || p == x[5] ? s.dim : times(s.dim, s.heads > 0 ? s.heads : 1)) : any64();
        for (int residual = 0; residual < 2; ++residual) {
            if (residual) s.heads = below(8) ? 1 : s.heads;
            g_launches.clear();
            const int rc = residual ? norm_residual(&s, buffer, buffer, buffer, buffer, buffer, buffer, buffer, nullptr)
                                    : norm_gated(&s, buffer, buffer, buffer, buffer, nullptr);
            if (rc != CV_OK) {
                check(g_launches.empty() && linattn_last_error()[0], "a refused norm launched", nullptr);
                continue;
            }
            ++taken;
            check((s.rows == 0) == g_launches.empty(), "norm launches", nullptr);
            if (s.rows == 0) continue;
            const Launch &l = g_launches[0];
            const wide groups = (wide)s.rows * (residual ? 1 : s.heads);
            const int per = residual ? (s.dim <= 512 ? 4 : 1) : s.dim <= 8 ? 256 : 4;
            check(l.grid <= INT32_MAX && (wide)l.grid == (groups + per - 1) / per, "norm grid", nullptr);
        }
    }
    std::printf("norms: %ld calls taken\n", taken);
    check(taken > n / 20, "norms taken", nullptr);
}
}  // namespace

int main(int argc, char **argv) {
    const long n = argc > 1 ? std::atol(argv[1]) : 1000;
    alignas(64) static char buffer[64];
    float *g = reinterpret_cast<float *>(buffer);
    int32_t *v = reinterpret_cast<int32_t *>(buffer);
    long taken[4] = {}, cut = 0;
    for (long i = 0; i < n; ++i) {
        const la_shape_t s = shape(below(2) != 0);
        const int call = (int)below(4);
        g_launches.clear();
        int rc;
        if (call == LA_CALL_PREFILL) {
            const int64_t need = linattn_prefill_workspace(&s);
            check(g_launches.empty(), "asking launched", &s);
            rc = linattn_prefill(&s, buffer, buffer, buffer, g, buffer, v, v, v, buffer, buffer, need < 0 ? 0 : need, nullptr);
            check(need >= 0 || rc == need, "workspace and call agree", &s);
            if (need > 0) {
                const size_t before = g_launches.size();
                check(linattn_prefill(&s, buffer, buffer, buffer, g, buffer, v, v, v, buffer, buffer, need - 1, nullptr) == CV_EINVAL &&
                          g_launches.size() == before, "a small workspace", &s);
            }
        } else if (call == LA_CALL_COMMIT) {
            rc = linattn_commit(&s, buffer, buffer, g, buffer, v, v, nullptr);
        } else {
            rc = call == LA_CALL_UPDATE ? linattn_update(&s, buffer, buffer, buffer, g, buffer, v, buffer, nullptr)
                                        : linattn_verify(&s, buffer, buffer, buffer, g, buffer, v, buffer, nullptr);
        }
        if (rc != CV_OK) {
            check(g_launches.empty(), "a refused call launched", &s);
            check(rc < 0 && linattn_last_error()[0] != 0, "its reason", &s);
            continue;
        }
        ++taken[call];
        cut += g_launches.size() == 3;
        accepted(call, &s);
    }
    std::printf("fuzz: %ld shapes, taken %ld %ld %ld %ld, cut %ld\n", n, taken[0], taken[1], taken[2], taken[3], cut);
    for (long t : taken) check(t > n / 50, "shapes taken", nullptr);
    check(cut > n / 200, "cut calls", nullptr);
    norms(n / 4);
    if (g_mismatches) std::printf("%ld mismatches\n", g_mismatches);
    else std::printf("ALL OK\n");
    return g_mismatches ? 1 : 0;
}

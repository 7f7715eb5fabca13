// The host side of libseqops.so (sq_api.cpp) under AddressSanitizer and UndefinedBehaviorSanitizer, with
// stand-ins for the kernels' pickers and for hipLaunchKernel, which records the launch instead of
// running it.  A fuzz of shapes over the full range of every field: a refused call launches nothing,
// an accepted one launches grids within the hardware limits that are exactly the workgroups its plan
// needs; and the segments of random rows fit the grid and the workspace that a call asks for.
#include <hip/hip_runtime_api.h>

#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <random>
#include <vector>

#include "sequence_ops.h"
#include "sq_internal.h"

using namespace sqimpl;
typedef __int128 wide;

namespace {
char g_marker[16];
const void *mark(int i) { return &g_marker[i]; }
struct Launch { int code; unsigned grid, block; ScanArgs scan; RotaryArgs rotary; AcceptArgs accept; };
std::vector<Launch> g_launches;
long g_mismatches = 0;

void check(bool ok, const char *what) {
    if (!ok && ++g_mismatches <= 20) std::printf("MISMATCH %s\n", what);
}
}  // namespace

namespace sqimpl {
// the real pickers' tiles
static int sixteens(int d_state) { return (d_state + 15) / 16; }
ScanPlan pick_scan(int, int, int d_state, bool, bool) { return {mark(0), d_state <= 16 ? 256 : d_state <= 32 ? 128 : 64, 256}; }
ScanPlan pick_groups(int, int, int, int) { return {mark(1), 64, 256}; }
PromptPlan pick_prompt(int, int, int d_state) {
    return {mark(2), mark(3), 64, 256, 16, 1024 * sixteens(d_state), 256};
}
RotaryPlan pick_rotary(int, int dim) {
    const int units = dim / 16;
    return {mark(5), 256, 64 / (units <= 1 ? 1 : units <= 2 ? 2 : units <= 4 ? 4 : units <= 8 ? 8 : 16)};
}
AcceptPlan pick_accept(int) { return {mark(6), mark(7), 256, 4}; }
}  // namespace sqimpl

extern "C" {
hipError_t hipLaunchKernel(const void *fn, dim3 grid, dim3 block, void **args, size_t, hipStream_t) {
    Launch l{};
    l.code = (int)(static_cast<const char *>(fn) - g_marker);
    l.grid = grid.x, l.block = block.x;
    check(l.code >= 0 && l.code < 8 && l.grid >= 1 && l.grid <= INT32_MAX && l.block == 256, "launch");
    if (l.code < 5) std::memcpy(&l.scan, args[0], sizeof l.scan);
    else if (l.code == 5) std::memcpy(&l.rotary, args[0], sizeof l.rotary);
    else std::memcpy(&l.accept, args[0], sizeof l.accept);
    g_launches.push_back(l);
    return hipSuccess;
}
const char *hipGetErrorString(hipError_t) { return "stub"; }
}

namespace {
std::mt19937_64 g_rng(11);
int64_t below(int64_t n) { return (int64_t)(g_rng() % (uint64_t)n); }
template <typename T, size_t N>
T one_of(const T (&v)[N]) { return v[g_rng() % N]; }
int32_t any32() {
    static const int32_t odd[] = {0, 1, -1, 2, 8, 31, 32, 33, 64, 256, INT32_MAX, INT32_MIN, INT32_MAX - 7, 1 << 24};
    return below(4) ? one_of(odd) : (int32_t)g_rng();
}
int64_t any64() {
    static const int64_t odd[] = {0, 8, 16, 64, 1024, -8, INT64_MAX, INT64_MAX - 7, INT64_MIN, 1LL << 28, 1LL << 31, 1LL << 40, 1LL << 62};
    return below(4) ? one_of(odd) : (int64_t)g_rng();
}
int32_t log_size(int bits) { return (int32_t)((g_rng() & ((1ull << (1 + below(bits))) - 1)) | (below(4) ? 1 : 0)); }
int64_t times(int64_t a, int64_t b) {
    int64_t r;
    return __builtin_mul_overflow(a, b, &r) ? INT64_MAX / 16 * 16 : r;
}
alignas(64) char g_buffer[64];
float *f32() { return reinterpret_cast<float *>(g_buffer); }
int32_t *i32() { return reinterpret_cast<int32_t *>(g_buffer); }

sq_scan_shape_t scan_shape(bool wild) {
    sq_scan_shape_t s{};
    s.d = 8 * (1 + log_size(below(8) ? 11 : 27) % (1 << 27));
    s.d_state = (int32_t)(8 + 8 * below(8));
    s.n_seq = log_size(below(4) ? 10 : 31);
    if (below(16) == 0) s.n_seq = INT32_MAX - (int32_t)below(9), s.d = 8;
    s.T = below(3) ? (int32_t)(1 + below(32)) : log_size(31);
    s.x_dtype = below(2) ? CV_BF16 : CV_F32;
    s.state_dtype = s.x_dtype == CV_F32 || below(2) ? CV_F32 : CV_BF16;
    s.n_slots = below(2) ? s.n_seq : log_size(31);
    s.softplus = (int32_t)below(2);
    int64_t *tok[] = {&s.x_tok_stride, &s.dt_tok_stride, &s.z_tok_stride, &s.out_tok_stride};
    int64_t *seq[] = {&s.x_seq_stride, &s.dt_seq_stride, &s.z_seq_stride, &s.out_seq_stride};
    for (int k = 0; k < 4; ++k) *tok[k] = s.d, *seq[k] = times(s.T, s.d);
    s.b_tok_stride = s.c_tok_stride = 2 * s.d_state + below(5);
    s.b_seq_stride = s.c_seq_stride = times(s.T, s.b_tok_stride);
    s.state_slot_stride = (int64_t)s.d * s.d_state;
    s.tokens = below(3) ? below((int64_t)1 << (1 + below(40))) : 0;
    for (int n = wild ? (int)below(4) : 0; n > 0; --n) {
        int32_t *w[] = {&s.n_seq, &s.T, &s.d, &s.d_state, &s.x_dtype, &s.state_dtype, &s.n_slots, &s.softplus};
        int64_t *x[] = {&s.x_seq_stride, &s.x_tok_stride, &s.dt_seq_stride, &s.dt_tok_stride, &s.z_seq_stride, &s.z_tok_stride,
                        &s.b_seq_stride, &s.b_tok_stride, &s.c_seq_stride, &s.c_tok_stride, &s.out_seq_stride, &s.out_tok_stride,
                        &s.state_slot_stride, &s.tokens};
        if (below(2)) *w[g_rng() % 8] = any32();
        else *x[g_rng() % 14] = any64();
    }
    return s;
}

// The launches of an accepted call against its description.
void scan_accepted(int call, const sq_scan_shape_t &s) {
    sq_scan_info_t info;
    check(selscan_describe(call, &s, &info) == CV_OK, "described");
    check((int)g_launches.size() == info.launches, "launches");
    if (s.n_seq == 0) return;
    const ScanArgs &a = g_launches.back().scan;
    check((int64_t)g_launches.back().grid == info.workgroups, "workgroups described");
    for (const Launch &l : g_launches) {
        check((wide)l.scan.tiles * info.channels >= s.d && (wide)(l.scan.tiles - 1) * info.channels < s.d, "tiles");
        check((wide)l.grid == (wide)a.segments * a.tiles, "workgroups");
    }
    check(g_launches.back().code == (call == SQ_SCAN_PREFILL ? 2 : g_launches.back().code == 1 ? 1 : 0), "kernel");
    if (g_launches.back().code >= 1) {             // four tokens lie within 2 GiB, and 16 of C
        const int xb = s.x_dtype == CV_F32 ? 4 : 2;
        for (int64_t t : {a.x_tok, a.dt_tok, a.z_tok, a.o_tok, a.b_tok, 5 * a.c_tok})
            check(((wide)3 * t + s.d) * xb <= INT32_MAX, "far tokens");
    }
    if (call != SQ_SCAN_PREFILL) return;
    if (info.launches != 2) {
        check(a.seg_len == s.T && a.segments == s.n_seq && info.workspace_bytes == 0, "whole rows");
        return;
    }
    check(g_launches[0].code == 3, "order of the launches");
    check(a.seg_len == info.segment_tokens && a.seg_len < s.T && a.seg_len % 16 == 0, "segments");
    const wide each = (wide)a.places * a.tiles, ws = (const char *)a.ws_total - (const char *)a.ws;
    check(a.places > 0 && ws == each * 4096 * sixteens(s.d_state) && ws + each * 1024 <= info.workspace_bytes, "workspace");
    // rows of at most T tokens, of all tokens together: what the device counts
    for (int turn = 0; turn < 3; ++turn) {
        wide left = s.tokens > 0 ? s.tokens : INT64_MAX, segments = 0, places = 0;
        const int64_t rows = s.n_seq < 4096 ? s.n_seq : 4096;
        for (int64_t i = 0; i < rows; ++i) {
            int64_t n = turn == 0 ? s.T : turn == 1 ? (int64_t)a.seg_len + 1 : below((int64_t)s.T + 1);
            if (n > s.T) n = s.T;
            if ((wide)n > left) n = (int64_t)left;
            left -= n;
            const int64_t own = n == 0 ? 1 : (n + a.seg_len - 1) / a.seg_len;
            segments += own;
            if (own > 1) places += own;
        }
        segments += s.n_seq - rows;
        check(segments <= a.segments && places <= a.places, "rows within the grid and the workspace");
    }
}

void scans(long n) {
    long taken[4] = {}, cut = 0;
    const sq_scan_data_t data{g_buffer, g_buffer, g_buffer, g_buffer, g_buffer, f32(), f32(), f32()};
    for (long i = 0; i < n; ++i) {
        const sq_scan_shape_t s = scan_shape(below(2) != 0);
        const int call = (int)below(4);
        g_launches.clear();
        int rc;
        if (call == SQ_SCAN_PREFILL) {
            const int64_t need = selscan_prefill_workspace(&s);
            check(g_launches.empty(), "asking launched");
            rc = selscan_prefill(&s, &data, g_buffer, i32(), i32(), i32(), g_buffer, g_buffer, need < 0 ? 0 : need, nullptr);
            check(need >= 0 || rc == need, "workspace and call agree");
            if (need > 0) {
                const size_t before = g_launches.size();
                check(selscan_prefill(&s, &data, g_buffer, i32(), i32(), i32(), g_buffer, g_buffer, need - 1, nullptr) == CV_EINVAL &&
                          g_launches.size() == before, "a small workspace");
            }
        } else if (call == SQ_SCAN_COMMIT) {
            rc = selscan_commit(&s, &data, g_buffer, i32(), i32(), nullptr);
        } else {
            rc = call == SQ_SCAN_UPDATE ? selscan_update(&s, &data, g_buffer, i32(), g_buffer, nullptr)
                                        : selscan_verify(&s, &data, g_buffer, i32(), g_buffer, nullptr);
        }
        if (rc != CV_OK) {
            check(g_launches.empty() && rc < 0 && seqops_last_error()[0], "a refused scan");
            continue;
        }
        ++taken[call];
        cut += g_launches.size() == 2;
        scan_accepted(call, s);
    }
    std::printf("fuzz: %ld shapes, taken %ld %ld %ld %ld, cut %ld\n", n, taken[0], taken[1], taken[2], taken[3], cut);
    for (long t : taken) check(t > n / 50, "shapes taken");
    check(cut > n / 500, "cut calls");
}

void rotaries(long n) {
    long taken = 0;
    for (long i = 0; i < n; ++i) {
        sq_rotary_shape_t s{};
        s.tokens = below(4) ? log_size(24) : any64();
        s.q_heads = below(8) ? 1 + log_size(6) : any32();
        s.k_heads = below(8) ? log_size(5) : any32();
        s.dim = below(8) ? (int32_t)(16 + 16 * below(16)) : any32();
        s.rot = below(8) && s.dim > 0 ? (int32_t)(16 * below(s.dim / 16 + 1)) : any32();
        s.eps = 1e-6f;
        s.x_dtype = below(8) ? (int32_t)below(2) : any32();
        s.wide_positions = (int32_t)below(2);
        int64_t *tok[] = {&s.q_tok_stride, &s.k_tok_stride, &s.q_out_tok_stride, &s.k_out_tok_stride};
        int64_t *head[] = {&s.q_head_stride, &s.k_head_stride, &s.q_out_head_stride, &s.k_out_head_stride};
        for (int k = 0; k < 4; ++k) {
            *head[k] = below(16) ? s.dim : any64();
            *tok[k] = below(16) ? times(s.dim, k % 2 ? s.k_heads : s.q_heads) : any64();
        }
        g_launches.clear();
        const int rc = norm_rotary(&s, g_buffer, g_buffer, g_buffer, g_buffer, g_buffer, f32(), g_buffer, g_buffer, nullptr);
        if (rc != CV_OK) {
            check(g_launches.empty() && seqops_last_error()[0], "a refused rotation");
            continue;
        }
        ++taken;
        check((s.tokens == 0) == g_launches.empty(), "rotation launches");
        if (s.tokens == 0) continue;
        const Launch &l = g_launches[0];
        const wide waves = (wide)s.tokens * l.rotary.blocks_per_token;
        check(l.rotary.blocks_per_token >= 1 && (wide)l.grid == (waves + 3) / 4, "rotation grid");
    }
    std::printf("rotations: %ld taken\n", taken);
    check(taken > n / 20, "rotations taken");
}

void accepts(long n) {
    long taken = 0;
    for (long i = 0; i < n; ++i) {
        sq_accept_shape_t s{};
        s.n_seq = below(4) ? log_size(16) : any32();
        s.T = below(8) ? (int32_t)(1 + below(33)) : any32();
        s.vocab = below(8) ? 1 + log_size(24) : any32();
        s.p_dtype = below(8) ? (int32_t)below(2) : any32();
        const int64_t T = s.T > 0 ? s.T : 1;
        s.tokens_stride = s.parent_stride = s.uniform_stride = s.path_stride = T;
        s.target_tok_stride = s.draft_tok_stride = s.vocab;
        s.target_seq_stride = times(T, s.vocab), s.draft_seq_stride = times(T - 1, s.vocab);
        if (below(4) == 0) {
            int64_t *x[] = {&s.tokens_stride, &s.parent_stride, &s.uniform_stride, &s.path_stride, &s.target_seq_stride,
                            &s.target_tok_stride, &s.draft_seq_stride, &s.draft_tok_stride};
            *x[g_rng() % 8] = any64();
        }
        const bool tree = below(3) == 0, draft = below(tree ? 8 : 2) == 0;
        const int64_t need = accept_drafts_workspace(&s);
        g_launches.clear();
        const int rc = accept_drafts(&s, i32(), tree ? i32() : nullptr, g_buffer, draft ? g_buffer : nullptr, f32(), i32(), i32(),
                                     i32(), i32(), i32(), g_buffer, need < 0 ? 0 : need, nullptr);
        if (rc != CV_OK) {
            check(g_launches.empty() && seqops_last_error()[0], "a refused verdict");
            continue;
        }
        ++taken;
        check(need >= 0 && (s.n_seq == 0) == g_launches.empty(), "verdict launches");
        if (s.n_seq == 0) continue;
        const AcceptArgs &a = g_launches[0].accept;
        check(g_launches.size() == 2 && g_launches[0].code == 6 && g_launches[1].code == 7, "verdict order");
        check((wide)a.parts * kPart >= s.vocab && (wide)(a.parts - 1) * kPart < s.vocab, "parts");
        check((wide)a.chunks * 4 >= a.parts && (wide)g_launches[0].grid == (wide)s.n_seq * a.chunks, "verdict grid");
        check((int64_t)g_launches[1].grid == s.n_seq, "draw grid");
        const wide sums = (const char *)a.sums - (const char *)a.verdicts;
        check(sums == (wide)s.n_seq * (wide)sizeof(Verdict) && sums % 8 == 0 && sums + (wide)s.n_seq * a.parts * 8 <= need, "verdict workspace");
    }
    std::printf("verdicts: %ld taken\n", taken);
    check(taken > n / 20, "verdicts taken");
}
}  // namespace

int main(int argc, char **argv) {
    const long n = argc > 1 ? std::atol(argv[1]) : 1000;
    scans(n);
    rotaries(n / 2);
    accepts(n / 2);
    if (g_mismatches) std::printf("%ld mismatches\n", g_mismatches);
    else std::printf("ALL OK\n");
    return g_mismatches ? 1 : 0;
}

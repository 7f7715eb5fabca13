// Packed prompts of bf16 tokens, in chunks of 64 on the matrix cores.  With G the running sum of
// a chunk's log decays and S the state that enters it, the recurrence is
//
//   out_t = scale * (exp(G_t) S^T q_t + sum_{s <= t} exp(G_t - G_s) (q_t . k_s) v_s)
//   S    <- exp(G_63) S + sum_s k_s (exp(G_63 - G_s) v_s)^T
//
// Every exponent is a difference of sums held in 64 bits (as a pair of floats in LDS), so
// strong decays cost their neighbours nothing.
//
// One workgroup of four wavefronts owns (row, v head, 64 * NC columns of the state), each
// wavefront 16 * NC of them over all dk rows, in 32-bit registers for the whole row.  The
// accumulators of the state's update hold, lane by lane, what the product with q takes as its
// operand (the sum over dk may run in any order, and q is read in the state's), so the state
// never passes through LDS.  32-bit factors enter the products as sums of bf16 parts: two for
// the state, the decayed products and (bf16 states) the decayed values, which leave 2^-17 of a
// factor where bf16 outputs or a bf16 state depend on it (2^-9 of theirs is rounded off; one output
// in a thousand ends on the neighbour of a 32-bit computation's), three (2^-24) for the decayed
// values that build an fp32 state.  q.k of a chunk is shared: each wavefront makes its part of
// the ten 16 x 16 tiles on and below the diagonal and leaves it in LDS in two parts.  k and v
// are stored as they come and read transposed where a product needs their tokens in a lane; rows
// in LDS are padded by 32 bytes (k, v), which both ways of reading take at their full rate (5 cycles an
// instruction, where rows of 256 bytes take 16 to 32), or by 16 (q, the products), which 8-byte reads do.
//
// Measured: 8 prompts of 2048 tokens with 48 heads of 128 x 128 (fp32 state) 211-216 us; one of 16384
// with 32 heads in 16 segments (bf16 state) 194-199 us, 58 of them the segments' own states and 13 their
// sums.  What bounds it: the traffic (565 MB) would take 94 us, and the matrix instructions that the
// parts make of it (a wavefront's 230 of 16 cycles a chunk) about 100; a chunk of two workgroups on a
// compute unit takes 13,000 cycles (12,000 alone), the matrix units busy for 42% of them: one
// wavefront's 560 vector instructions, at 4 to 5 cycles each, and its matrix instructions share the
// issue with the other's, and the clock goes from 2.4 GHz with a few workgroups to 1.9 with all of
// them.  Tried and slower: 8 wavefronts of 16 columns (288 for 238 us at the time), tiles of 64
// columns on a full chip (231 for 213), one XCD's blocks contiguous.  Without effect: priorities, the
// compiler's order inside steps, loads and stores past the caches.  Two parts instead of three for an
// fp32 state's values would save 9%, at 2^-18 of each token's contribution for 2^-24.
#include <type_traits>

#include "la_matrix.h"

namespace laimpl {
namespace {

constexpr int C = 64;              // tokens of a chunk: one per lane of the scan

struct __attribute__((aligned(16))) Decays {   // of one chunk
    float hi[C], lo[C];            // running sums in base 2, as pairs
    float in[C], left[C];          // scale * 2^(sum up to t), 2^(sum behind t)
    float total;                   // 2^(sum of all)
};

constexpr int W = 4;               // wavefronts of a workgroup

template <int KT, int NC>
struct Shared {
    static constexpr int QP = KT * 64 + 16, KP = KT * 64 + 32, VP = W * NC * 32 + 32, PP = C * 2 + 16;
    // the decayed products, in two parts, take q's place once q has been used
    union __attribute__((aligned(16))) { char q[C * QP]; char p[2][C * PP]; };
    __attribute__((aligned(16))) char k[C * KP], v[C * VP], zeros[16];
    Decays d[2];
    int64_t found[3];
};

// KT: dk in blocks of 32; W: wavefronts; NC: column tiles of 16 of each; OUT: outputs are wanted, else
// only what a segment's tokens leave in a state that starts from zeros, and, in the place of a row's
// last segment, the state that the row starts from.
template <int KT, int NC, typename ST, bool OUT>
__global__ __launch_bounds__(64 * W, KT <= 4 || NC == 1 ? 2 : 1) void chunked(const AttnArgs a) {
    constexpr int PARTS = sizeof(ST) == 4 ? 3 : 2;
    constexpr int DT = 2 * KT;                     // row tiles of the state
    using SH = Shared<KT, NC>;
    constexpr int COLS = 16 * W * NC;
    __shared__ SH sh;

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int j = lane & 15, g4 = 4 * (lane >> 4);
    int rest = shared_block(blockIdx.x, a.group * a.tiles, gridDim.x);
    const int tile = uniform(rest % a.tiles);
    rest /= a.tiles;
    const int h = uniform(rest % a.v_heads), id = uniform(rest / a.v_heads);
    const int hq = h / a.group;

    const Segment seg = find_segment<W>(a, id, sh.found);
    if (seg.row < 0) return;                       // same for the workgroup
    const Row row = uniform(row_of(a, seg.row));
    const bool init = !a.has_init || uniform(a.has_init[seg.row]) != 0;
    if (!OUT && seg.last && seg.index == 0) return;
    if (OUT && row.n == 0 && init) return;
    const int first = seg.index * a.seg_len;
    const int n = (row.n - first < a.seg_len ? row.n - first : a.seg_len);

    const int col0 = tile * COLS;                 // of the workgroup
    const int colw = 16 * NC * wave;               // of the wavefront, inside the tile
    // of column x of the wavefront's tile nc: with two tiles, groups of 4 in turn, so that the
    // outputs of a lane are 4 * NC columns side by side
    auto column = [&](int nc, int x) { return NC == 2 ? colw + 8 * (x / 4) + 4 * nc + x % 4 : colw + x; };

    // ---- the state that enters the segment.  Of a row in one segment it is in the pool.  Where a row
    // is cut its last segment writes the pool at a time that the others know nothing of, so the pool is
    // read before that, by the launch without outputs (the last segment's workgroup, which has nothing
    // else to do there), and every segment takes its state from the workspace.
    ST *state = static_cast<ST *>(a.state) + row.slot * a.s_slot + (int64_t)h * a.dk * a.dv;
    auto from_pool = [&](int nc, int d) {          // loads without branches, the first place where there is none
        f32x4 f;
        const int c = col0 + column(nc, j);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 16 * d + g4 + i;
            const bool in = r < a.dk && c < a.dv;
            const float x = load_one(state + (in ? r * a.dv + c : 0));
            f[i] = in ? x : 0.0f;
        }
        return f;
    };
    const int64_t ws_head = ((int64_t)(seg.place + seg.index) * a.v_heads + h) * a.tiles + tile;
    const int64_t ws_step = (int64_t)a.v_heads * a.tiles;          // from segment to segment
    constexpr int64_t WS = (int64_t)64 * W * NC * DT;              // f32x4 of one workgroup
    f32x4 S[NC][DT];
#pragma unroll
    for (int nc = 0; nc < NC; ++nc)
#pragma unroll
        for (int d = 0; d < DT; ++d) S[nc][d] = f32x4{0, 0, 0, 0};
    if constexpr (OUT) {
        const bool cut = seg.index > 0 || !seg.last;
#pragma unroll
        for (int nc = 0; nc < NC; ++nc)
#pragma unroll
            for (int d = 0; d < DT; ++d)
                if (init && !cut) S[nc][d] = from_pool(nc, d);
        if (cut) {                                 // the one before has it; the first one's is in the last one's place
            const int64_t at = seg.index > 0 ? ws_head - ws_step : ws_head + (row.n - 1) / a.seg_len * ws_step;
            const f32x4 *w = static_cast<const f32x4 *>(a.ws) + at * WS + tid;
#pragma unroll
            for (int nc = 0; nc < NC; ++nc)
#pragma unroll
                for (int d = 0; d < DT; ++d) S[nc][d] = w[(nc * DT + d) * 64 * W];
        }
    } else if (seg.last) {
        f32x4 *w = static_cast<f32x4 *>(a.ws) + ws_head * WS + tid;
#pragma unroll
        for (int nc = 0; nc < NC; ++nc)
#pragma unroll
            for (int d = 0; d < DT; ++d) w[(nc * DT + d) * 64 * W] = init ? from_pool(nc, d) : S[nc][d];
        return;
    }

    // ---- staging of a chunk: global memory -> registers -> LDS.  Eight lanes take 128 bytes of a
    // row, so a thread has 8 / W rows (from thread / 8 on, 8 * W apart) and the same channels of
    // each block of 64.  Rows and channels that are not there are read from the last ones that
    // are, and zeroed on the way to LDS.
    constexpr int U = 8 / W, B = KT / 2, VB = W * NC / 4;   // rows; blocks of q and k, of v
    u32x4 rq[U][OUT ? B : 1], rk[U][B], rv[U][VB];
    const char *gq = reinterpret_cast<const char *>(static_cast<const Bf16 *>(a.q) + row.q + hq * a.q_head + first * a.q_tok);
    const char *gk = reinterpret_cast<const char *>(static_cast<const Bf16 *>(a.k) + row.k + hq * a.k_head + first * a.k_tok);
    const char *gv = reinterpret_cast<const char *>(static_cast<const Bf16 *>(a.v) + row.v + h * a.v_head + col0 + first * a.v_tok);
    // bytes from token to token; a chunk's fit 32 bits
    const uint32_t q_step = 2 * (uint32_t)a.q_tok, k_step = 2 * (uint32_t)a.k_tok, v_step = 2 * (uint32_t)a.v_tok;
    const int dv_here = a.dv - col0 < COLS ? a.dv - col0 : COLS;
    const bool whole_tile = a.dk == 32 * KT && dv_here == COLS;
    // Piece `i` (row i / BLOCKS, block i % BLOCKS) of a chunk of which `left` tokens are there.
    auto fetch = [&](const char *from, uint32_t step, int here, auto &to, int i, int left, int place) {
        constexpr int BLOCKS = sizeof(to[0]) / sizeof(u32x4);
        const int u = i / BLOCKS, b = i % BLOCKS, row = (place >> 3) + 8 * W * u, c = 8 * (place & 7) + 64 * b;
        const uint32_t t = row < left ? row : left - 1;
        to[u][b] = *reinterpret_cast<const u32x4 *>(from + (t * step + (c < here ? 2 * c : 0)));
    };
    auto stage = [&](char *lds, int pitch, int here, auto &from, int left, int place) {
        constexpr int BLOCKS = sizeof(from[0]) / sizeof(u32x4);
        const int r0 = place >> 3, c0 = 8 * (place & 7);
        if (!whole_tile || left < C) {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int b = 0; b < BLOCKS; ++b)
                    if (r0 + 8 * W * u >= left || c0 + 64 * b >= here) from[u][b] = u32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int b = 0; b < BLOCKS; ++b)
                *reinterpret_cast<u32x4 *>(lds + (r0 + 8 * W * u) * pitch + 2 * c0 + 128 * b) = from[u][b];
    };
    // One wavefront, lane = token: the chunk's decays, from log decays loaded a chunk earlier.
    const float *gg = a.g ? a.g + row.g + h + (int64_t)first * a.g_tok : nullptr;
    float g_next = 0.0f;
    auto fetch_decays = [&](int t0) {
        // a line for each token: by the wavefront that sums them only
        if (wave == W - 1 && gg) g_next = t0 + lane < n ? gg[(int64_t)(t0 + lane) * a.g_tok] : 0.0f;
    };
    double whole = 0.0;                            // log2 of the segment's decay (that wavefront)
    auto scan = [&](Decays &d) {
        double x = 1.4426950408889634 * (double)finite_decay(g_next);
        x = running_sum(x);
        const double total = __shfl(x, C - 1);
        const float hi = (float)x;
        d.hi[lane] = hi;
        d.lo[lane] = (float)(x - hi);
        d.in[lane] = a.scale * __builtin_amdgcn_exp2f(hi);
        d.left[lane] = __builtin_amdgcn_exp2f((float)(total - x));
        if (lane == 0) d.total = __builtin_amdgcn_exp2f((float)total);
        whole += total;
    };

    if (n > 0) {
        fetch_decays(0);
#pragma unroll
        for (int i = 0; i < KT; ++i) fetch(gk, k_step, a.dk, rk, i, n, tid);
#pragma unroll
        for (int i = 0; i < U * VB; ++i) fetch(gv, v_step, dv_here, rv, i, n, tid);
        if constexpr (OUT)
#pragma unroll
            for (int i = 0; i < KT; ++i) fetch(gq, q_step, a.dk, rq, i, n, tid);
        if (wave == W - 1) scan(sh.d[0]);
        stage(sh.k, SH::KP, a.dk, rk, n, tid);
        stage(sh.v, SH::VP, dv_here, rv, n, tid);
    }
    if (tid < 4) reinterpret_cast<uint32_t *>(sh.zeros)[tid] = 0;
    char *out = OUT ? reinterpret_cast<char *>(static_cast<Bf16 *>(a.out) + row.o + h * a.o_head + col0 + first * a.o_tok)
                    : nullptr;
    const uint32_t o_step = 2 * (uint32_t)a.o_tok;

    // Each step below issues matrix instructions whose operands the step before it made, beside the
    // vector work and the reads that the next step needs: a wavefront issues in order, and there
    // are few of them.  A step is closed to the scheduler, which would otherwise hold more of the
    // next ones' operands than there are registers.
    for (int t0 = 0, turn = 0; t0 < n; t0 += C, turn ^= 1) {
        // The lane's place, hidden at each chunk: what is derived from it is computed again
        // rather than kept in registers, which are short here.
        int place = tid;
        asm volatile("" : "+v"(place));
        const int j = place & 15, g4 = (place & 48) >> 2;
        const u32x2 minus = minus_identity(place & 63);
        // the next chunk (this one again behind the last: what is fetched then is not used)
        const bool more = n - t0 > C;
        const int next = more ? n - t0 - C : n - t0;
        if (more) {
            gk += (int64_t)C * k_step;
            gv += (int64_t)C * v_step;
            if constexpr (OUT) gq += (int64_t)C * q_step;
        }
        if constexpr (OUT) stage(sh.q, SH::QP, a.dk, rq, n - t0, place);
        __syncthreads();                           // the chunk is there
        fetch_decays(t0 + C);
        const Decays &dec = sh.d[turn];
        const float keep = dec.total;

        auto read_v = [&](int nc, int x, int j) {  // this lane's tokens of the wavefront's columns
            const char *vp = sh.v + (32 * x + 2 * g4 + j / 4) * SH::VP + 2 * column(nc, 4 * (j % 4));
            return frag(read_transposed(vp), read_transposed(vp + 4 * SH::VP));
        };
        bf16x8 part[2][NC][PARTS];                 // decayed values, of 32 tokens at a time
        bf16x8 raw;
        float left[8];
        auto read_for_decay = [&](int x, int nc) {
            raw = read_v(nc, x, j);
            load_vec<8>(dec.left + 32 * x + 2 * g4, left);
        };
        auto decay_v = [&](int x, int nc) {
            const u32x4 w = __builtin_bit_cast(u32x4, raw);
            f32x4 f[2];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[i / 2][i % 2 * 2] = bf16_lo(w[i]) * left[2 * i];
                f[i / 2][i % 2 * 2 + 1] = bf16_hi(w[i]) * left[2 * i + 1];
            }
#pragma unroll
            for (int u = 0; u < PARTS; ++u) {
                const u32x2 a = part_of(f[0]), b = part_of(f[1]);
                part[x][nc][u] = frag(a, b);
                if (u + 1 < PARTS) f[0] = less(f[0], a, minus), f[1] = less(f[1], b, minus);
            }
        };

        f32x4 o[OUT ? 4 : 1][NC];                  // outputs, transposed: lane = token, 4 columns
        f32x4 p[OUT ? 3 : 1];                      // products q.k, transposed: lane = token t
        int ti[3], si[3];
        if constexpr (OUT) {
            // ---- q.k: of the ten tiles on and below the diagonal, three wavefronts make three each,
            // (3, 0..2); (2, 0..2); (1, 0..1), (3, 3), and the one that sums the next chunk's
            // decays has (0, 0) (three times, so that all run the same code)
#pragma unroll
            for (int u = 0; u < 3; ++u) {
                const bool third = wave == 2 && u == 2;
                ti[u] = third ? 3 : 3 - wave;
                si[u] = third ? 3 : wave == 3 ? 0 : u;
                p[u] = f32x4{0, 0, 0, 0};
            }
#pragma unroll
            for (int x = 0; x < KT; ++x)
#pragma unroll
                for (int u = 0; u < 3; ++u)
                    p[u] = mma(*reinterpret_cast<const bf16x8 *>(sh.k + (16 * si[u] + j) * SH::KP + 4 * g4 + 64 * x),
                               *reinterpret_cast<const bf16x8 *>(sh.q + (16 * ti[u] + j) * SH::QP + 4 * g4 + 64 * x),
                               p[u]);
            // ---- S^T q
            u32x2 qa[2][4], qb[2][4];
            bf16x8 s[2][NC][2];
            auto read_q = [&](int x) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const char *qp = sh.q + (16 * r + j) * SH::QP + 64 * x + 2 * g4;
                    qa[x & 1][r] = *reinterpret_cast<const u32x2 *>(qp);
                    qb[x & 1][r] = *reinterpret_cast<const u32x2 *>(qp + 32);
                }
            };
            auto split_state = [&](int x) {
#pragma unroll
                for (int nc = 0; nc < NC; ++nc) {
                    const u32x2 a = part_of(S[nc][2 * x]), b = part_of(S[nc][2 * x + 1]);
                    s[x & 1][nc][0] = frag(a, b);
                    s[x & 1][nc][1] = frag(part_of(less(S[nc][2 * x], a, minus)), part_of(less(S[nc][2 * x + 1], b, minus)));
#pragma unroll
                    for (int i = 0; i < 4; ++i) S[nc][2 * x][i] *= keep, S[nc][2 * x + 1][i] *= keep;
                }
            };
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int nc = 0; nc < NC; ++nc) o[r][nc] = f32x4{0, 0, 0, 0};
            read_q(0);
            split_state(0);
#pragma unroll
            for (int x = 0; x < KT; ++x) {
                __builtin_amdgcn_sched_barrier(0);
                fetch(gk, k_step, a.dk, rk, x, next, place);
                if (x + 1 < KT) read_q(x + 1);
                if (x >= KT - NC) {
                    read_for_decay(0, x - KT + NC);
                    decay_v(0, x - KT + NC);
                }
                if (x + 1 < KT) split_state(x + 1);
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
#pragma unroll
                        for (int nc = 0; nc < NC; ++nc)
                            o[r][nc] = mma(s[x & 1][nc][u], frag(qa[x & 1][r], qb[x & 1][r]), o[r][nc]);
            }
            __builtin_amdgcn_sched_barrier(0);
            __syncthreads();                       // q has been used: the products take its place
        } else {
#pragma unroll
            for (int x = 0; x < KT; ++x) fetch(gk, k_step, a.dk, rk, x, next, place);
#pragma unroll
            for (int nc = 0; nc < NC; ++nc) {
                read_for_decay(0, nc);
                decay_v(0, nc);
#pragma unroll
                for (int d = 0; d < DT; ++d)
#pragma unroll
                    for (int i = 0; i < 4; ++i) S[nc][d][i] *= keep;
            }
        }

        auto decay_products = [&](int u) {
            const int t = 16 * ti[u] + j, s = 16 * si[u] + g4;
            const float thi = dec.hi[t], tlo = dec.lo[t];
            const f32x4 shi = *reinterpret_cast<const f32x4 *>(dec.hi + s);
            const f32x4 slo = *reinterpret_cast<const f32x4 *>(dec.lo + s);
            f32x4 f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float e = __builtin_amdgcn_exp2f((thi - shi[i]) + (tlo - slo[i]));
                float x = a.scale * p[u][i] * e;
                asm("" : "+v"(x));                 // a select, not a branch round the products
                f[i] = s + i <= t ? x : 0.0f;
            }
#pragma unroll
            for (int part = 0; part < 2; ++part) {
                const u32x2 w = part_of(f);
                *reinterpret_cast<u32x2 *>(sh.p[part] + t * SH::PP + 2 * s) = w;
                if (part == 0) f = less(f, w, minus);
            }
        };
        // ---- the state's update, two row tiles a step
        bf16x8 kf[2][2];
        auto read_k = [&](int step) {
            const char *kp = sh.k + (32 * (step / KT) + 2 * g4 + j / 4) * SH::KP + 8 * (j % 4) + 64 * (step % KT);
#pragma unroll
            for (int e = 0; e < 2; ++e)
                kf[step & 1][e] = frag(read_transposed(kp + 32 * e), read_transposed(kp + 32 * e + 4 * SH::KP));
        };
        read_k(0);
        read_for_decay(1, 0);
#pragma unroll
        for (int step = 0; step < 2 * KT; ++step) {
            __builtin_amdgcn_sched_barrier(0);
            if (step < U * VB) fetch(gv, v_step, dv_here, rv, step, next, place);
            if constexpr (OUT)
                if (step >= KT) fetch(gq, q_step, a.dk, rq, step - KT, next, place);
            if (step + 1 < 2 * KT) read_k(step + 1);
            if (step < NC) {
                decay_v(1, step);
                if (step + 1 < NC) read_for_decay(1, step + 1);
            }
            if constexpr (OUT) {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (step == (NC + 1 + r < 2 * KT ? NC + 1 + r : 2 * KT - 1)) {
                        const float e = dec.in[16 * r + j];
#pragma unroll
                        for (int nc = 0; nc < NC; ++nc)
#pragma unroll
                            for (int i = 0; i < 4; ++i) o[r][nc][i] *= e;
                    }
                if (step == NC - 1) decay_products(0);
            }
#pragma unroll
            for (int u = 0; u < PARTS; ++u)
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int nc = 0; nc < NC; ++nc)
                        S[nc][2 * (step % KT) + e] = mma(kf[step & 1][e], part[step / KT][nc][u], S[nc][2 * (step % KT) + e]);
            if (step == NC) {
                __builtin_amdgcn_sched_barrier(0);
                if (wave == W - 1) {
                    if (more) scan(sh.d[turn ^ 1]);
                } else if constexpr (OUT) {
                    decay_products(1);
                    decay_products(2);
                }
            }
        }
        __builtin_amdgcn_sched_barrier(0);

        bf16x8 vf[NC][2];
        if constexpr (OUT) {
#pragma unroll
            for (int nc = 0; nc < NC; ++nc)
#pragma unroll
                for (int x = 0; x < 2; ++x) vf[nc][x] = read_v(nc, x, j);
        }
        // A v that is not finite makes its column of the state so (0 * inf is NaN): then such
        // values are taken out of the chunk's own products, for a masked product of 0 must not
        // carry them to the tokens before theirs, and what they reach is marked instead.
        bool any_bad = false;
        uint32_t marks[OUT ? NC : 1] = {};         // bit 4 * r + i: output o[r][nc][i]
        if constexpr (OUT) {
            bool bad = false;
#pragma unroll
            for (int nc = 0; nc < NC; ++nc) bad |= !(__builtin_fabsf(S[nc][0][0]) < INFINITY);
            any_bad = __any(bad);
            if (any_bad) {
                int token = j;                     // hidden: these masks are not worth registers
                asm volatile("" : "+v"(token));
#pragma unroll
                for (int nc = 0; nc < NC; ++nc) {
                    bf16x8 bf[2];
#pragma unroll
                    for (int x = 0; x < 2; ++x) bf[x] = take_bad(vf[nc][x]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        f32x4 reached = {0, 0, 0, 0};
#pragma unroll
                        for (int x = 0; x <= r / 2; ++x) {
                            u32x4 below;           // 1 where token s <= t
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int s = 32 * x + 2 * g4 + 2 * i, t = 16 * r + token;
                                below[i] = (s <= t ? 0x3F80u : 0u) | (s + 1 <= t ? 0x3F800000u : 0u);
                            }
                            reached = mma(bf[x], __builtin_bit_cast(bf16x8, below), reached);
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (reached[i] > 0.0f) marks[nc] |= 1u << (4 * r + i);
                    }
                }
            }
        }
        __syncthreads();                           // the products are there, k and v have been used
        if constexpr (OUT) {
            // ---- the chunk's own tokens
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int r = 2 * x; r < 4; ++r) {
                        const char *pp = sh.p[u] + (16 * r + j) * SH::PP + 64 * x + 4 * g4;
                        // the tile above the diagonal is not stored
                        if (r == 2 * x) pp = g4 >= 8 ? sh.zeros : pp;
                        const bf16x8 pf = *reinterpret_cast<const bf16x8 *>(pp);
#pragma unroll
                        for (int nc = 0; nc < NC; ++nc) o[r][nc] = mma(vf[nc][x], pf, o[r][nc]);
                    }
        }
        stage(sh.k, SH::KP, a.dk, rk, next, place);
        stage(sh.v, SH::VP, dv_here, rv, next, place);
        if constexpr (OUT) {
            if (any_bad)
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int nc = 0; nc < NC; ++nc)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (marks[nc] >> (4 * r + i) & 1) o[r][nc][i] = NAN;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float f[4 * NC];
#pragma unroll
                for (int nc = 0; nc < NC; ++nc)
#pragma unroll
                    for (int i = 0; i < 4; ++i) f[4 * nc + i] = o[r][nc][i];
                const int t = 16 * r + j, c = colw + NC * g4;
                if (t0 + t < n && col0 + c < a.dv)
                    store_vec<4 * NC>(reinterpret_cast<Bf16 *>(out + (t * o_step + 2 * c)), f);
            }
            out += (int64_t)C * o_step;
            __syncthreads();                       // the products have been used: q takes their place
        }
    }

    if constexpr (OUT) {
        if (!seg.last) return;
        auto store = [&](auto whole) {
#pragma unroll
            for (int nc = 0; nc < NC; ++nc)
#pragma unroll
                for (int d = 0; d < DT; ++d)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = 16 * d + g4 + i, c = col0 + column(nc, j);
                        if (decltype(whole)::value || (r < a.dk && c < a.dv)) store_one(state + (r * a.dv + c), S[nc][d][i]);
                    }
        };
        if (whole_tile) store(std::true_type{});
        else store(std::false_type{});
    } else {
        f32x4 *w = static_cast<f32x4 *>(a.ws) + ws_head * WS + tid;
#pragma unroll
        for (int nc = 0; nc < NC; ++nc)
#pragma unroll
            for (int d = 0; d < DT; ++d) w[(nc * DT + d) * 64 * W] = S[nc][d];
        if (tid == 64 * (W - 1)) a.ws_total[ws_head] = __builtin_amdgcn_exp2f((float)whole);
    }
}

// Between the two: each segment's place in the workspace, which holds what its own tokens leave in a
// state of zeros, is left with the state behind it, from the row's first state in the last one's place.
// A workgroup has 256 vectors of one (row, v head, tile), far apart from segment to segment; eight
// segments' are in flight at once.
__global__ __launch_bounds__(64 * W) void combine(const AttnArgs a, const int vectors) {
    const int parts = vectors / (64 * W);
    int rest = blockIdx.x;
    const int part = rest % parts;
    rest /= parts;
    const int ht = rest % (a.v_heads * a.tiles), i = rest / (a.v_heads * a.tiles);
    const int count = uniform(segments_of(a, i));
    if (count < 2) return;                         // same for the workgroup
    const int64_t place = first_place<W>(a, i);
    if (place + count > a.places) return;
    const int64_t step = (int64_t)a.v_heads * a.tiles, at = place * step + ht;
    f32x4 *w = static_cast<f32x4 *>(a.ws) + at * vectors + part * (64 * W) + threadIdx.x;
    const float *total = a.ws_total + at;
    f32x4 S = w[(count - 1) * step * vectors];
    constexpr int AHEAD = 8;
    for (int s0 = 0; s0 < count - 1; s0 += AHEAD) {
        f32x4 x[AHEAD];
        float keep[AHEAD];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            const int s = s0 + u < count - 1 ? s0 + u : count - 2;
            x[u] = w[s * step * vectors];
            keep[u] = total[s * step];
        }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
            if (s0 + u < count - 1) {
#pragma unroll
                for (int e = 0; e < 4; ++e) S[e] = fmaf(S[e], keep[u], x[u][e]);
                w[(s0 + u) * step * vectors] = S;
            }
    }
}

template <int KT, int NC, typename ST>
ChunkedPlan plan() {
    return {(const void *)chunked<KT, NC, ST, true>, (const void *)chunked<KT, NC, ST, false>,
            (const void *)combine, 16 * W * NC, 64 * W, C,
            (int64_t)64 * W * NC * 2 * KT * 16};
}

template <int NC, typename ST>
ChunkedPlan pick_for(int dk) {
    if (dk <= 64) return plan<2, NC, ST>();
    if (dk <= 128) return plan<4, NC, ST>();
    if (dk <= 192) return plan<6, NC, ST>();
    return plan<8, NC, ST>();
}

}  // namespace

ChunkedPlan pick_chunked(int state_bytes, int dk, bool wide) {
    if (state_bytes == 4) return wide ? pick_for<2, float>(dk) : pick_for<1, float>(dk);
    return wide ? pick_for<2, Bf16>(dk) : pick_for<1, Bf16>(dk);
}

}  // namespace laimpl

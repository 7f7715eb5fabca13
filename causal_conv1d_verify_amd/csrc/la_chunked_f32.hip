// Packed prompts of fp32 tokens (and 12 to 32 tokens of each row, as one chunk), in chunks of 32: the
// formulas and the division of la_chunked.hip with fp32 products of 16 x 16 x 4, so no factor is taken
// apart.  A wavefront owns 16 of the state's columns over all dk rows in registers, and its four rows
// of a register group are four places of the product with q, read 16 bytes a lane.  v goes from memory
// to the lanes that use it.  Measured: 5 prompts of up to 777 tokens, 6 heads of 96 x 72, in segments
// of 128: 36 us (12 + 5 + 21 in its three kernels, traced).  What bounds it there is the length of a
// chain, four chunks of some 5 us in few workgroups: the matrix units are busy for a third of a
// wavefront's time, and in the tile past column 64 one wavefront of four has columns (8).  With the
// card full the fp32 matrix rate (a sixteenth of bf16's) would be the bound; the state's two products
// take the most of it.
#include "la_matrix.h"

namespace laimpl {
namespace {

constexpr int C = 32, W = 4;       // tokens of a chunk, wavefronts

__device__ __forceinline__ f32x4 mma(float a, float b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

struct __attribute__((aligned(16))) Decays32 {
    float hi[C], lo[C], in[C], left[C], total;
};

template <int DT>
struct Shared {
    static constexpr int QP = DT * 16 + 4, PP = C + 4;             // floats of a row
    __attribute__((aligned(16))) float q[C * QP], k[C * QP], p[C * PP];
    Decays32 d[2];
    int64_t found[3];
};

// DT: row tiles of 16; OUT as in la_chunked.hip.
template <int DT, bool OUT>
__global__ __launch_bounds__(64 * W, 2) void chunked_f32(const AttnArgs a) {
    using SH = Shared<DT>;
    __shared__ SH sh;
    constexpr int COLS = 16 * W;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int j = lane & 15, g4 = 4 * (lane >> 4);
    int rest = blockIdx.x;
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
    const int n = row.n - first < a.seg_len ? row.n - first : a.seg_len;

    // ---- the state that enters the segment, as in la_chunked.hip
    const int col = tile * COLS + 16 * wave + j;
    const bool in_cols = col < a.dv;
    float *state = static_cast<float *>(a.state) + row.slot * a.s_slot + (int64_t)h * a.dk * a.dv + col;
    auto from_pool = [&](int d) {
        f32x4 f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool in = in_cols && 16 * d + g4 + i < a.dk;
            const float x = in_cols ? state[in ? (16 * d + g4 + i) * a.dv : 0] : 0.0f;
            f[i] = in ? x : 0.0f;
        }
        return f;
    };
    const int64_t ws_head = ((int64_t)(seg.place + seg.index) * a.v_heads + h) * a.tiles + tile;
    const int64_t ws_step = (int64_t)a.v_heads * a.tiles;
    constexpr int64_t WS = (int64_t)64 * W * DT;
    f32x4 S[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d) S[d] = f32x4{0, 0, 0, 0};
    if constexpr (OUT) {
        const bool cut = seg.index > 0 || !seg.last;
#pragma unroll
        for (int d = 0; d < DT; ++d)
            if (init && !cut) S[d] = from_pool(d);
        if (cut) {
            const int64_t at = seg.index > 0 ? ws_head - ws_step : ws_head + (row.n - 1) / a.seg_len * ws_step;
            const f32x4 *w = static_cast<const f32x4 *>(a.ws) + at * WS + tid;
#pragma unroll
            for (int d = 0; d < DT; ++d) S[d] = w[d * 64 * W];
        }
    } else if (seg.last) {
        f32x4 *w = static_cast<f32x4 *>(a.ws) + ws_head * WS + tid;
#pragma unroll
        for (int d = 0; d < DT; ++d) w[d * 64 * W] = init ? from_pool(d) : S[d];
        return;
    }

    // ---- a chunk's q and k: 8 threads a row, 32 floats apart by block
    const char *gk = reinterpret_cast<const char *>(static_cast<const float *>(a.k) + row.k + hq * a.k_head + first * a.k_tok);
    const char *gv = reinterpret_cast<const char *>(static_cast<const float *>(a.v) + row.v + h * a.v_head + first * a.v_tok);
    // (a commit has no q and no outputs: k stands in, and nothing of what it makes is stored)
    const char *gq = OUT && a.q ? reinterpret_cast<const char *>(static_cast<const float *>(a.q) + row.q + hq * a.q_head + first * a.q_tok)
                                : gk;
    const uint32_t k_step = 4 * (uint32_t)a.k_tok, v_step = 4 * (uint32_t)a.v_tok, q_step = a.q ? 4 * (uint32_t)a.q_tok : k_step;
    constexpr int B = DT / 2;
    const int r0 = tid >> 3, f0 = 4 * (tid & 7);
    f32x4 rq[OUT ? B : 1], rk[B];
    float rv[8];                                   // tokens 16 x + g4 + i of the lane's column
    auto fetch = [&](int left) {
        const uint32_t t = r0 < left ? r0 : left - 1;
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            const int at = 16 * (x / 4) + g4 + x % 4;
            const uint32_t tv = at < left ? at : left - 1;
            rv[x] = *reinterpret_cast<const float *>(gv + (tv * v_step + (in_cols ? 4 * col : 0)));
        }
        gv += (int64_t)C * v_step;
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const uint32_t c = f0 + 32 * b < a.dk ? 4 * (f0 + 32 * b) : 0;
            rk[b] = *reinterpret_cast<const f32x4 *>(gk + (t * k_step + c));
            if constexpr (OUT) rq[b] = *reinterpret_cast<const f32x4 *>(gq + (t * q_step + c));
        }
        gk += (int64_t)C * k_step;
        if constexpr (OUT) gq += (int64_t)C * q_step;
    };
    auto stage = [&](int left) {
        const bool there = r0 < left;
        const f32x4 zero = {0, 0, 0, 0};
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const bool in = there && f0 + 32 * b < a.dk;
            *reinterpret_cast<f32x4 *>(sh.k + r0 * SH::QP + f0 + 32 * b) = in ? rk[b] : zero;
            if constexpr (OUT) *reinterpret_cast<f32x4 *>(sh.q + r0 * SH::QP + f0 + 32 * b) = in ? rq[b] : zero;
        }
    };
    const float *gg = a.g ? a.g + row.g + h + (int64_t)first * a.g_tok : nullptr;
    float g_next = 0.0f;
    auto fetch_decays = [&](int t0) { g_next = gg && wave == W - 1 && lane < C && t0 + lane < n ? gg[(int64_t)(t0 + lane) * a.g_tok] : 0.0f; };
    double whole = 0.0;
    auto scan = [&](Decays32 &d) {
        const double x = running_sum(1.4426950408889634 * (double)finite_decay(g_next));
        const double total = __shfl(x, C - 1);
        if (lane < C) {
            const float hi = (float)x;
            d.hi[lane] = hi;
            d.lo[lane] = (float)(x - hi);
            d.in[lane] = a.scale * __builtin_amdgcn_exp2f(hi);
            d.left[lane] = __builtin_amdgcn_exp2f((float)(total - x));
        }
        if (lane == 0) d.total = __builtin_amdgcn_exp2f((float)total);
        whole += total;
    };
    if (n > 0) {
        fetch_decays(0);
        fetch(n);
        if (wave == W - 1) scan(sh.d[0]);
    }
    char *out = OUT ? reinterpret_cast<char *>(static_cast<float *>(a.out) + row.o + h * a.o_head + first * a.o_tok) : nullptr;
    const uint32_t o_step = 4 * (uint32_t)a.o_tok;

    for (int t0 = 0, turn = 0; t0 < n; t0 += C, turn ^= 1) {
        stage(n - t0);
        float v[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) v[x] = in_cols && t0 + 16 * (x / 4) + g4 + x % 4 < n ? rv[x] : 0.0f;
        __syncthreads();
        const Decays32 &dec = sh.d[turn];
        const float keep = dec.total;
        if (n - t0 > C) {
            fetch_decays(t0 + C);
            fetch(n - t0 - C);
        }
        f32x4 o[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
        if constexpr (OUT) {
            // q.k, decayed: tiles (0, 0), (1, 0), (1, 1) by three wavefronts, the next chunk's decays by
            // the fourth
            if (wave < 3) {
                const int ti = wave ? 1 : 0, si = wave == 2 ? 1 : 0;
                f32x4 p = {0, 0, 0, 0};
                const float *kp = sh.k + (16 * si + j) * SH::QP + g4, *qp = sh.q + (16 * ti + j) * SH::QP + g4;
#pragma unroll
                for (int d = 0; d < DT; ++d) {
                    const f32x4 x = *reinterpret_cast<const f32x4 *>(kp + 16 * d), y = *reinterpret_cast<const f32x4 *>(qp + 16 * d);
#pragma unroll
                    for (int i = 0; i < 4; ++i) p = mma(x[i], y[i], p);
                }
                const int t = 16 * ti + j, s = 16 * si + g4;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float e = __builtin_amdgcn_exp2f((dec.hi[t] - dec.hi[s + i]) + (dec.lo[t] - dec.lo[s + i]));
                    float x = a.scale * p[i] * e;
                    asm("" : "+v"(x));             // a select, not a branch round the products
                    p[i] = s + i <= t ? x : 0.0f;
                }
                *reinterpret_cast<f32x4 *>(sh.p + t * SH::PP + s) = p;
            } else if (n - t0 > C) {
                scan(sh.d[turn ^ 1]);
            }
            // S^T q, transposed outputs: lane = token, registers = 4 columns
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const f32x4 q = *reinterpret_cast<const f32x4 *>(sh.q + (16 * r + j) * SH::QP + 16 * d + g4);
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[r] = mma(S[d][i], q[i], o[r]);
                }
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[r][i] *= dec.in[16 * r + j];
        } else if (wave == W - 1 && n - t0 > C) {
            scan(sh.d[turn ^ 1]);
        }
        // ---- the state's update
        float w[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) w[x] = v[x] * dec.left[16 * (x / 4) + g4 + x % 4];
#pragma unroll
        for (int d = 0; d < DT; ++d) {
#pragma unroll
            for (int i = 0; i < 4; ++i) S[d][i] *= keep;
#pragma unroll
            for (int x = 0; x < 8; ++x)
                S[d] = mma(sh.k[(16 * (x / 4) + g4 + x % 4) * SH::QP + 16 * d + j], w[x], S[d]);
        }
        if constexpr (OUT) {
            // ---- the chunk's own tokens; values that are not finite as in la_chunked.hip
            float bad[8];
            bool some = false;
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const bool is = !(__builtin_fabsf(v[x]) < INFINITY);
                bad[x] = is ? 1.0f : 0.0f;
                some |= is;
                v[x] = is ? 0.0f : v[x];
            }
            const bool any_bad = __any(some);
            __syncthreads();                       // the products are there
#pragma unroll
            for (int r = 0; r < 2; ++r) {
#pragma unroll
                for (int x = 0; x <= r; ++x) {
                    const f32x4 p = *reinterpret_cast<const f32x4 *>(sh.p + (16 * r + j) * SH::PP + 16 * x + g4);
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[r] = mma(v[4 * x + i], p[i], o[r]);
                }
                if (any_bad) {
                    f32x4 reached = {0, 0, 0, 0};
#pragma unroll
                    for (int x = 0; x <= r; ++x)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            reached = mma(bad[4 * x + i], 16 * x + g4 + i <= 16 * r + j ? 1.0f : 0.0f, reached);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (reached[i] > 0.0f) o[r][i] = NAN;
                }
                const int t = 16 * r + j, c = tile * COLS + 16 * wave + g4;
                if (a.out && t0 + t < n && c < a.dv) *reinterpret_cast<f32x4 *>(out + (t * o_step + 4 * c)) = o[r];
            }
            out += (int64_t)C * o_step;
        }
        __syncthreads();                           // every wavefront is done with the tiles
    }

    if constexpr (OUT) {
        if (!seg.last || !a.write_state) return;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (in_cols && 16 * d + g4 + i < a.dk) state[(16 * d + g4 + i) * a.dv] = S[d][i];
    } else {
        f32x4 *w = static_cast<f32x4 *>(a.ws) + ws_head * WS + tid;
#pragma unroll
        for (int d = 0; d < DT; ++d) w[d * 64 * W] = S[d];
        if (tid == 64 * (W - 1)) a.ws_total[ws_head] = __builtin_amdgcn_exp2f((float)whole);
    }
}

template <int DT>
ChunkedPlan plan() {
    return {(const void *)chunked_f32<DT, true>, (const void *)chunked_f32<DT, false>, nullptr, 16 * W, 64 * W, C,
            (int64_t)64 * W * DT * 16};
}

}  // namespace

ChunkedPlan pick_chunked_f32(int dk) {
    ChunkedPlan p = dk <= 64 ? plan<4>() : dk <= 96 ? plan<6>() : dk <= 128 ? plan<8>() : dk <= 192 ? plan<12>() : plan<16>();
    p.combine = pick_chunked(4, dk, false).combine;
    return p;
}

}  // namespace laimpl

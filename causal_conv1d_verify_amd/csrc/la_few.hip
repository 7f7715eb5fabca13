// Up to 32 tokens of each row on the matrix cores, in one pass over the state:
//
//   out_t = scale * (exp(G_t) S^T q_t + sum_{s <= t} exp(G_t - G_s) (q_t . k_s) v_s)
//   S    <- exp(G) S + sum_s k_s (exp(G - G_s) v_s)^T        G_t the running sum of log decays
//
// which is bound by the state, read once and (but for verify) written once.  A workgroup of four
// wavefronts owns (row, v head, 128 of the state's columns), a wavefront half of the columns and
// half of the rows: a lane has four columns side by side of each of 8 * RB rows, so every load of
// the state is 16 bytes (8 of bf16) a lane, all are in flight at once, and the registers they come
// into are the accumulators of the update and the operands of the product with q.  The tokens are
// few enough to come straight from memory in the operands' order; only the update's k goes through
// LDS, to be read transposed.  Outputs are linear in the rows' share of both sums, so the two halves
// of the rows meet once, in LDS.  bf16 parts of 32-bit factors are as for prompts.
//
// Measured: one token for 256 rows x 32 heads of 128 x 128 (fp32 state, a tenth of the rows padded)
// 166 us, 6.0 TB/s; eight for 128 rows x 48 heads, verify and commit, 184-186 us, 6.2 TB/s.  States
// past the Infinity Cache's reach go past it (184 and 209 us through it).
#include <type_traits>

#include "la_matrix.h"

namespace laimpl {
namespace {

// RB: blocks of 32 rows of a wavefront; TT: tiles of 16 tokens; OUT: outputs are wanted; WRITE: the
// state is written.
template <int RB, int TT, typename ST, bool OUT, bool WRITE>
__global__ __launch_bounds__(256) void few(const AttnArgs a) {
    constexpr int NC = 4;                          // column tiles of a wavefront: column 4 * j + nc
    constexpr int PARTS = sizeof(ST) == 4 ? 3 : 2; // of the decayed values
    constexpr int SPARTS = sizeof(ST) == 4 ? 2 : 1;
    constexpr int KP = 128 * RB + 32;              // bytes of a token's k in LDS
    __shared__ __attribute__((aligned(16))) char sk[WRITE ? 16 * TT * KP : 16];
    __shared__ struct __attribute__((aligned(16))) {       // each wavefront's own: it waits for no other's
        float hi[4][32], lo[4][32], in[4][32], left[4][32];
    } dec;
    __shared__ f32x4 half[OUT ? 2 * TT * NC * kWave : 1];

    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int j = lane & 15, g4 = 4 * (lane >> 4);
    int rest = blockIdx.x;
    const int tile = rest % a.tiles;
    rest /= a.tiles;
    const int h = rest % a.v_heads, i = rest / a.v_heads;
    const Row row = uniform(row_of(a, i));
    const int n = row.n;
    if (n <= 0) return;                            // same for the workgroup; no tokens: no change
    const int hq = h / a.group;
    const int r0 = 32 * RB * (wave >> 1);          // of the wavefront
    const int c0 = 128 * tile + 64 * (wave & 1) + 4 * j;   // of the lane
    const bool in_cols = c0 < a.dv;

    // ---- the state: row r0 + 32 b + 16 e + g4 + u, columns c0 + nc
    f32x4 S[RB][2][NC];
    auto rows_of_state = [&](auto each) {
#pragma unroll
        for (int b = 0; b < RB; ++b)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int r = r0 + 32 * b + 16 * e + g4 + u;
                    each(b, e, u, r, in_cols && r < a.dk);
                }
    };
    ST *state = static_cast<ST *>(a.state) + row.slot * a.s_slot + (int64_t)h * a.dk * a.dv;
    auto load = [&](auto stream) {
        rows_of_state([&](int b, int e, int u, int r, bool in) {
            float f[4] = {};
            if (decltype(stream)::value ? in : true) load_vec<4, decltype(stream)::value>(state + (in ? r * a.dv + c0 : 0), f);
#pragma unroll
            for (int nc = 0; nc < NC; ++nc) S[b][e][nc][u] = in ? f[nc] : 0.0f;
        });
    };
    // Where states are streamed they are the call's work and go first; where they are few the tokens'
    // own products are made while the state is on its way (8 rows x 17 tokens, 32 heads, verify and
    // commit: 12.5 us for 17.8).
    if (a.streaming) load(std::true_type{});

    // ---- the tokens, at the places 4g + u and 16 + 4g + u of a sum over 32.  What is not there is read
    // from the first place that is, without a branch, and zeroed.
    const Bf16 *gk = static_cast<const Bf16 *>(a.k) + row.k + hq * a.k_head;
    const u32x2 none = {0, 0};
    bf16x8 qf[OUT ? TT : 1][RB], kf[OUT ? TT : 1][RB];
    if constexpr (OUT) {
        const Bf16 *gq = static_cast<const Bf16 *>(a.q) + row.q + hq * a.q_head;
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int b = 0; b < RB; ++b) {
                u32x2 q[2], k[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int at = r0 + g4 + 32 * b + 16 * e;
                    const bool in = 16 * t + j < n && at < a.dk;
                    q[e] = *reinterpret_cast<const u32x2 *>(gq + (in ? (16 * t + j) * a.q_tok + at : 0));
                    k[e] = *reinterpret_cast<const u32x2 *>(gk + (in ? (16 * t + j) * a.k_tok + at : 0));
                    q[e] = in ? q[e] : none;
                    k[e] = in ? k[e] : none;
                }
                qf[t][b] = frag(q[0], q[1]);
                kf[t][b] = frag(k[0], k[1]);
            }
    }
    const Bf16 *gv = static_cast<const Bf16 *>(a.v) + row.v + h * a.v_head;
    u32x2 v[2][4];                                 // tokens 16 t + g4 + u, columns c0 to c0 + 3
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            v[t][u] = none;
            if (t >= TT) continue;
            const bool in = in_cols && 16 * t + g4 + u < n;
            v[t][u] = *reinterpret_cast<const u32x2 *>(gv + (in ? (16 * t + g4 + u) * a.v_tok + c0 : 0));
            v[t][u] = in ? v[t][u] : none;
        }
    const float g = a.g && lane < n ? a.g[row.g + h + lane * a.g_tok] : 0.0f;
    constexpr int PIECES = WRITE ? (16 * TT * 8 * RB + 255) / 256 : 0;   // of k for LDS, of a thread
    u32x4 rk[WRITE ? PIECES : 1];
#pragma unroll
    for (int p = 0; p < PIECES; ++p) {
        const int at = tid + 256 * p, t = at / (8 * RB), c = 8 * (at % (8 * RB));
        const bool in = t < n && c < a.dk;
        const u32x4 zero = {0, 0, 0, 0};
        rk[p] = *reinterpret_cast<const u32x4 *>(gk + (in ? t * a.k_tok + c : 0));
        rk[p] = in ? rk[p] : zero;
    }

    if (!a.streaming) load(std::false_type{});

    if constexpr (WRITE) {
#pragma unroll
        for (int p = 0; p < PIECES; ++p) {
            const int at = tid + 256 * p, t = at / (8 * RB), c = 8 * (at % (8 * RB));
            if (at < 16 * TT * 8 * RB) *reinterpret_cast<u32x4 *>(sk + t * KP + 2 * c) = rk[p];
        }
        __syncthreads();
    }
    bf16x8 vf[NC];                                 // the same, a column's tokens together
#pragma unroll
    for (int nc = 0; nc < NC; ++nc) {
        const uint32_t pick = nc % 2 ? 0x07060302u : 0x05040100u;
        u32x4 w;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int u = 0; u < 2; ++u)
                w[2 * t + u] = __builtin_amdgcn_perm(v[t][2 * u + 1][nc / 2], v[t][2 * u][nc / 2], pick);
        vf[nc] = __builtin_bit_cast(bf16x8, w);
    }

    // ---- the decays, lane = token
    double sum = running_sum(1.4426950408889634 * (double)finite_decay(g));
    const double total = __shfl(sum, kWave - 1);
    if (lane < 32) {
        const float hi = (float)sum;
        dec.hi[wave][lane] = hi;
        dec.lo[wave][lane] = (float)(sum - hi);
        dec.in[wave][lane] = a.scale * __builtin_amdgcn_exp2f(hi);
        dec.left[wave][lane] = __builtin_amdgcn_exp2f((float)(total - sum));
    }

    f32x4 o[OUT ? TT : 1][NC];
    if constexpr (OUT) {
        // ---- the tokens' own products.  Values that are not finite are taken out: a masked product
        // of 0 must not carry them to the tokens before theirs; what they reach is marked.
        bf16x8 clean[NC], bad[NC];
        uint32_t some = 0;
#pragma unroll
        for (int nc = 0; nc < NC; ++nc) {
            clean[nc] = vf[nc];
            bad[nc] = take_bad(clean[nc]);
            const u32x4 w = __builtin_bit_cast(u32x4, bad[nc]);
            some |= w[0] | w[1] | w[2] | w[3];
        }
        const bool any_bad = __any(some != 0);
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            const float thi = dec.hi[wave][16 * t + j], tlo = dec.lo[wave][16 * t + j];
#pragma unroll
            for (int nc = 0; nc < NC; ++nc) o[t][nc] = f32x4{0, 0, 0, 0};
            float f[8] = {};
            u32x4 below = {0, 0, 0, 0};            // 1 where token s <= t
#pragma unroll
            for (int s = 0; s <= t; ++s) {
                f32x4 p = {0, 0, 0, 0};            // transposed: lane = t
#pragma unroll
                for (int b = 0; b < RB; ++b) p = mma(kf[s][b], qf[t][b], p);
                const f32x4 shi = *reinterpret_cast<const f32x4 *>(&dec.hi[wave][16 * s + g4]);
                const f32x4 slo = *reinterpret_cast<const f32x4 *>(&dec.lo[wave][16 * s + g4]);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int at = 16 * s + g4 + u;
                    const float e = __builtin_amdgcn_exp2f((thi - shi[u]) + (tlo - slo[u]));
                    float x = a.scale * p[u] * e;
                    asm("" : "+v"(x));             // a select, not a branch round the products
                    const bool on = at <= 16 * t + j;
                    f[4 * s + u] = on ? x : 0.0f;
                    below[2 * s + u / 2] |= on ? 0x3F80u << 16 * (u % 2) : 0u;
                }
            }
#pragma unroll
            for (int part = 0; part < 2; ++part) {
                const bf16x8 p = take_part(f);
#pragma unroll
                for (int nc = 0; nc < NC; ++nc) o[t][nc] = mma(clean[nc], p, o[t][nc]);
            }
            if (any_bad)
#pragma unroll
                for (int nc = 0; nc < NC; ++nc) {
                    const f32x4 reached = mma(bad[nc], __builtin_bit_cast(bf16x8, below), f32x4{0, 0, 0, 0});
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        if (reached[u] > 0.0f) o[t][nc][u] = NAN;
                }
        }
        // ---- S^T q, transposed: lane = token
        f32x4 old[TT][NC];
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int nc = 0; nc < NC; ++nc) old[t][nc] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int b = 0; b < RB; ++b)
#pragma unroll
            for (int nc = 0; nc < NC; ++nc) {
                float f[8];
#pragma unroll
                for (int u = 0; u < 4; ++u) f[u] = S[b][0][nc][u], f[4 + u] = S[b][1][nc][u];
#pragma unroll
                for (int part = 0; part < SPARTS; ++part) {
                    const bf16x8 s = take_part(f);
#pragma unroll
                    for (int t = 0; t < TT; ++t) old[t][nc] = mma(s, qf[t][b], old[t][nc]);
                }
            }
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            const float in = dec.in[wave][16 * t + j];
#pragma unroll
            for (int nc = 0; nc < NC; ++nc)
#pragma unroll
                for (int u = 0; u < 4; ++u) o[t][nc][u] = fmaf(old[t][nc][u], in, o[t][nc][u]);
        }
        if (wave >= 2)
#pragma unroll
            for (int t = 0; t < TT; ++t)
#pragma unroll
                for (int nc = 0; nc < NC; ++nc) half[((wave - 2) * TT * NC + t * NC + nc) * kWave + lane] = o[t][nc];
        __syncthreads();
        if (wave < 2) {
            // a lane has the columns 4 * (g4 + u) + nc of the wavefront's 64
            const int c = 128 * tile + 64 * wave + 4 * g4;
            Bf16 *out = static_cast<Bf16 *>(a.out) + row.o + h * a.o_head + c;
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                float f[16];
#pragma unroll
                for (int nc = 0; nc < NC; ++nc) {
                    const f32x4 x = half[(wave * TT * NC + t * NC + nc) * kWave + lane];
#pragma unroll
                    for (int u = 0; u < 4; ++u) f[4 * u + nc] = o[t][nc][u] + x[u];
                }
                if (16 * t + j >= n) continue;
                Bf16 *p = out + (16 * t + j) * a.o_tok;
                const float lower[8] = {f[0], f[1], f[2], f[3], f[4], f[5], f[6], f[7]};
                const float upper[8] = {f[8], f[9], f[10], f[11], f[12], f[13], f[14], f[15]};
                if (c < a.dv) store_vec<8>(p, lower);
                if (c + 8 < a.dv) store_vec<8>(p + 8, upper);
            }
        }
    }

    if constexpr (WRITE) {
        const float keep = __builtin_amdgcn_exp2f((float)total);
        float by[8];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int u = 0; u < 4; ++u) by[4 * t + u] = t < TT ? dec.left[wave][16 * t + g4 + u] : 0.0f;
        bf16x8 part[NC][PARTS];
#pragma unroll
        for (int nc = 0; nc < NC; ++nc) {
            const u32x4 w = __builtin_bit_cast(u32x4, vf[nc]);
            float f[8];
#pragma unroll
            for (int u = 0; u < 4; ++u) f[2 * u] = bf16_lo(w[u]) * by[2 * u], f[2 * u + 1] = bf16_hi(w[u]) * by[2 * u + 1];
#pragma unroll
            for (int p = 0; p < PARTS; ++p) part[nc][p] = take_part(f);
        }
#pragma unroll
        for (int b = 0; b < RB; ++b)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const char *kp = sk + (g4 + j / 4) * KP + 2 * (r0 + 32 * b + 16 * e + 4 * (j % 4));
                const bf16x8 k = frag(read_transposed(kp), TT == 2 ? read_transposed(kp + (TT - 1) * 16 * KP) : none);
#pragma unroll
                for (int nc = 0; nc < NC; ++nc)
#pragma unroll
                    for (int u = 0; u < 4; ++u) S[b][e][nc][u] *= keep;
#pragma unroll
                for (int p = 0; p < PARTS; ++p)
#pragma unroll
                    for (int nc = 0; nc < NC; ++nc) S[b][e][nc] = mma(k, part[nc][p], S[b][e][nc]);
            }
        auto store = [&](auto stream) {
            rows_of_state([&](int b, int e, int u, int r, bool in) {
                const float f[4] = {S[b][e][0][u], S[b][e][1][u], S[b][e][2][u], S[b][e][3][u]};
                if (in) store_vec<4, decltype(stream)::value>(state + (r * a.dv + c0), f);
            });
        };
        if (a.streaming) store(std::true_type{});
        else store(std::false_type{});
    }
}

template <int RB, int TT, typename ST>
const void *pick(bool out, bool write) {
    return !out ? (const void *)few<RB, TT, ST, false, true> : write ? (const void *)few<RB, TT, ST, true, true>
                                                                     : (const void *)few<RB, TT, ST, true, false>;
}

template <typename ST>
const void *pick(int dk, int T, bool out, bool write) {
    if (dk <= 64) return T <= 16 ? pick<1, 1, ST>(out, write) : pick<1, 2, ST>(out, write);
    if (dk <= 128) return T <= 16 ? pick<2, 1, ST>(out, write) : pick<2, 2, ST>(out, write);
    return T <= 16 ? pick<4, 1, ST>(out, write) : pick<4, 2, ST>(out, write);
}

}  // namespace

const void *pick_few(int state_bytes, int dk, int T, bool out, bool write) {
    return state_bytes == 4 ? pick<float>(dk, T, out, write) : pick<Bf16>(dk, T, out, write);
}

}  // namespace laimpl

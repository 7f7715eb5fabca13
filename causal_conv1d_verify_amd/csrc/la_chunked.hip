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
// the state, the decayed products and (bf16 states) the decayed values, three for the decayed
// values that build an fp32 state.  q.k of a chunk is shared: each wavefront makes its part of
// the ten 16 x 16 tiles on and below the diagonal and leaves it in LDS in two parts.  k and v
// are stored as they come and read transposed where a product needs their tokens in a lane.
#include <type_traits>

#include "la_device.h"

namespace laimpl {
namespace {

constexpr int C = 64;              // tokens of a chunk: one per lane of the scan

typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// Row 4g + i (i = 0..3) of column j for lane (g, j), from 4 rows of 16 columns for each g: lane
// (g, j) points at row 4g + j / 4, columns 4 * (j % 4) to + 3.
__device__ __forceinline__ u32x2 read_transposed(const char *p) {
    const s16x4 r = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
    return __builtin_bit_cast(u32x2, r);
}

__device__ __forceinline__ bf16x8 frag(u32x2 a, u32x2 b) {
    const u32x4 w = {a[0], a[1], b[0], b[1]};
    return __builtin_bit_cast(bf16x8, w);
}

__device__ __forceinline__ f32x4 mma(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// x less the low (high) bf16 of w, exact: one dot product with (-1, 0) or (0, -1), which are kept
// in scalar registers (as an inline constant of a packed operand they would mean something else).
__device__ __forceinline__ float less_lo(float x, uint32_t w) {
    uint32_t m = 0xBF80u;
    asm("" : "+s"(m));
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, w), __builtin_bit_cast(bf16x2, m), x, false);
}
__device__ __forceinline__ float less_hi(float x, uint32_t w) {
    uint32_t m = 0xBF800000u;
    asm("" : "+s"(m));
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, w), __builtin_bit_cast(bf16x2, m), x, false);
}

// The next bf16 part of eight values, taken off them.
__device__ __forceinline__ bf16x8 take_part(float (&x)[8]) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
        x[2 * i] = less_lo(x[2 * i], w[i]);
        x[2 * i + 1] = less_hi(x[2 * i + 1], w[i]);
    }
    return __builtin_bit_cast(bf16x8, w);
}

// Non-finite elements of eight bf16 values: zeroed in v, 1 in the returned indicator.
__device__ __forceinline__ bf16x8 take_bad(bf16x8 &v) {
    u32x4 w = __builtin_bit_cast(u32x4, v), bad;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = (w[i] & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u;
        const uint32_t hi = (w[i] & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u;
        bad[i] = (lo & 0x3F80u) | (hi & 0x3F800000u);
        w[i] &= ~(lo | hi);
    }
    v = __builtin_bit_cast(bf16x8, w);
    return __builtin_bit_cast(bf16x8, bad);
}

struct __attribute__((aligned(16))) Decays {   // of one chunk
    float hi[C], lo[C];            // running sums in base 2, as pairs
    float in[C], left[C];          // scale * 2^(sum up to t), 2^(sum behind t)
    float total;                   // 2^(sum of all)
};

template <int KT, int NC>
struct Shared {
    static constexpr int QP = KT * 64 + 16, KP = KT * 64 + 32, VP = NC * 128 + 32, PP = C * 2 + 16;
    __attribute__((aligned(16))) char q[C * QP], k[C * KP], v[C * VP], p[2][C * PP];
    Decays d[2];
    int64_t found[2];
};

// KT: dk in blocks of 32; NC: column tiles of 16 per wavefront; OUT: outputs are wanted, else
// only what a segment's tokens leave in a state that starts from zeros.
template <int KT, int NC, typename ST, bool OUT>
__global__ __launch_bounds__(256, KT <= 4 ? 2 : 1) void chunked(const AttnArgs a) {
    constexpr int PARTS = sizeof(ST) == 4 ? 3 : 2;
    constexpr int DT = 2 * KT;                     // row tiles of the state
    using SH = Shared<KT, NC>;
    __shared__ SH sh;

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int j = lane & 15, g4 = 4 * (lane >> 4);
    int rest = blockIdx.x;
    const int tile = rest % a.tiles;
    rest /= a.tiles;
    const int h = rest % a.v_heads, id = rest / a.v_heads;
    const int hq = h / a.group;

    const Segment seg = find_segment(a, id, sh.found);
    if (seg.row < 0) return;                       // same for the workgroup
    const Row row = row_of(a, seg.row);
    const bool init = !a.has_init || a.has_init[seg.row] != 0;
    if (!OUT && seg.last) return;
    if (OUT && row.n == 0 && init) return;
    const int first = seg.index * a.seg_len;
    const int n = (row.n - first < a.seg_len ? row.n - first : a.seg_len);

    const int col0 = tile * 64 * NC;               // of the workgroup
    const int colw = 16 * NC * wave;               // of the wavefront, inside the tile
    auto column = [&](int nc) {                    // of lane j's column of tile nc, inside the tile
        return NC == 2 ? colw + 8 * (j / 4) + 4 * nc + j % 4 : colw + j;
    };

    // ---- the state that enters the segment
    f32x4 S[NC][DT];
    ST *state = static_cast<ST *>(a.state) + row.slot * a.s_slot + (int64_t)h * a.dk * a.dv;
#pragma unroll
    for (int nc = 0; nc < NC; ++nc)
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            S[nc][d] = f32x4{0, 0, 0, 0};
            if (!OUT || !init) continue;
            const int c = col0 + column(nc);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 16 * d + g4 + i;
                if (r < a.dk && c < a.dv) S[nc][d][i] = load_one(state + (int64_t)r * a.dv + c);
            }
        }
    const int64_t ws_head = ((int64_t)id * a.v_heads + h) * a.tiles + tile;
    const int64_t ws_step = (int64_t)a.v_heads * a.tiles;          // from segment to segment
    constexpr int64_t WS = (int64_t)256 * NC * DT;                 // f32x4 of one workgroup
    if constexpr (OUT) {
        for (int s = seg.index; s > 0; --s) {
            const int64_t at = ws_head - s * ws_step;
            const float keep = a.ws_total[at];
            const f32x4 *w = static_cast<const f32x4 *>(a.ws) + at * WS + tid;
#pragma unroll
            for (int nc = 0; nc < NC; ++nc)
#pragma unroll
                for (int d = 0; d < DT; ++d) {
                    const f32x4 x = w[(nc * DT + d) * 256];
#pragma unroll
                    for (int i = 0; i < 4; ++i) S[nc][d][i] = fmaf(S[nc][d][i], keep, x[i]);
                }
        }
    }

    // ---- staging of a chunk: global memory -> registers -> LDS.  Eight lanes take 128 bytes of a
    // row, so a thread has two rows (r0 = thread / 8 and r0 + 32) and the same channels of each block.  Rows
    // and channels that are not there are read from the last ones that are, and zeroed on the
    // way to LDS.
    u32x4 rq[OUT ? KT : 1], rk[KT], rv[2 * NC];
    const Bf16 *gq = static_cast<const Bf16 *>(a.q) + row.q + hq * a.q_head + first * a.q_tok;
    const Bf16 *gk = static_cast<const Bf16 *>(a.k) + row.k + hq * a.k_head + first * a.k_tok;
    const Bf16 *gv = static_cast<const Bf16 *>(a.v) + row.v + h * a.v_head + col0 + first * a.v_tok;
    const int dv_here = a.dv - col0 < 64 * NC ? a.dv - col0 : 64 * NC;
    const bool whole_tile = a.dk == 32 * KT && dv_here == 64 * NC;
    auto fetch = [&](int left, int place) {        // the chunk at gq, gk, gv: `left` tokens of it on
        const int r0 = place >> 3, c0 = 8 * (place & 7);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int r = r0 + 32 * u < left ? r0 + 32 * u : left - 1;
            const Bf16 *pk = gk + r * a.k_tok, *pv = gv + r * a.v_tok, *pq = OUT ? gq + r * a.q_tok : nullptr;
#pragma unroll
            for (int b = 0; b < KT / 2; ++b) {
                const int c = c0 + 64 * b < a.dk ? c0 + 64 * b : 0;
                rk[u * (KT / 2) + b] = *reinterpret_cast<const u32x4 *>(pk + c);
                if constexpr (OUT) rq[u * (KT / 2) + b] = *reinterpret_cast<const u32x4 *>(pq + c);
            }
#pragma unroll
            for (int b = 0; b < NC; ++b) {
                const int c = c0 + 64 * b < dv_here ? c0 + 64 * b : 0;
                rv[u * NC + b] = *reinterpret_cast<const u32x4 *>(pv + c);
            }
        }
        gk += C * a.k_tok;
        gv += C * a.v_tok;
        if constexpr (OUT) gq += C * a.q_tok;
    };
    auto stage = [&](int left, int place) {
        const int r0 = place >> 3, c0 = 8 * (place & 7);
        if (!whole_tile || left < C) {
            const u32x4 zero = {0, 0, 0, 0};
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const bool there = r0 + 32 * u < left;
#pragma unroll
                for (int b = 0; b < KT / 2; ++b)
                    if (!there || c0 + 64 * b >= a.dk) {
                        rk[u * (KT / 2) + b] = zero;
                        if constexpr (OUT) rq[u * (KT / 2) + b] = zero;
                    }
#pragma unroll
                for (int b = 0; b < NC; ++b)
                    if (!there || c0 + 64 * b >= dv_here) rv[u * NC + b] = zero;
            }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int r = r0 + 32 * u;
#pragma unroll
            for (int b = 0; b < KT / 2; ++b) {
                *reinterpret_cast<u32x4 *>(sh.k + r * SH::KP + 2 * c0 + 128 * b) = rk[u * (KT / 2) + b];
                if constexpr (OUT)
                    *reinterpret_cast<u32x4 *>(sh.q + r * SH::QP + 2 * c0 + 128 * b) = rq[u * (KT / 2) + b];
            }
#pragma unroll
            for (int b = 0; b < NC; ++b)
                *reinterpret_cast<u32x4 *>(sh.v + r * SH::VP + 2 * c0 + 128 * b) = rv[u * NC + b];
        }
    };
    // One wavefront, lane = token: the chunk's decays, from log decays loaded a chunk earlier.
    const float *gg = a.g ? a.g + row.g + h + (int64_t)(first + lane) * a.g_tok : nullptr;
    float g_next = 0.0f;
    auto fetch_decays = [&](int t0) {
        g_next = gg && t0 + lane < n ? gg[(int64_t)t0 * a.g_tok] : 0.0f;
    };
    double whole = 0.0;                            // log2 of the segment's decay (that wavefront)
    auto scan = [&](Decays &d) {
        double x = 1.4426950408889634 * (double)finite_decay(g_next);
#pragma unroll
        for (int s = 1; s < C; s *= 2) {
            const double y = __shfl_up(x, s);
            if (lane >= s) x += y;
        }
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
        if (wave == 3) fetch_decays(0);
        fetch(n, tid);
        if (wave == 3) {
            scan(sh.d[0]);
            fetch_decays(C);
        }
    }
    if constexpr (OUT) {
        // the tiles just above the diagonal that the products read: zeros for good
        const int t = 32 * (tid >> 7) + ((tid >> 3) & 15), c = 16 + (tid & 7) * 2;
        const int at = t * SH::PP + (32 * (tid >> 7) + c) * 2;
        *reinterpret_cast<uint32_t *>(sh.p[0] + at) = 0;
        *reinterpret_cast<uint32_t *>(sh.p[1] + at) = 0;
    }
    Bf16 *out = OUT ? static_cast<Bf16 *>(a.out) + row.o + h * a.o_head + col0 : nullptr;

    for (int t0 = 0, turn = 0; t0 < n; t0 += C, turn ^= 1) {
        // The lane's place, hidden at each chunk: what is derived from it is computed again
        // rather than kept in registers, which are short here.
        int place = tid;
        asm volatile("" : "+v"(place));
        const int j = place & 15, g4 = (place & 48) >> 2;
        stage(n - t0, place);
        __syncthreads();
        const Decays &dec = sh.d[turn];
        if (wave == 3 && t0 + C < n) {
            scan(sh.d[turn ^ 1]);
            fetch_decays(t0 + 2 * C);
        }

        f32x4 o[OUT ? 4 : 1][NC];
        if constexpr (OUT) {
            // ---- this wavefront's tiles of the decayed products, transposed (lane = token t):
            // 3 or (the one that scans) 1 of the ten, (3, 0..2); (2, 0..2); (1, 0..1), (3, 3); (0, 0)
            auto products = [&](auto tiles) {
                constexpr int N = decltype(tiles)::value;
                f32x4 p[N];
                int ti[N], si[N];
#pragma unroll
                for (int u = 0; u < N; ++u) {
                    const bool lone = wave == 2 && u == 2;
                    ti[u] = lone ? 3 : 3 - wave;
                    si[u] = lone ? 3 : u;
                    p[u] = f32x4{0, 0, 0, 0};
                }
#pragma unroll
                for (int x = 0; x < KT; ++x)
#pragma unroll
                    for (int u = 0; u < N; ++u)
                        p[u] = mma(*reinterpret_cast<const bf16x8 *>(sh.k + (16 * si[u] + j) * SH::KP + 4 * g4 + 64 * x),
                                   *reinterpret_cast<const bf16x8 *>(sh.q + (16 * ti[u] + j) * SH::QP + 4 * g4 + 64 * x),
                                   p[u]);
#pragma unroll
                for (int u = 0; u < N; ++u) {
                    const int t = 16 * ti[u] + j, s = 16 * si[u] + g4;
                    const float thi = dec.hi[t], tlo = dec.lo[t];
                    const f32x4 shi = *reinterpret_cast<const f32x4 *>(dec.hi + s);
                    const f32x4 slo = *reinterpret_cast<const f32x4 *>(dec.lo + s);
                    float f[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float e = __builtin_amdgcn_exp2f((thi - shi[i]) + (tlo - slo[i]));
                        f[i] = s + i <= t ? a.scale * p[u][i] * e : 0.0f;
                    }
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
                        const u32x2 w = {pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3])};
                        *reinterpret_cast<u32x2 *>(sh.p[part] + t * SH::PP + 2 * s) = w;
                        f[0] = less_lo(f[0], w[0]), f[1] = less_hi(f[1], w[0]);
                        f[2] = less_lo(f[2], w[1]), f[3] = less_hi(f[3], w[1]);
                    }
                }
            };
            if (wave == 3) products(std::integral_constant<int, 1>{});
            else products(std::integral_constant<int, 3>{});

            // ---- S^T q, transposed outputs: lane = token, registers = 4 columns.  q is read one
            // step ahead; a product's accumulator comes round after 4 * NC products.
            u32x2 qa[2][4], qb[2][4];
            auto read_q = [&](int x) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const char *qp = sh.q + (16 * r + j) * SH::QP + 64 * x + 2 * g4;
                    qa[x & 1][r] = *reinterpret_cast<const u32x2 *>(qp);
                    qb[x & 1][r] = *reinterpret_cast<const u32x2 *>(qp + 32);
                }
            };
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int nc = 0; nc < NC; ++nc) o[r][nc] = f32x4{0, 0, 0, 0};
            read_q(0);
#pragma unroll
            for (int x = 0; x < KT; ++x) {
                __builtin_amdgcn_sched_barrier(0);
                if (x + 1 < KT) read_q(x + 1);
                bf16x8 s[2][NC];
#pragma unroll
                for (int nc = 0; nc < NC; ++nc) {
                    float f[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) f[i] = S[nc][2 * x][i], f[4 + i] = S[nc][2 * x + 1][i];
                    s[0][nc] = take_part(f);
                    s[1][nc] = take_part(f);
                }
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
#pragma unroll
                        for (int nc = 0; nc < NC; ++nc)
                            o[r][nc] = mma(s[part][nc], frag(qa[x & 1][r], qb[x & 1][r]), o[r][nc]);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float e = dec.in[16 * r + j];
#pragma unroll
                for (int nc = 0; nc < NC; ++nc)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[r][nc][i] *= e;
            }
            __syncthreads();                       // the products are there
        }
        if (t0 + C < n) fetch(n - t0 - C, place);

        // ---- the state's update
        bf16x8 vf[NC][2];
        const float keep = dec.total;
#pragma unroll
        for (int nc = 0; nc < NC; ++nc)
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int i = 0; i < 4; ++i) S[nc][d][i] *= keep;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            __builtin_amdgcn_sched_barrier(0);
            const int t = 32 * x + 2 * g4 + j / 4;  // this lane's row of the transposing reads
            float left[8];
            load_vec<8>(dec.left + 32 * x + 2 * g4, left);
            bf16x8 part[NC][PARTS];
#pragma unroll
            for (int nc = 0; nc < NC; ++nc) {
                const int c = NC == 2 ? colw + 8 * (j % 4) + 4 * nc : colw + 4 * (j % 4);
                const char *vp = sh.v + t * SH::VP + 2 * c;
                vf[nc][x] = frag(read_transposed(vp), read_transposed(vp + 4 * SH::VP));
                const u32x4 w = __builtin_bit_cast(u32x4, vf[nc][x]);
                float f[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f[2 * i] = bf16_lo(w[i]) * left[2 * i];
                    f[2 * i + 1] = bf16_hi(w[i]) * left[2 * i + 1];
                }
#pragma unroll
                for (int u = 0; u < PARTS; ++u) part[nc][u] = take_part(f);
            }
            const char *kp = sh.k + t * SH::KP + 8 * (j % 4);
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                const bf16x8 kf = frag(read_transposed(kp + 32 * d), read_transposed(kp + 32 * d + 4 * SH::KP));
#pragma unroll
                for (int nc = 0; nc < NC; ++nc)
#pragma unroll
                    for (int u = 0; u < PARTS; ++u) S[nc][d] = mma(kf, part[nc][u], S[nc][d]);
            }
        }

        if constexpr (OUT) {
            // ---- the chunk's own tokens.  A v that is not finite makes its column of the state
            // so (0 * inf is NaN): then such values are taken out, for a masked product of 0 must
            // not carry them to the tokens before theirs, and what they reach is marked instead.
            __builtin_amdgcn_sched_barrier(0);
            bool bad = false;
#pragma unroll
            for (int nc = 0; nc < NC; ++nc) bad |= !(__builtin_fabsf(S[nc][0][0]) < INFINITY);
            const bool any_bad = __any(bad);
            bf16x8 bf[NC][2];
            if (any_bad) {
                asm volatile("");                  // not to be computed where it is not needed
#pragma unroll
                for (int nc = 0; nc < NC; ++nc)
#pragma unroll
                    for (int x = 0; x < 2; ++x) bf[nc][x] = take_bad(vf[nc][x]);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int x = 0; x <= r / 2; ++x)
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
                        const bf16x8 pf = *reinterpret_cast<const bf16x8 *>(
                            sh.p[part] + (16 * r + j) * SH::PP + 64 * x + 4 * g4);
#pragma unroll
                        for (int nc = 0; nc < NC; ++nc) o[r][nc] = mma(vf[nc][x], pf, o[r][nc]);
                    }
            if (any_bad) {
                int token = j;                     // hidden: these masks are not worth registers
                asm volatile("" : "+v"(token));
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int nc = 0; nc < NC; ++nc) {
                        f32x4 marks = {0, 0, 0, 0};
#pragma unroll
                        for (int x = 0; x <= r / 2; ++x) {
                            u32x4 below;           // 1 where token s <= t
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int s = 32 * x + 2 * g4 + 2 * i, t = 16 * r + token;
                                below[i] = (s <= t ? 0x3F80u : 0u) | (s + 1 <= t ? 0x3F800000u : 0u);
                            }
                            marks = mma(bf[nc][x], __builtin_bit_cast(bf16x8, below), marks);
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (marks[i] > 0.0f) o[r][nc][i] = NAN;
                    }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float f[4 * NC];
#pragma unroll
                for (int nc = 0; nc < NC; ++nc)
#pragma unroll
                    for (int i = 0; i < 4; ++i) f[4 * nc + i] = o[r][nc][i];
                const int t = 16 * r + j, c = colw + NC * g4;
                if (t0 + t < n && col0 + c < a.dv)
                    store_vec<4 * NC>(out + (int64_t)(first + t0 + t) * a.o_tok + c, f);
            }
        }
        __syncthreads();                           // every wavefront is done with the tiles
    }

    if constexpr (OUT) {
        if (!seg.last) return;
#pragma unroll
        for (int nc = 0; nc < NC; ++nc)
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = 16 * d + g4 + i, c = col0 + column(nc);
                    if (r < a.dk && c < a.dv) store_one(state + (int64_t)r * a.dv + c, S[nc][d][i]);
                }
    } else {
        f32x4 *w = static_cast<f32x4 *>(a.ws) + ws_head * WS + tid;
#pragma unroll
        for (int nc = 0; nc < NC; ++nc)
#pragma unroll
            for (int d = 0; d < DT; ++d) w[(nc * DT + d) * 256] = S[nc][d];
        if (tid == 192) a.ws_total[ws_head] = __builtin_amdgcn_exp2f((float)whole);
    }
}

template <int KT, int NC, typename ST>
ChunkedPlan plan() {
    return {(const void *)chunked<KT, NC, ST, true>, (const void *)chunked<KT, NC, ST, false>, 64 * NC,
            (int64_t)256 * NC * 2 * KT * 16};
}

template <typename ST>
ChunkedPlan pick(int dk, int dv) {
    if (dv <= 64) {
        if (dk <= 64) return plan<2, 1, ST>();
        if (dk <= 128) return plan<4, 1, ST>();
        if (dk <= 192) return plan<6, 1, ST>();
        return plan<8, 1, ST>();
    }
    if (dk <= 64) return plan<2, 2, ST>();
    if (dk <= 128) return plan<4, 2, ST>();
    if (dk <= 192) return plan<6, 2, ST>();
    return plan<8, 2, ST>();
}

}  // namespace

ChunkedPlan pick_chunked(int state_bytes, int dk, int dv) {
    return state_bytes == 4 ? pick<float>(dk, dv) : pick<Bf16>(dk, dv);
}

}  // namespace laimpl

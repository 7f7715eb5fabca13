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

// The next bf16 part of eight values, taken off them.
__device__ __forceinline__ bf16x8 take_part(float (&x)[8]) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
        x[2 * i] -= bf16_lo(w[i]);
        x[2 * i + 1] -= bf16_hi(w[i]);
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
    float in[C], left[C];          // 2^(sum up to t), 2^(sum behind t)
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

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
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

    // ---- staging of a chunk: global memory -> registers -> LDS
    constexpr int QCH = KT * 4, VCH = NC * 8;      // 16-byte pieces of a row
    u32x4 rq[OUT ? KT : 1], rk[KT], rv[2 * NC];
    const Bf16 *gq = static_cast<const Bf16 *>(a.q) + row.q + hq * a.q_head;
    const Bf16 *gk = static_cast<const Bf16 *>(a.k) + row.k + hq * a.k_head;
    const Bf16 *gv = static_cast<const Bf16 *>(a.v) + row.v + h * a.v_head + col0;
    const float *gg = a.g ? a.g + row.g + h : nullptr;
    auto fetch = [&](int t0, int left) {           // tokens first + t0 .., `left` of them there
        const u32x4 zero = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < KT; ++i) {
            const int at = tid + 256 * i, r = at / QCH, c = 8 * (at % QCH);
            const bool in = r < left && c < a.dk;
            const int64_t t = first + t0 + r;
            rk[i] = in ? *reinterpret_cast<const u32x4 *>(gk + t * a.k_tok + c) : zero;
            if constexpr (OUT) rq[i] = in ? *reinterpret_cast<const u32x4 *>(gq + t * a.q_tok + c) : zero;
        }
#pragma unroll
        for (int i = 0; i < 2 * NC; ++i) {
            const int at = tid + 256 * i, r = at / VCH, c = 8 * (at % VCH);
            const int64_t t = first + t0 + r;
            rv[i] = r < left && col0 + c < a.dv ? *reinterpret_cast<const u32x4 *>(gv + t * a.v_tok + c) : zero;
        }
    };
    auto stage = [&]() {
#pragma unroll
        for (int i = 0; i < KT; ++i) {
            const int at = tid + 256 * i, r = at / QCH, c = 16 * (at % QCH);
            *reinterpret_cast<u32x4 *>(sh.k + r * SH::KP + c) = rk[i];
            if constexpr (OUT) *reinterpret_cast<u32x4 *>(sh.q + r * SH::QP + c) = rq[i];
        }
#pragma unroll
        for (int i = 0; i < 2 * NC; ++i) {
            const int at = tid + 256 * i, r = at / VCH, c = 16 * (at % VCH);
            *reinterpret_cast<u32x4 *>(sh.v + r * SH::VP + c) = rv[i];
        }
    };
    // one wavefront, lane = token: the chunk's decays
    double whole = 0.0;                            // log2 of the segment's decay (that wavefront)
    auto scan = [&](int t0, int left, Decays &d) {
        double x = gg && lane < left
                       ? 1.4426950408889634 * (double)finite_decay(gg[(int64_t)(first + t0 + lane) * a.g_tok])
                       : 0.0;
#pragma unroll
        for (int s = 1; s < C; s *= 2) {
            const double y = __shfl_up(x, s);
            if (lane >= s) x += y;
        }
        const double total = __shfl(x, C - 1);
        const float hi = (float)x;
        d.hi[lane] = hi;
        d.lo[lane] = (float)(x - hi);
        d.in[lane] = __builtin_amdgcn_exp2f(hi);
        d.left[lane] = __builtin_amdgcn_exp2f((float)(total - x));
        if (lane == 0) d.total = __builtin_amdgcn_exp2f((float)total);
        whole += total;
    };

    if (n > 0) {
        fetch(0, n);
        if (wave == 3) scan(0, n, sh.d[0]);
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
        stage();
        __syncthreads();
        const Decays &dec = sh.d[turn];
        const bool more = t0 + C < n;
        if (more) {
            fetch(t0 + C, n - t0 - C);
            if (wave == 3) scan(t0 + C, n - t0 - C, sh.d[turn ^ 1]);
        }

        f32x4 o[OUT ? 4 : 1][NC];
        if constexpr (OUT) {
            // ---- this wavefront's tiles of the decayed products, transposed (lane = token t)
            for (int u = 0; u < 3; ++u) {
                int ti, si;                        // 3 + 3 + 3 + 1 of the ten tiles
                if (wave == 0) ti = 3, si = u;
                else if (wave == 1) ti = 2, si = u;
                else if (wave == 2) ti = u < 2 ? 1 : 3, si = u < 2 ? u : 3;
                else { if (u) break; ti = 0, si = 0; }
                f32x4 p = {0, 0, 0, 0};
                const char *kp = sh.k + (16 * si + j) * SH::KP + 4 * g4;
                const char *qp = sh.q + (16 * ti + j) * SH::QP + 4 * g4;
#pragma unroll
                for (int x = 0; x < KT; ++x)
                    p = mma(*reinterpret_cast<const bf16x8 *>(kp + 64 * x),
                            *reinterpret_cast<const bf16x8 *>(qp + 64 * x), p);
                const int t = 16 * ti + j, s = 16 * si + g4;
                const float thi = dec.hi[t], tlo = dec.lo[t];
                const f32x4 shi = *reinterpret_cast<const f32x4 *>(dec.hi + s);
                const f32x4 slo = *reinterpret_cast<const f32x4 *>(dec.lo + s);
                float f[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float e = __builtin_amdgcn_exp2f((thi - shi[i]) + (tlo - slo[i]));
                    f[i] = s + i <= t ? p[i] * e : 0.0f;
                }
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    const u32x2 w = {pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3])};
                    *reinterpret_cast<u32x2 *>(sh.p[part] + t * SH::PP + 2 * s) = w;
                    f[0] -= bf16_lo(w[0]), f[1] -= bf16_hi(w[0]);
                    f[2] -= bf16_lo(w[1]), f[3] -= bf16_hi(w[1]);
                }
            }
            // ---- S^T q, transposed outputs: lane = token, registers = 4 columns
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int nc = 0; nc < NC; ++nc) o[r][nc] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int x = 0; x < KT; ++x) {
                bf16x8 hi[NC], lo[NC];
#pragma unroll
                for (int nc = 0; nc < NC; ++nc) {
                    float f[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) f[i] = S[nc][2 * x][i], f[4 + i] = S[nc][2 * x + 1][i];
                    hi[nc] = take_part(f);
                    lo[nc] = take_part(f);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const char *qp = sh.q + (16 * r + j) * SH::QP + 64 * x + 2 * g4;
                    const bf16x8 qf = frag(*reinterpret_cast<const u32x2 *>(qp),
                                           *reinterpret_cast<const u32x2 *>(qp + 32));
#pragma unroll
                    for (int nc = 0; nc < NC; ++nc) {
                        o[r][nc] = mma(hi[nc], qf, o[r][nc]);
                        o[r][nc] = mma(lo[nc], qf, o[r][nc]);
                    }
                }
            }
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
            bool bad = false;
#pragma unroll
            for (int nc = 0; nc < NC; ++nc) bad |= !(__builtin_fabsf(S[nc][0][0]) < INFINITY);
            const bool any_bad = __any(bad);
            bf16x8 bf[NC][2];
            if (any_bad)
#pragma unroll
                for (int nc = 0; nc < NC; ++nc)
#pragma unroll
                    for (int x = 0; x < 2; ++x) bf[nc][x] = take_bad(vf[nc][x]);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                f32x4 marks[NC];
#pragma unroll
                for (int nc = 0; nc < NC; ++nc) marks[nc] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int x = 0; x <= r / 2; ++x) {
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
                        const bf16x8 pf = *reinterpret_cast<const bf16x8 *>(
                            sh.p[part] + (16 * r + j) * SH::PP + 64 * x + 4 * g4);
#pragma unroll
                        for (int nc = 0; nc < NC; ++nc) o[r][nc] = mma(vf[nc][x], pf, o[r][nc]);
                    }
                    if (any_bad) {
                        u32x4 below;               // 1 where token s <= t
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int s = 32 * x + 2 * g4 + 2 * i, t = 16 * r + j;
                            below[i] = (s <= t ? 0x3F80u : 0u) | (s + 1 <= t ? 0x3F800000u : 0u);
                        }
#pragma unroll
                        for (int nc = 0; nc < NC; ++nc)
                            marks[nc] = mma(bf[nc][x], __builtin_bit_cast(bf16x8, below), marks[nc]);
                    }
                }
                float f[4 * NC];
#pragma unroll
                for (int nc = 0; nc < NC; ++nc)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        f[4 * nc + i] = a.scale * o[r][nc][i];
                        if (any_bad && marks[nc][i] > 0.0f) f[4 * nc + i] = NAN;
                    }
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

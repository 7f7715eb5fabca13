// The selective scan: for each channel c and state n
//
//   h <- exp(delta A[c,n]) h + (delta x) B[n],   y = sum_n C[n] h + D x,   out = y silu(z)
//
// The decay is another one for every channel and state, so no product of matrices makes it: each
// state update is an exponential and four multiply-adds of its own (the exponent, delta x B, the
// two of the sums), which bound the prompts.
//
// Four neighbouring lanes hold the states of one channel, NL each, and stay with it from the row's
// first token to its last; a wavefront has 16 channels and a workgroup 64 (of bf16 one 128-byte
// line a token).  Tokens go in groups of four: each of a channel's lanes loads x, dt and z of one
// of them and makes its delta and, behind the sums, its gate, so that none is made twice; the four
// steps take delta and delta x from the lane that has them by quad permutes, which are free operands
// of the multiplies.  B and C go through LDS, a stage of 16 tokens for each wavefront: a lane reads
// its own states' share in vectors.  Loads are a stage ahead.  No barrier: wavefronts are alone.
#include "la_device.h"
#include "sq_internal.h"

namespace sqimpl {
namespace {

using namespace laimpl;

constexpr int kStage = 16;        // tokens
constexpr int kChannels = 64;     // of a workgroup
constexpr float kLog2e = 1.4426950408889634f;

enum { OUTPUTS, STATE, FIRST };   // what a launch makes

// Elements of 2 or 4 bytes in vectors that are aligned to an element only.
typedef uint32_t u32_2 __attribute__((ext_vector_type(1), aligned(2)));
typedef uint32_t u32x2_2 __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32x2_4 __attribute__((ext_vector_type(2), aligned(4)));
typedef uint32_t u32x4_4 __attribute__((ext_vector_type(4), aligned(4)));

// NL consecutive elements as they lie in memory, the ones from `left` on as 0.  (NL a multiple of 4:
// `left` is one too.  Else all are there.)
template <typename XT, int NL>
struct Run {
    static constexpr int W = NL * (int)sizeof(XT) / 4;
    uint32_t w[W];
    __device__ __forceinline__ void load(const XT *p, int left) {
        if constexpr (NL % 4 == 0) {
#pragma unroll
            for (int i = 0; i < NL; i += 4)
                if constexpr (sizeof(XT) == 2) {
                    u32x2_2 v = {0, 0};
                    if (i < left) v = *reinterpret_cast<const u32x2_2 *>(p + i);
                    w[i / 2] = v[0], w[i / 2 + 1] = v[1];
                } else {
                    u32x4_4 v = {0, 0, 0, 0};
                    if (i < left) v = *reinterpret_cast<const u32x4_4 *>(p + i);
                    w[i] = v[0], w[i + 1] = v[1], w[i + 2] = v[2], w[i + 3] = v[3];
                }
        } else {
#pragma unroll
            for (int i = 0; i < NL; i += 2)
                if constexpr (sizeof(XT) == 2) {
                    w[i / 2] = (*reinterpret_cast<const u32_2 *>(p + i))[0];
                } else {
                    const u32x2_4 v = *reinterpret_cast<const u32x2_4 *>(p + i);
                    w[i] = v[0], w[i + 1] = v[1];
                }
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = 0;
    }
    __device__ __forceinline__ float operator[](int i) const {
        if constexpr (sizeof(XT) == 2) return i & 1 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
        else return __uint_as_float(w[i]);
    }
};

template <typename ST, int NL>
__device__ __forceinline__ void store_run(ST *p, const float (&h)[NL], int left) {
    if constexpr (NL % 4 == 0) {
#pragma unroll
        for (int i = 0; i < NL; i += 4) {
            const float f[4] = {h[i], h[i + 1], h[i + 2], h[i + 3]};
            if (i < left) store_vec<4>(p + i, f);
        }
    } else {
#pragma unroll
        for (int i = 0; i < NL; i += 2)
            if constexpr (sizeof(ST) == 2) *reinterpret_cast<uint32_t *>(p + i) = pack_bf16(h[i], h[i + 1]);
            else *reinterpret_cast<u32x2 *>(p + i) = u32x2{__float_as_uint(h[i]), __float_as_uint(h[i + 1])};
    }
}

// log(1 + 2^(-|v| log2 e)) + max(v, 0).  With e the power, log(1 + e) = 2 artanh(s), s = e / (2 + e) <=
// 1/3, by its series up to s^15 (the rest is below 2^-26 of it), which keeps its relative accuracy
// where e is small, as 1 + e would not.
__device__ __forceinline__ float softplus(float v) {
    const float e = __builtin_amdgcn_exp2f(__builtin_fabsf(v) * -kLog2e);
    const float s = e * __builtin_amdgcn_rcpf(2.0f + e);
    const float s2 = s * s;
    float p = 2.0f / 15;
    p = fmaf(p, s2, 2.0f / 13);
    p = fmaf(p, s2, 2.0f / 11);
    p = fmaf(p, s2, 2.0f / 9);
    p = fmaf(p, s2, 2.0f / 7);
    p = fmaf(p, s2, 2.0f / 5);
    p = fmaf(p, s2, 2.0f / 3);
    p = fmaf(p, s2, 2.0f);
    return fmaf(p, s, v > 0.0f ? v : 0.0f);
}

template <int J>
__device__ __forceinline__ float of_quad(float v) { return cvimpl::dpp<J * 0x55>(v); }
__device__ __forceinline__ float quad_sum(float v) {
    v += cvimpl::dpp<0xB1>(v);     // lane ^ 1
    return v + cvimpl::dpp<0x4E>(v);   // lane ^ 2
}

template <typename XT>
struct Token { XT x, dt, z; };

template <typename XT, typename ST, int NL, int MAKES>
__global__ __launch_bounds__(256) void scan(const ScanArgs a) {
    constexpr int NP = 4 * NL;
    constexpr bool OUT = MAKES == OUTPUTS;
    __shared__ float low[4][kStage][OUT ? 2 : 1][NP];
    __shared__ int64_t found[3];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int sub = lane & 3;
    const int tile = uniform((int)(blockIdx.x % a.tiles)), id = uniform((int)(blockIdx.x / a.tiles));
    const Segment seg = find_segment<4>(a, id, found);
    if (seg.row < 0) return;                       // same for the workgroup
    Span row = span_of(a, seg.row);
    row = Span{uniform(row.n), uniform(row.slot), uniform(row.first), uniform(row.seq)};
    const bool init = !a.has_init || uniform(a.has_init[seg.row]) != 0;
    const bool cut = !seg.last || seg.index > 0;
    if (MAKES == FIRST && !cut) return;
    if (row.n == 0 && (init || !a.write_state)) return;
    const int c0 = tile * kChannels + 16 * wave;
    if (c0 >= a.d) return;                         // a whole wavefront
    const int c = c0 + (lane >> 2) < a.d ? c0 + (lane >> 2) : a.d - 1;
    const bool own = c0 + (lane >> 2) < a.d;

    // ---- the states that enter
    const int n0 = sub * NL, left = a.d_state - n0;
    ST *state = static_cast<ST *>(a.state) + row.slot * a.s_slot + (int64_t)c * a.d_state + n0;
    float h[NL], decay[NL];
#pragma unroll
    for (int i = 0; i < NL; ++i) h[i] = 0.0f;
    auto from_pool = [&]() {
        Run<ST, NL> r;
        r.load(state, left);
#pragma unroll
        for (int i = 0; i < NL; ++i) h[i] = r[i];
    };
    auto place = [&](int index) {
        return ((int64_t)(seg.place + index) * a.tiles + tile) * 256 + tid;
    };
    if (MAKES == FIRST) {
        if (seg.last) {                            // the row's first state, in its last place
            if (init) from_pool();
            float *ws = a.ws + place(seg.index) * NL;
#pragma unroll
            for (int i = 0; i < NL; ++i) ws[i] = h[i];
            return;
        }
    } else if (cut) {
        const float *ws = a.ws + place(seg.index > 0 ? seg.index - 1 : segments_of(a, seg.row) - 1) * NL;
#pragma unroll
        for (int i = 0; i < NL; ++i) h[i] = ws[i];
    } else if (init) {
        from_pool();
    }
    {
        Run<float, NL> r;
        r.load(a.A + (int64_t)c * a.d_state + n0, left);
#pragma unroll
        for (int i = 0; i < NL; ++i) decay[i] = r[i] * kLog2e;
    }
    const float bias = a.dt_bias ? a.dt_bias[c] : 0.0f, skip = OUT && a.D ? a.D[c] : 0.0f;

    // ---- the tokens
    const int begin = seg.index * a.seg_len;
    const int n = row.n - begin < a.seg_len ? row.n - begin : a.seg_len;
    const int64_t t0 = row.first + begin;
    const XT *x = static_cast<const XT *>(a.x) + row.seq * a.x_seq + (t0 + sub) * a.x_tok + c;
    const XT *dt = static_cast<const XT *>(a.dt) + row.seq * a.dt_seq + (t0 + sub) * a.dt_tok + c;
    const XT *z = nullptr;
    XT *out = nullptr;
    const int tb = lane >> 2;                      // the token of the stage whose B and C are this lane's
    const XT *B = static_cast<const XT *>(a.B) + row.seq * a.b_seq + (t0 + tb) * a.b_tok + n0, *C = nullptr;
    if constexpr (OUT) {
        if (a.z) z = static_cast<const XT *>(a.z) + row.seq * a.z_seq + (t0 + sub) * a.z_tok + c;
        out = static_cast<XT *>(a.out) + row.seq * a.o_seq + (t0 + sub) * a.o_tok + c;
        C = static_cast<const XT *>(a.C) + row.seq * a.c_seq + (t0 + tb) * a.c_tok + n0;
    }
    Token<XT> next[4] = {};
    Run<XT, NL> next_b, next_c;
    auto fetch = [&](int s) {                      // the stage from token s on
        const int64_t at = s;
        next_b.clear();
        if (OUT) next_c.clear();
        if (s + tb < n) {
            next_b.load(B + at * a.b_tok, left);
            if constexpr (OUT) next_c.load(C + at * a.c_tok, left);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (s + 4 * k + sub < n) {
                next[k].x = x[(at + 4 * k) * a.x_tok];
                next[k].dt = dt[(at + 4 * k) * a.dt_tok];
                if constexpr (OUT)
                    if (z) next[k].z = z[(at + 4 * k) * a.z_tok];
            }
    };
    float total = 0.0f;
    fetch(0);
    for (int s = 0; s < n; s += kStage) {
        Token<XT> now[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) now[k] = next[k];
        // LDS of a wavefront is written and read in its own order
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            low[wave][tb][0][n0 + i] = next_b[i];
            if constexpr (OUT) low[wave][tb][1][n0 + i] = next_c[i];
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (s + kStage < n) fetch(s + kStage);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (s + 4 * k >= n) break;
            // a token past the last changes nothing: its delta is 0
            const bool there = s + 4 * k + sub < n;
            const float xv = load_one(&now[k].x);
            float delta = load_one(&now[k].dt) + bias;
            if (a.softplus) delta = softplus(delta);
            delta = there ? delta : 0.0f;
            const float dx = there ? delta * xv : 0.0f;
            if (MAKES == FIRST) total += delta;
            float y = 0.0f;
            auto step = [&](auto J) {
                constexpr int j = decltype(J)::value;
                const float *b = low[wave][4 * k + j][0] + n0;
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < NL; ++i) {
                    const float keep = __builtin_amdgcn_exp2f(of_quad<j>(delta) * decay[i]);
                    h[i] = fmaf(h[i], keep, of_quad<j>(dx) * b[i]);
                    if constexpr (OUT) sum = fmaf(b[NP + i], h[i], sum);
                }
                if constexpr (OUT) {
                    sum = quad_sum(sum);
                    y = sub == j ? sum : y;
                }
            };
            step(std::integral_constant<int, 0>{});
            step(std::integral_constant<int, 1>{});
            step(std::integral_constant<int, 2>{});
            step(std::integral_constant<int, 3>{});
            if constexpr (OUT) {
                y = fmaf(skip, xv, y);
                if (z) y *= cvimpl::silu(load_one(&now[k].z));
                if (there && own) store_one(out + ((int64_t)s + 4 * k) * a.o_tok, y);
            }
        }
    }
    if (MAKES == FIRST) {
        float *ws = a.ws + place(seg.index) * NL;
#pragma unroll
        for (int i = 0; i < NL; ++i) ws[i] = h[i];
        a.ws_total[place(seg.index)] = quad_sum(total);
        return;
    }
    if (seg.last && a.write_state && own) store_run<ST, NL>(state, h, left);
}

// Between the two: each segment's place in the workspace, which holds what its own tokens leave in a
// state of zeros, is left with the state behind it, from the row's first state in the last one's place.
template <int NL>
__global__ __launch_bounds__(256) void combine(const ScanArgs a) {
    const int tid = threadIdx.x;
    const int tile = blockIdx.x % a.tiles, i = blockIdx.x / a.tiles;
    const int count = uniform(segments_of(a, i));
    if (count < 2) return;                         // same for the workgroup
    const int64_t first = first_place<4>(a, i);
    if (first + count > a.places) return;
    const int c = tile * kChannels + (tid >> 2), n0 = (tid & 3) * NL;
    if (c >= a.d) return;
    Run<float, NL> r;
    r.load(a.A + (int64_t)c * a.d_state + n0, a.d_state - n0);
    const int64_t step = (int64_t)a.tiles * 256, at = first * step + tile * 256 + tid;
    float h[NL];
#pragma unroll
    for (int e = 0; e < NL; ++e) h[e] = a.ws[(at + (count - 1) * step) * NL + e];
#pragma unroll 4
    for (int s = 0; s < count - 1; ++s) {
        float *ws = a.ws + (at + s * step) * NL;
        const float total = a.ws_total[at + s * step];
#pragma unroll
        for (int e = 0; e < NL; ++e) {
            h[e] = fmaf(h[e], __builtin_amdgcn_exp2f(total * (r[e] * kLog2e)), ws[e]);
            ws[e] = h[e];
        }
    }
}

template <typename XT, typename ST, int NL>
ScanPlan plan(bool out) {
    return {out ? (const void *)scan<XT, ST, NL, OUTPUTS> : (const void *)scan<XT, ST, NL, STATE>,
            (const void *)scan<XT, ST, NL, FIRST>, (const void *)combine<NL>, kChannels, 256, kStage, 256 * NL, 256};
}

template <typename XT, typename ST>
ScanPlan pick(int d_state, bool out) {
    if (d_state <= 8) return plan<XT, ST, 2>(out);
    if (d_state <= 16) return plan<XT, ST, 4>(out);
    if (d_state <= 24) return plan<XT, ST, 6>(out);
    if (d_state <= 32) return plan<XT, ST, 8>(out);
    if (d_state <= 48) return plan<XT, ST, 12>(out);
    return plan<XT, ST, 16>(out);
}

}  // namespace

ScanPlan pick_scan(int x_bytes, int state_bytes, int d_state, bool out) {
    if (x_bytes == 4) return pick<float, float>(d_state, out);
    return state_bytes == 4 ? pick<Bf16, float>(d_state, out) : pick<Bf16, Bf16>(d_state, out);
}

}  // namespace sqimpl

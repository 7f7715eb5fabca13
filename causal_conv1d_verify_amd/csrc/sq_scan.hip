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
#include "sq_scan_device.h"

namespace sqimpl {
namespace {

template <int J>
__device__ __forceinline__ float of_quad(float v) { return cvimpl::dpp<J * 0x55>(v); }
__device__ __forceinline__ float quad_sum(float v) {
    v += cvimpl::dpp<0xB1>(v);     // lane ^ 1
    return v + cvimpl::dpp<0x4E>(v);   // lane ^ 2
}

template <typename XT>
struct Token { XT x, dt, z; };

template <typename XT, typename ST, int NL, bool OUT>
__global__ __launch_bounds__(256) void scan(const ScanArgs a) {
    constexpr int NP = 4 * NL;
    __shared__ float low[4][kStage][OUT ? 2 : 1][NP];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int sub = lane & 3;
    const int tile = uniform((int)(blockIdx.x % a.tiles)), i = uniform((int)(blockIdx.x / a.tiles));
    Span row = span_of(a, i);
    row = Span{uniform(row.n), uniform(row.slot), uniform(row.first), uniform(row.seq)};
    const int n = row.n;
    const int c0 = tile * kChannels + 16 * wave;
    if (n <= 0 || c0 >= a.d) return;               // a whole wavefront
    const int c = c0 + (lane >> 2) < a.d ? c0 + (lane >> 2) : a.d - 1;
    const bool own = c0 + (lane >> 2) < a.d;

    // ---- the states that enter
    const int n0 = sub * NL, left = a.d_state - n0;
    ST *state = static_cast<ST *>(a.state) + row.slot * a.s_slot + (int64_t)c * a.d_state + n0;
    Run<ST, NL> first;
    Run<float, NL> rate;
    first.load(state, left);
    rate.load(a.A + (int64_t)c * a.d_state + n0, left);
    float h[NL], decay[NL];
#pragma unroll
    for (int e = 0; e < NL; ++e) h[e] = first[e], decay[e] = rate[e] * kLog2e;
    const float bias = a.dt_bias ? a.dt_bias[c] : 0.0f, skip = OUT && a.D ? a.D[c] : 0.0f;

    // ---- the tokens
    const XT *x = static_cast<const XT *>(a.x) + row.seq * a.x_seq + sub * a.x_tok + c;
    const XT *dt = static_cast<const XT *>(a.dt) + row.seq * a.dt_seq + sub * a.dt_tok + c;
    const XT *z = nullptr;
    XT *out = nullptr;
    const int tb = lane >> 2;                      // the token of the stage whose B and C are this lane's
    const XT *B = static_cast<const XT *>(a.B) + row.seq * a.b_seq + tb * a.b_tok + n0, *C = nullptr;
    if constexpr (OUT) {
        if (a.z) z = static_cast<const XT *>(a.z) + row.seq * a.z_seq + sub * a.z_tok + c;
        out = static_cast<XT *>(a.out) + row.seq * a.o_seq + sub * a.o_tok + c;
        C = static_cast<const XT *>(a.C) + row.seq * a.c_seq + tb * a.c_tok + n0;
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
                if (z) y *= gate(load_one(&now[k].z));
                if (there && own) store_one(out + ((int64_t)s + 4 * k) * a.o_tok, y);
            }
        }
    }
    if (a.write_state && own) store_run<ST, NL>(state, h, left);
}

template <typename XT, typename ST, int NL>
ScanPlan plan(bool out) {
    return {out ? (const void *)scan<XT, ST, NL, true> : (const void *)scan<XT, ST, NL, false>, kChannels, 256};
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

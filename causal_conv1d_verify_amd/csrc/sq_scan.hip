// The selective scan of up to 32 tokens of each row: for each channel c and state n
//
//   h <- exp(delta A[c,n]) h + (delta x) B[n],   y = sum_n C[n] h + D x,   out = y silu(z)
//
// For one token the state's traffic bounds it: 256 rows of 12288 channels with 16 fp32 states, 395 MB, 79 us,
// 5.0 TB/s (a large copy: 5.3).  From some four on the vector units do (sq_prompt.hip).
//
// Four neighbouring lanes hold the states of one channel, NL each, so that a state is loaded and stored
// in whole runs; a lane holds U such shares, of channels 16 apart, and a wavefront has 16 U channels for
// all tokens.  x, dt and z come a channel a lane, and delta and the gate are made there; delta and
// delta x go to the channel's four lanes, and the four lanes' sum back, through LDS.  G tokens are
// loaded at once, the next G while these are computed.  No barrier: wavefronts are alone.
//
// 16 states in U = 4 shares: 16 loads of a lane are in flight at once and delta is made once for each
// channel (one share a wavefront, four tokens a channel's lanes: 134 us; 128 rows of one token with U = 4, 2, 1:
// 33.4, 35.8, 37.9 us, one row 3.2 to 3.5).  Loads and stores of the state past the caches: no change.
#include "sq_scan_device.h"

namespace sqimpl {
namespace {

__device__ __forceinline__ float quad_sum(float v) {
    v += cvimpl::dpp<0xB1>(v);         // lane ^ 1
    return v + cvimpl::dpp<0x4E>(v);   // lane ^ 2
}

template <typename XT, typename ST, int NL, int U, int G, bool OUT>
__global__ __launch_bounds__(256) void scan(const ScanArgs a) {
    constexpr int CH = 16 * U;                     // channels of a wavefront
    constexpr bool FITS = NL <= 8;                 // 4 NL is d_state; above, 40 and 56 go as 48 and 64
    __shared__ float2 steps[4][G][64];
    __shared__ float sums[4][G][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int sub = lane & 3, quad = lane >> 2;
    const int tile = uniform((int)(blockIdx.x % a.tiles)), i = uniform((int)(blockIdx.x / a.tiles));
    Span row = span_of(a, i);
    const int n = uniform(row.n);
    const int64_t slot = uniform(row.slot);
    const int c0 = (tile * 4 + wave) * CH;
    if (n <= 0 || c0 >= a.d) return;               // a whole wavefront

    // ---- tokens: a channel a lane
    const bool mine = lane < CH && c0 + lane < a.d;
    const int c = mine ? c0 + lane : a.d - 1, n0 = sub * NL;
    const XT *x = static_cast<const XT *>(a.x) + i * a.x_seq, *dt = static_cast<const XT *>(a.dt) + i * a.dt_seq;
    const XT *B = static_cast<const XT *>(a.B) + i * a.b_seq, *z = nullptr, *C = nullptr;
    if constexpr (OUT) {
        z = a.z ? static_cast<const XT *>(a.z) + i * a.z_seq : x;
        C = static_cast<const XT *>(a.C) + i * a.c_seq;
    }
    const int64_t z_tok = OUT && a.z ? a.z_tok : a.x_tok;
    struct Raw {
        XT x, dt, z;
        Run<XT, NL, FITS> B, C;
    } next[G];
    auto fetch = [&](int s) {                      // past the last token it again: loads without branches
#pragma unroll
        for (int k = 0; k < G; ++k) {
            const int64_t t = s + k < n ? s + k : n - 1;
            next[k].x = (x + t * a.x_tok)[c];
            next[k].dt = (dt + t * a.dt_tok)[c];
            if constexpr (OUT) next[k].z = (z + t * z_tok)[c];
            next[k].B.load(B + t * a.b_tok, n0, a.d_state);
            if constexpr (OUT) next[k].C.load(C + t * a.c_tok, n0, a.d_state);
        }
    };
    fetch(0);
    const float bias = a.dt_bias ? a.dt_bias[c] : 0.0f, skip = OUT && a.D ? a.D[c] : 0.0f;

    // ---- the states
    ST *state = static_cast<ST *>(a.state) + slot * a.s_slot;
    float h[U][NL], decay[U][NL];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int cu = c0 + 16 * u + quad < a.d ? c0 + 16 * u + quad : a.d - 1;
        const int64_t at = (int64_t)cu * a.d_state;
        Run<ST, NL, FITS> first;
        Run<float, NL, FITS> rate;
        first.load(state + at, n0, a.d_state);
        rate.load(a.A + at, n0, a.d_state);
        first.end(n0, a.d_state);
        rate.end(n0, a.d_state);
#pragma unroll
        for (int e = 0; e < NL; ++e) h[u][e] = first[e], decay[u][e] = rate[e] * kLog2e;
    }

    for (int s = 0; s < n; s += G) {
        Raw now[G];
        float xv[G], gates[G];
#pragma unroll
        for (int k = 0; k < G; ++k) {
            now[k] = next[k];
            now[k].B.end(n0, a.d_state);
            if constexpr (OUT) now[k].C.end(n0, a.d_state);
        }
        // LDS of a wavefront is written and read in its own order
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int k = 0; k < G; ++k) {
            xv[k] = load_one(&now[k].x);
            float delta = load_one(&now[k].dt) + bias;
            if (a.softplus) delta = softplus(delta);
            steps[wave][k][lane] = make_float2(delta, delta * xv[k]);
            if constexpr (OUT) gates[k] = a.z ? gate(load_one(&now[k].z)) : 1.0f;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (s + G < n) fetch(s + G);
#pragma unroll
        for (int k = 0; k < G; ++k) {
            if (s + k >= n) break;
            float y = 0.0f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float2 step = steps[wave][k][16 * u + quad];
                float sum = 0.0f;
#pragma unroll
                for (int e = 0; e < NL; ++e) {
                    const float keep = __builtin_amdgcn_exp2f(exponent(step.x, decay[u][e]));
                    h[u][e] = fmaf(h[u][e], keep, step.y * now[k].B[e]);
                    if constexpr (OUT) sum = fmaf(now[k].C[e], h[u][e], sum);
                }
                if constexpr (OUT) {
                    sum = quad_sum(sum);
                    y = u == 0 || (sub & (U - 1)) == u ? sum : y;
                }
            }
            if constexpr (OUT) sums[wave][k][16 * (sub & (U - 1)) + quad] = y;
        }
        if constexpr (OUT) {
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            XT *out = static_cast<XT *>(a.out) + i * a.o_seq + s * a.o_tok;
#pragma unroll
            for (int k = 0; k < G; ++k) {
                if (s + k >= n) break;
                const float y = sums[wave][k][lane & (CH - 1)], with = fmaf(skip, xv[k], y);
                if (mine) store_one(out + k * a.o_tok + c, (a.D ? with : y) * gates[k]);
            }
        }
    }
    if (!a.write_state) return;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int cu = c0 + 16 * u + quad;
        if (cu >= a.d) continue;
        store_run(state + (int64_t)cu * a.d_state + n0, h[u], a.d_state - n0);
    }
}

template <typename XT, typename ST, int NL, int U, int G>
ScanPlan plan(bool one, bool out) {
    const void *fn = one ? out ? (const void *)scan<XT, ST, NL, U, 1, true> : (const void *)scan<XT, ST, NL, U, 1, false>
                         : out ? (const void *)scan<XT, ST, NL, U, G, true> : (const void *)scan<XT, ST, NL, U, G, false>;
    return {fn, 64 * U, 256};
}

template <typename XT, typename ST>
ScanPlan pick(int d_state, bool one, bool out) {
    if (d_state <= 8) return plan<XT, ST, 2, 4, 4>(one, out);
    if (d_state <= 16) return plan<XT, ST, 4, 4, 4>(one, out);
    if (d_state <= 24) return plan<XT, ST, 6, 2, 2>(one, out);
    if (d_state <= 32) return plan<XT, ST, 8, 2, 2>(one, out);
    if (d_state <= 48) return plan<XT, ST, 12, 1, 2>(one, out);
    return plan<XT, ST, 16, 1, 2>(one, out);
}

}  // namespace

ScanPlan pick_scan(int x_bytes, int state_bytes, int d_state, bool one, bool out) {
    if (x_bytes == 4) return pick<float, float>(d_state, one, out);
    return state_bytes == 4 ? pick<Bf16, float>(d_state, one, out) : pick<Bf16, Bf16>(d_state, one, out);
}

}  // namespace sqimpl

// The norm of each head of q and k and its rotation by the token's position, in one pass: a head is
// read once and written once, and that traffic bounds it (16384 tokens of 32 heads of 128 channels, half of
// them rotated, bf16: 54.4 us, 4.9 TB/s, where a large copy has 5.3).
//
// A wavefront has one token (or some of its heads) and makes its angles once, one or two a lane, for
// all heads: the product position * inv_freq and its remainder modulo a turn in fp64, then sine and
// cosine by their series on an eighth of a turn.  They go through LDS.  A head lies across LG lanes, 16
// channels each, in two vectors of 8: from channels 8u and rot/2 + 8u on for unit u, which hold both halves
// of 8 rotated pairs (interleaved: four whole pairs each); behind the rotated ones likewise.
#include "la_device.h"
#include "sq_internal.h"

namespace sqimpl {
namespace {

using namespace laimpl;

// Sine and cosine of `position * freq`.
__device__ __forceinline__ void turn(double position, double freq, float &cos, float &sin) {
    constexpr double kTurn = 0x1.45f306dc9c883p-3, kTurnLow = -0x1.6b01ec5417056p-57;   // 1 / 2 pi
    const double angle = position * freq;
    const double turns = angle * kTurn;
    // what the product's rounding leaves, and the rest of 1 / 2 pi
    const double low = fma(angle, kTurn, -turns) + angle * kTurnLow;
    double part = (turns - rint(turns)) + low;                    // of a turn, in about [-1/2, 1/2]
    const double quarter = rint(4.0 * part);
    part -= 0.25 * quarter;                                       // in [-1/8, 1/8]
    const float t = (float)(part * 6.283185307179586), t2 = t * t;
    // the series: the next terms are below 2^-29 (sine) and 2^-33 (cosine) of a value at pi / 4
    float s = 2.7557319e-6f;
    s = fmaf(s, t2, -1.9841270e-4f);
    s = fmaf(s, t2, 8.3333333e-3f);
    s = fmaf(s, t2, -1.6666667e-1f);
    s = fmaf(s * t2, t, t);
    float c = -2.7557319e-7f;
    c = fmaf(c, t2, 2.4801587e-5f);
    c = fmaf(c, t2, -1.3888889e-3f);
    c = fmaf(c, t2, 4.1666667e-2f);
    c = fmaf(c, t2, -0.5f);
    c = fmaf(c, t2, 1.0f);
    const int q = (int)quarter;
    const float a = q & 1 ? s : c, b = q & 1 ? c : s;
    cos = ((q + 1) & 2) ? -a : a;
    sin = (q & 2) ? -b : b;
}

// The sum over groups of LG neighbouring lanes, on each of them.
template <int LG>
__device__ __forceinline__ float group_sum(float v) {
    if constexpr (LG > 1) v += cvimpl::dpp<0xB1>(v);              // lane ^ 1
    if constexpr (LG > 2) v += cvimpl::dpp<0x4E>(v);              // lane ^ 2
    if constexpr (LG > 4) v += cvimpl::dpp<0x141>(v);             // the other four of eight
    if constexpr (LG > 8) v += cvimpl::dpp<0x140>(v);             // the other eight of sixteen
    return v;
}

// 1 / sqrt(sum / dim + eps) of a head's squares.  A head whose sum leaves fp32's range is scaled by a
// power of two and summed again.
template <int LG>
__device__ __forceinline__ float inverse_norm(float (&v)[16], float per_dim, float eps) {
    auto total = [&]() {
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < 16; ++j) s = fmaf(v[j], v[j], s);
        return group_sum<LG>(s);
    };
    float sum = total(), e = eps;
    const bool high = !(sum < INFINITY), low = sum < 0x1p-100f && eps < 0x1p-100f;
    if (__builtin_expect(high || low, 0)) {
        const float scale = high ? 0x1p-80f : 0x1p100f;   // a square of 2^-149 2^100 is no subnormal, which rsq takes for 0
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] *= scale;
        sum = total();
        e = (eps * scale) * scale;
    }
    return __builtin_amdgcn_rsqf(fmaf(sum, per_dim, e));
}

// Eight channels as they lie in memory.
template <typename XT>
struct Eight {
    u32x4 w[sizeof(XT) / 2];
    __device__ __forceinline__ void load(const XT *p) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(XT) / 2; ++i) w[i] = reinterpret_cast<const u32x4 *>(p)[i];
    }
    __device__ __forceinline__ float operator[](int j) const {
        if constexpr (sizeof(XT) == 2) return j & 1 ? bf16_hi(w[0][j / 2]) : bf16_lo(w[0][j / 2]);
        else return __uint_as_float(w[j / 4][j % 4]);
    }
};

template <typename XT, int LG>
__global__ __launch_bounds__(256) void rotary(const RotaryArgs a) {
    constexpr int SIDE = kWave / LG;               // heads side by side
    constexpr int BATCH = 4;                       // of each lane, in flight at once
    __shared__ alignas(16) float cs[4][2][128];
    const int lane = threadIdx.x & 63, wave = uniform((int)(threadIdx.x >> 6));
    const int64_t id = (int64_t)blockIdx.x * 4 + wave;
    const int64_t token = id / a.blocks_per_token;
    if (token >= a.tokens) return;                 // a whole wavefront, and no barrier below
    const int part = (int)(id - token * a.blocks_per_token);
    const int heads = a.heads[0] + a.heads[1], units = a.dim / 16, turned = a.rot / 16;
    const int u = lane % LG;
    const bool in = u < units, turns = u < turned;
    // both halves of what is rotated, and of what is not
    const int c0 = turns ? 8 * u : a.rot + 8 * (u - turned), c1 = c0 + (turns ? a.rot : a.dim - a.rot) / 2;
    const int first = part * SIDE + lane / LG, step = a.blocks_per_token * SIDE;

    const XT *from[2];
    XT *to[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        from[i] = static_cast<const XT *>(a.x[i]) + token * a.tok[i];
        to[i] = static_cast<XT *>(a.out[i]) + token * a.out_tok[i];
    }
    Eight<XT> raw[BATCH][2];
    auto load = [&](int h0) {
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            const int h = h0 + b * step, i = h >= a.heads[0];
            raw[b][0] = raw[b][1] = Eight<XT>{};
            if (in && h < heads) {
                const XT *p = (i ? from[1] : from[0]) + (h - (i ? a.heads[0] : 0)) * (i ? a.head[1] : a.head[0]);
                raw[b][0].load(p + c0);
                raw[b][1].load(p + c1);
            }
        }
    };
    load(first);

    // ---- the angles
    if (a.rot) {
        const double position = a.wide ? (double)static_cast<const int64_t *>(a.positions)[token]
                                       : (double)static_cast<const int32_t *>(a.positions)[token];
#pragma unroll
        for (int i = lane; i < 128; i += kWave)
            if (i < a.rot / 2) turn(position, (double)a.inv_freq[i], cs[wave][0][i], cs[wave][1][i]);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
    float cos[8], sin[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) cos[j] = sin[j] = 0.0f;
    if (turns) {
        // pairs 8u to 8u + 7, or of neighbours those of either half
        const int p0 = a.interleaved ? 4 * u : 8 * u, p1 = a.interleaved ? 4 * u + a.rot / 4 : 8 * u + 4;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            cos[j] = cs[wave][0][p0 + j], cos[4 + j] = cs[wave][0][p1 + j];
            sin[j] = cs[wave][1][p0 + j], sin[4 + j] = cs[wave][1][p1 + j];
        }
    }

    const float per_dim = 1.0f / (float)a.dim;
    for (int h0 = first; h0 - lane / LG < heads; h0 += BATCH * step) {
        if (h0 != first) load(h0);
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            const int h = h0 + b * step, i = h >= a.heads[0];
            const XT *w = static_cast<const XT *>(i ? a.weight[1] : a.weight[0]);
            float v[16];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = raw[b][0][j], v[8 + j] = raw[b][1][j];
            if (w) {                               // the same for a head's lanes
                const float mult = inverse_norm<LG>(v, per_dim, a.eps);
                float f[16] = {};
                if (in) {
                    float lo[8], hi[8];
                    load_vec<8>(w + c0, lo);
                    load_vec<8>(w + c1, hi);
#pragma unroll
                    for (int j = 0; j < 8; ++j) f[j] = lo[j], f[8 + j] = hi[j];
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = (v[j] * mult) * f[j];
            }
            if (!in || h >= heads) continue;
            float lo[8], hi[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) lo[j] = v[j], hi[j] = v[8 + j];
            if (turns && a.interleaved) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float e = lo[2 * j], f = lo[2 * j + 1], g = hi[2 * j], k = hi[2 * j + 1];
                    lo[2 * j] = fmaf(e, cos[j], -(f * sin[j]));
                    lo[2 * j + 1] = fmaf(f, cos[j], e * sin[j]);
                    hi[2 * j] = fmaf(g, cos[4 + j], -(k * sin[4 + j]));
                    hi[2 * j + 1] = fmaf(k, cos[4 + j], g * sin[4 + j]);
                }
            } else if (turns) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float e = lo[j], f = hi[j];
                    lo[j] = fmaf(e, cos[j], -(f * sin[j]));
                    hi[j] = fmaf(f, cos[j], e * sin[j]);
                }
            }
            XT *p = (i ? to[1] : to[0]) + (h - (i ? a.heads[0] : 0)) * (i ? a.out_head[1] : a.out_head[0]);
            // past the caches' usual order: alone 4-20% faster (16384 tokens of 32 heads of 128: 54.4 us for
            // 58.4), with a reader behind it from 6% faster to 5% slower
            store_vec<8, true>(p + c0, lo);
            store_vec<8, true>(p + c1, hi);
        }
    }
}

template <typename XT>
RotaryPlan pick(int dim) {
    const int units = dim / 16;
    if (units <= 1) return {(const void *)rotary<XT, 1>, 256, 64};
    if (units <= 2) return {(const void *)rotary<XT, 2>, 256, 32};
    if (units <= 4) return {(const void *)rotary<XT, 4>, 256, 16};
    if (units <= 8) return {(const void *)rotary<XT, 8>, 256, 8};
    return {(const void *)rotary<XT, 16>, 256, 4};
}

}  // namespace

RotaryPlan pick_rotary(int x_bytes, int dim) { return x_bytes == 4 ? pick<float>(dim) : pick<Bf16>(dim); }

}  // namespace sqimpl

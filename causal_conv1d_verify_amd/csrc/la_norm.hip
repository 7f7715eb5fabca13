// The gated RMS norm of each head, and the norm at a block's end.  Both hold a row in registers
// between the sum of its squares and its scaling, so every element is read once and written
// once, and both are bound by that traffic.  Measured: the gated norm of 16384 x 48 heads of 128 (bf16)
// 116 us, 5.2 TB/s; the residual norm of 16384 x 4096 with an fp32 stream 163 us, 5.75 TB/s, of 1024 x
// 5120 10.3 us.  Tried and no faster: two and four heads a lane group (118 and 132 us), stores past the
// caches (no change), the weights asked for before the first sum (10.3 -> 11.8, 163 -> 169 us: fewer
// wavefronts).
#include "la_device.h"

namespace laimpl {
namespace {

// 1 / (1 + e) or e / (1 + e) with e = 2^(-|z| log2 e): the reciprocal's argument stays in
// [1, 2].  Results below fp32's normal range come out as 0.
__device__ __forceinline__ float sigmoid(float z) {
    const float e = __builtin_amdgcn_exp2f(__builtin_fabsf(z) * -1.4426950408889634f);
    const float r = __builtin_amdgcn_rcpf(1.0f + e);
    return z < 0.0f ? e * r : r;
}

// A group (one head of one row) lies across LG lanes, each holding E vectors of 8 channels,
// vector e of lane l at channel 8 * (l + LG * e); 256 / LG groups per workgroup.
template <typename XT, int LG, int E>
__global__ __launch_bounds__(256) void gated(const NormArgs a) {
    const int lane = threadIdx.x % LG;
    const int64_t at = (int64_t)blockIdx.x * (256 / LG) + threadIdx.x / LG;
    if (at >= a.rows * a.heads) return;      // whole groups leave: no sum below loses a lane
    const int64_t row = at / a.heads;
    const int head = (int)(at - row * a.heads);
    const XT *y = static_cast<const XT *>(a.y) + row * a.y_row + head * a.y_head;
    const XT *z = static_cast<const XT *>(a.gate) + row * a.gate_row + head * a.gate_head;
    const XT *w = static_cast<const XT *>(a.weight);
    XT *out = static_cast<XT *>(a.out) + row * a.out_row + head * a.out_head;

    float v[E][8], m[E][8];                  // the values to normalise, and their factors
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int c = 8 * (lane + LG * e);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[e][j] = m[e][j] = 0.0f;
        if (c < a.dim) {
            load_vec<8>(y + c, v[e]);
            load_vec<8>(w + c, m[e]);
            if (a.gate) {
                float f[8];
                load_vec<8>(z + c, f);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float act = a.sigmoid ? sigmoid(f[j]) : cvimpl::silu(f[j]);
                    if (a.gate_first) v[e][j] *= act; else m[e][j] *= act;
                }
            }
        }
    }
    float mult, pre;
    inverse_rms([&](float scale) {
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e)
#pragma unroll
            for (int j = 0; j < 8; ++j) s = fmaf(v[e][j] * scale, v[e][j] * scale, s);
#pragma unroll
        for (int d = LG / 2; d > 0; d /= 2) s += __shfl_xor(s, d);
        return s;
    }, a.dim, a.eps, mult, pre);
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int c = 8 * (lane + LG * e);
        if (c < a.dim) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[e][j] = ((v[e][j] * pre) * mult) * m[e][j];
            store_vec<8>(out + c, v[e]);
        }
    }
}

// A row lies across TPR lanes (one wavefront's 64, or the whole workgroup), E vectors of 8
// channels each.  A row shared by several wavefronts is summed through LDS.
template <typename XT, typename RT, int TPR, int E>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void residual(const NormArgs a) {
    constexpr int THREADS = TPR < 256 ? 256 : TPR;
    constexpr int WAVES = TPR / kWave;       // of a row
    __shared__ float part[2][THREADS / kWave];
    const int lane = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * (THREADS / TPR) + threadIdx.x / TPR;
    if (row >= a.rows) return;               // whole wavefronts; the only row where TPR >= 256
    const XT *y = static_cast<const XT *>(a.y) + row * a.y_row;
    const XT *z = static_cast<const XT *>(a.gate) + row * a.gate_row;
    const XT *w = static_cast<const XT *>(a.weight), *pw = static_cast<const XT *>(a.post_weight);
    const RT *res = static_cast<const RT *>(a.residual) + row * a.res_row;
    RT *res_out = static_cast<RT *>(a.residual_out) + row * a.res_out_row;
    XT *out = static_cast<XT *>(a.out) + row * a.out_row;

    int turn = 0;
    auto row_sum = [&](float s) {
#pragma unroll
        for (int d = kWave / 2; d > 0; d /= 2) s += __shfl_xor(s, d);
        if constexpr (WAVES > 1) {
            // two buffers in turn: the one of a sum is next written behind the barrier of the
            // next sum, which every wavefront reaches after reading this one
            if (threadIdx.x % kWave == 0) part[turn][threadIdx.x / kWave] = s;
            __syncthreads();
            s = 0.0f;
#pragma unroll
            for (int i = 0; i < WAVES; ++i) s += part[turn][i];
            turn ^= 1;
        }
        return s;
    };

    float v[E][8], r[E][8];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int c = 8 * (lane + TPR * e);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[e][j] = r[e][j] = 0.0f;
        if (c < a.dim) {
            load_vec<8>(y + c, v[e]);
            load_vec<8>(res + c, r[e]);
        }
    }
    auto square_sum = [&](const float (&x)[E][8], float scale) {
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e)
#pragma unroll
            for (int j = 0; j < 8; ++j) s = fmaf(x[e][j] * scale, x[e][j] * scale, s);
        return row_sum(s);
    };
    float mult = 1.0f, pre = 1.0f;
    if (a.post_weight)
        inverse_rms([&](float scale) { return square_sum(v, scale); }, a.dim, a.eps, mult, pre);
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int c = 8 * (lane + TPR * e);
        if (c < a.dim) {
            float f[8];
            if (a.post_weight) {
                load_vec<8>(pw + c, f);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[e][j] = ((v[e][j] * pre) * mult) * f[j];
            }
            if (a.gate) {
                load_vec<8>(z + c, f);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[e][j] *= f[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) r[e][j] = fmaf(a.scale, v[e][j], r[e][j]);
            store_vec<8>(res_out + c, r[e]);
        }
    }
    if (!a.out) return;
    inverse_rms([&](float scale) { return square_sum(r, scale); }, a.dim, a.eps, mult, pre);
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int c = 8 * (lane + TPR * e);
        if (c < a.dim) {
            float f[8];
            load_vec<8>(w + c, f);
#pragma unroll
            for (int j = 0; j < 8; ++j) r[e][j] = ((r[e][j] * pre) * mult) * f[j];
            store_vec<8>(out + c, r[e]);
        }
    }
}

template <typename XT>
NormPlan gated_for(int dim) {
    const int vecs = dim / 8;
    if (vecs <= 1) return {(const void *)gated<XT, 1, 1>, 256, 256};
    if (vecs <= 2) return {(const void *)gated<XT, 2, 1>, 256, 128};
    if (vecs <= 4) return {(const void *)gated<XT, 4, 1>, 256, 64};
    if (vecs <= 8) return {(const void *)gated<XT, 8, 1>, 256, 32};
    if (vecs <= 16) return {(const void *)gated<XT, 16, 1>, 256, 16};
    if (vecs <= 32) return {(const void *)gated<XT, 32, 1>, 256, 8};
    if (vecs <= 64) return {(const void *)gated<XT, 64, 1>, 256, 4};
    if (vecs <= 128) return {(const void *)gated<XT, 64, 2>, 256, 4};
    return {(const void *)gated<XT, 64, 4>, 256, 4};
}

template <typename XT, typename RT>
NormPlan residual_for(int dim) {
    if (dim <= 512) return {(const void *)residual<XT, RT, 64, 1>, 256, 4};
    if (dim <= 2048) return {(const void *)residual<XT, RT, 256, 1>, 256, 1};
    if (dim <= 4096) return {(const void *)residual<XT, RT, 512, 1>, 512, 1};
    if (dim <= 8192) return {(const void *)residual<XT, RT, 512, 2>, 512, 1};
    return {(const void *)residual<XT, RT, 1024, 2>, 1024, 1};
}

}  // namespace

NormPlan pick_gated(int x_bytes, int dim) {
    return x_bytes == 4 ? gated_for<float>(dim) : gated_for<Bf16>(dim);
}

NormPlan pick_residual(int x_bytes, int res_bytes, int dim) {
    if (x_bytes == 4) return residual_for<float, float>(dim);
    return res_bytes == 4 ? residual_for<Bf16, float>(dim) : residual_for<Bf16, Bf16>(dim);
}

}  // namespace laimpl

// The recurrence token by token, with a tile of the state held in registers:
//
//   S <- exp(g_t) S + k_t v_t^T,   out_t = scale * S^T q_t
//
// One workgroup of 256 lanes owns (row, v head, a tile of the state's columns) from the row's
// first token to its last.  A lane holds 16 bytes of each of R state rows (VC columns), LPR
// lanes lie across the tile's columns and 256 / LPR lane groups along the rows, so a load of
// the state is whole 128- or 256-byte runs and all of a lane's R loads are in flight at once.
// out sums over the rows: in the lane, across the wavefront's groups, and across the four
// wavefronts through LDS (always in the same order).
//
// It takes few fp32 tokens one after the other, the single tokens of few rows, where
// it starts sooner than the matrix form (one row of 48 heads, 128 x 128, fp32 state: 4.4 us a call,
// 5.0 of the kernel traced alone, for 6.5 us), and prompts whose tokens lie too far apart for 32-bit
// offsets.  For one token it is bound by the state, read and written once.
#include "la_device.h"

namespace laimpl {
namespace {

template <typename XT, typename ST, int LPR, int R>
__global__ __launch_bounds__(256) void recurrent(const AttnArgs a) {
    constexpr int VC = 16 / sizeof(ST);
    constexpr int COLS = LPR * VC;
    constexpr int RU = R < 8 ? R : 8;          // rows per guard: dk is a multiple of 8
    __shared__ float part[2][4][COLS];

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = threadIdx.x % LPR, rg = threadIdx.x / LPR;
    const int tile = blockIdx.x % a.tiles;
    const int rest = blockIdx.x / a.tiles;
    const int h = rest % a.v_heads, i = rest / a.v_heads;
    const Row row = row_of(a, i);
    const bool init = !a.has_init || a.has_init[i] != 0;
    if (row.n < 0 || (row.n == 0 && (init || !a.write_state))) return;   // same for the workgroup

    const int c0 = tile * COLS + col * VC, r0 = rg * R;
    const bool in_cols = c0 < a.dv;
    ST *s = static_cast<ST *>(a.state) + row.slot * a.s_slot +
            ((int64_t)h * a.dk + r0) * a.dv + c0;
    float S[R][VC];
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int c = 0; c < VC; ++c) S[r][c] = 0.0f;
        if (init && in_cols && r0 + r < a.dk) load_vec<VC>(s + (int64_t)r * a.dv, S[r]);
    }

    const int hq = h / a.group;
    const XT *q = static_cast<const XT *>(a.q) + row.q + hq * a.q_head + r0;
    const XT *k = static_cast<const XT *>(a.k) + row.k + hq * a.k_head + r0;
    const XT *v = static_cast<const XT *>(a.v) + row.v + h * a.v_head + c0;
    XT *out = static_cast<XT *>(a.out) + row.o + h * a.o_head + c0;
    const float *g = a.g ? a.g + row.g + h : nullptr;
    for (int t = 0; t < row.n; ++t) {
        const float decay = g ? expf(finite_decay(g[t * a.g_tok])) : 1.0f;
        float kt[R] = {}, qt[R] = {}, vt[VC] = {}, o[VC] = {};
#pragma unroll
        for (int u = 0; u < R; u += RU)
            if (r0 + u < a.dk) {
                float w[RU];
                load_vec<RU>(k + t * a.k_tok + u, w);
#pragma unroll
                for (int r = 0; r < RU; ++r) kt[u + r] = w[r];
                if (a.out) {
                    load_vec<RU>(q + t * a.q_tok + u, w);
#pragma unroll
                    for (int r = 0; r < RU; ++r) qt[u + r] = w[r];
                }
            }
        if (in_cols) load_vec<VC>(v + t * a.v_tok, vt);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int c = 0; c < VC; ++c) {
                S[r][c] = fmaf(S[r][c], decay, kt[r] * vt[c]);
                o[c] = fmaf(qt[r], S[r][c], o[c]);
            }
        if (!a.out) continue;
#pragma unroll
        for (int d = LPR; d < kWave; d *= 2)
#pragma unroll
            for (int c = 0; c < VC; ++c) o[c] += __shfl_xor(o[c], d);
        if (lane < LPR)
#pragma unroll
            for (int c = 0; c < VC; ++c) part[t & 1][wave][col * VC + c] = o[c];
        __syncthreads();   // the buffer of token t is next written behind token t + 1's barrier
        if (threadIdx.x < LPR && in_cols) {
#pragma unroll
            for (int c = 0; c < VC; ++c) {
                const int at = col * VC + c;
                o[c] = a.scale * ((part[t & 1][0][at] + part[t & 1][1][at]) +
                                  (part[t & 1][2][at] + part[t & 1][3][at]));
            }
            store_vec<VC>(out + t * a.o_tok, o);
        }
    }
    if (!a.write_state || !in_cols) return;
#pragma unroll
    for (int r = 0; r < R; ++r)
        if (r0 + r < a.dk) store_vec<VC>(s + (int64_t)r * a.dv, S[r]);
}

template <typename XT, typename ST>
RecurrentPlan pick(int dk, bool wide) {
    constexpr int VC = 16 / sizeof(ST);
    // the smallest R whose lane groups cover dk rows
    if (wide) {
        if (dk <= 64) return {(const void *)recurrent<XT, ST, 16, 4>, 16 * VC, 256};
        if (dk <= 128) return {(const void *)recurrent<XT, ST, 16, 8>, 16 * VC, 256};
        return {(const void *)recurrent<XT, ST, 16, 16>, 16 * VC, 256};
    }
    if (dk <= 128) return {(const void *)recurrent<XT, ST, 8, 4>, 8 * VC, 256};
    return {(const void *)recurrent<XT, ST, 8, 8>, 8 * VC, 256};
}

}  // namespace

RecurrentPlan pick_recurrent(int x_bytes, int state_bytes, int dk, bool wide) {
    if (x_bytes == 4) return pick<float, float>(dk, wide);
    return state_bytes == 4 ? pick<Bf16, float>(dk, wide) : pick<Bf16, Bf16>(dk, wide);
}

}  // namespace laimpl

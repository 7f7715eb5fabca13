// What the kernels on the matrix cores share: operands of 16 x 16 x 32 products of bf16 and sums
// over lanes.  Lane (g, j) = (lane / 16, lane % 16) holds row (column) j of the left (right)
// operand at eight of the 32 places of the sum, which may be any, if both sides agree; of a
// result it holds column j, rows 4g to 4g + 3.  Internal; included by the .hip sources only.
#pragma once

#include "la_device.h"

namespace laimpl {
namespace {

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

// Four 32-bit values to bf16, and what that leaves of them: x - part, exact.  In the order of a
// result's registers the difference is a product with minus the identity (`minus`, of this lane),
// which costs the wavefront one issue where the vector unit would take eight.
__device__ __forceinline__ u32x2 part_of(f32x4 x) { return u32x2{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])}; }
__device__ __forceinline__ u32x2 minus_identity(int lane) {
    const uint32_t one = lane / 16 == lane % 16 / 4 ? 0xBF80u << 16 * (lane % 2) : 0u;
    return lane & 2 ? u32x2{0, one} : u32x2{one, 0};
}
__device__ __forceinline__ f32x4 less(f32x4 x, u32x2 part, u32x2 minus) {
    return __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(s16x4, minus), __builtin_bit_cast(s16x4, part), x,
                                                     0, 0, 0);
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

template <int CTRL, int ROWS>
__device__ __forceinline__ double add_from(double x) {
    const uint64_t w = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)w, CTRL, ROWS, 0xF, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(w >> 32), CTRL, ROWS, 0xF, false);
    return x + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// The sum over the lanes up to each one, by data moves between lanes: inside rows of 16 from 1, 2,
// 4 and 8 lanes before (zeros from outside), then row 0's to row 1 and 2's to 3, then 0 and 1's
// to 2 and 3.
__device__ __forceinline__ double running_sum(double x) {
    x = add_from<0x111, 0xF>(x);
    x = add_from<0x112, 0xF>(x);
    x = add_from<0x114, 0xF>(x);
    x = add_from<0x118, 0xF>(x);
    x = add_from<0x142, 0xA>(x);
    return add_from<0x143, 0xC>(x);
}

}  // namespace
}  // namespace laimpl

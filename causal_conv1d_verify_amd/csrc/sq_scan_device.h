// Device-side pieces that both kernels of the scan share.  Internal; included by sq_scan.hip and
// sq_prompt.hip only.
#pragma once

#include "la_device.h"
#include "sq_internal.h"

namespace sqimpl {
namespace {

using namespace laimpl;

constexpr int kChannels = 64;     // of a workgroup, 16 of a wavefront
constexpr float kLog2e = 1.4426950408889634f;

// Elements of 2 or 4 bytes in vectors that are aligned to an element only.
typedef uint32_t u32_2 __attribute__((ext_vector_type(1), aligned(2)));
typedef uint32_t u32x2_2 __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32x2_4 __attribute__((ext_vector_type(2), aligned(4)));
typedef uint32_t u32x4_4 __attribute__((ext_vector_type(4), aligned(4)));

// The NL consecutive elements from n0 on of a row of `count` (a multiple of 8), as they lie in memory.
// Four lanes share a row, from 0, NL, 2 NL and 3 NL on.  FITS: that is the row exactly, as for sq_scan.hip's
// rows of up to 32.  Otherwise runs may reach past it (its rows of 40 and 56, and sq_prompt.hip's, rounded up
// to sixteens, of 8, 24, 40 and 56): for quads behind the row its first is loaded, without a branch among
// loads, and `end` makes them 0, where the loads are waited for anyway.
template <typename XT, int NL, bool FITS = false>
struct Run {
    static constexpr int W = NL * (int)sizeof(XT) / 4;
    static_assert(FITS || NL % 4 == 0, "only quads are held against the row's end");
    uint32_t w[W];
    __device__ __forceinline__ void load(const XT *row, int n0, int count) {
        if constexpr (NL % 4 == 0) {
#pragma unroll
            for (int i = 0; i < NL; i += 4) {
                const XT *p = row + (FITS || n0 + i < count ? n0 + i : 0);
                if constexpr (sizeof(XT) == 2) {
                    const u32x2_2 v = load_as<false, u32x2_2>(p);
#pragma unroll
                    for (int e = 0; e < 2; ++e) w[i / 2 + e] = v[e];
                } else {
                    const u32x4_4 v = load_as<false, u32x4_4>(p);
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[i + e] = v[e];
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < NL; i += 2)
                if constexpr (sizeof(XT) == 2) {
                    w[i / 2] = load_as<false, u32_2>(row + n0 + i)[0];
                } else {
                    const u32x2_4 v = load_as<false, u32x2_4>(row + n0 + i);
                    w[i] = v[0], w[i + 1] = v[1];
                }
        }
    }
    __device__ __forceinline__ void end(int n0, int count) {
        if constexpr (!FITS)
#pragma unroll
            for (int i = 0; i < W; ++i) w[i] = n0 + i * NL / W / 4 * 4 < count ? w[i] : 0;
    }
    __device__ __forceinline__ float operator[](int i) const {
        if constexpr (sizeof(XT) == 2) return i & 1 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
        else return __uint_as_float(w[i]);
    }
};

// A state's run back, `left` of it.
template <typename ST, int NL>
__device__ __forceinline__ void store_run(ST *p, const float (&h)[NL], int left) {
    if constexpr (NL % 4 == 0) {
#pragma unroll
        for (int i = 0; i < NL; i += 4) {
            const float f[4] = {h[i], h[i + 1], h[i + 2], h[i + 3]};
            if (NL <= 8 || i < left) store_vec<4>(p + i, f);
        }
    } else {
#pragma unroll
        for (int i = 0; i < NL; i += 2)
            if constexpr (sizeof(ST) == 2) store_as<false>(p + i, pack_bf16(h[i], h[i + 1]));
            else store_as<false>(p + i, u32x2{__float_as_uint(h[i]), __float_as_uint(h[i + 1])});
    }
}

// What a step, or a sum of steps, makes of a rate: the state keeps 2^ of it.  0 times anything is 0 here: a
// step of nothing keeps a state also where its rate times log2 e is past fp32 (A of fp32's lowest value), and
// a rate of 0 keeps it where a sum of steps is.  One instruction (for which the compiler has no builtin), no
// slower than another product.
extern "C" __device__ float scan_mul_legacy(float, float) __asm("llvm.amdgcn.fmul.legacy");
__device__ __forceinline__ float exponent(float step, float rate) { return scan_mul_legacy(step, rate); }

// max(v, 0) + log(1 + e) with e = 2^(-|v| log2 e).  log(1 + e) = 2 artanh(s), s = e / (2 + e) <= 1/3: a
// polynomial in s^2 keeps its relative accuracy where e is small, as 1 + e would not.
__device__ __forceinline__ float softplus(float v) {
    const float e = __builtin_amdgcn_exp2f(__builtin_fabsf(v) * -kLog2e);
    const float s = e * __builtin_amdgcn_rcpf(2.0f + e);
    const float s2 = s * s;
    float p = 0.28191546f;
    p = fmaf(p, s2, 0.27957666f);
    p = fmaf(p, s2, 0.40025115f);
    p = fmaf(p, s2, 0.6666631f);
    p = fmaf(p, s2, 2.0f);
    return fmaf(p, s, __int_as_float(max(__float_as_int(v), 0)));   // (and NaN stays)
}

// z / (1 + 2^(-z log2 e)).  Where its sigmoid is below fp32's normal range (z under -87) it is 0.
__device__ __forceinline__ float gate(float z) {
    return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -kLog2e));
}

}  // namespace
}  // namespace sqimpl

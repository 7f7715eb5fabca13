// Device-side pieces that both kernels of the scan share.  Internal; included by sq_scan.hip and
// sq_prompt.hip only.
#pragma once

#include "la_device.h"
#include "sq_internal.h"

namespace sqimpl {
namespace {

using namespace laimpl;

constexpr int kStage = 16;        // tokens
constexpr int kChannels = 64;     // of a workgroup, 16 of a wavefront
constexpr float kLog2e = 1.4426950408889634f;

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
    // The run from n0 on of a row of `count`; quads past the row are its first one instead.
    __device__ __forceinline__ void load_near(const XT *row, int n0, int count) {
        static_assert(NL % 4 == 0);
#pragma unroll
        for (int i = 0; i < NL; i += 4) {
            const XT *p = row + (n0 + i < count ? n0 + i : 0);
            if constexpr (sizeof(XT) == 2) {
                const u32x2_2 v = *reinterpret_cast<const u32x2_2 *>(p);
                w[i / 2] = v[0], w[i / 2 + 1] = v[1];
            } else {
                const u32x4_4 v = *reinterpret_cast<const u32x4_4 *>(p);
                w[i] = v[0], w[i + 1] = v[1], w[i + 2] = v[2], w[i + 3] = v[3];
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
    return fmaf(p, s, __builtin_amdgcn_fmed3f(v, 0.0f, INFINITY));
}

// z / (1 + 2^(-z log2 e)).  Where its sigmoid is below fp32's normal range (z under -87) it is 0.
__device__ __forceinline__ float gate(float z) {
    return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -kLog2e));
}

}  // namespace
}  // namespace sqimpl

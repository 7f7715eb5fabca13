// Device-side helpers shared by the kernels of liblinattn.so.  Internal; included by the .hip
// sources only.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "cv_device.h"
#include "la_internal.h"

namespace laimpl {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

struct Bf16 { uint16_t bits; };

// Two floats to packed bf16, to nearest even (one instruction on gfx950).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const bf16x2 p = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, p);
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// 4, 8 or 16 bytes; with STREAM past the caches' usual order, for what no cache can hold until it is
// read again.
template <bool STREAM, typename V>
__device__ __forceinline__ V load_as(const void *p) {
    if constexpr (STREAM) return __builtin_nontemporal_load(static_cast<const V *>(p));
    else return *static_cast<const V *>(p);
}
template <bool STREAM, typename V>
__device__ __forceinline__ void store_as(void *p, V x) {
    if constexpr (STREAM) __builtin_nontemporal_store(x, static_cast<V *>(p));
    else *static_cast<V *>(p) = x;
}

// N consecutive elements (N a multiple of 4 for float, 4 or a multiple of 8 for bf16) as floats.
template <int N, bool STREAM = false>
__device__ __forceinline__ void load_vec(const float *p, float (&f)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const f32x4 w = load_as<STREAM, f32x4>(p + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) f[i + j] = w[j];
    }
}
template <int N, bool STREAM = false>
__device__ __forceinline__ void load_vec(const Bf16 *p, float (&f)[N]) {
    if constexpr (N == 4) {
        const u32x2 w = load_as<STREAM, u32x2>(p);
#pragma unroll
        for (int j = 0; j < 2; ++j) f[2 * j] = bf16_lo(w[j]), f[2 * j + 1] = bf16_hi(w[j]);
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 8) {
            const u32x4 w = load_as<STREAM, u32x4>(p + i);
#pragma unroll
            for (int j = 0; j < 4; ++j) f[i + 2 * j] = bf16_lo(w[j]), f[i + 2 * j + 1] = bf16_hi(w[j]);
        }
    }
}
template <int N, bool STREAM = false>
__device__ __forceinline__ void store_vec(float *p, const float (&f)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const f32x4 w = {f[i], f[i + 1], f[i + 2], f[i + 3]};
        store_as<STREAM>(p + i, w);
    }
}
template <int N, bool STREAM = false>
__device__ __forceinline__ void store_vec(Bf16 *p, const float (&f)[N]) {
    if constexpr (N == 4) {
        const u32x2 w = {pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3])};
        store_as<STREAM>(p, w);
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 8) {
            const u32x4 w = {pack_bf16(f[i], f[i + 1]), pack_bf16(f[i + 2], f[i + 3]),
                             pack_bf16(f[i + 4], f[i + 5]), pack_bf16(f[i + 6], f[i + 7])};
            store_as<STREAM>(p + i, w);
        }
    }
}

// A log decay with -inf (and anything whose exp() is 0 many times over) made finite, so that
// differences of sums of decays stay defined; NaN stays NaN.
__device__ __forceinline__ float finite_decay(float g) { return g < -1e6f ? -1e6f : g; }

// A value that is the same in every lane, for the compiler to keep in scalar registers.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int64_t uniform(int64_t x) {
    const uint32_t lo = (uint32_t)uniform((int)(uint32_t)x), hi = (uint32_t)uniform((int)(x >> 32));
    return (int64_t)((uint64_t)hi << 32 | lo);
}

// Workgroups go round the chip's 8 dies in turn, each with an L2 of its own.  Blocks in sets of
// `set` that read the same q and k, in this order, lie on one die one after the other, and the sets
// go round the dies (prompts: 1-3% faster, a third of q's and k's traffic with three v heads to one).
__device__ __forceinline__ int shared_block(int b, int set, int blocks) {
    const int round = 8 * set;
    if (b >= blocks / round * round) return b;
    return b / round * round + b % 8 * set + b / 8 % set;
}

// One row of a batch: its token count (-1: skip the row), its slot and its first elements.
struct Row {
    int n;
    int64_t slot, q, k, v, o, g;
};
__device__ __forceinline__ Row uniform(const Row &r) {
    return Row{uniform(r.n), uniform(r.slot), uniform(r.q), uniform(r.k), uniform(r.v), uniform(r.o), uniform(r.g)};
}
__device__ __forceinline__ Row row_of(const AttnArgs &a, int i) {
    Row r;
    r.slot = a.slot_idx ? a.slot_idx[i] : i;
    int64_t first = 0, seq = i;
    r.n = a.T;
    if (a.cu_seqlens) {
        first = a.cu_seqlens[i];
        const int64_t n = (int64_t)a.cu_seqlens[i + 1] - first;
        r.n = n >= 0 && n <= a.T ? (int)n : -1;
        seq = 0;
    } else if (a.num_tokens) {
        const int n = a.num_tokens[i];
        r.n = n >= 0 && n <= a.T ? n : -1;
    }
    if (r.slot < 0 || r.slot >= a.n_slots) r.n = -1;
    r.q = seq * a.q_seq + first * a.q_tok;
    r.k = seq * a.k_seq + first * a.k_tok;
    r.v = seq * a.v_seq + first * a.v_tok;
    r.o = seq * a.o_seq + first * a.o_tok;
    r.g = seq * a.g_seq + first * a.g_tok;
    return r;
}

__device__ __forceinline__ float load_one(const float *p) { return *p; }
__device__ __forceinline__ float load_one(const Bf16 *p) { return __uint_as_float((uint32_t)p->bits << 16); }
__device__ __forceinline__ void store_one(float *p, float x) { *p = x; }
__device__ __forceinline__ void store_one(Bf16 *p, float x) {
    p->bits = __builtin_bit_cast(uint16_t, (__bf16)x);
}

// Segment `id` of the rows in order, each row cut into ceil(tokens / seg_len) of them and one
// where it has no tokens; row -1 where there are fewer.  Rows that are skipped have none, nor
// has a row that would end past a.segments or a.places (more tokens than the caller declared).
// `place` is the row's first place in the workspace, where rows of one segment have none.  Called
// by a whole workgroup of W wavefronts, `shared` is three words of LDS.
struct Segment { int row, index; bool last; int place; };
__device__ __forceinline__ int segments_of(const AttnArgs &a, int i) {
    const Row r = row_of(a, i);
    return r.n < 0 ? 0 : r.n == 0 ? 1 : (int)(((uint32_t)r.n + (uint32_t)a.seg_len - 1) / (uint32_t)a.seg_len);
}
__device__ __forceinline__ int places_of(int segments) { return segments > 1 ? segments : 0; }
template <int W>
__device__ __forceinline__ Segment find_segment(const AttnArgs &a, int id, int64_t *shared) {
    if (a.seg_len >= a.T) return row_of(a, id).n < 0 ? Segment{-1, 0, true, 0} : Segment{id, 0, true, 0};
    __shared__ int sums[2][W];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int64_t before = 0, places = 0;                // of the rows before these
    if (threadIdx.x == 0) shared[0] = -1;
    for (int i0 = 0; i0 < a.n_seq && before <= id; i0 += 64 * W) {
        const int i = i0 + threadIdx.x;
        const int own = i < a.n_seq ? segments_of(a, i) : 0, held = places_of(own);
        int upto = own, held_upto = held;
#pragma unroll
        for (int d = 1; d < kWave; d *= 2) {
            const int y = __shfl_up(upto, d), z = __shfl_up(held_upto, d);
            if (lane >= d) upto += y, held_upto += z;
        }
        __syncthreads();                           // the sums of the last turn are read
        if (lane == kWave - 1) sums[0][wave] = upto, sums[1][wave] = held_upto;
        __syncthreads();
        int64_t at = before + upto - own, place = places + held_upto - held;
        for (int w = 0; w < wave; ++w) at += sums[0][w], place += sums[1][w];
        if (id >= at && id < at + own && at + own <= a.segments && place + held <= a.places) {
            shared[0] = i;
            shared[1] = (id - at) * 2 + (id - at == own - 1);
            shared[2] = place;
        }
        for (int w = 0; w < W; ++w) before += sums[0][w], places += sums[1][w];
    }
    __syncthreads();
    const int64_t at = uniform(shared[1]);
    return Segment{uniform((int)shared[0]), (int)(at >> 1), (at & 1) != 0, uniform((int)shared[2])};
}

// The first place of row i in the workspace (i the same for the workgroup).
template <int W>
__device__ __forceinline__ int64_t first_place(const AttnArgs &a, int i) {
    __shared__ int64_t sums[W];
    int64_t own = 0;
    for (int r = threadIdx.x; r < i; r += 64 * W) own += places_of(segments_of(a, r));
#pragma unroll
    for (int d = kWave / 2; d > 0; d /= 2) own += __shfl_xor(own, d);
    if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = own;
    __syncthreads();
    int64_t all = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) all += sums[w];
    return uniform(all);
}

}  // namespace
}  // namespace laimpl

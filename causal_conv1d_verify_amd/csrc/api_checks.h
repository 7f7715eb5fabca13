// Shared by the host sides of liblinattn.so and libseqops.so (one translation unit of each): the
// error detail, checks of sizes, strides and pointers, and the launch.  Internal.
#pragma once

#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "conv_verify.h"

namespace {

thread_local char g_detail[512];

int fail(int code, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_detail, sizeof(g_detail), fmt, ap);
    va_end(ap);
    return code;
}

int dtype_bytes(int32_t dt) { return dt == CV_F32 ? 4 : dt == CV_BF16 ? 2 : 0; }
bool aligned(const void *p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// Size arithmetic on caller-supplied values (>= 0), saturating at INT64_MAX: the results are
// only compared against limits.
int64_t sat_mul(int64_t a, int64_t b) {
    int64_t r;
    return __builtin_mul_overflow(a, b, &r) ? INT64_MAX : r;
}
int64_t sat_add(int64_t a, int64_t b) {
    int64_t r;
    return __builtin_add_overflow(a, b, &r) ? INT64_MAX : r;
}

struct Dim { int64_t count, stride; };

// Whether the elements of an array are all apart: inner elements contiguous, then the
// dimensions of more than one index, by rising stride, each past what lies inside it.
bool apart(int64_t inner, Dim *dims, int n) {
    std::sort(dims, dims + n, [](const Dim &a, const Dim &b) { return a.stride < b.stride; });
    int64_t span = inner;
    for (int i = 0; i < n; ++i) {
        if (dims[i].count <= 1) continue;
        if (dims[i].stride < span) return false;
        span = sat_add(sat_mul(dims[i].count - 1, dims[i].stride), span);
    }
    return true;
}

struct Pointer { const char *name; const void *p; bool needed; int align; };

template <int N>
int check_pointers(const Pointer (&ps)[N]) {
    for (const auto &p : ps) {
        if (p.needed && !p.p) return fail(CV_EINVAL, "%s is NULL", p.name);
        if (p.p && !aligned(p.p, p.align))
            return fail(CV_ENOTSUP, "%s is not %d-byte aligned", p.name, p.align);
    }
    return CV_OK;
}

int launch(const void *fn, int64_t blocks, int threads, int64_t lds, void *args, void *stream, void *more = nullptr) {
    if (blocks > INT32_MAX) return fail(CV_ENOTSUP, "%lld workgroups in one launch", (long long)blocks);
    void *kargs[] = {args, more};
    const hipError_t e = hipLaunchKernel(fn, dim3((unsigned)blocks), dim3((unsigned)threads), kargs,
                                         (size_t)lds, (hipStream_t)stream);
    if (e != hipSuccess)
        return fail(CV_EHIP_BASE - (int)e, "kernel launch failed: %s", hipGetErrorString(e));
    return CV_OK;
}

}  // namespace

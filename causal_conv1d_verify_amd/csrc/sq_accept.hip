// The verdict on a row's drafts and the token behind the accepted ones.
//
// What it has to read is the one row of probabilities (with a draft two) that the next token is drawn
// from, and at most 31 single ones.  Which row that is only the verdict tells, so every workgroup
// makes it for itself, in one wavefront: lane t holds token t, its parent and both probabilities, a
// chain's verdict is the number of ones in front of a ballot, a tree's a walk over ballots of children.
//
// `sums` has a wavefront add up kPart weights each, over the whole card also for a single row; `pick`,
// one workgroup a row, finds the part and then the weight at which the running sum passes the given
// share of the total.  Sums are fp64, in an order that the sizes alone set.
//
// 128 rows of 128000 probabilities with drafts, 122 MB: 23 us, the copy's rate.  A few rows are latency: 7.8 us, 4.0
// and 3.0 of the two kernels, three dependent loads each.  All of a row in one workgroup of 16 wavefronts and
// one launch was no faster for 4000 probabilities (8.1 us for 8.2) and slower for more (32000: 10.0 for 8.8).
#include "la_device.h"
#include "sq_internal.h"

namespace sqimpl {
namespace {

using namespace laimpl;

__device__ __forceinline__ double lane_value(double v, int lane) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)b, lane), hi = __builtin_amdgcn_readlane((uint32_t)(b >> 32), lane);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Row i's verdict, by one wavefront; `tell`: it goes to the outputs and to the workspace too.
template <typename PT>
__device__ __forceinline__ void judge(const AcceptArgs &a, int i, bool tell, Verdict *v) {
    const int t = threadIdx.x & 63;
    const bool in = t < a.T;
    const int token = in ? a.tokens[i * a.tokens_row + t] : -1;
    const int parent = in ? a.parent ? a.parent[i * a.parent_row + t] : t - 1 : -2;
    const bool bad = in && (parent < -1 || parent >= (t ? t : 0));
    const bool skip = (a.slot_idx && a.slot_idx[i] < 0) || __builtin_amdgcn_ballot_w64(bad) != 0;
    const bool tried = in && t > 0 && !bad && parent >= 0 && token >= 0 && token < a.vocab;
    double p = 0.0, q = 1.0, u = 0.0;
    if (tried) {
        p = load_one(static_cast<const PT *>(a.target) + i * a.target_seq + parent * a.target_tok + token);
        if (a.draft) q = load_one(static_cast<const PT *>(a.draft) + i * a.draft_seq + parent * a.draft_tok + token);
        u = a.uniform[i * a.uniform_row + t - 1];
    }
    int last = 0;
    uint64_t way = 1, gone = 0;
    bool against = false;
    if (!a.parent) {
        const uint64_t ok = __builtin_amdgcn_ballot_w64(tried && u * q < p);
        last = __builtin_ctzll(~(ok >> 1));
        way = (2ull << last) - 1;
        const uint64_t child = __builtin_amdgcn_ballot_w64(tried) & (2ull << last);
        against = a.draft && child;
        if (!a.draft) gone = child;
    } else {
        bool more = true;
        while (more) {                             // at each turn the current token has moved on
            more = false;
            double left = 1.0;
            gone = 0;
            uint64_t children = __builtin_amdgcn_ballot_w64(tried && parent == last);
            while (children) {
                const int j = __builtin_ctzll(children);
                children &= children - 1;
                const int its = __builtin_amdgcn_readlane(token, j);
                if (__builtin_amdgcn_ballot_w64((gone >> t & 1) && token == its)) continue;
                const double pj = lane_value(p, j);
                if (lane_value(u, j) * left < pj) {
                    last = j;
                    way |= 1ull << j;
                    more = true;
                    break;
                }
                left -= pj;
                gone |= 1ull << j;
            }
        }
    }
    const int num = skip ? 0 : __builtin_popcountll(way), removed = __builtin_popcountll(gone);
    auto put = [&](Verdict *to) {
        if (gone >> t & 1) to->token[__builtin_popcountll(gone & ((1ull << t) - 1))] = token;
        if (t == 0) to->num = num, to->last = last, to->against = against, to->removed = removed;
    };
    put(v);
    if (!tell) return;
    put(a.verdicts + i);
    if (skip) return;
    if (a.path && in) {
        if (way >> t & 1) a.path[i * a.path_row + __builtin_popcountll(way & ((1ull << t) - 1))] = t;
        if (t >= num) a.path[i * a.path_row + t] = -1;
    }
    if (t == 0) {
        a.num[i] = num;
        if (a.last) a.last[i] = last;
    }
}

// The weights of four neighbouring tokens from `at` on, those past the vocabulary 0.
typedef float f32x4_4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x2_2 __attribute__((ext_vector_type(2), aligned(2)));
__device__ __forceinline__ f32x4 four(const float *p, int at, int vocab) {
    if (at + 4 <= vocab) return *reinterpret_cast<const f32x4_4 *>(p + at);
    f32x4 f = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 3; ++e)
        if (at + e < vocab) f[e] = p[at + e];
    return f;
}
__device__ __forceinline__ f32x4 four(const Bf16 *p, int at, int vocab) {
    if (at + 4 <= vocab) {
        const u32x2_2 w = *reinterpret_cast<const u32x2_2 *>(p + at);
        return f32x4{bf16_lo(w[0]), bf16_hi(w[0]), bf16_lo(w[1]), bf16_hi(w[1])};
    }
    f32x4 f = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 3; ++e)
        if (at + e < vocab) f[e] = load_one(p + at + e);
    return f;
}

// What row i's next token is drawn from.
template <typename PT>
struct Weights {
    const PT *p, *q;              // q NULL: p alone
    int vocab, removed;
    const int *token;
    __device__ __forceinline__ Weights(const AcceptArgs &a, int i, const Verdict &v)
        : p(static_cast<const PT *>(a.target) + i * a.target_seq + v.last * a.target_tok),
          q(v.against ? static_cast<const PT *>(a.draft) + i * a.draft_seq + v.last * a.draft_tok : nullptr),
          vocab(a.vocab), removed(v.removed), token(v.token) {}
    struct Raw { f32x4 p, q; };
    __device__ __forceinline__ Raw load(int at) const {
        Raw r;
        r.p = four(p, at, vocab);
        r.q = q ? four(q, at, vocab) : f32x4{0, 0, 0, 0};
        return r;
    }
    __device__ __forceinline__ void of(const Raw &r, double (&w)[4]) const {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const double x = (double)r.p[e] - (double)r.q[e];
            w[e] = x > 0.0 && x < (double)INFINITY ? x : 0.0;
        }
    }
    // tokens tried, among those from `begin` up to `end`
    __device__ __forceinline__ bool any_removed(int begin, int end) const {
        bool any = false;
        for (int r = 0; r < removed; ++r) any |= token[r] >= begin && token[r] < end;
        return any;
    }
    __device__ __forceinline__ void take_removed(int at, double (&w)[4]) const {
        for (int r = 0; r < removed; ++r)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (token[r] == at + e) w[e] = 0.0;
    }
};

// The value of the lane that CTRL names, in the rows that ROWS has, and 0 in others: DPP moves, a few
// cycles each where a shuffle through LDS takes some sixty.
template <int CTRL, int ROWS>
__device__ __forceinline__ double moved(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS, 0xF, true);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROWS, 0xF, true);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// The running sums over a wavefront: of each row of 16 lanes, then with the rows before.
__device__ __forceinline__ double wave_upto(double s) {
    s += moved<0x111, 0xF>(s);    // the lane before
    s += moved<0x112, 0xF>(s);    // two, four and eight before
    s += moved<0x114, 0xF>(s);
    s += moved<0x118, 0xF>(s);
    s += moved<0x142, 0xA>(s);    // the last of the row before, in the second and the fourth
    s += moved<0x143, 0xC>(s);    // the last of the second, in the third and the fourth
    return s;
}

// The sum of part `part`'s weights, by one wavefront.
template <typename PT>
__device__ __forceinline__ double part_sum(const Weights<PT> &weights, int part) {
    constexpr int PER = kPart / (4 * kWave);
    const int lane = threadIdx.x & 63, begin = part * kPart;
    typename Weights<PT>::Raw raw[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) raw[k] = weights.load(begin + 4 * (lane + kWave * k));
    const bool slow = weights.any_removed(begin, begin + kPart);
    double s = 0.0;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        double w[4];
        weights.of(raw[k], w);
        if (slow) weights.take_removed(begin + 4 * (lane + kWave * k), w);
        s += (w[0] + w[1]) + (w[2] + w[3]);
    }
    return lane_value(wave_upto(s), kWave - 1);
}

template <typename PT>
__global__ __launch_bounds__(256) void sums(const AcceptArgs a) {
    __shared__ Verdict v;
    const int chunk = blockIdx.x % a.chunks, i = blockIdx.x / a.chunks;
    const int wave = uniform((int)(threadIdx.x >> 6));
    if (wave == 0) judge<PT>(a, i, chunk == 0, &v);
    __syncthreads();
    if (v.num == 0) return;                        // same for the workgroup
    const Weights<PT> weights(a, i, v);
    const int part = chunk * 4 + wave;
    if (part >= a.parts) return;
    const double s = part_sum(weights, part);
    if ((threadIdx.x & 63) == 0) a.sums[(int64_t)i * a.parts + part] = s;
}

// The running sums of each lane's `own` over the workgroup's 256 lanes: what is before it, and all.
__device__ __forceinline__ double before_lane(double own, double *waves, double &all) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const double upto = wave_upto(own), y = moved<0x138, 0xF>(upto);   // (of the lane before)
    __syncthreads();                               // the last sums are read
    if (lane == kWave - 1) waves[wave] = upto;
    __syncthreads();
    double base = 0.0;
    all = 0.0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        if (w < wave) base += waves[w];
        all += waves[w];
    }
    return base + y;
}

// Of the workgroup's lanes in order, the value of the first that has one, and that of the last that
// has another; -1 where none has.
struct Ends { int first, last; };
__device__ __forceinline__ Ends ends_of(bool first, int value, bool last, int other, int (*slots)[4]) {
    const int wave = threadIdx.x >> 6;
    const uint64_t f = __builtin_amdgcn_ballot_w64(first), l = __builtin_amdgcn_ballot_w64(last);
    const int from = __builtin_amdgcn_readlane(value, f ? __builtin_ctzll(f) : 0);
    const int to = __builtin_amdgcn_readlane(other, l ? 63 - __builtin_clzll(l) : 0);
    if ((threadIdx.x & 63) == 0) slots[0][wave] = f ? from : -1, slots[1][wave] = l ? to : -1;
    __syncthreads();
    Ends e{-1, -1};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        if (e.first < 0) e.first = slots[0][w];
        if (slots[1][w] >= 0) e.last = slots[1][w];
    }
    return e;
}

template <typename PT>
__global__ __launch_bounds__(256) void pick(const AcceptArgs a) {
    __shared__ Verdict v;
    __shared__ double waves[4], start;
    __shared__ int slots[2][2][4];
    const int i = blockIdx.x, tid = threadIdx.x, wave = uniform(tid >> 6);
    double *sums = a.sums + (int64_t)i * a.parts;
    const int per = (a.parts + 255) / 256;
    const int first = tid * per < a.parts ? tid * per : a.parts, last = first + per < a.parts ? first + per : a.parts;
    double own = 0.0, base, all;
    for (int k = first; k < last; ++k) own += sums[k];
    const double share = a.uniform[i * a.uniform_row + a.T - 1];
    if (tid < (int)(sizeof(Verdict) / 4)) reinterpret_cast<int *>(&v)[tid] = reinterpret_cast<const int *>(a.verdicts + i)[tid];
    __syncthreads();
    if (v.num == 0) return;                        // same for the workgroup
    Weights<PT> weights(a, i, v);
    base = before_lane(own, waves, all);
    if (!(all > 0.0) && (weights.q || weights.removed)) {
        // nothing is left beside the tokens tried: the target's own probabilities
        weights.q = nullptr;
        weights.removed = 0;
        for (int k = wave; k < a.parts; k += 4) {
            const double s = part_sum(weights, k);
            if ((tid & 63) == 0) sums[k] = s;
        }
        __syncthreads();                           // (the row's sums are this workgroup's alone)
        own = 0.0;
        for (int k = first; k < last; ++k) own += sums[k];
        base = before_lane(own, waves, all);
    }
    if (!(all > 0.0)) {
        if (tid == 0) a.next[i] = -1;
        return;
    }
    const double passed = share * all;

    // ---- the part
    int over = -1, some = -1;
    double at = base;
    for (int k = first; k < last && over < 0; ++k) {
        const double s = sums[k];
        if (s > 0.0) some = k;
        // (`base` may be past `passed` where the sums before it, in their own order, are not: an empty
        // part is not the one)
        if ((s > 0.0) & (at + s > passed)) over = k;
        else at += s;
    }
    const Ends parts = ends_of(over >= 0, over, some >= 0, some, slots[0]);
    const bool none = parts.first < 0;             // rounding: the last weight that there is
    const int part = none ? parts.last : parts.first;
    if (part >= first && part < last) {
        double s = base;
        for (int k = first; k < part; ++k) s += sums[k];
        start = s;
    }

    // ---- the weight
    const int begin = part * kPart;
    double w[4];
    weights.of(weights.load(begin + 4 * tid), w);
    if (weights.any_removed(begin, begin + kPart)) weights.take_removed(begin + 4 * tid, w);
    double whole;
    at = before_lane((w[0] + w[1]) + (w[2] + w[3]), waves, whole);
    at += start;                                   // written before the barriers of the sums
    over = some = -1;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        at += w[e];
        if (w[e] > 0.0) {
            some = 4 * tid + e;
            if (!none && over < 0 && at > passed) over = 4 * tid + e;
        }
    }
    const Ends which = ends_of(over >= 0, over, some >= 0, some, slots[1]);
    if (tid == 0) a.next[i] = begin + (which.first >= 0 ? which.first : which.last);
}

}  // namespace

AcceptPlan pick_accept(int p_bytes) {
    if (p_bytes == 4) return {(const void *)sums<float>, (const void *)pick<float>, 256, 4};
    return {(const void *)sums<Bf16>, (const void *)pick<Bf16>, 256, 4};
}

}  // namespace sqimpl

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
#include "la_device.h"
#include "sq_internal.h"

namespace sqimpl {
namespace {

using namespace laimpl;

struct Verdict {
    int num, last;                // num 0: the row is skipped
    int against;                  // 1: the weights are what the draft leaves of the target
    int removed;                  // tokens tried without a draft, which weigh nothing
    uint64_t way;                 // the accepted tokens' places
    int token[32];
};

__device__ __forceinline__ double lane_value(double v, int lane) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)b, lane), hi = __builtin_amdgcn_readlane((uint32_t)(b >> 32), lane);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Row i's verdict, by one wavefront.
template <typename PT>
__device__ __forceinline__ void judge(const AcceptArgs &a, int i, Verdict *v) {
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
    int last = 0, removed = 0;
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
    removed = __builtin_popcountll(gone);
    if (gone >> t & 1) v->token[__builtin_popcountll(gone & ((1ull << t) - 1))] = token;
    if (t == 0) {
        v->num = skip ? 0 : __builtin_popcountll(way);
        v->last = last;
        v->against = against;
        v->removed = removed;
        v->way = way;
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

__device__ __forceinline__ double wave_sum(double s) {
#pragma unroll
    for (int d = kWave / 2; d > 0; d /= 2) s += __shfl_xor(s, d);
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
    return wave_sum(s);
}

template <typename PT>
__global__ __launch_bounds__(256) void sums(const AcceptArgs a) {
    __shared__ Verdict v;
    const int chunk = blockIdx.x % a.chunks, i = blockIdx.x / a.chunks;
    const int wave = uniform((int)(threadIdx.x >> 6));
    if (wave == 0) judge<PT>(a, i, &v);
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
    double upto = own;
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) {
        const double y = __shfl_up(upto, d);
        if (lane >= d) upto += y;
    }
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
    const double y = __shfl_up(upto, 1);
    return base + (lane ? y : 0.0);
}

template <typename PT>
__global__ __launch_bounds__(256) void pick(const AcceptArgs a) {
    __shared__ Verdict v;
    __shared__ double waves[4];
    __shared__ double start;
    __shared__ int found, final;
    const int i = blockIdx.x, tid = threadIdx.x, wave = uniform(tid >> 6);
    if (wave == 0) judge<PT>(a, i, &v);
    __syncthreads();
    if (v.num == 0) return;                        // same for the workgroup
    if (tid < a.T) {
        if (a.path) {
            if (v.way >> tid & 1) a.path[i * a.path_row + __builtin_popcountll(v.way & ((1ull << tid) - 1))] = tid;
            if (tid >= v.num) a.path[i * a.path_row + tid] = -1;
        }
        if (tid == 0) {
            a.num[i] = v.num;
            if (a.last) a.last[i] = v.last;
        }
    }
    Weights<PT> weights(a, i, v);
    double *sums = a.sums + (int64_t)i * a.parts;
    const double share = a.uniform[i * a.uniform_row + a.T - 1];
    const int per = (a.parts + 255) / 256;
    const int first = tid * per < a.parts ? tid * per : a.parts, last = first + per < a.parts ? first + per : a.parts;

    double own, base, all;
    for (bool again = false;; again = true) {
        own = 0.0;
        for (int k = first; k < last; ++k) own += sums[k];
        base = before_lane(own, waves, all);
        if (all > 0.0 || again || (!weights.q && !weights.removed)) break;
        // nothing is left beside the tokens tried: the target's own probabilities
        weights.q = nullptr;
        weights.removed = 0;
        for (int k = wave; k < a.parts; k += 4) {
            const double s = part_sum(weights, k);
            if ((tid & 63) == 0) sums[k] = s;
        }
        __syncthreads();                           // (the row's sums are this workgroup's alone)
    }
    if (!(all > 0.0)) {
        if (tid == 0) a.next[i] = -1;
        return;
    }
    const double passed = share * all;

    // ---- the part
    if (tid == 0) found = a.parts, final = -1;
    __syncthreads();
    double at = base;
    for (int k = first; k < last; ++k) {
        const double s = sums[k];
        if (s > 0.0) atomicMax(&final, k);
        if (at + s > passed) {
            atomicMin(&found, k);
            break;
        }
        at += s;
    }
    __syncthreads();
    const bool none = found == a.parts;            // rounding: the last weight that there is
    const int part = none ? final : found;
    if (part >= first && part < last) {
        double s = base;
        for (int k = first; k < part; ++k) s += sums[k];
        start = s;
    }
    __syncthreads();
    const double from = start;
    __syncthreads();
    if (tid == 0) found = 4 * 256, final = -1;
    __syncthreads();

    // ---- the weight
    const int begin = part * kPart;
    double w[4];
    weights.of(weights.load(begin + 4 * tid), w);
    if (weights.any_removed(begin, begin + kPart)) weights.take_removed(begin + 4 * tid, w);
    double whole;
    at = from + before_lane((w[0] + w[1]) + (w[2] + w[3]), waves, whole);
    bool over = false;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        at += w[e];
        if (w[e] > 0.0) atomicMax(&final, 4 * tid + e);
        if (!none && !over && at > passed && w[e] > 0.0) {
            atomicMin(&found, 4 * tid + e);
            over = true;
        }
    }
    __syncthreads();
    if (tid == 0) a.next[i] = begin + (found < 4 * 256 ? found : final);
}

}  // namespace

AcceptPlan pick_accept(int p_bytes) {
    if (p_bytes == 4) return {(const void *)sums<float>, (const void *)pick<float>, 256, 4};
    return {(const void *)sums<Bf16>, (const void *)pick<Bf16>, 256, 4};
}

}  // namespace sqimpl

// The selective scan of packed prompts, and of 8 and more tokens of each row: for each channel c and
// state n
//
//   h <- exp(delta A[c,n]) h + (delta x) B[n],   y = sum_n C[n] h + D x,   out = y silu(z)
//
// The decay is another one for every channel and state, so no product of matrices makes it: each
// state update is a multiply, an exponential and two multiply-adds on the vector units (4 + 8 + 4 + 4
// cycles of a wavefront).  They bound this kernel: 8 x 2048 tokens of 8192 channels with 16 states take 498
// us, of which the updates alone are 273 at 2.4 GHz; the stream of x, dt, z and out would take 204.  A
// wavefront has 402 vector instructions for 64 updates of a lane, 256 of them theirs, 36 for each token of
// a channel (conversions, softplus, gate, the sum across lanes); the vector units are 82-90% busy, at 2.1 to
// 2.2 GHz.  What could be taken off them: the products (delta x) B are a rank-one product for each
// token, four tokens of 16 states x 16 channels in one matrix instruction beside them (656 -> 591 us,
// together with the layout below).
//
// A wavefront has 16 channels from a segment's first token to its last, lane l channel l % 16 and, of
// every 16 states, the four from 4 (l / 16) on; tokens go in groups of four, of which lane l loads x, dt
// and z of token l / 16 and makes its delta and gate.  The deltas of a group come back through LDS in
// one vector, as C does (a stage of 16 tokens, converted once).  The four lanes' sums of four tokens
// are added and dealt out in three lane swaps, to the lane that has the token.  Loads are a stage
// ahead, without branches among them and waited for alone (591 -> 494 us with the instructions that
// this saves).  No barrier: wavefronts are alone, four on a SIMD (of NT 1).
//
// States come in sixteens: 8, 24, 40 and 56 of them take the time of 16, 32, 48 and 64, with zeros in the last
// places (8 x 1024 tokens of 8192 channels: 249 and 253 us with 8 and 16 states, 408 and 409 with 24 and
// 32, 596 with 40 and 48, 831 with 56 and 64).
//
// Where rows are cut, `first` passes over all segments but a row's last one for what each adds to a state
// of zeros, and each segment joins those before it: 1 x 16384 tokens of 4096 channels 418 us, 166 and 252
// of the two kernels; uncut a token takes 99 ns.
//
// Tried and slower: the sums with C as 4 x 4 x 1 matrix instructions (678 us for 540: each keeps the SIMD for
// some 13 cycles); the few tokens' states brought to their lanes through LDS from whole runs (128 rows of 8
// tokens: 64.7 us for 59.4).
#include "sq_scan_device.h"

namespace sqimpl {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));

// p[i] of lanes 16 g + j for the four g added up, token i's on the lanes of g = i.
__device__ __forceinline__ float deal_sums(const float (&p)[4]) {
    auto swap32 = [](float a, float b) {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
        return __uint_as_float(r[0]) + __uint_as_float(r[1]);
    };
    const float even = swap32(p[0], p[2]), odd = swap32(p[1], p[3]);   // tokens 0 | 2, 1 | 3
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(even), __float_as_uint(odd), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// The elements of a segment's tokens that a wavefront loads or stores in groups of four tokens, each
// through a buffer resource that ends with the segment's last token: loads past it are 0 (or, where a
// token's stride is below its width, of what overlaps with it), and stores are dropped, as at the
// offset kNowhere.
constexpr uint32_t kNowhere = 0x80000000u;
template <typename XT>
struct Tokens {
    const XT *p;
    uint32_t tok, width;          // of a token; four tokens lie within 2 GiB
    __device__ __forceinline__ uint32_t offset(int token, int element) const {
        return (token * tok + element) * (uint32_t)sizeof(XT);
    }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t from(int s4, int n) const {
        const int left = n - s4 < 4 ? n - s4 : 4;
        const uint32_t bytes = ((left - 1) * tok + width) * (uint32_t)sizeof(XT);
        return cvimpl::make_rsrc(p + (int64_t)s4 * tok, left > 0 ? bytes : 0u);
    }
};
template <typename XT>
__device__ __forceinline__ XT load_from(__amdgpu_buffer_rsrc_t r, uint32_t offset) {
    if constexpr (sizeof(XT) == 2) return __builtin_bit_cast(XT, __builtin_amdgcn_raw_buffer_load_b16(r, (int)offset, 0, 0));
    else return __builtin_bit_cast(XT, __builtin_amdgcn_raw_buffer_load_b32(r, (int)offset, 0, 0));
}
template <typename XT>
__device__ __forceinline__ void store_to(__amdgpu_buffer_rsrc_t r, uint32_t offset, float y) {
    XT v;
    store_one(&v, y);
    if constexpr (sizeof(XT) == 2) __builtin_amdgcn_raw_buffer_store_b16(v.bits, r, (int)offset, 0, 0);
    else __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), r, (int)offset, 0, 0);
}

// What a launch makes.  PROMPT: the outputs and the last state of packed prompts.  FIRST: what each
// segment of a cut row adds to a state of zeros, and the row's first state, in the workspace.  FEW: the
// outputs of up to 32 tokens and, if it is wanted, the state behind them.
enum { PROMPT, FIRST, FEW };

// NT: sixteens of states; K: groups of four tokens in a stage.
template <typename XT, typename ST, int NT, int K, int MAKES>
__global__ __launch_bounds__(256, NT == 1 ? 4 : NT == 2 ? 3 : 2) void prompt(const ScanArgs a) {
    constexpr int NP = 16 * NT, NL = 4 * NT, STAGE = 4 * K;
    constexpr bool OUT = MAKES == PROMPT || MAKES == FEW, CUTS = MAKES == PROMPT || MAKES == FIRST;
    __shared__ alignas(16) float deltas[4][K][16][4];             // [wave][group][channel][token]
    __shared__ alignas(16) float cs[4][OUT ? STAGE : 1][OUT ? NP : 4];
    __shared__ int64_t found[CUTS ? 3 : 1];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int j = lane & 15, g = lane >> 4;
    const int tile = uniform((int)(blockIdx.x % a.tiles)), id = uniform((int)(blockIdx.x / a.tiles));
    Segment seg{id, 0, true, 0};
    if constexpr (CUTS) seg = find_segment<4>(a, id, found);
    if (seg.row < 0) return;                       // same for the workgroup
    Span row = span_of(a, seg.row);
    row = Span{uniform(row.n), uniform(row.slot), uniform(row.first), uniform(row.seq)};
    const bool init = !CUTS || !a.has_init || uniform(a.has_init[seg.row]) != 0;
    const bool cut = CUTS && (!seg.last || seg.index > 0);
    if (MAKES == FIRST && !cut) return;
    if (row.n < 0 || (row.n == 0 && (init || !a.write_state))) return;
    const int c0 = tile * kChannels + 16 * wave;
    if (c0 >= a.d) return;                         // a whole wavefront
    const bool own = c0 + j < a.d;
    const int c = own ? c0 + j : a.d - 1;

    // ---- the states that enter
    ST *state = static_cast<ST *>(a.state) + row.slot * a.s_slot + (int64_t)c * a.d_state + 4 * g;
    float h[NT][4], decay[NT][4];
#pragma unroll
    for (int q = 0; q < NT; ++q)
#pragma unroll
        for (int r = 0; r < 4; ++r) h[q][r] = decay[q][r] = 0.0f;
    auto from_pool = [&]() {
#pragma unroll
        for (int q = 0; q < NT; ++q)
            if (16 * q + 4 * g < a.d_state) load_vec<4>(state + 16 * q, h[q]);
    };
    auto place = [&](int index) {
        return ((int64_t)(seg.place + index) * a.tiles + tile) * 256 + tid;
    };
    auto from_workspace = [&](int index) {
        const float *ws = a.ws + place(index) * NL;
#pragma unroll
        for (int q = 0; q < NT; ++q) load_vec<4>(ws + 4 * q, h[q]);
    };
    auto to_workspace = [&]() {
        float *ws = a.ws + place(seg.index) * NL;
#pragma unroll
        for (int q = 0; q < NT; ++q) store_vec<4>(ws + 4 * q, h[q]);
    };
    if (MAKES == FIRST) {
        if (seg.last) {                            // the row's first state, in its last place
            if (init) from_pool();
            to_workspace();
            return;
        }
    } else if (cut) {
        from_workspace(segments_of(a, seg.row) - 1);
    } else if (init) {
        from_pool();
    }
#pragma unroll
    for (int q = 0; q < NT; ++q)
        if (16 * q + 4 * g < a.d_state) {
            load_vec<4>(a.A + (int64_t)c * a.d_state + 16 * q + 4 * g, decay[q]);
#pragma unroll
            for (int r = 0; r < 4; ++r) decay[q][r] *= kLog2e;
        }
    if (MAKES == PROMPT && cut) {                  // and what the segments before this one add to them
        constexpr int AHEAD = NT == 1 ? 8 : NT == 2 ? 4 : 2;   // segments that are in flight at once
        for (int s0 = 0; s0 < seg.index; s0 += AHEAD) {
            float add[AHEAD][NT][4], total[AHEAD];
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) {
                const int64_t from = place(s0 + u < seg.index ? s0 + u : seg.index - 1);
                total[u] = a.ws_total[from];
#pragma unroll
                for (int q = 0; q < NT; ++q) load_vec<4>(a.ws + from * NL + 4 * q, add[u][q]);
            }
#pragma unroll
            for (int u = 0; u < AHEAD; ++u)
                if (s0 + u < seg.index)
#pragma unroll
                    for (int q = 0; q < NT; ++q)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            // 2^e in two factors: a whole segment's may leave fp32's range where the state
                            // does not, and 0 stays 0 (a token's delta that is not finite is in `add` as well)
                            const float e = __builtin_amdgcn_fmed3f(exponent(total[u], decay[q][r]), -1024.0f, 1024.0f);
                            const float whole = rintf(e), grown = h[q][r] * __builtin_amdgcn_exp2f(e - whole);
                            h[q][r] = __builtin_ldexpf(grown, (int)whole) + add[u][q][r];
                        }
        }
    }
    const float bias = a.dt_bias ? a.dt_bias[c] : 0.0f, skip = OUT && a.D ? a.D[c] : 0.0f;

    // ---- the tokens
    const int begin = CUTS ? seg.index * a.seg_len : 0;
    const int n = !CUTS || row.n - begin < a.seg_len ? row.n - begin : a.seg_len;
    const int64_t t0 = row.first + begin;
    auto tokens_of = [&](const void *p, int64_t seq, int64_t tok, int width) {
        return Tokens<XT>{static_cast<const XT *>(p) + row.seq * seq + t0 * tok, (uint32_t)tok, (uint32_t)width};
    };
    const Tokens<XT> x = tokens_of(a.x, a.x_seq, a.x_tok, a.d), dt = tokens_of(a.dt, a.dt_seq, a.dt_tok, a.d);
    const Tokens<XT> z = a.z ? tokens_of(a.z, a.z_seq, a.z_tok, a.d) : x, out = tokens_of(a.out, a.o_seq, a.o_tok, a.d);
    const Tokens<XT> B = tokens_of(a.B, a.b_seq, a.b_tok, a.d_state);
    const uint32_t off_x = own ? x.offset(g, c) : kNowhere, off_dt = own ? dt.offset(g, c) : kNowhere;
    const uint32_t off_z = own ? z.offset(g, c) : kNowhere, off_out = own ? out.offset(g, c) : kNowhere;
    const uint32_t off_b = B.offset(g, j);
    const int tc = (lane >> 2) % STAGE, n0 = (lane & 3) * NL;   // C: the token of the stage and the states that this lane brings
    const XT *C = OUT ? static_cast<const XT *>(a.C) + row.seq * a.c_seq + t0 * a.c_tok : nullptr;
    const uint32_t off_c = tc * (uint32_t)a.c_tok;
    XT next_x[K], next_dt[K], next_z[K], next_b[K][NT];
    Run<XT, NL> next_c;
    // The stage from token s on.  There is no branch among its loads, which would wait for them:
    // past the row's end C is the last token's, for outputs that nobody has.
    auto fetch = [&](int s) {
        if constexpr (OUT) {
            const XT *p = C + s * a.c_tok + off_c;
            if (s + STAGE > n) p = C + (int64_t)(s + tc < n ? s + tc : n - 1) * a.c_tok;
            next_c.load(p, n0, a.d_state);
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int s4 = s + 4 * k;
            next_x[k] = load_from<XT>(x.from(s4, n), off_x);
            next_dt[k] = load_from<XT>(dt.from(s4, n), off_dt);
            if constexpr (OUT) next_z[k] = load_from<XT>(z.from(s4, n), off_z);
            const auto b = B.from(s4, n);
#pragma unroll
            for (int q = 0; q < NT; ++q)
                next_b[k][q] = load_from<XT>(b, 16 * q + j < a.d_state ? off_b + 16 * q * (uint32_t)sizeof(XT) : kNowhere);
        }
    };
    float total = 0.0f;
    if (n > 0) fetch(0);                           // (a row of no tokens has no last one to load)
    // The first stage's loads are waited for here: with none under way into the loop, its own wait is for
    // a stage's loads alone and not for the stores behind them.
    if (CUTS) __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
    for (int s = 0; s < n; s += STAGE) {
        float xv[K], dx[K], gates[K], b[K][NT];
        // LDS of a wavefront is written and read in its own order
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if constexpr (OUT) {
            next_c.end(n0, a.d_state);
#pragma unroll
            for (int i = 0; i < NL; i += 4) {
                const float f[4] = {next_c[i], next_c[i + 1], next_c[i + 2], next_c[i + 3]};
                store_vec<4>(&cs[wave][tc][n0 + i], f);
            }
        }
        float delta[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            xv[k] = load_one(&next_x[k]);
            if constexpr (OUT) gates[k] = load_one(&next_z[k]);
            delta[k] = load_one(&next_dt[k]) + bias;
#pragma unroll
            for (int q = 0; q < NT; ++q) b[k][q] = load_one(&next_b[k][q]);
        }
        if (a.softplus)
#pragma unroll
            for (int k = 0; k < K; ++k) delta[k] = softplus(delta[k]);
        if constexpr (OUT)
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const float open = gate(gates[k]);   // (without z that of x, which nobody has)
                gates[k] = a.z ? open : 1.0f;
            }
        if (s + STAGE > n)                        // past the last token nothing changes, whatever lies there
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const bool is = s + 4 * k + g < n;
                delta[k] = is ? delta[k] : 0.0f;
                xv[k] = is ? xv[k] : 0.0f;
#pragma unroll
                for (int q = 0; q < NT; ++q) b[k][q] = is ? b[k][q] : 0.0f;
            }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            deltas[wave][k][j][g] = delta[k];
            dx[k] = delta[k] * xv[k];
            if (MAKES == FIRST) total += delta[k];
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (CUTS || s + STAGE < n) fetch(s + STAGE);   // (past the row's end: no bytes)
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (!CUTS && s + 4 * k >= n) break;    // (prompts: no branch; tokens past the end change nothing)
            const f32x4 step = *reinterpret_cast<const f32x4 *>(deltas[wave][k][j]);
            float sum[4] = {};
#pragma unroll
            for (int q = 0; q < NT; ++q) {
                f32x16 add = {};
                add = __builtin_amdgcn_mfma_f32_16x16x1f32(b[k][q], dx[k], add, 0, 0, 0);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    f32x4 w = {};
                    if constexpr (OUT) w = *reinterpret_cast<const f32x4 *>(&cs[wave][4 * k + t][16 * q + 4 * g]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float keep = __builtin_amdgcn_exp2f(exponent(step[t], decay[q][r]));
                        h[q][r] = fmaf(h[q][r], keep, add[4 * t + r]);
                        if constexpr (OUT) sum[t] = fmaf(w[r], h[q][r], sum[t]);
                    }
                }
            }
            if constexpr (OUT) {
                const float y = deal_sums(sum), with = fmaf(skip, xv[k], y);
                store_to<XT>(out.from(s + 4 * k, n), off_out, (a.D ? with : y) * gates[k]);
            }
        }
    }
    if (MAKES == FIRST) {
        to_workspace();
        total += __shfl_xor(total, 16);
        a.ws_total[place(seg.index)] = total + __shfl_xor(total, 32);
        return;
    }
    if (seg.last && a.write_state && own)
#pragma unroll
        for (int q = 0; q < NT; ++q)
            if (16 * q + 4 * g < a.d_state) store_vec<4>(state + 16 * q, h[q]);
}

template <typename XT, typename ST, int NT>
PromptPlan plan() {
    return {(const void *)prompt<XT, ST, NT, 4, PROMPT>, (const void *)prompt<XT, ST, NT, 4, FIRST>,
            kChannels, 256, 16, 256 * 4 * NT, 256};
}
template <typename XT, typename ST, int NT>
ScanPlan plan_few(int T) {
    // The stage that leaves the fewest groups without a token: of 3 for 3, 5 and 6 groups of four tokens
    // (8 rows of 17: 9.5 us for 10.0 in stages of 4; 128 rows of 9: 91 for 102, of 17: 129 for 142).
    const int groups = (T + 3) / 4;
    const void *run = groups <= 2 ? (const void *)prompt<XT, ST, NT, 2, FEW>
                      : groups == 3 || groups == 5 || groups == 6 ? (const void *)prompt<XT, ST, NT, 3, FEW>
                                                                  : (const void *)prompt<XT, ST, NT, 4, FEW>;
    return {run, kChannels, 256};
}

template <typename XT, typename ST>
PromptPlan pick(int d_state) {
    if (d_state <= 16) return plan<XT, ST, 1>();
    if (d_state <= 32) return plan<XT, ST, 2>();
    if (d_state <= 48) return plan<XT, ST, 3>();
    return plan<XT, ST, 4>();
}
template <typename XT, typename ST>
ScanPlan pick_few(int d_state, int T) {
    if (d_state <= 16) return plan_few<XT, ST, 1>(T);
    if (d_state <= 32) return plan_few<XT, ST, 2>(T);
    if (d_state <= 48) return plan_few<XT, ST, 3>(T);
    return plan_few<XT, ST, 4>(T);
}

}  // namespace

PromptPlan pick_prompt(int x_bytes, int state_bytes, int d_state) {
    if (x_bytes == 4) return pick<float, float>(d_state);
    return state_bytes == 4 ? pick<Bf16, float>(d_state) : pick<Bf16, Bf16>(d_state);
}
ScanPlan pick_groups(int x_bytes, int state_bytes, int d_state, int T) {
    if (x_bytes == 4) return pick_few<float, float>(d_state, T);
    return state_bytes == 4 ? pick_few<Bf16, float>(d_state, T) : pick_few<Bf16, Bf16>(d_state, T);
}

}  // namespace sqimpl

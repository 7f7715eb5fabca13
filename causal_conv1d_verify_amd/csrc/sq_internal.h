// Shared by the host side (sq_api.cpp) and the kernels of libseqops.so: kernel arguments and the
// pickers that map a launch plan to a compiled kernel.  Internal.
#pragma once

#include <stdint.h>

namespace sqimpl {

// One batch of rows of the scan.  Strides in elements.
struct ScanArgs {
    const void *x, *dt, *z, *B, *C;     // z NULL: no gate
    const float *A, *D, *dt_bias;       // D, dt_bias NULL: 0
    void *state, *out;
    const int32_t *slot_idx;      // NULL: row i uses slot i
    const int32_t *cu_seqlens;    // packed rows, or NULL
    const int32_t *num_tokens;    // tokens of each row, or NULL (T)
    const int32_t *has_init;      // NULL: every row starts from its state
    int64_t x_seq, x_tok, dt_seq, dt_tok, z_seq, z_tok, b_seq, b_tok, c_seq, c_tok, o_seq, o_tok;
    int64_t s_slot;
    int32_t n_seq, T, d, d_state, n_slots;
    int32_t tiles;                // workgroups across the channels of a row
    int32_t softplus, write_state;
    // prompts: a row is cut into segments of seg_len tokens (a multiple of the stage; rows of at
    // most seg_len tokens are one)
    int32_t seg_len, segments;    // segments that the grid holds
    int32_t places;               // segments of cut rows that the workspace holds
    float *ws;                    // what each segment adds to a state (a row's last: the row's
                                  // first state)
    float *ws_total;              // each channel's sum of delta over each
};

// Up to 32 tokens of each row (one: a single one; out false: the state only).
struct ScanPlan {
    const void *run;
    int channels, threads;              // of a workgroup
};
ScanPlan pick_scan(int x_bytes, int state_bytes, int d_state, bool one, bool out);
ScanPlan pick_groups(int x_bytes, int state_bytes, int d_state, int T);

// Packed prompts.  run makes the outputs and the last state; where rows are cut, first leaves what
// each segment adds to a state of zeros, and the row's first state, in the workspace.
struct PromptPlan {
    const void *run, *first;
    int channels, threads, stage;       // of a workgroup; tokens of a stage
    int64_t ws_floats, total_floats;    // of one workgroup's state, and of its sums of delta
};
PromptPlan pick_prompt(int x_bytes, int state_bytes, int d_state);

struct RotaryArgs {
    const void *x[2], *weight[2];       // q, k
    void *out[2];
    const void *positions;
    const float *inv_freq;
    int64_t tok[2], head[2], out_tok[2], out_head[2];
    int64_t tokens;
    int32_t heads[2], dim, rot;
    int32_t blocks_per_token;           // wavefronts that share a token's heads
    float eps;
    int32_t interleaved, wide;
};
struct RotaryPlan {
    const void *fn;
    int threads, heads;                 // wavefronts of a workgroup times 64; heads side by side in one
};
RotaryPlan pick_rotary(int x_bytes, int dim);

// What is known of a row before its next token is drawn.
struct Verdict {
    int32_t num, last;                  // num 0: the row is skipped
    int32_t against;                    // 1: the weights are what the draft leaves of the target
    int32_t removed;                    // tokens tried without a draft, which weigh nothing
    int32_t token[32];                  // they
};
struct AcceptArgs {
    const int32_t *tokens, *parent;
    const void *target, *draft;
    const float *uniform;
    const int32_t *slot_idx;
    int32_t *num, *next, *last, *path;
    int64_t tokens_row, parent_row, uniform_row, path_row, target_seq, target_tok, draft_seq, draft_tok;
    Verdict *verdicts;                  // [n_seq]
    double *sums;                       // [n_seq, parts]: of kPart consecutive weights each
    int32_t n_seq, T, vocab, parts, chunks;
};
constexpr int kPart = 1024;             // weights of one sum of the workspace
struct AcceptPlan {
    const void *sums, *pick;
    int threads, parts;                 // of a workgroup of `sums`
};
AcceptPlan pick_accept(int p_bytes);

}  // namespace sqimpl

// Shared by the host side (la_api.cpp) and the kernels of liblinattn.so: kernel arguments and
// the pickers that map a launch plan to a compiled kernel.  Internal.
#pragma once

#include <stdint.h>

namespace laimpl {

constexpr int kWave = 64;

// One batch of rows of the recurrence.  Strides in elements.
struct AttnArgs {
    const void *q, *k, *v;
    const float *g;               // NULL: no decay
    void *state;
    void *out;                    // NULL: outputs not wanted
    const int32_t *slot_idx;      // NULL: row i uses slot i
    const int32_t *cu_seqlens;    // packed rows, or NULL
    const int32_t *num_tokens;    // tokens of each row, or NULL (T)
    const int32_t *has_init;      // NULL: every row starts from its state
    int64_t q_seq, q_tok, q_head;
    int64_t k_seq, k_tok, k_head;
    int64_t v_seq, v_tok, v_head;
    int64_t o_seq, o_tok, o_head;
    int64_t g_seq, g_tok;
    int64_t s_slot;
    int32_t n_seq, T, v_heads, group;   // group = v heads that share a q/k head
    int32_t dk, dv, n_slots, tiles;     // tiles = workgroups along dv of a head
    float scale;
    int32_t write_state;
    int32_t streaming;            // the states of this call are more than the caches keep
    // prompts in chunks: a row is cut into segments of seg_len tokens (a multiple of the chunk;
    // rows of at most seg_len tokens are one)
    int32_t seg_len, segments;          // segments that the grid holds
    int32_t places;                     // segments of cut rows that the workspace holds
    void *ws;                           // what each segment adds to a state (a row's last: the row's
                                        // first state), then the state behind it
    float *ws_total;                    // the decay over each
};

struct NormArgs {
    const void *y, *gate, *weight, *post_weight, *residual;
    void *out, *residual_out;
    int64_t rows;
    int64_t y_row, y_head, gate_row, gate_head, out_row, out_head, res_row, res_out_row;
    int32_t heads, dim;
    float eps, scale;
    int32_t sigmoid, gate_first;
};

// Columns of the state (channels of v) that one workgroup of the recurrent kernel holds.
struct RecurrentPlan {
    const void *fn;
    int cols, threads;
};
// wide: 16 lanes across the state's columns (64 fp32 / 128 bf16 columns a workgroup), else 8.
RecurrentPlan pick_recurrent(int x_bytes, int state_bytes, int dk, bool wide);

// Prompts in chunks.  Where rows are cut, `first` leaves what each segment's tokens add to a state
// and the row's first state in the workspace, `combine` makes the state behind each segment of them;
// `run` makes the outputs and the last state, and of a cut row it does not read the pool that it writes.
struct ChunkedPlan {
    const void *run, *first, *combine;
    int cols, threads, chunk;     // columns of the state per workgroup; tokens of a chunk
    int64_t ws_bytes;             // of one workgroup's state
};
// wide: 128 columns per workgroup, else 64.
ChunkedPlan pick_chunked(int state_bytes, int dk, bool wide);
ChunkedPlan pick_chunked_f32(int dk);        // fp32 tokens and state

// Up to 32 tokens of bf16 in one pass over the state: 128 columns per workgroup of 256 lanes.
const void *pick_few(int state_bytes, int dk, int T, bool out, bool write);

struct NormPlan {
    const void *fn;
    int threads, per_block;       // groups (gated) or rows (residual) per workgroup
};
NormPlan pick_gated(int x_bytes, int dim);
NormPlan pick_residual(int x_bytes, int res_bytes, int dim);

}  // namespace laimpl

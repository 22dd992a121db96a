// Internal host-side interface of the serving-step operators (page maps, rotary
// positions, the block-scaled cache), and what they share with smla_api.cu. Not
// installed; not part of the ABI.
#pragma once

#include "smla_internal.h"

#include <cuda_bf16.h>

namespace smla {

// Records a CUDA error for smla_last_error_string and maps it to a status.
smla_status cuda_status(cudaError_t e);
// SM count of the current device (cached per device).
cudaError_t current_sm_count(int *out);

// Block tables and slot maps of a step, validated by the ABI layer.
struct TablesArgs {
    const int32_t *seq_lens, *query_lens, *blocks_held; // [B]
    int32_t *blocks_held_out;                           // [B], may be blocks_held
    int B, block_size, block_shift;
    int32_t *block_table; // [B, table_width], row stride
    int64_t table_stride;
    int table_width;
    int32_t *free_ring;
    int ring_size;
    const int32_t *ring_state; // head, count
    int32_t *ring_state_out;   // may be ring_state
    int32_t *query_start;      // [B + 1]
    int64_t *positions, *slot_mapping;
    int32_t *token_request; // or nullptr
    int64_t num_tokens;
    int32_t *counts; // [4]
    // workspace: the scan's plan for the fill
    int4 *plan;          // [B] first block taken, blocks held, blocks after, length
    int32_t *give_start; // [B]
    int32_t *state;      // [2] ring head and count before the call
};
cudaError_t launch_block_tables(const TablesArgs &a, int sm_count, cudaStream_t stream);

// A rotary table's frequencies: turns per position times 2^64, and the factor of its values.
constexpr int kMaxRopePairs = 128;
struct RopeFrequencies {
    unsigned long long frac[kMaxRopePairs];
    int pairs;
    float factor;
};
cudaError_t launch_rope_table(float *table, int64_t rows, int64_t first, const RopeFrequencies &f, int sm_count,
                              cudaStream_t stream);

// The rotation of q and k, validated by the ABI layer.
struct RopeArgs {
    const void *q, *k;
    void *q_out, *k_out;
    int64_t q_st, q_sh, qo_st, qo_sh, k_st, k_sh, ko_st, ko_sh;
    const int64_t *positions;
    const float *cos_sin;
    int64_t max_position;
    int T, H, H_k, D, rot_dim, rot_offset;
    bool neox, inverse;
};
cudaError_t launch_rope(const RopeArgs &a, int dtype, int sm_count, cudaStream_t stream);
cudaError_t read_rope_error(int *out, bool reset);

// The write of the block-scaled cache, validated by the ABI layer.
struct Kv8AppendArgs {
    const __nv_bfloat16 *k, *v; // [T, H_kv, D], strides
    int64_t k_st, k_sh, v_st, v_sh;
    const int64_t *slot_mapping;
    int T, H_kv, block_shift;
    uint8_t *k_cache, *v_cache; // [num_blocks, H_kv, block_size, D]
    float *k_scale, *v_scale;   // [num_blocks, H_kv]
    int64_t num_blocks;
    int window; // tokens whose runs one block takes (set by the launch)
};
cudaError_t launch_kv8_append(const Kv8AppendArgs &a, int D, int sm_count, cudaStream_t stream);
cudaError_t read_append_error(int *out, bool reset);

// Attention over the block-scaled cache, validated by the ABI layer.
struct Kv8AttnArgs {
    const void *q; // bf16 [T, H, D], strides
    int64_t q_st, q_sh;
    const uint8_t *k_cache, *v_cache;
    const float *k_scale, *v_scale;
    int64_t num_blocks;
    const int32_t *block_table;
    int64_t table_stride;
    int table_width;
    const int32_t *seq_lens, *query_start;
    int B, T, H, H_kv, G; // G = H / H_kv
    int block_size, block_shift, window;
    float scale;
    const float *sinks; // [H] or nullptr
    void *out;          // bf16 [T, H, D]
    float *lse;         // [T, H] or nullptr
};
size_t kv8_tile_workspace(int B, int T, int H, int H_kv, int D, int max_query_len, int sm_count);
cudaError_t launch_kv8_tile(const Kv8AttnArgs &a, int D, int max_query_len, void *workspace, int sm_count, cudaStream_t stream);
cudaError_t read_kv8_error(int *out, bool reset);
cudaError_t read_kv8_stream_error(int *out, bool reset);
// positions: those that the block table has at most
size_t kv8_stream_workspace(int B, int T, int G, int H_kv, int D, int max_query_len, int64_t positions, int sm_count);
cudaError_t launch_kv8_stream(const Kv8AttnArgs &a, int D, int max_query_len, void *workspace, int sm_count,
                              cudaStream_t stream);

} // namespace smla

// Internal host-side interface of the serving-step operators (page maps, rotary
// positions, the block-scaled cache), and what they share with smla_api.cu. Not
// installed; not part of the ABI.
#pragma once

#include "smla_internal.h"

#include <cuda_bf16.h>

namespace smla {

// What the ABI layer's checks share.
inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline size_t up256(size_t x) { return (x + 255) & ~size_t(255); }
// log2 of a supported block size, -1 otherwise
inline int block_shift(int block_size)
{
    switch (block_size) {
    case 16:
        return 4;
    case 32:
        return 5;
    case 64:
        return 6;
    case 128:
        return 7;
    default:
        return -1;
    }
}
constexpr int64_t kMostPositions = 1 << 30; // of a block table
constexpr int kMostRequests = 1 << 30, kMostWidth = 1 << 30; // loops over them step past their ends in 31 bits
// Rows over one another would be written by several threads: heads lie within a token's row, or tokens within a
// head's (any other order of rows apart is refused with those that overlap).
inline bool rows_overlap(int T, int heads, int D, int64_t st, int64_t sh)
{
    if ((heads > 1 && sh < D) || (T > 1 && st < D))
        return true;
    return heads > 1 && T > 1 && st < (heads - 1) * sh + D && sh < (T - 1) * st + D;
}

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
cudaError_t read_rope_error(int *out, bool reset); // and smla_qk_norm_rope's

// Norms of q's and k's heads with the rotation, validated by the ABI layer.
struct NormRopeArgs {
    const void *q, *k;
    void *q_out, *k_out;
    int64_t q_st, q_sh, qo_st, qo_sh, k_st, k_sh, ko_st, ko_sh;
    const void *q_weight, *k_weight; // [D] (stride 0) or a row to a head; nullptr: ones
    int64_t qw_sh, kw_sh;
    float weight_offset, eps, inv_D;
    const int64_t *positions;
    const float *cos_sin;
    int64_t max_position;
    int T, H, H_k, D, rot_dim, rot_offset;
    bool neox;
};
// weight_f32: the weights are binary32 (otherwise of the tensors' type)
cudaError_t launch_norm_rope(const NormRopeArgs &a, int dtype, bool weight_f32, int sm_count, cudaStream_t stream);
cudaError_t read_norm_rope_error(int *out, bool reset);

// Masks and positions of drafted trees, validated by the ABI layer.
constexpr int kMostTreeWords = 16;
struct TreeMaskArgs {
    const int32_t *parents, *seq_lens, *query_start; // [T], [B], [B + 1]
    int B, T, words, window;
    uint64_t *mask;     // [T, words]
    int64_t *positions; // [T]
};
cudaError_t launch_tree_masks(const TreeMaskArgs &a, int sm_count, cudaStream_t stream);
cudaError_t read_tree_error(int *out, bool reset);

// The move of kept tokens' rows, and copies of blocks: the pools of one launch.
constexpr int kMostPools = 128;
struct KeepArgs {
    const int32_t *block_table;
    int64_t table_stride;
    int table_width;
    const int32_t *seq_lens, *query_lens; // [B]
    const int32_t *kept;                  // [B, kept_width], row stride
    int64_t kept_stride;
    int kept_width;
    const int32_t *kept_lens; // [B]
    int32_t *seq_lens_out;    // [B], or nullptr (not by this launch)
    int B, heads, block_shift, row_bytes;
    int64_t num_blocks;
    int pools;
    uint8_t *codes[kMostPools]; // [num_blocks, heads, block_size, row_bytes]
    float *scales[kMostPools];  // [num_blocks, heads], or nullptr
};
cudaError_t launch_keep_tokens(const KeepArgs &a, bool scaled, int sm_count, cudaStream_t stream);
cudaError_t read_keep_error(int *out, bool reset);
struct CopyArgs {
    const int32_t *from, *to; // [n]
    int n, pools;
    int64_t num_blocks;
    uint8_t *pool[kMostPools];
    int64_t block_bytes[kMostPools];
};
cudaError_t launch_copy_blocks(const CopyArgs &a, int sm_count, cudaStream_t stream);

// Forked block tables, validated by the ABI layer.
constexpr int kForkUnit = 256; // entries of a row that a warp takes
// Units of the old and new rows: at least one to a row, however narrow.
constexpr int64_t fork_units(int64_t rows, int table_width)
{
    return rows * (table_width > kForkUnit ? ((int64_t)table_width + kForkUnit - 1) / kForkUnit : 1);
}
// Up to this many units one block does it all, a warp to a unit, without the launches of the phases: its rounds of 32 units
// take 3 us each, the launches as good as nothing. By one block and by launches, rows being old and new ones together: 5 rows
// of 32 entries 6.5 us and 9.9, 32 of 8 7.6 and 10.4, 2 of 4000 15.6 and 14.6; 64 of 2 10.2 and 10.7, 64 of 100 14.9 and 12.4,
// 128 of 8 15.6 and 10.4, 512 of 8 48 and 10.9, 2000 of 2 175 and 13.5. (A cluster of eight blocks: 264 entries 9.6, 4000 11.0.)
constexpr int64_t kForkOneBlockUnits = 32;
constexpr bool fork_by_one_block(int B_old, int B, int table_width)
{
    return fork_units((int64_t)B + B_old, table_width) <= kForkOneBlockUnits;
}
struct ForkArgs {
    const int32_t *source_rows, *seq_lens; // [B]
    int B;
    const int32_t *blocks_held; // [B_old]
    int B_old;
    const int32_t *block_table; // [B_old, table_width], row stride
    int64_t table_stride;
    int32_t *blocks_held_out; // [B]
    int32_t *block_table_out; // [B, table_width], row stride
    int64_t out_stride;
    int table_width, block_shift;
    int64_t num_blocks;
    int32_t *free_ring;
    int ring_size;
    const int32_t *ring_state;
    int32_t *ring_state_out;    // may be ring_state
    int32_t *copy_from, *copy_to; // [B]
    int32_t *counts;            // [4]
    // workspace
    uint32_t *marks;     // [num_blocks]
    int32_t *gives;      // [B_old * units] blocks that the unit gives back, then where its first one goes
    int4 *plan;          // [B] source row, blocks, the number of its new last block (-1: none)
    int32_t *state;      // [4] ring head and count before the call, whether blocks lack, blocks done
};
cudaError_t launch_fork_tables(const ForkArgs &a, int sm_count, cudaStream_t stream);

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
cudaError_t read_append_error(int *out, bool reset); // and those of tree masks and kept tokens

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
    // drafted trees (nullptr: none, causal): which of its request's new tokens each token sees
    const uint64_t *tree_mask; // [T, tree_words]
    int tree_words;
    const int64_t *tree_positions; // [T], for the window
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

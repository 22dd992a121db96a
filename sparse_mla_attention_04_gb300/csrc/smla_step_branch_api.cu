// C ABI of the operators of a step that drafts and branches (norms with the
// rotation, tree masks, kept tokens, forked block tables, block copies): argument
// checks on the host, then the launch. Declared and documented in
// include/sparse_mla.h.
#include "smla_step.h"

#include <climits>
#include <cmath>

namespace {

using smla::aligned;
using smla::block_shift;
using smla::cuda_status;
using smla::current_sm_count;
using smla::up256;

bool fork_sizes(int B_old, int B, int table_width, int64_t num_blocks)
{
    return B_old >= 0 && B >= 0 && table_width >= 0 && num_blocks >= 0;
}

bool fork_supported(int B_old, int B, int table_width, int64_t num_blocks)
{
    return B_old <= smla::kMostRequests && B <= smla::kMostRequests && table_width <= smla::kMostWidth &&
           (int64_t)B_old * table_width <= INT_MAX && (int64_t)B * table_width <= INT_MAX && num_blocks <= INT_MAX;
}

// workspace of smla_fork_block_tables: state, the rows' plans, the units' sums, the marks
size_t fork_workspace(int B_old, int B, int table_width, int64_t num_blocks)
{
    return 256 + up256((size_t)B * sizeof(int4)) + up256((size_t)smla::fork_units(B_old, table_width) * sizeof(int32_t)) +
           up256((size_t)num_blocks * sizeof(uint32_t));
}

// Whether x[0, n) and y[0, m) have words in common.
bool overlap(const int32_t *x, int64_t n, const int32_t *y, int64_t m)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y);
    return a < b + (uintptr_t)m * 4 && b < a + (uintptr_t)n * 4;
}

} // namespace

extern "C" {

SMLA_API smla_status smla_qk_norm_rope(const smla_qk_norm_rope_params *p)
{
    if (p == nullptr)
        return SMLA_ERR_NULL_POINTER;
    if (p->size < sizeof(smla_qk_norm_rope_params))
        return SMLA_ERR_BAD_SHAPE;
    if ((p->dtype != SMLA_BF16 && p->dtype != SMLA_F16 && p->dtype != SMLA_F32) ||
        (p->weight_dtype != p->dtype && p->weight_dtype != SMLA_F32))
        return SMLA_ERR_BAD_DTYPE;
    if (p->T < 0 || p->H < 0 || p->H_k < 0 || p->D < 0 || p->D > 65536 || p->rot_dim < 2 || p->rot_dim % 2 != 0 ||
        p->rot_dim > 2 * smla::kMaxRopePairs || p->rot_offset < 0 || p->rot_offset > p->D - p->rot_dim ||
        p->max_position < 0 || p->H > (1 << 20) || p->H_k > (1 << 20) || !std::isfinite(p->weight_offset) ||
        !std::isfinite(p->eps) || !(p->eps >= 0x1p-100f))
        return SMLA_ERR_BAD_SHAPE;
    if (p->q_stride_t < 0 || p->q_stride_h < 0 || p->q_out_stride_t < 0 || p->q_out_stride_h < 0 || p->k_stride_t < 0 ||
        p->k_stride_h < 0 || p->k_out_stride_t < 0 || p->k_out_stride_h < 0 || p->q_weight_stride_h < 0 ||
        p->k_weight_stride_h < 0)
        return SMLA_ERR_BAD_SHAPE;
    if (p->T == 0 || p->H + p->H_k == 0)
        return SMLA_OK;
    if ((p->H > 0 && (p->q == nullptr || p->q_out == nullptr)) || (p->H_k > 0 && (p->k == nullptr || p->k_out == nullptr)) ||
        p->positions == nullptr || (p->cos_sin_cache == nullptr && p->max_position > 0))
        return SMLA_ERR_NULL_POINTER;
    const int size = p->dtype == SMLA_F32 ? 4 : 2, wsize = p->weight_dtype == SMLA_F32 ? 4 : 2;
    if ((p->H > 0 && (!aligned(p->q, size) || !aligned(p->q_out, size))) ||
        (p->H_k > 0 && (!aligned(p->k, size) || !aligned(p->k_out, size))) || !aligned(p->positions, 8) ||
        !aligned(p->cos_sin_cache, 4) || !aligned(p->q_weight, wsize) || !aligned(p->k_weight, wsize))
        return SMLA_ERR_MISALIGNED;
    // in place: the same strides, or a row would be written over before it is read
    if ((p->H > 0 && p->q == p->q_out && (p->q_stride_t != p->q_out_stride_t || p->q_stride_h != p->q_out_stride_h)) ||
        (p->H_k > 0 && p->k == p->k_out && (p->k_stride_t != p->k_out_stride_t || p->k_stride_h != p->k_out_stride_h)))
        return SMLA_ERR_BAD_SHAPE;
    if ((p->H > 0 && smla::rows_overlap(p->T, p->H, p->D, p->q_out_stride_t, p->q_out_stride_h)) ||
        (p->H_k > 0 && smla::rows_overlap(p->T, p->H_k, p->D, p->k_out_stride_t, p->k_out_stride_h)))
        return SMLA_ERR_BAD_SHAPE;
    smla::NormRopeArgs a{};
    if (p->H > 0) {
        a.q = p->q;
        a.q_out = p->q_out;
        a.q_st = p->q_stride_t;
        a.q_sh = p->q_stride_h;
        a.qo_st = p->q_out_stride_t;
        a.qo_sh = p->q_out_stride_h;
        a.q_weight = p->q_weight;
        a.qw_sh = p->q_weight ? p->q_weight_stride_h : 0;
    }
    if (p->H_k > 0) {
        a.k = p->k;
        a.k_out = p->k_out;
        a.k_st = p->k_stride_t;
        a.k_sh = p->k_stride_h;
        a.ko_st = p->k_out_stride_t;
        a.ko_sh = p->k_out_stride_h;
        a.k_weight = p->k_weight;
        a.kw_sh = p->k_weight ? p->k_weight_stride_h : 0;
    }
    a.weight_offset = p->weight_offset;
    a.eps = p->eps;
    a.inv_D = 1.0f / (float)p->D;
    a.positions = p->positions;
    a.cos_sin = p->cos_sin_cache;
    a.max_position = p->max_position;
    a.T = p->T;
    a.H = p->H;
    a.H_k = p->H_k;
    a.D = p->D;
    a.rot_dim = p->rot_dim;
    a.rot_offset = p->rot_offset;
    a.neox = p->is_neox != 0;
    int sms = 0;
    if (const cudaError_t e = current_sm_count(&sms); e != cudaSuccess)
        return cuda_status(e);
    const cudaError_t e =
        smla::launch_norm_rope(a, p->dtype, p->weight_dtype == SMLA_F32, sms, reinterpret_cast<cudaStream_t>(p->stream));
    return e == cudaErrorInvalidValue ? SMLA_ERR_UNSUPPORTED : cuda_status(e);
}

SMLA_API smla_status smla_build_tree_masks(const int32_t *parents, const int32_t *seq_lens, const int32_t *query_start,
                                           int B, int T, int tree_words, int window, uint64_t *tree_mask,
                                           int64_t *positions, smla_stream_t stream)
{
    if (B < 0 || T < 0 || tree_words < 1 || window < 0)
        return SMLA_ERR_BAD_SHAPE;
    if (tree_words > smla::kMostTreeWords || B > smla::kMostRequests || T > INT_MAX - 1024)
        return SMLA_ERR_UNSUPPORTED;
    if (T == 0)
        return SMLA_OK;
    if (tree_mask == nullptr || positions == nullptr ||
        (B > 0 && (parents == nullptr || seq_lens == nullptr || query_start == nullptr)))
        return SMLA_ERR_NULL_POINTER;
    if (!aligned(parents, 4) || !aligned(seq_lens, 4) || !aligned(query_start, 4) || !aligned(tree_mask, 8) ||
        !aligned(positions, 8))
        return SMLA_ERR_MISALIGNED;
    const smla::TreeMaskArgs a{parents, seq_lens, query_start, B, T, tree_words, window, tree_mask, positions};
    int sms = 0;
    if (const cudaError_t e = current_sm_count(&sms); e != cudaSuccess)
        return cuda_status(e);
    return cuda_status(smla::launch_tree_masks(a, sms, reinterpret_cast<cudaStream_t>(stream)));
}

SMLA_API smla_status smla_keep_tokens(const smla_keep_tokens_params *p)
{
    if (p == nullptr)
        return SMLA_ERR_NULL_POINTER;
    if (p->size < sizeof(smla_keep_tokens_params) || p->B < 0 || p->num_pools < 1 || p->heads < 1 || p->row_bytes < 1 ||
        p->num_blocks < 0 || p->table_width < 0 || p->table_stride < p->table_width || p->kept_width < 0 ||
        p->kept_stride < p->kept_width)
        return SMLA_ERR_BAD_SHAPE;
    const bool scaled = p->scales != nullptr;
    const int shift = block_shift(p->block_size);
    if (shift < 0 || (scaled ? p->row_bytes != 64 && p->row_bytes != 128 : p->row_bytes % 8 != 0 || p->row_bytes > 65536) ||
        p->B > smla::kMostRequests || ((int64_t)p->table_width << shift) > smla::kMostPositions || p->num_blocks > INT_MAX ||
        p->heads > INT_MAX / 2)
        return SMLA_ERR_UNSUPPORTED;
    if (p->B == 0)
        return SMLA_OK;
    if ((p->block_table == nullptr && p->table_width > 0) || p->seq_lens == nullptr || p->query_lens == nullptr ||
        (p->kept == nullptr && p->kept_width > 0) || p->kept_lens == nullptr || p->pools == nullptr)
        return SMLA_ERR_NULL_POINTER;
    if (!aligned(p->block_table, 4) || !aligned(p->seq_lens, 4) || !aligned(p->query_lens, 4) || !aligned(p->kept, 4) ||
        !aligned(p->kept_lens, 4) || !aligned(p->seq_lens_out, 4))
        return SMLA_ERR_MISALIGNED;
    for (int i = 0; i < p->num_pools; ++i) {
        if (p->num_blocks > 0 && (p->pools[i] == nullptr || (scaled && p->scales[i] == nullptr)))
            return SMLA_ERR_NULL_POINTER;
        if (!aligned(p->pools[i], scaled ? 16 : 8) || (scaled && !aligned(p->scales[i], 4)))
            return SMLA_ERR_MISALIGNED;
    }
    if ((int64_t)p->B * p->heads > INT_MAX / smla::kMostPools)
        return SMLA_ERR_UNSUPPORTED;
    // (lengths, lists and tables are read by every team of the launch, the new lengths written by one)
    const auto meets_out = [&](const int32_t *x, int64_t n) { return overlap(x, n, p->seq_lens_out, p->B); };
    if (p->seq_lens_out != nullptr &&
        (meets_out(p->seq_lens, p->B) || meets_out(p->query_lens, p->B) || meets_out(p->kept_lens, p->B) ||
         (p->kept_width > 0 && meets_out(p->kept, (p->B - 1) * p->kept_stride + p->kept_width)) ||
         (p->table_width > 0 && meets_out(p->block_table, (p->B - 1) * p->table_stride + p->table_width))))
        return SMLA_ERR_BAD_SHAPE;
    smla::KeepArgs a;
    a.block_table = p->block_table;
    a.table_stride = p->table_stride;
    a.table_width = p->table_width;
    a.seq_lens = p->seq_lens;
    a.query_lens = p->query_lens;
    a.kept = p->kept;
    a.kept_stride = p->kept_stride;
    a.kept_width = p->kept_width;
    a.kept_lens = p->kept_lens;
    a.seq_lens_out = p->seq_lens_out;
    a.B = p->B;
    a.heads = p->heads;
    a.block_shift = shift;
    a.row_bytes = p->row_bytes;
    a.num_blocks = p->num_blocks;
    int sms = 0;
    if (const cudaError_t e = current_sm_count(&sms); e != cudaSuccess)
        return cuda_status(e);
    for (int i0 = 0; i0 < p->num_pools; i0 += smla::kMostPools) {
        a.pools = p->num_pools - i0 < smla::kMostPools ? p->num_pools - i0 : smla::kMostPools;
        for (int i = 0; i < a.pools; ++i) {
            a.codes[i] = static_cast<uint8_t *>(p->pools[i0 + i]);
            a.scales[i] = scaled ? p->scales[i0 + i] : nullptr;
        }
        const cudaError_t e = smla::launch_keep_tokens(a, scaled, sms, reinterpret_cast<cudaStream_t>(p->stream));
        if (e != cudaSuccess)
            return cuda_status(e);
        a.seq_lens_out = nullptr;
    }
    return SMLA_OK;
}

SMLA_API smla_status smla_copy_blocks(void *const *pools, const int64_t *block_bytes, int num_pools,
                                      const int32_t *copy_from, const int32_t *copy_to, int n, int64_t num_blocks,
                                      smla_stream_t stream)
{
    if (num_pools < 0 || n < 0 || num_blocks < 0)
        return SMLA_ERR_BAD_SHAPE;
    if (num_blocks > INT_MAX)
        return SMLA_ERR_UNSUPPORTED;
    if (num_pools == 0 || n == 0 || num_blocks == 0)
        return SMLA_OK;
    if (pools == nullptr || block_bytes == nullptr || copy_from == nullptr || copy_to == nullptr)
        return SMLA_ERR_NULL_POINTER;
    for (int i = 0; i < num_pools; ++i) {
        if (block_bytes[i] < 0 || block_bytes[i] > ((int64_t)1 << 40))
            return SMLA_ERR_BAD_SHAPE;
        if (pools[i] == nullptr && block_bytes[i] > 0)
            return SMLA_ERR_NULL_POINTER;
    }
    if (!aligned(copy_from, 4) || !aligned(copy_to, 4))
        return SMLA_ERR_MISALIGNED;
    int sms = 0;
    if (const cudaError_t e = current_sm_count(&sms); e != cudaSuccess)
        return cuda_status(e);
    smla::CopyArgs a;
    a.from = copy_from;
    a.to = copy_to;
    a.n = n;
    a.num_blocks = num_blocks;
    for (int i0 = 0; i0 < num_pools; i0 += smla::kMostPools) {
        a.pools = num_pools - i0 < smla::kMostPools ? num_pools - i0 : smla::kMostPools;
        for (int i = 0; i < a.pools; ++i) {
            a.pool[i] = static_cast<uint8_t *>(pools[i0 + i]);
            a.block_bytes[i] = block_bytes[i0 + i];
        }
        const cudaError_t e = smla::launch_copy_blocks(a, sms, reinterpret_cast<cudaStream_t>(stream));
        if (e != cudaSuccess)
            return cuda_status(e);
    }
    return SMLA_OK;
}

SMLA_API size_t smla_fork_block_tables_workspace_size(int B_old, int B, int table_width, int64_t num_blocks)
{
    return fork_sizes(B_old, B, table_width, num_blocks) && fork_supported(B_old, B, table_width, num_blocks)
               ? fork_workspace(B_old, B, table_width, num_blocks)
               : (size_t)-1;
}

SMLA_API smla_status smla_fork_block_tables(const smla_fork_block_tables_params *p)
{
    if (p == nullptr)
        return SMLA_ERR_NULL_POINTER;
    if (p->size < sizeof(smla_fork_block_tables_params) || !fork_sizes(p->B_old, p->B, p->table_width, p->num_blocks) ||
        p->table_stride < p->table_width || p->table_out_stride < p->table_width || p->ring_size < 1)
        return SMLA_ERR_BAD_SHAPE;
    const int shift = block_shift(p->block_size);
    if (shift < 0 || !fork_supported(p->B_old, p->B, p->table_width, p->num_blocks) ||
        ((int64_t)p->table_width << shift) > smla::kMostPositions)
        return SMLA_ERR_UNSUPPORTED;
    if (p->free_ring == nullptr || p->ring_state == nullptr || p->ring_state_out == nullptr || p->counts == nullptr ||
        p->workspace == nullptr ||
        (p->B > 0 && (p->source_rows == nullptr || p->seq_lens == nullptr || p->blocks_held_out == nullptr ||
                      p->copy_from == nullptr || p->copy_to == nullptr ||
                      (p->block_table_out == nullptr && p->table_width > 0))) ||
        (p->B_old > 0 && (p->blocks_held == nullptr || (p->block_table == nullptr && p->table_width > 0))))
        return SMLA_ERR_NULL_POINTER;
    if (!aligned(p->source_rows, 4) || !aligned(p->seq_lens, 4) || !aligned(p->blocks_held, 4) ||
        !aligned(p->block_table, 4) || !aligned(p->blocks_held_out, 4) || !aligned(p->block_table_out, 4) ||
        !aligned(p->free_ring, 4) || !aligned(p->ring_state, 4) || !aligned(p->ring_state_out, 4) ||
        !aligned(p->copy_from, 4) || !aligned(p->copy_to, 4) || !aligned(p->counts, 4) || !aligned(p->workspace, 16))
        return SMLA_ERR_MISALIGNED;
    if (p->workspace_bytes < fork_workspace(p->B_old, p->B, p->table_width, p->num_blocks))
        return SMLA_ERR_WORKSPACE_TOO_SMALL;
    // Rows are read while others are written: the old tables and the new ones are apart.
    if (p->B > 0 && p->B_old > 0) {
        const int64_t old_end = (p->B_old - 1) * p->table_stride + p->table_width,
                      new_end = (p->B - 1) * p->table_out_stride + p->table_width;
        if (overlap(p->blocks_held, p->B_old, p->blocks_held_out, p->B) ||
            (p->table_width > 0 && overlap(p->block_table, old_end, p->block_table_out, new_end)))
            return SMLA_ERR_BAD_SHAPE;
    }
    smla::ForkArgs a;
    a.source_rows = p->source_rows;
    a.seq_lens = p->seq_lens;
    a.B = p->B;
    a.blocks_held = p->blocks_held;
    a.B_old = p->B_old;
    a.block_table = p->block_table;
    a.table_stride = p->table_stride;
    a.blocks_held_out = p->blocks_held_out;
    a.block_table_out = p->block_table_out;
    a.out_stride = p->table_out_stride;
    a.table_width = p->table_width;
    a.block_shift = shift;
    a.num_blocks = p->num_blocks;
    a.free_ring = p->free_ring;
    a.ring_size = p->ring_size;
    a.ring_state = p->ring_state;
    a.ring_state_out = p->ring_state_out;
    a.copy_from = p->copy_from;
    a.copy_to = p->copy_to;
    a.counts = p->counts;
    uint8_t *ws = static_cast<uint8_t *>(p->workspace);
    a.state = reinterpret_cast<int32_t *>(ws);
    ws += 256;
    a.plan = reinterpret_cast<int4 *>(ws);
    ws += up256((size_t)p->B * sizeof(int4));
    a.gives = reinterpret_cast<int32_t *>(ws);
    ws += up256((size_t)smla::fork_units(p->B_old, p->table_width) * sizeof(int32_t));
    a.marks = reinterpret_cast<uint32_t *>(ws);
    int sms = 0;
    if (const cudaError_t e = current_sm_count(&sms); e != cudaSuccess)
        return cuda_status(e);
    return cuda_status(smla::launch_fork_tables(a, sms, reinterpret_cast<cudaStream_t>(p->stream)));
}

} // extern "C"

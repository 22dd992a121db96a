// C ABI of the serving-step operators (block tables, rotary, the block-scaled
// cache's write and attention): argument checks on the host, then the launch.
// Declared and documented in include/sparse_mla.h.
#include "smla_step.h"

#include <cfloat>
#include <climits>
#include <cmath>

namespace {

using smla::aligned;
using smla::block_shift;
using smla::cuda_status;
using smla::current_sm_count;
using smla::kMostPositions;
using smla::kMostRequests;
using smla::kMostWidth;
using smla::up256;

// workspace of smla_build_block_tables: the ring state, then the plan of each request
size_t tables_workspace(int B) { return 256 + up256((size_t)B * sizeof(int4)) + up256((size_t)B * sizeof(int32_t)); }

// Rows of a request that the streaming kernel takes in one unit; more go to the tile
// kernel. 64 requests of 4096 positions, 4 kv heads of 128 columns: 8 rows 73 us against
// 88 by the tile kernel, 16 rows 92 against 92 (one of 32768: 37 against 56; but 32
// requests of 16384: 156 against 136); 20 rows, 32 requests of 8192 and 8 kv heads: 288
// against 143, since K and V are read twice and the second unit, of 4 rows, is not full.
// By the bound alone: requests with fewer rows than it says have units that are not full,
// whose steps all go through the masks (8 rows under a bound of 16: 293 against 141).
bool few_rows(int H, int H_kv, int max_query_len) { return (int64_t)(H / H_kv) * max_query_len <= 16; }

size_t kv8_workspace(int B, int T, int H, int H_kv, int D, int max_query_len, int64_t positions, int sms)
{
    return few_rows(H, H_kv, max_query_len) ? smla::kv8_stream_workspace(B, T, H / H_kv, H_kv, D, max_query_len, positions, sms)
                                            : smla::kv8_tile_workspace(B, T, H, H_kv, D, max_query_len, sms);
}

smla_status check_kv8_shape(int B, int T, int H, int H_kv, int D, int max_query_len)
{
    if (B < 0 || T < 0 || H <= 0 || H_kv <= 0 || H % H_kv != 0 || D <= 0 || max_query_len < 0)
        return SMLA_ERR_BAD_SHAPE;
    if (D != 64 && D != 128)
        return SMLA_ERR_UNSUPPORTED;
    // row and unit counts stay in 31 bits
    if (B > kMostRequests || (int64_t)T * (H / H_kv) > INT_MAX / 2 || ((int64_t)T * (H / H_kv) / 8 + B) * H_kv > INT_MAX)
        return SMLA_ERR_UNSUPPORTED;
    return SMLA_OK;
}

// The masks of drafted trees, for smla_kv8_tree_attn_fwd (mask NULL: none).
struct Tree {
    const uint64_t *mask;
    int words;
    const int64_t *positions;
};

smla_status kv8_attn(const smla_kv8_attn_params *p, const Tree *tree)
{
    if (p->size < sizeof(smla_kv8_attn_params))
        return SMLA_ERR_BAD_SHAPE;
    if (const smla_status s = check_kv8_shape(p->B, p->T, p->H, p->H_kv, p->D, p->max_query_len); s != SMLA_OK)
        return s;
    if (p->num_blocks < 0 || p->table_width < 0 || p->table_stride < p->table_width || p->window < 0 ||
        p->q_stride_t < 0 || p->q_stride_h < 0 || !std::isfinite(p->scale))
        return SMLA_ERR_BAD_SHAPE;
    if (block_shift(p->block_size) < 0 || ((int64_t)p->table_width << block_shift(p->block_size)) > kMostPositions ||
        p->num_blocks > INT_MAX / p->H_kv)
        return SMLA_ERR_UNSUPPORTED;
    if (p->T == 0 || p->B == 0)
        return SMLA_OK;
    if (p->q == nullptr || p->out == nullptr || p->seq_lens == nullptr || p->query_start == nullptr ||
        (p->table_width > 0 && p->block_table == nullptr) ||
        (p->num_blocks > 0 && (p->k_cache == nullptr || p->v_cache == nullptr || p->k_scale == nullptr || p->v_scale == nullptr)) ||
        p->workspace == nullptr || (tree && (tree->mask == nullptr || (p->window > 0 && tree->positions == nullptr))))
        return SMLA_ERR_NULL_POINTER;
    const int64_t q_st = p->T > 1 ? p->q_stride_t : 0, q_sh = p->H > 1 ? p->q_stride_h : 0; // (of one row none is used)
    if (q_st % 8 != 0 || q_sh % 8 != 0 || !aligned(p->q, 16) || !aligned(p->out, 16) ||
        !aligned(p->k_cache, 16) || !aligned(p->v_cache, 16) || !aligned(p->k_scale, 4) || !aligned(p->v_scale, 4) ||
        !aligned(p->block_table, 4) || !aligned(p->seq_lens, 4) || !aligned(p->query_start, 4) || !aligned(p->lse, 4) ||
        !aligned(p->sinks, 4) || !aligned(p->workspace, 256) ||
        (tree && (!aligned(tree->mask, 8) || !aligned(tree->positions, 8))))
        return SMLA_ERR_MISALIGNED;
    int sms = 0;
    if (const cudaError_t e = current_sm_count(&sms); e != cudaSuccess)
        return cuda_status(e);
    if (p->workspace_bytes < kv8_workspace(p->B, p->T, p->H, p->H_kv, p->D, p->max_query_len,
                                           (int64_t)p->table_width << block_shift(p->block_size), sms))
        return SMLA_ERR_WORKSPACE_TOO_SMALL;
    smla::Kv8AttnArgs a;
    a.q = p->q;
    a.q_st = q_st;
    a.q_sh = q_sh;
    a.k_cache = static_cast<const uint8_t *>(p->k_cache);
    a.v_cache = static_cast<const uint8_t *>(p->v_cache);
    a.k_scale = p->k_scale;
    a.v_scale = p->v_scale;
    a.num_blocks = p->num_blocks;
    a.block_table = p->block_table;
    a.table_stride = p->table_stride;
    a.table_width = p->table_width;
    a.seq_lens = p->seq_lens;
    a.query_start = p->query_start;
    a.B = p->B;
    a.T = p->T;
    a.H = p->H;
    a.H_kv = p->H_kv;
    a.G = p->H / p->H_kv;
    a.block_size = p->block_size;
    a.block_shift = block_shift(p->block_size);
    // a window of all positions that the table has is none, and sums with others stay in 31 bits
    a.window = p->window < (int64_t)p->table_width << a.block_shift ? p->window : 0;
    a.scale = p->scale;
    a.sinks = p->sinks;
    a.out = p->out;
    a.lse = p->lse;
    a.tree_mask = tree ? tree->mask : nullptr;
    a.tree_words = tree ? tree->words : 0;
    a.tree_positions = tree ? tree->positions : nullptr;
    if (!few_rows(p->H, p->H_kv, p->max_query_len))
        return cuda_status(smla::launch_kv8_tile(a, p->D, p->max_query_len, p->workspace, sms,
                                                 reinterpret_cast<cudaStream_t>(p->stream)));
    return cuda_status(smla::launch_kv8_stream(a, p->D, p->max_query_len, p->workspace, sms,
                                               reinterpret_cast<cudaStream_t>(p->stream)));
}

} // namespace

extern "C" {

SMLA_API size_t smla_build_block_tables_workspace_size(int B)
{
    return B < 0 || B > kMostRequests ? (size_t)-1 : tables_workspace(B);
}

SMLA_API smla_status smla_build_block_tables(const int32_t *seq_lens, const int32_t *query_lens,
                                             const int32_t *blocks_held, int32_t *blocks_held_out, int B,
                                             int block_size, int32_t *block_table, int64_t table_stride,
                                             int table_width, int32_t *free_ring, int ring_size,
                                             const int32_t *ring_state, int32_t *ring_state_out,
                                             int32_t *query_start, int64_t *positions, int64_t *slot_mapping,
                                             int32_t *token_request, int64_t num_tokens, int32_t *counts,
                                             void *workspace, size_t workspace_bytes, smla_stream_t stream)
{
    if (B < 0 || num_tokens < 0 || num_tokens > INT_MAX || table_width < 0 || table_stride < table_width || ring_size < 1)
        return SMLA_ERR_BAD_SHAPE;
    // (with B * table_width, what is given back stays in 31 bits whatever blocks_held says)
    if (block_shift(block_size) < 0 || B > kMostRequests || table_width > kMostWidth || (int64_t)B * table_width > INT_MAX)
        return SMLA_ERR_UNSUPPORTED;
    if (ring_state == nullptr || ring_state_out == nullptr || query_start == nullptr || counts == nullptr ||
        free_ring == nullptr || workspace == nullptr ||
        (B > 0 && (seq_lens == nullptr || query_lens == nullptr || blocks_held == nullptr ||
                   blocks_held_out == nullptr || (block_table == nullptr && table_width > 0))) ||
        (num_tokens > 0 && (positions == nullptr || slot_mapping == nullptr)))
        return SMLA_ERR_NULL_POINTER;
    if (!aligned(seq_lens, 4) || !aligned(query_lens, 4) || !aligned(blocks_held, 4) || !aligned(blocks_held_out, 4) ||
        !aligned(block_table, 4) || !aligned(free_ring, 4) || !aligned(ring_state, 4) || !aligned(ring_state_out, 4) ||
        !aligned(query_start, 4) || !aligned(positions, 8) || !aligned(slot_mapping, 8) ||
        !aligned(token_request, 4) || !aligned(counts, 4) || !aligned(workspace, 16))
        return SMLA_ERR_MISALIGNED;
    if (workspace_bytes < tables_workspace(B))
        return SMLA_ERR_WORKSPACE_TOO_SMALL;
    smla::TablesArgs a;
    a.seq_lens = seq_lens;
    a.query_lens = query_lens;
    a.blocks_held = blocks_held;
    a.blocks_held_out = blocks_held_out;
    a.B = B;
    a.block_size = block_size;
    a.block_shift = block_shift(block_size);
    a.block_table = block_table;
    a.table_stride = table_stride;
    a.table_width = table_width;
    a.free_ring = free_ring;
    a.ring_size = ring_size;
    a.ring_state = ring_state;
    a.ring_state_out = ring_state_out;
    a.query_start = query_start;
    a.positions = positions;
    a.slot_mapping = slot_mapping;
    a.token_request = token_request;
    a.num_tokens = num_tokens;
    a.counts = counts;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    a.state = reinterpret_cast<int32_t *>(ws);
    a.plan = reinterpret_cast<int4 *>(ws + 256);
    a.give_start = reinterpret_cast<int32_t *>(ws + 256 + up256((size_t)B * sizeof(int4)));
    int sms = 0;
    if (const cudaError_t e = current_sm_count(&sms); e != cudaSuccess)
        return cuda_status(e);
    return cuda_status(smla::launch_block_tables(a, sms, reinterpret_cast<cudaStream_t>(stream)));
}

SMLA_API smla_status smla_rope_cos_sin_cache(float *table, int64_t num_positions, int64_t first_position,
                                             int rot_dim, double base, int scaling, double factor,
                                             int64_t original_max_position, double beta_fast, double beta_slow,
                                             double attention_factor, smla_stream_t stream)
{
    constexpr int64_t kMostPositions = (int64_t)1 << 31;
    if (num_positions < 0 || first_position < 0 || num_positions > kMostPositions ||
        first_position > kMostPositions - num_positions || rot_dim < 2 || rot_dim % 2 != 0 ||
        rot_dim > 2 * smla::kMaxRopePairs)
        return SMLA_ERR_BAD_SHAPE;
    if (scaling < SMLA_ROPE_NONE || scaling > SMLA_ROPE_YARN)
        return SMLA_ERR_BAD_DTYPE;
    if (!(base > 1.0) || !std::isfinite(base) || !(attention_factor >= 0.0 && attention_factor <= FLT_MAX))
        return SMLA_ERR_BAD_SHAPE;
    if (scaling != SMLA_ROPE_NONE && (!(factor >= 1.0) || !std::isfinite(factor)))
        return SMLA_ERR_BAD_SHAPE;
    if (scaling == SMLA_ROPE_NTK && rot_dim < 4)
        return SMLA_ERR_BAD_SHAPE;
    if (scaling == SMLA_ROPE_YARN && (original_max_position < 1 || !(beta_slow > 0.0) || !(beta_fast > beta_slow) ||
                                      !std::isfinite(beta_fast)))
        return SMLA_ERR_BAD_SHAPE;
    if (num_positions == 0)
        return SMLA_OK;
    if (table == nullptr)
        return SMLA_ERR_NULL_POINTER;
    if (!aligned(table, 4))
        return SMLA_ERR_MISALIGNED;
    const double d = rot_dim, two_pi = 6.283185307179586476925;
    const double b = scaling == SMLA_ROPE_NTK ? base * std::pow(factor, d / (d - 2.0)) : base;
    if (!std::isfinite(b))
        return SMLA_ERR_BAD_SHAPE;
    double lo = 0.0, hi = 0.0;
    if (scaling == SMLA_ROPE_YARN) {
        const auto pair_of = [&](double turns) {
            return d * std::log((double)original_max_position / (turns * two_pi)) / (2.0 * std::log(base));
        };
        lo = std::fmax(std::floor(pair_of(beta_fast)), 0.0);
        hi = std::fmin(std::ceil(pair_of(beta_slow)), d - 1.0);
    }
    smla::RopeFrequencies f;
    f.pairs = rot_dim / 2;
    for (int i = 0; i < f.pairs; ++i) {
        double w = std::pow(b, -2.0 * i / d); // radians per position, in (0, 1]
        if (scaling == SMLA_ROPE_LINEAR)
            w /= factor;
        if (scaling == SMLA_ROPE_YARN) {
            const double ramp = std::fmin(std::fmax((i - lo) / std::fmax(hi - lo, 0.001), 0.0), 1.0);
            w = w / factor * ramp + w * (1.0 - ramp);
        }
        f.frac[i] = (unsigned long long)std::nearbyint(w / two_pi * 18446744073709551616.0); // below 2^62: w <= 1
    }
    const double m = attention_factor > 0.0 ? attention_factor
                                            : (scaling == SMLA_ROPE_YARN ? 0.1 * std::log(factor) + 1.0 : 1.0);
    f.factor = (float)m;
    int sms = 0;
    if (const cudaError_t e = current_sm_count(&sms); e != cudaSuccess)
        return cuda_status(e);
    return cuda_status(smla::launch_rope_table(table, num_positions, first_position, f, sms,
                                               reinterpret_cast<cudaStream_t>(stream)));
}

SMLA_API smla_status smla_rope(const smla_rope_params *p)
{
    if (p == nullptr)
        return SMLA_ERR_NULL_POINTER;
    if (p->size < sizeof(smla_rope_params))
        return SMLA_ERR_BAD_SHAPE;
    if (p->dtype != SMLA_BF16 && p->dtype != SMLA_F16 && p->dtype != SMLA_F32)
        return SMLA_ERR_BAD_DTYPE;
    if (p->T < 0 || p->H < 0 || p->H_k < 0 || p->D < 0 || p->D > 65536 || p->rot_dim < 2 || p->rot_dim % 2 != 0 ||
        p->rot_dim > 2 * smla::kMaxRopePairs || p->rot_offset < 0 || p->rot_offset > p->D - p->rot_dim ||
        p->max_position < 0 || p->H > (1 << 20) || p->H_k > (1 << 20))
        return SMLA_ERR_BAD_SHAPE;
    if (p->q_stride_t < 0 || p->q_stride_h < 0 || p->q_out_stride_t < 0 || p->q_out_stride_h < 0 ||
        p->k_stride_t < 0 || p->k_stride_h < 0 || p->k_out_stride_t < 0 || p->k_out_stride_h < 0)
        return SMLA_ERR_BAD_SHAPE;
    if (p->T == 0 || p->H + p->H_k == 0)
        return SMLA_OK;
    if ((p->H > 0 && (p->q == nullptr || p->q_out == nullptr)) || (p->H_k > 0 && (p->k == nullptr || p->k_out == nullptr)) ||
        p->positions == nullptr || (p->cos_sin_cache == nullptr && p->max_position > 0))
        return SMLA_ERR_NULL_POINTER;
    const int size = p->dtype == SMLA_F32 ? 4 : 2;
    if ((p->H > 0 && (!aligned(p->q, size) || !aligned(p->q_out, size))) ||
        (p->H_k > 0 && (!aligned(p->k, size) || !aligned(p->k_out, size))) || !aligned(p->positions, 8) ||
        !aligned(p->cos_sin_cache, 4))
        return SMLA_ERR_MISALIGNED;
    // in place: the same strides, or a row would be written over before it is read
    if ((p->H > 0 && p->q == p->q_out && (p->q_stride_t != p->q_out_stride_t || p->q_stride_h != p->q_out_stride_h)) ||
        (p->H_k > 0 && p->k == p->k_out && (p->k_stride_t != p->k_out_stride_t || p->k_stride_h != p->k_out_stride_h)))
        return SMLA_ERR_BAD_SHAPE;
    if ((p->H > 0 && smla::rows_overlap(p->T, p->H, p->D, p->q_out_stride_t, p->q_out_stride_h)) ||
        (p->H_k > 0 && smla::rows_overlap(p->T, p->H_k, p->D, p->k_out_stride_t, p->k_out_stride_h)))
        return SMLA_ERR_BAD_SHAPE;
    smla::RopeArgs a{};
    if (p->H > 0) {
        a.q = p->q;
        a.q_out = p->q_out;
        a.q_st = p->q_stride_t;
        a.q_sh = p->q_stride_h;
        a.qo_st = p->q_out_stride_t;
        a.qo_sh = p->q_out_stride_h;
    }
    if (p->H_k > 0) {
        a.k = p->k;
        a.k_out = p->k_out;
        a.k_st = p->k_stride_t;
        a.k_sh = p->k_stride_h;
        a.ko_st = p->k_out_stride_t;
        a.ko_sh = p->k_out_stride_h;
    }
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
    a.inverse = p->inverse != 0;
    int sms = 0;
    if (const cudaError_t e = current_sm_count(&sms); e != cudaSuccess)
        return cuda_status(e);
    return cuda_status(smla::launch_rope(a, p->dtype, sms, reinterpret_cast<cudaStream_t>(p->stream)));
}

SMLA_API smla_status smla_kv8_append(const void *k, int64_t k_stride_t, int64_t k_stride_h, const void *v,
                                     int64_t v_stride_t, int64_t v_stride_h, const int64_t *slot_mapping, int T,
                                     int H_kv, int D, int block_size, void *k_cache, void *v_cache, float *k_scale,
                                     float *v_scale, int64_t num_blocks, smla_stream_t stream)
{
    if (T < 0 || H_kv <= 0 || num_blocks < 0 || k_stride_t < 0 || k_stride_h < 0 || v_stride_t < 0 || v_stride_h < 0)
        return SMLA_ERR_BAD_SHAPE;
    if ((D != 64 && D != 128) || block_shift(block_size) < 0 || num_blocks > INT_MAX || H_kv > INT_MAX / 2 ||
        T > INT_MAX - 128)
        return SMLA_ERR_UNSUPPORTED;
    if (T == 0)
        return SMLA_OK;
    if (k == nullptr || v == nullptr || slot_mapping == nullptr || k_cache == nullptr || v_cache == nullptr ||
        k_scale == nullptr || v_scale == nullptr)
        return SMLA_ERR_NULL_POINTER;
    if (T == 1) // of one row no stride is used
        k_stride_t = v_stride_t = 0;
    if (H_kv == 1)
        k_stride_h = v_stride_h = 0;
    if (k_stride_t % 8 != 0 || k_stride_h % 8 != 0 || v_stride_t % 8 != 0 || v_stride_h % 8 != 0 || !aligned(k, 16) ||
        !aligned(v, 16) || !aligned(slot_mapping, 8) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(k_scale, 4) || !aligned(v_scale, 4))
        return SMLA_ERR_MISALIGNED;
    smla::Kv8AppendArgs a;
    a.k = static_cast<const __nv_bfloat16 *>(k);
    a.v = static_cast<const __nv_bfloat16 *>(v);
    a.k_st = k_stride_t;
    a.k_sh = k_stride_h;
    a.v_st = v_stride_t;
    a.v_sh = v_stride_h;
    a.slot_mapping = slot_mapping;
    a.T = T;
    a.H_kv = H_kv;
    a.block_shift = block_shift(block_size);
    a.k_cache = static_cast<uint8_t *>(k_cache);
    a.v_cache = static_cast<uint8_t *>(v_cache);
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.num_blocks = num_blocks;
    a.window = 1;
    int sms = 0;
    if (const cudaError_t e = current_sm_count(&sms); e != cudaSuccess)
        return cuda_status(e);
    const cudaError_t e = smla::launch_kv8_append(a, D, sms, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaErrorInvalidValue ? SMLA_ERR_UNSUPPORTED : cuda_status(e);
}

SMLA_API size_t smla_kv8_attn_workspace_size(int B, int T, int H, int H_kv, int D, int max_query_len)
{
    int sms = 0;
    if (check_kv8_shape(B, T, H, H_kv, D, max_query_len) != SMLA_OK || current_sm_count(&sms) != cudaSuccess)
        return (size_t)-1;
    return kv8_workspace(B, T, H, H_kv, D, max_query_len, kMostPositions, sms);
}

SMLA_API size_t smla_kv8_attn_workspace_size_of(const smla_kv8_attn_params *p)
{
    int sms = 0;
    if (p == nullptr || p->size < sizeof(smla_kv8_attn_params) ||
        check_kv8_shape(p->B, p->T, p->H, p->H_kv, p->D, p->max_query_len) != SMLA_OK || p->table_width < 0 ||
        block_shift(p->block_size) < 0 || ((int64_t)p->table_width << block_shift(p->block_size)) > kMostPositions ||
        current_sm_count(&sms) != cudaSuccess)
        return (size_t)-1;
    return kv8_workspace(p->B, p->T, p->H, p->H_kv, p->D, p->max_query_len,
                         (int64_t)p->table_width << block_shift(p->block_size), sms);
}

SMLA_API smla_status smla_kv8_attn_fwd(const smla_kv8_attn_params *p)
{
    return p == nullptr ? SMLA_ERR_NULL_POINTER : kv8_attn(p, nullptr);
}

SMLA_API smla_status smla_kv8_tree_attn_fwd(const smla_kv8_tree_attn_params *p)
{
    if (p == nullptr)
        return SMLA_ERR_NULL_POINTER;
    if (p->size < sizeof(smla_kv8_tree_attn_params) || p->tree_words < 1 || p->tree_words > (1 << 20))
        return SMLA_ERR_BAD_SHAPE;
    const Tree tree{p->tree_mask, p->tree_words, p->positions};
    return kv8_attn(&p->attn, &tree);
}

} // extern "C"

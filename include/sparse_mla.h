/*
 * sparse_mla.h — C ABI of libsparse_mla.so, a GB300 (sm_103a) sparse MLA
 * attention forward and its companion fp8 cache writer.
 *
 * Sources (by page title and section):
 *   [P1] "[ROCm][Perf][GLM-5.3-Flash] Enable AITER sparse MLA on gfx942,
 *        including FP8 KV" (vLLM PR 60583): Overview, Claims, Details
 *        ("FP8 KV on gfx942": q quantized per tile inside the kernel, fp8 dots;
 *        the optional dot_precision argument; "Numerics").
 *   [P3] "[ROCm][DSv4.1][Perf] Route gfx942 sparse MLA prefill to AITER
 *        pa_prefill_sparse" (vLLM PR 60102): What changed (one KV pool, output
 *        of q's dtype), Gating and the jin-amd A/B (split-K decode vs no split).
 *   [P4] "[ROCm][MLA][Perf] Fuse decode QK-RoPE + Q-concat + KV-concat +
 *        KV-cache write for sparse MLA" (vLLM PR 47757): Test plan (cache row =
 *        concat(latent, rope); fp8 storage = x / scale, scaled_fp8_quant
 *        convention), "Why positions is a real argument" (graph safety), and the
 *        non-contiguous-input hazard.
 *
 * Conventions shared by every entry point:
 *   - Pointers marked "device" are CUDA device pointers on the current device.
 *     The caller owns every buffer; the library never allocates, frees or
 *     synchronizes, so every call may be captured into a CUDA graph.
 *   - Calls are asynchronous on `stream` (NULL = the legacy default stream).
 *   - Arguments are checked on the host before anything is launched. A failed
 *     check returns its status and writes nothing. SMLA_ERR_CUDA reports a
 *     CUDA runtime error seen at launch.
 *   - Tensors are dense and row-major (contiguous). Strided views are not
 *     accepted: a strided input once produced silently wrong results [P4].
 *   - bf16 is IEEE binary32's upper half; fp8 is OCP E4M3 ("e4m3fn": max 448,
 *     S.1111.111 = NaN, no infinities).
 */
#ifndef SPARSE_MLA_H
#define SPARSE_MLA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define SMLA_API __attribute__((visibility("default")))
#else
#define SMLA_API
#endif

/* A cudaStream_t, declared without the CUDA headers. */
typedef struct CUstream_st *smla_stream_t;

typedef enum {
    SMLA_OK = 0,
    SMLA_ERR_NULL_POINTER = 1,        /* a required pointer is NULL                   */
    SMLA_ERR_BAD_SHAPE = 2,           /* a size is negative or inconsistent            */
    SMLA_ERR_BAD_DTYPE = 3,           /* unknown dtype / precision, or a bad pairing    */
    SMLA_ERR_MISALIGNED = 4,          /* a pointer lacks the alignment stated below    */
    SMLA_ERR_UNSUPPORTED = 5,         /* valid arguments the library has no kernel for */
    SMLA_ERR_WORKSPACE_TOO_SMALL = 6, /* workspace_bytes below the required size       */
    SMLA_ERR_CUDA = 7                 /* CUDA runtime error (device query or launch)   */
} smla_status;

typedef enum {
    SMLA_KV_BF16 = 0,
    SMLA_KV_FP8_E4M3 = 1
} smla_kv_dtype;

/* Precision of the QK dot products [P1 Details: optional dot_precision; when
 * omitted the precision follows q's dtype, which is bf16 here].
 *   AUTO = BF16.
 *   BF16: bf16 q . K, with K the bf16 cache or the fp8 cache's values
 *         code * kv_scale.
 *   FP8 : q quantized inside the kernel per (row, head) tile to E4M3 with
 *         s_q = amax|q[t,h,:]| / 448 (1.0 if amax == 0), q8 = RNE_sat(q / s_q),
 *         dotted with the E4M3 cache; requires an fp8 cache.
 * The PV product always runs on 16-bit operands with fp32 accumulation. */
typedef enum {
    SMLA_DOT_AUTO = 0,
    SMLA_DOT_BF16 = 1,
    SMLA_DOT_FP8 = 2
} smla_dot_precision;

/* Which kernel serves a forward call (smla_fwd_params.kernel).
 *   AUTO     : the library's choice (described under sparse_mla_fwd).
 *   WARP_MMA : the warp-level mma.sync kernel, for every supported shape and
 *              precision (a comparison path: slower, same results within the
 *              stated tolerances).
 *   TCGEN05_BASIC : the first tcgen05 kernels, whose CTAs take a whole SM:
 *              for 16 heads over an E4M3 cache one CTA per SM (AUTO runs two
 *              lean ones per SM); otherwise as AUTO. */
typedef enum {
    SMLA_KERNEL_AUTO = 0,
    SMLA_KERNEL_WARP_MMA = 1,
    SMLA_KERNEL_TCGEN05_BASIC = 2
} smla_kernel_choice;

/* Human-readable name of a status. Never NULL. */
SMLA_API const char *smla_status_string(int status);

/* ABI version, (major << 16) | minor. */
SMLA_API int smla_version(void);

/* Text of the last CUDA runtime error behind an SMLA_ERR_CUDA returned to the
 * calling thread ("no CUDA error" if there was none). Never NULL. */
SMLA_API const char *smla_last_error_string(void);

/* Number of splits of the top-k list ("split-K", [P3] jin-amd A/B: decode-sized
 * calls need it) that sparse_mla_fwd uses when num_splits == 0, for a device
 * with `sm_count` SMs. Host-only arithmetic; returns >= 1, or 0 for invalid
 * arguments. A caller that runs independent calls concurrently (each on its
 * own stream with its own buffers) can pass the SMs one call will get, e.g.
 * half the device's with two or more in flight, and give the result as the
 * calls' num_splits. */
SMLA_API int smla_plan_num_splits(int T, int H, int D_qk, int topk, int kv_dtype,
                                  int sm_count);

/* Bytes of workspace sparse_mla_fwd needs with `num_splits` splits
 * (num_splits == 0: the automatic plan for the current device, which queries
 * the device), for any dot precision the cache allows (the largest of their
 * needs). 0 means no workspace is needed. Returns (size_t)-1 on invalid
 * arguments or a failed device query. (The boundary's first sketch took
 * (T, H, D_v, topk, sm_count); D_qk and kv_dtype are needed because the
 * 128-head E4M3 kernel keeps its quantized q in the workspace, and
 * num_splits because an explicit split count decides the merge path.) */
SMLA_API size_t sparse_mla_fwd_workspace_size(int T, int H, int D_qk, int D_v, int topk,
                                              int kv_dtype, int num_splits);

/*
 * Sparse MLA attention forward ([P1] Overview and Details, [P3] per-call
 * benchmark shapes, [P4] cache layout).
 *
 * For each query row t in [0, T) and head h in [0, H):
 *   I      = { indices[t, i] : indices[t, i] != -1 }            (order free,
 *            duplicates count; entries < -1 or >= num_slots are masked and
 *            never dereferenced — smla_validate_indices reports them)
 *   K(j)   = dequant(kv_cache[j, 0:D_qk]),  V(j) = dequant(kv_cache[j, 0:D_v])
 *            (MLA: one latent row serves as key and value; for D_qk = 576 the
 *            last 64 columns are the rope part, used by QK only)
 *   s_i    = scale * q[t, h, :] . K(I_i)
 *   out[t, h, :] = sum_i softmax(s)_i V(I_i)      (bf16, round to nearest even)
 *   lse[t, h]    = ln sum_i exp(s_i)              (natural log; scale included)
 *   An empty I gives out = 0 and lse = -inf.
 *
 * q            device, bf16 [T, H, D_qk], 16-byte aligned (q and out may be
 *              NULL when T == 0).
 * kv_cache     device, [num_slots, D_qk] of bf16 or E4M3 (kv_dtype): the paged
 *              pool with its blocks flattened (slot = block * block_size +
 *              offset), 16-byte aligned.
 * kv_dtype     smla_kv_dtype.
 * kv_scale     device pointer to one float (dequant = code * kv_scale);
 *              required for SMLA_KV_FP8_E4M3, ignored (may be NULL) for bf16.
 *              Read on the device, so a graph replays the current value.
 * indices      device, int32 [T, topk], 4-byte aligned (may be NULL when topk == 0).
 * T, H, D_qk, D_v, num_slots, topk
 *              supported: H a multiple of 16, D_v = 512, D_qk in {512, 576}.
 *              T = 0 is a no-op. topk = 0 gives empty rows.
 * scale        softmax scale (e.g. 1/sqrt(D_qk)).
 * dot_precision smla_dot_precision (FP8 needs an fp8 cache). AUTO or BF16
 *              with an fp8 cache keeps q in bf16 and dots it with the cache
 *              values code * kv_scale ([P1 Details, "Numerics": the BF16-dots
 *              option]); this runs on the warp-MMA kernel, with at most 8
 *              automatic splits.
 * out          device, bf16 [T, H, D_v], 16-byte aligned, written.
 * lse          device, float [T, H], or NULL to skip.
 * workspace    device, >= sparse_mla_fwd_workspace_size(...) bytes, 256-byte
 *              aligned; may be NULL when that size is 0, which is the case for
 *              up to 8 splits with 16 heads: the splits of a row form one
 *              thread-block cluster and merge through distributed shared
 *              memory. The workspace opens with a fixed region of merge
 *              counters, which must be zero-filled before the buffer's first
 *              use; every call leaves that region zero, so one buffer serves
 *              later calls of any shape on the same stream. With more than 8
 *              splits, after the region, every split writes its partial output
 *              in binary16 (T*H*S*D_v*2 bytes in all) and its lse, then takes a
 *              counter ticket; the split that takes a row's last ticket merges
 *              the row's partials (no split waits for another). The binary16
 *              partials hold averages of value rows: a bf16 cache with values
 *              beyond +-65504 is not supported with more than 8 splits.
 *              The 128-head E4M3 kernel (below) also needs a workspace, after
 *              that region: q quantized per (row, head), T*H*D_qk bytes, and
 *              its T*H scales.
 *              Calls that overlap in time must not share a workspace.
 * Kernels: 16 heads with D_qk = D_v = 512 run on tcgen05 kernels (keys on
 *              the MMA's M axis, accumulators in tensor memory, TMA row
 *              gathers): a bf16 cache on one that takes a whole SM per CTA,
 *              an E4M3 cache with fp8 dots on a lean one that runs two CTAs
 *              per SM (its splits fill twice as many CTAs); H a multiple of
 *              128 with D_qk = 576, D_v = 512 and an E4M3 cache runs, when the
 *              call does not ask for more than one split, on a tcgen05 kernel
 *              with heads on M (two CTAs per row, each owning half of the
 *              value dims; a first pass quantizes q into the workspace); every
 *              other supported shape runs on a warp-MMA (mma.sync) kernel
 *              (sparse_mla_fwd_ex can ask for it for any shape: its `kernel`
 *              field).
 * num_splits   0 = automatic (smla_plan_num_splits for the current device);
 *              otherwise the number of top-k splits to use, 1..128. More than 8
 *              splits need T * H / 16 <= 16384 (else SMLA_ERR_UNSUPPORTED).
 *              For 128 heads over an E4M3 cache with fp8 dots the automatic
 *              plan (0) also spreads the rows' key tiles evenly over pairs of
 *              SMs when the rows outnumber the pairs (a row cut between two
 *              pairs is merged through the workspace); 1 keeps one pair of
 *              CTAs per row.
 * stream       CUDA stream.
 */
SMLA_API smla_status sparse_mla_fwd(const void *q, const void *kv_cache, int kv_dtype,
                                    const float *kv_scale, const int32_t *indices,
                                    int T, int H, int D_qk, int D_v, int64_t num_slots,
                                    int topk, float scale, int dot_precision,
                                    void *out, float *lse,
                                    void *workspace, size_t workspace_bytes,
                                    int num_splits, smla_stream_t stream);

/*
 * The forward with every option in one versioned structure (set `size` to
 * sizeof(smla_fwd_params)); the fields mean what sparse_mla_fwd's arguments
 * mean, plus:
 *   q_scale  NULL for a bf16 q; else q holds E4M3 codes [T, H, D_qk] with this
 *            per-tensor scale (as sparse_mla_fwd_q8: an E4M3 cache, fp8 dots;
 *            dot_precision AUTO or FP8, else SMLA_ERR_BAD_DTYPE).
 *   sinks    NULL, or device float [H], 4-byte aligned: per-head attention
 *            sink logits [P1 Limitations: sinks are passed through], in the
 *            units of scale * q.k. The sink joins each row's softmax
 *            denominator and has no value row:
 *              out = sum_i e^{s_i} v_i / (e^{sink_h} + sum_j e^{s_j}),
 *              lse = log(e^{sink_h} + sum_j e^{s_j});
 *            a row with no valid index gives out = 0 and lse = sink_h.
 */
typedef struct smla_fwd_params {
    size_t size;
    const void *q;
    const float *q_scale;
    const void *kv_cache;
    int kv_dtype;
    const float *kv_scale;
    const int32_t *indices;
    int T, H, D_qk, D_v;
    int64_t num_slots;
    int topk;
    float scale;
    int dot_precision;
    const float *sinks;
    void *out;
    float *lse;
    void *workspace;
    size_t workspace_bytes;
    int num_splits;
    smla_stream_t stream;
    int kernel;          /* smla_kernel_choice (ABI 1.1; a structure of the 1.0
                            size, without this field, means AUTO) */
} smla_fwd_params;

SMLA_API smla_status sparse_mla_fwd_ex(const smla_fwd_params *params);

/* The exact workspace bytes the call described by `params` needs (its dot
 * precision, q form, kernel choice and split count; pointers are not read).
 * 0 = none. Returns (size_t)-1 for arguments sparse_mla_fwd_ex would reject
 * or a failed device query. */
SMLA_API size_t sparse_mla_fwd_ex_workspace_size(const smla_fwd_params *params);

/*
 * The same forward with a pre-quantized q [P1 Details, "FP8 KV on gfx942":
 * gfx950 keeps the pre-quantized q]: q8 holds E4M3 codes [T, H, D_qk] (as
 * written, for example, by smla_fused_qk_rope_cache with an E4M3 q_out) and
 * *q_scale is their per-tensor scale, so q enters the dots as code * q_scale.
 * The cache must be E4M3 (kv_scale as above); the dots run in fp8, as with
 * SMLA_DOT_FP8, without quantizing q again. Every other argument, the
 * workspace and the kernels are as for sparse_mla_fwd.
 * q8       device, uint8 [T, H, D_qk], 16-byte aligned.
 * q_scale  device, one float, 4-byte aligned.
 */
SMLA_API smla_status sparse_mla_fwd_q8(const void *q8, const float *q_scale, const void *kv_cache,
                                       const float *kv_scale, const int32_t *indices, int T, int H, int D_qk,
                                       int D_v, int64_t num_slots, int topk, float scale, void *out, float *lse,
                                       void *workspace, size_t workspace_bytes, int num_splits,
                                       smla_stream_t stream);


/*
 * Maximum workspace bytes sparse_mla_fwd_no_alloc can serve from its static
 * device array (8 MiB): every GPU that loads the library holds this much.
 */
#define SMLA_NO_ALLOC_SCRATCH_BYTES ((size_t)8 << 20)

/*
 * sparse_mla_fwd without a caller-provided workspace (the pages have no
 * counterpart; it exists for callers of this library that cannot allocate
 * device memory: a serving engine that reserved nearly all of HBM for its
 * KV-cache pool up front, or a host framework that only lets a plug-in use
 * the buffers it hands over).
 *
 * Arguments and results are those of sparse_mla_fwd; q, kv_cache, indices,
 * out and lse remain the caller's. When the call's own plan needs a workspace
 * the library uses a static device array of SMLA_NO_ALLOC_SCRATCH_BYTES
 * instead, and returns SMLA_ERR_WORKSPACE_TOO_SMALL (nothing launched) when
 * the call would need more. Two kinds of call need it:
 *   - more than 8 splits of a row (merge counters, then T * S * H * 1 KB of
 *     binary16 partial results);
 *   - the 128-head E4M3 kernel with fp8 dots (H a multiple of 128, D_qk = 576,
 *     one split), at any split plan: its quantized q, T * H * 580 bytes after
 *     a 64 KB counter region. When its automatic plan spreads the rows over
 *     CTA pairs (more rows than pairs) it also keeps partials of shared rows;
 *     if those do not fit, this entry point runs the call with one CTA pair
 *     per row, which needs the quantized q only. T * H must stay below about
 *     14,300: 128 rows of 128 heads (9.5 MB) do not fit and are rejected.
 * Calls with bf16 dots or a bf16 cache and at most 8 splits use no workspace
 * and never touch the array. Nothing is allocated or freed. Each call looks
 * the array's device address up (cudaGetSymbolAddress) with its device
 * current; make a device's first call before any stream capture, since that
 * lookup may load the module. A call that merges through the counters clears
 * them on `stream` before launching. All calls share the one array: calls
 * that can run at the same time on the GPU (unordered streams) race on it and
 * must not overlap.
 */
SMLA_API smla_status sparse_mla_fwd_no_alloc(const void *q, const void *kv_cache, int kv_dtype,
                                             const float *kv_scale, const int32_t *indices,
                                             int T, int H, int D_qk, int D_v, int64_t num_slots,
                                             int topk, float scale, int dot_precision,
                                             void *out, float *lse, int num_splits,
                                             smla_stream_t stream);

/*
 * ---------------------------------------------------------------------------
 * The serving step around the forward: page maps, rotary tables and rotations,
 * a block-scaled 8-bit cache and attention over it. The pool is paged as for
 * the forward: block `j` of a request holds its tokens [j * block_size,
 * (j + 1) * block_size), block_table[b, j] names the pool block, and a slot is
 * block * block_size + offset. block_size is 16, 32, 64 or 128 here.
 * ---------------------------------------------------------------------------
 *
 * Block tables and slot maps of one step, from the requests' lengths, on the
 * device. With need_b = ceil(max(seq_lens[b], 0) / block_size):
 *   - request b takes max(0, need_b - held_b) new blocks and gives back
 *     max(0, held_b - need_b) (all of them when it has ended: seq_lens[b] = 0);
 *   - free blocks are a ring: free_ring[(head + i) % ring_size], i < count, with
 *     (head, count) = ring_state. The batch's k-th new block (requests in
 *     order, then blocks in order) is the ring's k-th; given-back blocks (in
 *     the same order) go behind its end, for later calls;
 *   - token i of request b's query_lens[b] new tokens (clamped to
 *     [0, seq_lens[b]]; its last ones) is flat token query_start[b] + i, at
 *     position p = seq_lens[b] - query_lens[b] + i, with slot
 *     block_table[b, p / block_size] * block_size + p % block_size.
 * If a request needs more than table_width blocks, or the ring holds fewer than
 * the batch needs, nothing is taken or given back (tables, ring, held counts
 * and ring state keep their values), counts[3] is the number of blocks lacking
 * (those beyond the rows' width, plus those that the ring holds too few) and
 * tokens in blocks not held get slot -1: the caller can free requests and call
 * again.
 *
 * seq_lens, query_lens   device, int32 [B].
 * blocks_held            device, int32 [B]: blocks each request has in its row.
 * blocks_held_out        device, int32 [B], written; may be blocks_held.
 * block_table            device, int32 [B, table_width], row stride
 *                        table_stride; entries [held, need) of a row written.
 *                        Entries past a row's blocks keep what they hold.
 * free_ring              device, int32 [ring_size], ring_size >= every block of
 *                        the pool (so that what is taken and what is given back
 *                        never meet); entries behind the ring's end written.
 * ring_state             device, int32 [2] (head, count).
 * ring_state_out         device, int32 [2], written; may be ring_state.
 * query_start            device, int32 [B + 1], written: exclusive sums.
 * positions              device, int64 [num_tokens], written (0 past the last
 *                        token: a padded step's rows stay valid positions).
 * slot_mapping           device, int64 [num_tokens], written (-1 past it).
 * token_request          device, int32 [num_tokens] or NULL, written (-1 past it).
 * counts                 device, int32 [4], written: tokens, blocks taken, given
 *                        back, lacking (each at most 2^31 - 1).
 * workspace              device, smla_build_block_tables_workspace_size(B)
 *                        bytes, 16-byte aligned; need not be initialised.
 *                        Calls that overlap in time must not share it.
 * B and table_width at most 2^30, B * table_width and num_tokens below 2^31.
 */
SMLA_API size_t smla_build_block_tables_workspace_size(int B);
SMLA_API smla_status smla_build_block_tables(const int32_t *seq_lens, const int32_t *query_lens,
                                             const int32_t *blocks_held, int32_t *blocks_held_out, int B,
                                             int block_size, int32_t *block_table, int64_t table_stride,
                                             int table_width, int32_t *free_ring, int ring_size,
                                             const int32_t *ring_state, int32_t *ring_state_out,
                                             int32_t *query_start, int64_t *positions, int64_t *slot_mapping,
                                             int32_t *token_request, int64_t num_tokens, int32_t *counts,
                                             void *workspace, size_t workspace_bytes, smla_stream_t stream);

/* How smla_rope_cos_sin_cache scales the frequencies base^(-2i / rot_dim) for
 * contexts longer than those a model was trained on:
 *   LINEAR : divided by factor (positions interpolated).
 *   NTK    : base replaced by base * factor^(rot_dim / (rot_dim - 2)).
 *   YARN   : pairs that turn more than beta_fast times over
 *            original_max_position stay, those that turn less than beta_slow
 *            times are divided by factor, a linear ramp over the pair index
 *            between: with c(n) = rot_dim ln(original_max_position / (2 pi n)) /
 *            (2 ln base), lo = max(floor(c(beta_fast)), 0), hi =
 *            min(ceil(c(beta_slow)), rot_dim - 1), the ramp of pair i is
 *            clamp((i - lo) / max(hi - lo, 0.001), 0, 1). */
typedef enum {
    SMLA_ROPE_NONE = 0,
    SMLA_ROPE_LINEAR = 1,
    SMLA_ROPE_NTK = 2,
    SMLA_ROPE_YARN = 3
} smla_rope_scaling;

/*
 * The rotary table that smla_rope and smla_fused_qk_rope_cache read: row r
 * holds, for position p = first_position + r and pairs i < n = rot_dim / 2,
 * m cos(p f_i) in column i and m sin(p f_i) in column n + i, in binary32, each to
 * 6 * 2^-24 of itself for the angle that it is taken at. The angle is carried as a
 * 64-bit fraction of a turn, and whole turns leave it without a rounding; what moves
 * it is the frequency's own, in binary64 (some 2^-50 of it, so p f_i 2^-50: 2^-19
 * radians at position 2^31 for f = 1) and to 2^-65 of a turn a position.
 *
 * table              device, float [num_positions, rot_dim], 4-byte aligned, written.
 * num_positions, first_position  >= 0, first_position + num_positions <= 2^31.
 * rot_dim            even, 2..256 (NTK: at least 4).
 * base               > 1 and finite.
 * scaling            smla_rope_scaling; factor >= 1 (ignored for NONE);
 *                    original_max_position >= 1, beta_fast > beta_slow > 0 (YARN).
 * attention_factor   m, finite in binary32; 0 = the scaling's own:
 *                    0.1 ln(factor) + 1 for YARN, else 1.
 */
SMLA_API smla_status smla_rope_cos_sin_cache(float *table, int64_t num_positions, int64_t first_position,
                                             int rot_dim, double base, int scaling, double factor,
                                             int64_t original_max_position, double beta_fast, double beta_slow,
                                             double attention_factor, smla_stream_t stream);

/* Element type of smla_rope's tensors. */
typedef enum {
    SMLA_BF16 = 0,
    SMLA_F16 = 1,
    SMLA_F32 = 2
} smla_dtype;

/*
 * Rotary positions on part of each head, for a query and (optionally) a key
 * tensor in one launch. For token t, head h, p = positions[t] and pairs
 * i < n = rot_dim / 2 of the columns [rot_offset, rot_offset + rot_dim):
 *   (a, b) -> (a cos - b sin, b cos + a sin),
 * pair i being elements (i, n + i) (is_neox != 0) or (2i, 2i + 1), cos and sin
 * from row p of cos_sin_cache. In binary32, each product and the difference or
 * sum rounded (as smla_fused_qk_rope_cache), then rounded once to the type.
 * inverse != 0 turns by the opposite angle: the transpose, which is also the
 * gradient of the forward rotation. Other columns are copied.
 *
 * q, k            device, [T, H, D] and [T, H_k, D] of `dtype`, element strides
 *                 (t, h), last dimension contiguous. k (and k_out) NULL with
 *                 H_k = 0: q alone.
 * q_out, k_out    device, the same shapes, strides of their own. An output may
 *                 be its input (then with the same strides: rotated in place);
 *                 otherwise it must not overlap an input. Its rows must not
 *                 overlap: st >= (H - 1) sh + D or sh >= (T - 1) st + D.
 * positions       device, int64 [T].
 * cos_sin_cache   device, float [max_position, rot_dim], 4-byte aligned.
 * rot_dim even, 2..256, rot_offset >= 0, rot_offset + rot_dim <= D <= 65536.
 * A token whose position is outside [0, max_position) is not written and sets
 * bit 4 of smla_device_error.
 */
typedef struct smla_rope_params {
    size_t size; /* sizeof(smla_rope_params) */
    int dtype;
    const void *q;
    int64_t q_stride_t, q_stride_h;
    void *q_out;
    int64_t q_out_stride_t, q_out_stride_h;
    const void *k;
    int64_t k_stride_t, k_stride_h;
    void *k_out;
    int64_t k_out_stride_t, k_out_stride_h;
    const int64_t *positions;
    const float *cos_sin_cache;
    int64_t max_position;
    int T, H, H_k, D, rot_dim, rot_offset, is_neox, inverse;
    smla_stream_t stream;
} smla_rope_params;

SMLA_API smla_status smla_rope(const smla_rope_params *params);

/*
 * The block-scaled 8-bit cache: keys and values of H_kv heads in two pools
 * k_cache, v_cache, uint8 [num_blocks, H_kv, block_size, D] of E4M3 codes, each
 * (block, head) with its own scale in k_scale, v_scale, float [num_blocks,
 * H_kv]: value = code * scale.
 *
 * smla_kv8_append writes the rows of T new tokens at their slots. A run is a
 * maximal stretch of consecutive tokens t whose slots lie in one block. For each
 * run, head and cache, with amax the largest finite |x| of the run's rows there
 * (0 if there is none) and s_new = max(amax / 448, 2^-60), in binary32:
 *   - if the run's smallest offset o is above 0, the block holds o older tokens:
 *     scale = max(old scale, s_new), and when it grew their codes become
 *     E4M3_RNE(code * old / scale); otherwise scale = s_new (so rows of zeros
 *     change no block that holds other rows);
 *   - the run's codes are E4M3_RNE_satfinite(x / scale) (infinities saturate,
 *     NaN is the NaN code).
 * A negative slot skips its token (and ends a run); a slot >= num_blocks *
 * block_size writes nothing and sets bit 8 of smla_device_error. The new tokens
 * of a block must be one run with distinct slots (as smla_build_block_tables
 * lays them out): two runs of one call in one block race on its scale.
 *
 * k, v          device, bf16 [T, H_kv, D], element strides (t, h) multiples of
 *               8, 16-byte aligned, last dimension contiguous.
 * slot_mapping  device, int64 [T].
 * caches 16-byte aligned, scales 4-byte aligned. D is 64 or 128; num_blocks
 * below 2^31.
 */
SMLA_API smla_status smla_kv8_append(const void *k, int64_t k_stride_t, int64_t k_stride_h, const void *v,
                                     int64_t v_stride_t, int64_t v_stride_h, const int64_t *slot_mapping, int T,
                                     int H_kv, int D, int block_size, void *k_cache, void *v_cache, float *k_scale,
                                     float *v_scale, int64_t num_blocks, smla_stream_t stream);

/*
 * Attention over the block-scaled cache, for prompts, chunks of prompts and
 * single tokens. Request b's new tokens are the flat tokens [query_start[b],
 * query_start[b + 1]); its token i has position p = seq_lens[b] - (its number of
 * new tokens) + i. For query head h, which reads kv head h / (H / H_kv):
 *   s_j  = scale * q[t, h] . K_j over the visible positions j: j <= p, j <
 *          seq_lens[b], and j > p - window when window > 0;
 *   out[t, h] = sum_j softmax(s)_j V_j (bf16), lse[t, h] = ln sum_j exp(s_j).
 * With sinks, e^{sinks[h]} joins the denominator and the lse. A row that sees
 * nothing gives out = 0 and lse = -inf (sinks[h] with sinks). Positions whose
 * block_table entry is outside [0, num_blocks) are not read and see no one;
 * nothing beyond seq_lens[b] is read. Sums are in binary32. q is carried by two
 * E4M3 parts: its bf16 values whole down to 2^-9 of the largest |q| of their row
 * (token and head), to 2^-17 of that below. Weights are rounded to binary16 with
 * their block's value scale in them: softmax weight times v_scale is kept to 2^-11
 * of itself down to 2^-19 of the row's largest such product, to 2^-30 of that
 * product below; the denominator and lse have every weight in binary32. (So a
 * block whose scale is 2^19 times the others', but not its values, still leaves
 * the others theirs.) Scales are read of the blocks that a token of the request
 * sees; of one request and head they must be positive, at least 2^-60 (as
 * smla_kv8_append gives them) and within a factor of 2^100.
 *
 * q             device, bf16 [T, H, D], element strides (t, h) multiples of 8,
 *               16-byte aligned, last dimension contiguous; D is 64 or 128.
 * block_table   device, int32 [B, table_width], row stride table_stride;
 *               seq_lens above table_width * block_size are cut to that.
 * seq_lens      device, int32 [B]. query_start device, int32 [B + 1], ascending,
 *               within [0, T]; rows of q at or past query_start[B] are not read
 *               and their out and lse not written.
 * max_query_len a bound of the requests' new tokens: it chooses the kernel (a
 *               streaming kernel that splits the requests' tokens evenly over
 *               the SMs, or one with 128 query rows to a tile). A request with
 *               more is still computed in full.
 * out           device, bf16 [T, H, D] contiguous, 16-byte aligned; must not
 *               overlap q. lse device, float [T, H] or NULL.
 * sinks         device, float [H] or NULL, in the units of scale * q . k.
 * workspace     device, >= smla_kv8_attn_workspace_size(...) bytes, or
 *               smla_kv8_attn_workspace_size_of(params) (for the current
 *               device), 256-byte aligned, need not be initialised.
 *               Calls that overlap in time must not share it.
 * H a multiple of H_kv; B >= 0, T >= 0 (0: a no-op); 0 <= window;
 * num_blocks * H_kv below 2^31, B and table_width * block_size at most 2^30.
 */
typedef struct smla_kv8_attn_params {
    size_t size; /* sizeof(smla_kv8_attn_params) */
    const void *q;
    int64_t q_stride_t, q_stride_h;
    const void *k_cache, *v_cache;
    const float *k_scale, *v_scale;
    int64_t num_blocks;
    const int32_t *block_table;
    int64_t table_stride;
    int table_width;
    const int32_t *seq_lens, *query_start;
    int B, T, H, H_kv, D, block_size, max_query_len, window;
    float scale;
    const float *sinks;
    void *out;
    float *lse;
    void *workspace;
    size_t workspace_bytes;
    smla_stream_t stream;
} smla_kv8_attn_params;

/* (size_t)-1 on invalid arguments or a failed device query. */
SMLA_API size_t smla_kv8_attn_workspace_size(int B, int T, int H, int H_kv, int D, int max_query_len);
/* The bytes that one call needs: its block table's width bounds the work, so they
 * may be fewer (pointers, strides and the workspace are not looked at). */
SMLA_API size_t smla_kv8_attn_workspace_size_of(const smla_kv8_attn_params *params);
SMLA_API smla_status smla_kv8_attn_fwd(const smla_kv8_attn_params *params);

/*
 * ---------------------------------------------------------------------------
 * Steps that draft and branch: norms of queries and keys with their rotation, trees
 * of drafted tokens verified at once, their accepted tokens kept, and requests whose
 * block tables go on from one another (samples of one prompt, beams).
 * ---------------------------------------------------------------------------
 *
 * Root-mean-square norms of each query and key head, and smla_rope's rotation behind
 * them, in one pass. For token t and head h of q (and of k with k_weight):
 *   y_d = x_d r (weight_d + weight_offset), r = (mean over the head's D columns of
 *   x^2 + eps)^-1/2, then the columns [rot_offset, rot_offset + rot_dim) turned as
 * smla_rope turns them, in binary32 (squares that pass it are taken of the row scaled
 * by a power of two), rounded once to the type. A head with an infinity has zeros
 * beside it and NaN in its place, one with a NaN is all NaN, and what is rotated with
 * a NaN is one.
 *
 * q, k, q_out, k_out, positions, cos_sin_cache, T, H, H_k, D, rot_dim, rot_offset,
 *              is_neox: as for smla_rope (strided, in place, q alone, tokens out of
 *              range not written and bit 4 of smla_device_error set).
 * q_weight, k_weight  device, of weight_dtype (dtype, or SMLA_F32): [D] for all heads
 *              (stride_h 0) or a row of D to a head, stride_h elements apart; NULL:
 *              factors of 1 (weight_offset is not added).
 * weight_offset  finite; 1 for weights that are held less one.
 * eps          finite, at least 2^-100.
 */
typedef struct smla_qk_norm_rope_params {
    size_t size; /* sizeof(smla_qk_norm_rope_params) */
    int dtype, weight_dtype;
    const void *q;
    int64_t q_stride_t, q_stride_h;
    void *q_out;
    int64_t q_out_stride_t, q_out_stride_h;
    const void *k;
    int64_t k_stride_t, k_stride_h;
    void *k_out;
    int64_t k_out_stride_t, k_out_stride_h;
    const void *q_weight;
    int64_t q_weight_stride_h;
    const void *k_weight;
    int64_t k_weight_stride_h;
    float weight_offset, eps;
    const int64_t *positions;
    const float *cos_sin_cache;
    int64_t max_position;
    int T, H, H_k, D, rot_dim, rot_offset, is_neox;
    smla_stream_t stream;
} smla_qk_norm_rope_params;

SMLA_API smla_status smla_qk_norm_rope(const smla_qk_norm_rope_params *params);

/*
 * Masks and positions of drafted trees. A request's new tokens are the nodes of its
 * tree, in the order of the flat tokens [query_start[b], query_start[b + 1]); they lie
 * in the cache behind its context as any new tokens do, at ctx + i with ctx =
 * seq_lens[b] - (their number). parents[t] is the number in the tree of the node that
 * token t follows, -1 where it follows the context; it is below its own. Token t's
 * mask has the bits of itself and of the nodes that it descends from (bit i % 64 of
 * word i / 64 for node i), with window > 0 only of those fewer than `window`
 * generations up; its position is ctx + the number of nodes that it descends from (0
 * if that is negative).
 *
 * parents      device, int32 [T]. One that is not in [-1, its own number) counts as
 *              -1, and sets bit 16 of smla_device_error.
 * seq_lens     device, int32 [B]; query_start int32 [B + 1], ascending, within [0, T].
 * tree_words   1..16: 64-bit words of a mask. Nodes from 64 tree_words on have an empty
 *              mask and position ctx, and set bit 16 of smla_device_error.
 * tree_mask    device, uint64 [T, tree_words], 8-byte aligned; positions device, int64
 *              [T]; both written, with 0 for rows behind the last request.
 */
SMLA_API smla_status smla_build_tree_masks(const int32_t *parents, const int32_t *seq_lens,
                                           const int32_t *query_start, int B, int T, int tree_words, int window,
                                           uint64_t *tree_mask, int64_t *positions, smla_stream_t stream);

/*
 * smla_kv8_attn_fwd for trees of drafted tokens: token t of request b sees the context
 * [0, ctx) (ctx = seq_lens[b] - its number of new tokens; with window > 0 the
 * positions above positions[t] - window of it) and those of its request's new tokens
 * whose bits are set in its row of tree_mask: position ctx + i for bit i % 64 of word
 * i / 64, whether before or behind it, itself included only by its own bit; the window
 * does not apply to them. Bits of nodes that the request does not have are not looked
 * at, nodes without a bit are seen by none. Everything else (masked rows, sinks, pages
 * outside the pool, precision, workspace) is as for smla_kv8_attn_fwd, whose causal
 * mask is that of trees without branches.
 *
 * attn         the call; its `size` is sizeof(smla_kv8_attn_params), its workspace by
 *              smla_kv8_attn_workspace_size(_of).
 * tree_mask    device, uint64 [T, tree_words], 8-byte aligned; tree_words 1..2^20.
 * positions    device, int64 [T], or NULL without a window: the tokens' positions in
 *              their branches. One outside [ctx, seq_lens[b]) counts as the nearest.
 */
typedef struct smla_kv8_tree_attn_params {
    size_t size; /* sizeof(smla_kv8_tree_attn_params) */
    smla_kv8_attn_params attn;
    const uint64_t *tree_mask;
    int tree_words;
    const int64_t *positions;
} smla_kv8_tree_attn_params;

SMLA_API smla_status smla_kv8_tree_attn_fwd(const smla_kv8_tree_attn_params *params);

/*
 * Keeps some of each request's new tokens (the accepted path of a drafted tree): the
 * cache rows of the kept ones move together behind the context, in every layer's pools
 * at once and in place, and seq_lens_out[b] = ctx + their number is the request's new
 * length, ctx = seq_lens[b] - query_lens[b] (query_lens clamped to [0, seq_lens]). Kept
 * token i of request b is its new token kept[b, i]: the row of position ctx + kept[b, i]
 * goes to position ctx + i, both found through block_table. The numbers ascend strictly
 * and lie below query_lens[b]; the first that does not ends the list and sets bit 16 of
 * smla_device_error, as does a kept_lens[b] above the most there can be (which is cut; one
 * below 0 keeps none).
 * Rows whose old or new block is outside the pool do not move. The blocks written to
 * must be this request's alone (see smla_fork_block_tables), and no block may stand
 * twice in its row.
 *
 * scales NULL: rows of row_bytes bytes as they are (a multiple of 8, at most 65536), in
 * pools [num_blocks, heads, block_size, row_bytes]: the latent cache with heads = 1.
 * Otherwise the block-scaled cache: each K and each V is a pool of codes
 * [num_blocks, heads, block_size, D] with row_bytes = D = 64 or 128, and its scales
 * [num_blocks, heads]. There the scale of a block that rows go to becomes the largest
 * of its own and of those of the blocks that they come from; if that is larger, the
 * older codes in it (below the first row that is moved there) become
 * E4M3_RNE(code * old / scale), as do all moved ones whose block's scale was another:
 * codes under the same scale are copied. (Two operations in binary32, then the
 * rounding; positive scales.) Rows of the block behind the kept ones are left as they
 * are.
 *
 * block_table  device, int32 [B, table_width], row stride table_stride; positions past
 *              it do not move.
 * seq_lens, query_lens, kept_lens  device, int32 [B]; kept int32 [B, kept_width], row
 *              stride kept_stride.
 * seq_lens_out device, int32 [B], or NULL; apart from the other lengths, the lists and
 *              the tables.
 * pools, scales  arrays on the HOST, [num_pools], of device pointers: 16-byte aligned
 *              (rows as they are: 8), scales 4-byte. Read during the call only. No two
 *              of the pools and scales share memory.
 * B * heads below 2^24, table_width * block_size at most 2^30.
 */
typedef struct smla_keep_tokens_params {
    size_t size; /* sizeof(smla_keep_tokens_params) */
    const int32_t *block_table;
    int64_t table_stride;
    int table_width;
    const int32_t *seq_lens, *query_lens, *kept;
    int64_t kept_stride;
    int kept_width;
    const int32_t *kept_lens;
    int32_t *seq_lens_out;
    int B, heads, block_size, row_bytes;
    int64_t num_blocks;
    int num_pools;
    void *const *pools;
    float *const *scales;
    smla_stream_t stream;
} smla_keep_tokens_params;

SMLA_API smla_status smla_keep_tokens(const smla_keep_tokens_params *params);

/*
 * Block tables that go on from others: new row b holds the first blocks of old row
 * source_rows[b] (shared with it and with whatever other rows hold them), as many as
 * its first n = seq_lens[b] tokens need (at most those that blocks_held says are
 * there); source_rows[b] outside [0, B_old) makes an empty row. One call forks requests
 * (several rows from one), reorders beams, cuts requests back, ends them:
 *   - a last block that is not full will be written to, so it must be its row's alone.
 *     Where other new rows hold it as well, one that holds it full keeps it, else the
 *     first row that ends in it; every other row that ends in it gets a new block, the
 *     free ring's next (rows in order), and copy_from[b], copy_to[b] name both blocks
 *     for smla_copy_blocks (-1, -1 for rows that need no copy);
 *   - blocks of the old rows that no new row holds go back to the ring, behind its end,
 *     each once, in the order of their first places (old rows in order, then entries).
 * The ring is that of smla_build_block_tables. Nothing is counted between calls: every
 * row that holds blocks is among the old rows, and every old row that is to live on is
 * some new row's source. Rows that share blocks end and shrink by this call;
 * smla_build_block_tables may then let all rows grow (but would give a shared block back
 * while others hold it). If the ring holds too few blocks, counts[3] says how many lack,
 * the copies are all -1 and nothing else changes (block_table_out and blocks_held_out
 * are not written).
 *
 * source_rows, seq_lens  device, int32 [B].
 * blocks_held  device, int32 [B_old]; block_table device, int32 [B_old, table_width],
 *              row stride table_stride.
 * blocks_held_out  device, int32 [B], block_table_out device, int32 [B, table_width],
 *              row stride table_out_stride: written (the entries of blocks held; others
 *              keep what they hold). They must not overlap the old ones.
 * num_blocks   of the pool: entries outside [0, num_blocks) are carried on, never
 *              copied and never given back.
 * free_ring, ring_size, ring_state, ring_state_out  as for smla_build_block_tables.
 * copy_from, copy_to  device, int32 [B], written.
 * counts       device, int32 [4], written: tokens that the new rows hold, blocks taken,
 *              given back, lacking.
 * workspace    device, smla_fork_block_tables_workspace_size(...) bytes, 16-byte
 *              aligned; need not be initialised. Calls that overlap in time must not
 *              share it.
 * B, B_old and table_width at most 2^30, their products with table_width below 2^31,
 * table_width * block_size at most 2^30, num_blocks below 2^31.
 */
typedef struct smla_fork_block_tables_params {
    size_t size; /* sizeof(smla_fork_block_tables_params) */
    const int32_t *source_rows, *seq_lens;
    int B;
    const int32_t *blocks_held;
    int B_old;
    const int32_t *block_table;
    int64_t table_stride;
    int32_t *blocks_held_out;
    int32_t *block_table_out;
    int64_t table_out_stride;
    int table_width, block_size;
    int64_t num_blocks;
    int32_t *free_ring;
    int ring_size;
    const int32_t *ring_state;
    int32_t *ring_state_out;
    int32_t *copy_from, *copy_to, *counts;
    void *workspace;
    size_t workspace_bytes;
    smla_stream_t stream;
} smla_fork_block_tables_params;

/* (size_t)-1 on invalid arguments. */
SMLA_API size_t smla_fork_block_tables_workspace_size(int B_old, int B, int table_width, int64_t num_blocks);
SMLA_API smla_status smla_fork_block_tables(const smla_fork_block_tables_params *params);

/*
 * Copies blocks within each of several pools (every layer's keys, values and scales in
 * one call): block copy_from[i] to block copy_to[i], i < n. A pair with a number outside
 * [0, num_blocks), or the same twice, copies nothing. A block that is copied to must not
 * stand among the others of either list that copy (a block may be copied from many
 * times).
 *
 * pools, block_bytes  arrays on the HOST, [num_pools]: the device pointer to a pool and
 *              the bytes of one of its blocks (any; whole 16-byte pieces move fastest).
 *              Read during the call only.
 * copy_from, copy_to  device, int32 [n].
 */
SMLA_API smla_status smla_copy_blocks(void *const *pools, const int64_t *block_bytes, int num_pools,
                                      const int32_t *copy_from, const int32_t *copy_to, int n, int64_t num_blocks,
                                      smla_stream_t stream);

/*
 * Error word of the device-side checks (0 = none). The tcgen05 kernels wait on
 * the tensor core and on their own warps with a time limit (about 2 s); a wait
 * that gives up sets a bit here (1 = an awaited barrier never completed,
 * 2 = the copies or MMAs in flight did not drain), abandons the call's
 * arithmetic, frees its tensor memory and returns, leaving the context usable.
 * smla_fused_qk_rope_cache, smla_rope and smla_qk_norm_rope set 4 for a position
 * outside [0, max_position); smla_fused_qk_rope_cache and smla_kv8_append set 8 for a
 * slot past the pool; smla_build_tree_masks and smla_keep_tokens both set 16, for trees
 * and for lists of kept tokens that are none (a caller that has to tell them apart reads
 * the word between the two). The waits of smla_kv8_attn_fwd and smla_kv8_tree_attn_fwd
 * for their copies and products have the same limit and bits as the forward's.
 * Synchronous (copies the word from the device): unlike every other entry point it waits for the device, since the word is
 * read on the host. reset != 0 clears it.
 */
SMLA_API smla_status smla_device_error(int *code, int reset);

/*
 * Per-tensor fp8 scale of a bf16 tensor [P4 Test plan: scaled_fp8_quant with a
 * per-tensor scale]: *scale_out = amax(|x|) / 448 in binary32, or 1.0 when
 * amax == 0. NaN elements are ignored.
 * x          device, bf16 [n], 16-byte aligned (may be NULL when n == 0).
 * scale_out  device, one float, 4-byte aligned; used as the reduction cell
 *            during the call.
 */
SMLA_API smla_status smla_compute_fp8_scale(const void *x, int64_t n, float *scale_out,
                                            smla_stream_t stream);

/*
 * Quantizing cache write [P4 Summary and Test plan: concat_and_cache_mla into
 * an fp8 cache]: for n in [0, N) with slot = slot_mapping[n] in [0, num_slots):
 *   kv_cache[slot, d] = E4M3_RNE_satfinite(src[n, d] / *kv_scale)   (binary32
 *   division), d in [0, D). slot == -1 skips the row, as does any slot outside
 *   [0, num_slots) (a contract violation).
 * src          device, bf16 [N, D], 16-byte aligned, D a multiple of 8.
 * slot_mapping device, int64 [N].
 * kv_scale     device, one float.
 * kv_cache     device, uint8 [num_slots, D], 8-byte aligned.
 */
SMLA_API smla_status smla_fp8_cache_write(const void *src, const int64_t *slot_mapping,
                                          int64_t N, int D, const float *kv_scale,
                                          void *kv_cache, int64_t num_slots,
                                          smla_stream_t stream);

/*
 * The fused producer step of sparse MLA decode [P4 Summary: main RoPE on
 * q_pe/k_pe, the query concat, the KV concat and the fp8 KV-cache write in one
 * kernel; Test plan: parity with the split chain]. For each token t, with
 * p = positions[t] and R = the rotation below:
 *   q_out[t, h, :]  = concat(ql_nope[t, h, 0:512], R_p(q_pe[t, h, 0:64]))   h in [0, H)
 *   kv_cache[slot_mapping[t], :] = concat(kv_c[t, 0:512], R_p(k_pe[t, 0:64]))
 * stored as bf16, or (q_out_dtype / kv_dtype = SMLA_KV_FP8_E4M3) as the codes
 * E4M3_RNE_satfinite(x / *q_scale) resp. (x / *kv_scale), binary32 division of
 * the bf16 value x (the scaled_fp8_quant convention).
 * R_p rotates each pair (a, b) to (a cos - b sin, b cos + a sin) with
 * cos = cos_sin_cache[p, i], sin = cos_sin_cache[p, 32 + i] for pair i: in
 * binary32, each product and the difference or sum rounded (no fused
 * multiply-add), then rounded to bf16 before any quantization, as the split
 * chain stores it. is_neox != 0 pairs element i with i + 32, else 2i with
 * 2i + 1.
 *
 * ql_nope        device, bf16 [T, H, 512], element strides (ql_stride_t,
 *                ql_stride_h), the last dimension contiguous; strides
 *                multiples of 8, pointer 16-byte aligned (a transposed
 *                [H, T, 512] buffer is stride_t = 512, stride_h = T * 512).
 * q_pe           device, bf16 [T, H, 64] pre-RoPE, strides (qpe_stride_t,
 *                qpe_stride_h), even, pointer 4-byte aligned.
 * kv_c           device, bf16 [T, 512], row stride kvc_stride_t (multiple of
 *                8), 16-byte aligned.
 * k_pe           device, bf16 [T, 64] pre-RoPE, row stride kpe_stride_t (even),
 *                4-byte aligned.
 * positions      device, int64 [T].
 * cos_sin_cache  device, float [max_position, 64]: 32 cosines then 32 sines.
 * slot_mapping   device, int64 [T]; a negative slot writes no cache row.
 * kv_cache       device, [num_slots, 576] bf16 or E4M3 (kv_dtype), 16-byte aligned.
 * kv_scale       device, one float; required for an E4M3 cache.
 * q_out          device, [T, H, 576] bf16 or E4M3 (q_out_dtype), contiguous,
 *                16-byte aligned; must not overlap the inputs.
 * q_scale        device, one float; required for E4M3 q_out.
 * H may be 0 (cache rows only; the q pointers may then be NULL); H above
 * 524279 is SMLA_ERR_BAD_SHAPE.
 * A token whose position is outside [0, max_position) gets neither its q rows
 * nor its cache row, and sets bit 4 of smla_device_error; a slot >= num_slots
 * writes no row and sets bit 8. Asynchronous on `stream`.
 */
SMLA_API smla_status smla_fused_qk_rope_cache(const void *ql_nope, int64_t ql_stride_t, int64_t ql_stride_h,
                                              const void *q_pe, int64_t qpe_stride_t, int64_t qpe_stride_h,
                                              const void *kv_c, int64_t kvc_stride_t, const void *k_pe,
                                              int64_t kpe_stride_t, const int64_t *positions,
                                              const float *cos_sin_cache, int64_t max_position, int is_neox,
                                              const int64_t *slot_mapping, void *kv_cache, int kv_dtype,
                                              int64_t num_slots, const float *kv_scale, void *q_out,
                                              int q_out_dtype, const float *q_scale, int T, int H,
                                              smla_stream_t stream);

/*
 * Measurement kernels (not part of the forward; bench.py reports them beside
 * the forward's rate as the ceilings it is held against).
 *
 * smla_gather_probe: a pure indexed-row copy at the forward kernels' gather
 * pattern. The n_indices entries of `indices` are taken as consecutive tiles
 * of 64 rows, split evenly over ctas_per_sm CTAs on each SM; each CTA copies
 * its tiles' rows [idx, 0:row_bytes) of the pool [num_rows, row_bytes]
 * (row_bytes a multiple of 16, at most 1024) into a ring of `stages` tiles in
 * shared memory (128-byte column blocks, 128-byte swizzle): copy_mode 0 by TMA
 * tile::gather4 (128-byte boxes), copy_mode 1 by 16-byte cp.async copies from
 * eight warps (pair_mode and issue_warps 0, else SMLA_ERR_UNSUPPORTED). -1
 * and out-of-range entries are zero-filled without a read. A consumer folds
 * the first 4 bytes of each row into checksum[cta] (XOR, written; device
 * uint32 [sm_count * ctas_per_sm]) and holds each tile hold_ns nanoseconds
 * before releasing it. SMLA_ERR_UNSUPPORTED when `stages` tiles do not fit
 * ctas_per_sm CTAs on one SM; ctas_per_sm in 1..4, stages in 1..8.
 * pair_mode (with ctas_per_sm = 1): 0 = single CTAs; 1 or 2 = CTAs in pairs,
 * each pair a thread-block cluster of two that takes the tiles one CTA would:
 * each CTA gathers half of every tile's rows (so every row is read once) and
 * delivers it to both CTAs: its landed half goes into the peer's ring by a
 * warp's 16-byte stores (1) or by a bulk copy (2); a stage is refilled
 * once both consumers released it (the patterns of a pair that shares its key
 * rows). Only the first CTA of a pair writes its checksum (the second writes
 * 0). 3 = single CTAs launched in clusters of two (a control for 1 and 2).
 * issue_warps: 0 = copy c of a tile (c < 16 * boxes per row, boxes =
 * row_bytes / 128 rounded up; half that in pair modes 1 and 2) is issued by
 * producer thread c of four warps; 1..8 = the copies are spread evenly over
 * that many warps, ceil(copies / issue_warps) lanes each, which must not
 * exceed 32 (else SMLA_ERR_BAD_SHAPE).
 *
 * smla_l2_read_probe: `blocks` blocks of 512 threads read the first `bytes`
 * of `buf` (a multiple of 16, 16-byte aligned) `reps` times with 16-byte
 * loads that bypass L1, and write one word per block to checksum[block]. With
 * a buffer smaller than L2 its rate is the L2 -> SM read bandwidth.
 */
SMLA_API smla_status smla_gather_probe(const void *pool, int64_t num_rows, int row_bytes,
                                       const int32_t *indices, int64_t n_indices, int ctas_per_sm,
                                       int stages, int hold_ns, int pair_mode, int issue_warps, int copy_mode,
                                       uint32_t *checksum, smla_stream_t stream);
SMLA_API smla_status smla_l2_read_probe(const void *buf, int64_t bytes, int reps, uint32_t *checksum,
                                        int blocks, smla_stream_t stream);

/*
 * Counts the entries of indices [T, topk] that are neither -1 nor inside
 * [0, num_slots) and stores the count in *bad_count (device int, overwritten).
 */
SMLA_API smla_status smla_validate_indices(const int32_t *indices, int T, int topk,
                                           int64_t num_slots, int *bad_count,
                                           smla_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SPARSE_MLA_H */

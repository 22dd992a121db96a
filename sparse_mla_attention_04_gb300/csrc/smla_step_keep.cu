// The rows of kept tokens moved together behind their request's context, and copies
// of whole blocks, in many layers' pools at once (sm_103a).
//
// Kept token i, drafted as node kept[i], goes from position ctx + kept[i] to ctx + i.
// The nodes ascend strictly, so kept[i] >= i: rows move towards the front, and no row
// is written over before it is read as long as rows go in order and a batch of them
// is read whole before it is written. So one warp (block-scaled: of one head of one
// pool) or one block (plain rows) moves a request's rows in place, and nothing is
// shared between teams.
//
// Block-scaled: a block's scale becomes the largest of its own and of those of the
// blocks that rows come from; where that grew, the codes that stay follow. A later
// block is a source of an earlier one, never the other way round, so blocks in order
// find the scales of their sources as they were. Bound: latency (lengths, then the
// table, then scales, then rows, each behind the last), and for many layers the rows.
// Measured on the device: 64 requests that keep some four of up to 32 nodes, in eight
// layers of 8 heads of 128 columns (a launch of 8192 warps), in 7.0 us; one request in two
// latent pools 3.2 us.
//
// Copies: a block to 16 KB of a block's copy, four 16-byte pieces of a thread in flight.
// Bound: HBM. Measured: 173 blocks of 64 positions, 8 heads of 128 columns, in 16 layers'
// keys and values (725 MB read and written) in 98.5 us, 7.4 TB/s: a third of them are
// copies of one block, which the L2 cache holds.
#include "smla_device.cuh"
#include "smla_kv8_codes.cuh"
#include "smla_step.h"

#include <algorithm>
#include <climits>

namespace smla {

__device__ int g_keep_error = 0; // bit 16: kept nodes that do not ascend, or past the request's new tokens

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;

// A request's new tokens and how many of them are kept.
struct Kept {
    int ctx, count;
    const int32_t *nodes;
};

// By a whole warp.
__device__ __forceinline__ Kept kept_of(const KeepArgs &a, int b, int lane, bool report)
{
    const int len = max(a.seq_lens[b], 0), n = min(max(a.query_lens[b], 0), len);
    Kept k{len - n, min(max(a.kept_lens[b], 0), min(a.kept_width, n)), a.kept + b * a.kept_stride};
    int before = -1;
    bool bad = a.kept_lens[b] > min(a.kept_width, n); // (more than there can be)
    for (int i0 = 0; i0 < k.count; i0 += 32) {
        const int x = i0 + lane < k.count ? k.nodes[i0 + lane] : INT_MAX;
        int up = __shfl_up_sync(0xffffffffu, x, 1);
        up = lane == 0 ? before : up;
        const unsigned wrong = __ballot_sync(0xffffffffu, i0 + lane < k.count && (x <= up || x >= n));
        if (wrong) {
            k.count = i0 + __ffs(wrong) - 1;
            bad = true;
            break;
        }
        before = __shfl_sync(0xffffffffu, x, 31);
    }
    if (bad && report && lane == 0)
        atomicOr(&g_keep_error, 16);
    return k;
}

// The pool block of a position (-1: none).
__device__ __forceinline__ int block_at(const KeepArgs &a, int b, int pos)
{
    const int j = pos >> a.block_shift;
    const int e = j < a.table_width ? a.block_table[b * a.table_stride + j] : -1;
    return e >= 0 && e < a.num_blocks ? e : -1;
}

// Sixteen codes under another scale.
__device__ __forceinline__ uint4 rescaled(const uint4 &v, float old, float now)
{
    return make_uint4(requant4(v.x, old, now), requant4(v.y, old, now), requant4(v.z, old, now), requant4(v.w, old, now));
}

// Block-scaled pools: a warp to a request, head and pool.
__global__ void __launch_bounds__(kThreads) keep_scaled_kernel(const __grid_constant__ KeepArgs a)
{
    const int lane = threadIdx.x & 31;
    const int64_t team = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int pool = (int)(team % a.pools);
    const int64_t rest = team / a.pools;
    const int h = (int)(rest % a.heads), b = (int)min(rest / a.heads, (int64_t)INT_MAX);
    if (b >= a.B)
        return;
    const bool first = pool == 0 && h == 0;
    const Kept k = kept_of(a, b, lane, first);
    if (first && lane == 0 && a.seq_lens_out)
        a.seq_lens_out[b] = k.ctx + k.count;
    const int vecs = a.row_bytes / 16, per = 32 / vecs; // of a row; rows of a round
    const int vec = lane % vecs, row_in = lane / vecs;
    const int bs = 1 << a.block_shift;
    uint8_t *codes = a.codes[pool];
    float *scales = a.scales[pool];
    const auto base_of = [&](int block) {
        return reinterpret_cast<uint4 *>(codes + ((((int64_t)block * a.heads + h) << a.block_shift)) * a.row_bytes);
    };
    for (int i0 = 0; i0 < k.count;) {
        const int d0 = k.ctx + i0, off = d0 & (bs - 1);
        const int i1 = min(k.count, i0 + bs - off); // the rows that go to this block
        const int to = block_at(a, b, d0);
        if (to < 0) {
            i0 = i1;
            continue;
        }
        float *scale = scales + (int64_t)to * a.heads + h;
        const float old = *scale;
        float now = old;
        int from = -1, at = 0; // of row c0 + lane: its block and row there, the block's scale
        float was = 0.f;
        const auto look = [&](int c0) {
            const int i = c0 + lane;
            from = -1;
            if (i < i1) {
                const int s = k.ctx + k.nodes[i];
                from = block_at(a, b, s);
                at = s & (bs - 1);
                was = from < 0 ? 0.f : from == to ? old : scales[(int64_t)from * a.heads + h];
            }
        };
        for (int c0 = i0; c0 < i1; c0 += 32) {
            look(c0);
            now = fmaxf(now, warp_max(from < 0 ? 0.f : was));
        }
        const bool grown = now > old;
        if (grown)
            for (int x = lane; x < off * vecs; x += 32) {
                uint4 *p = base_of(to) + x;
                *p = rescaled(*p, old, now);
            }
        for (int c0 = i0; c0 < i1; c0 += 32) {
            if (i1 - i0 > 32) // (else what was looked at stands)
                look(c0);
            for (int r0 = 0; r0 < min(32, i1 - c0); r0 += per) {
                const int r = r0 + row_in; // (beyond the last: nothing)
                const int f = __shfl_sync(0xffffffffu, from, r), o = __shfl_sync(0xffffffffu, at, r);
                const float w = __shfl_sync(0xffffffffu, was, r);
                const int d = (off + c0 - i0 + r) & (bs - 1);
                const bool moves = f >= 0 && (f != to || o != d || w != now);
                uint4 v = make_uint4(0, 0, 0, 0);
                if (moves)
                    v = base_of(f)[o * vecs + vec];
                __syncwarp();
                if (moves)
                    base_of(to)[d * vecs + vec] = w == now ? v : rescaled(v, w, now);
            }
            __syncwarp();
        }
        if (grown && lane == 0)
            *scale = now;
        __syncwarp();
        i0 = i1;
    }
}

// Plain rows of kVec-byte pieces: a block to a request, head and pool.
template <typename V>
__global__ void __launch_bounds__(kThreads) keep_rows_kernel(const __grid_constant__ KeepArgs a)
{
    constexpr int kHeld = 4; // pieces of a thread between reading and writing
    __shared__ int s_count;
    const int pool = (int)((int64_t)blockIdx.x % a.pools), rest = (int)((int64_t)blockIdx.x / a.pools);
    const int h = rest % a.heads, b = rest / a.heads;
    const bool first = pool == 0 && h == 0;
    if (threadIdx.x < 32) {
        const Kept k = kept_of(a, b, threadIdx.x, first);
        if (threadIdx.x == 0) {
            s_count = k.count;
            if (first && a.seq_lens_out)
                a.seq_lens_out[b] = k.ctx + k.count;
        }
    }
    __syncthreads();
    const int len = max(a.seq_lens[b], 0), ctx = len - min(max(a.query_lens[b], 0), len);
    const int vecs = a.row_bytes / (int)sizeof(V), bs = 1 << a.block_shift;
    const int64_t total = (int64_t)s_count * vecs;
    const int32_t *nodes = a.kept + b * a.kept_stride;
    const auto row = [&](int pos) {
        const int e = block_at(a, b, pos);
        return e < 0 ? nullptr
                     : reinterpret_cast<V *>(a.codes[pool] +
                                             ((((int64_t)e * a.heads + h) << a.block_shift) + (pos & (bs - 1))) * a.row_bytes);
    };
    for (int64_t x0 = 0; x0 < total; x0 += kThreads * kHeld) {
        V v[kHeld];
        V *to[kHeld];
#pragma unroll
        for (int j = 0; j < kHeld; ++j) {
            const int64_t x = x0 + j * kThreads + threadIdx.x;
            to[j] = nullptr;
            if (x < total) {
                const int i = (int)(x / vecs), p = (int)(x % vecs), node = nodes[i];
                const V *from = node != i ? row(ctx + node) : nullptr; // (where it is already: nothing)
                if (from) {
                    to[j] = row(ctx + i);
                    if (to[j]) {
                        to[j] += p;
                        v[j] = from[p];
                    }
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kHeld; ++j)
            if (to[j])
                *to[j] = v[j];
    }
}

// Block from[i] of every pool to to[i]. V: what the pools' blocks are whole numbers of.
constexpr int kCopyThreads = 256, kCopyHeld = 4;
template <typename V>
__device__ __forceinline__ void copy_block(uint8_t *pool, int64_t bytes, int from, int to)
{
    const int64_t n = bytes / (int64_t)sizeof(V);
    const V *src = reinterpret_cast<const V *>(pool + from * bytes);
    V *dst = reinterpret_cast<V *>(pool + to * bytes);
    for (int64_t x0 = (int64_t)blockIdx.z * kCopyThreads * kCopyHeld; x0 < n; x0 += (int64_t)gridDim.z * kCopyThreads * kCopyHeld) {
        V v[kCopyHeld];
#pragma unroll
        for (int j = 0; j < kCopyHeld; ++j)
            if (const int64_t x = x0 + j * kCopyThreads + threadIdx.x; x < n)
                v[j] = src[x];
#pragma unroll
        for (int j = 0; j < kCopyHeld; ++j)
            if (const int64_t x = x0 + j * kCopyThreads + threadIdx.x; x < n)
                dst[x] = v[j];
    }
}

__global__ void __launch_bounds__(kCopyThreads) copy_blocks_kernel(const __grid_constant__ CopyArgs a)
{
    const int from = a.from[blockIdx.x], to = a.to[blockIdx.x];
    if (from < 0 || to < 0 || from >= a.num_blocks || to >= a.num_blocks || from == to)
        return;
    uint8_t *pool = a.pool[blockIdx.y];
    const int64_t bytes = a.block_bytes[blockIdx.y];
    const uint64_t bits = reinterpret_cast<uintptr_t>(pool) | (uint64_t)bytes;
    if (bits % 16 == 0)
        copy_block<uint4>(pool, bytes, from, to);
    else if (bits % 4 == 0)
        copy_block<uint32_t>(pool, bytes, from, to);
    else
        copy_block<uint8_t>(pool, bytes, from, to);
}

} // namespace

cudaError_t launch_keep_tokens(const KeepArgs &a, bool scaled, int sm_count, cudaStream_t stream)
{
    (void)sm_count;
    const int64_t teams = (int64_t)a.B * a.heads * a.pools;
    const int64_t blocks = scaled ? (teams + kWarps - 1) / kWarps : teams;
    if (blocks > INT_MAX)
        return cudaErrorInvalidValue;
    if (scaled) {
        keep_scaled_kernel<<<(unsigned)blocks, kThreads, 0, stream>>>(a);
        return cudaGetLastError();
    }
    uintptr_t bits = a.row_bytes;
    for (int i = 0; i < a.pools; ++i)
        bits |= reinterpret_cast<uintptr_t>(a.codes[i]);
    if (bits % 16 == 0)
        keep_rows_kernel<uint4><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
    else
        keep_rows_kernel<uint2><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_copy_blocks(const CopyArgs &a, int sm_count, cudaStream_t stream)
{
    (void)sm_count;
    int64_t most = 0;
    for (int i = 0; i < a.pools; ++i)
        most = std::max(most, a.block_bytes[i]);
    const int64_t chunk = 16 * kCopyThreads * kCopyHeld;
    const dim3 grid((unsigned)a.n, (unsigned)a.pools, (unsigned)std::min<int64_t>(std::max<int64_t>(1, (most + chunk - 1) / chunk), 64));
    copy_blocks_kernel<<<grid, kCopyThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t read_keep_error(int *out, bool reset)
{
    cudaError_t e = cudaMemcpyFromSymbol(out, g_keep_error, sizeof(int));
    if (e == cudaSuccess && reset) {
        const int zero = 0;
        e = cudaMemcpyToSymbol(g_keep_error, &zero, sizeof(int));
    }
    return e;
}

} // namespace smla

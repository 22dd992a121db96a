// Block tables and slot maps of a serving step, from the requests' lengths
// (sm_103a): two running sums over the requests (new tokens; blocks taken and
// given back), then independent fills of tokens and table entries.
//
// Work and bound: 12 bytes read per request, 20 written per token. A decode
// step is a few kilobytes, so it is one launch of one block, whose scan and
// fill meet in block barriers; past kOneBlockTokens tokens the fill is a second
// launch over the whole GPU and the plan passes through the workspace. No
// entry that one thread writes is read by another within the fill: a token
// whose block is new takes it from the ring, as the table's writer does.
#include "smla_device.cuh"
#include "smla_internal.h"

#include <climits>

namespace smla {
namespace {

constexpr int kThreads = 1024;
// Above this many tokens the fill runs on the whole GPU.
constexpr int kOneBlockTokens = 4096;

struct Sums {
    long long q, take, give;
};

__device__ __forceinline__ Sums add(const Sums &a, const Sums &b) { return {a.q + b.q, a.take + b.take, a.give + b.give}; }

__device__ __forceinline__ Sums shfl_up(const Sums &a, int d)
{
    return {__shfl_up_sync(0xffffffffu, a.q, d), __shfl_up_sync(0xffffffffu, a.take, d),
            __shfl_up_sync(0xffffffffu, a.give, d)};
}

// Exclusive sum over the block's threads; `total` gets the whole sum.
__device__ Sums block_exclusive(const Sums &v, Sums *total, Sums *warp_sums)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Sums inc = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const Sums o = shfl_up(inc, d);
        if (lane >= d)
            inc = add(inc, o);
    }
    if (lane == 31)
        warp_sums[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        Sums w = warp_sums[lane];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const Sums o = shfl_up(w, d);
            if (lane >= d)
                w = add(w, o);
        }
        warp_sums[lane] = w;
    }
    __syncthreads();
    const Sums base = warp > 0 ? warp_sums[warp - 1] : Sums{0, 0, 0};
    *total = warp_sums[31];
    __syncthreads();
    return {base.q + inc.q - v.q, base.take + inc.take - v.take, base.give + inc.give - v.give};
}

struct Request {
    int len, q, held, need;
};

__device__ __forceinline__ Request request(const TablesArgs &a, int b)
{
    Request r;
    r.len = max(a.seq_lens[b], 0);
    r.q = min(max(a.query_lens[b], 0), r.len);
    r.held = min(max(a.blocks_held[b], 0), a.table_width);
    r.need = (int)(((long long)r.len + a.block_size - 1) >> a.block_shift);
    return r;
}

__device__ __forceinline__ int clamp31(long long v) { return (int)min(v, (long long)INT_MAX); }

__device__ __forceinline__ int ring_at(const TablesArgs &a, int head, long long i)
{
    return a.free_ring[(head + i) % a.ring_size];
}

// One token's position, slot and request. plan[b] = {first taken block of the
// batch, held blocks, blocks after the call, length}.
__device__ __forceinline__ void fill_token(const TablesArgs &a, int64_t t, int b, int start, int4 p, int q, int head)
{
    const int pos = p.w - q + (int)(t - start);
    const int j = pos >> a.block_shift;
    int block = -1;
    if (j < p.z)
        block = j < p.y ? a.block_table[b * a.table_stride + j] : ring_at(a, head, p.x + j - p.y);
    a.positions[t] = pos;
    a.slot_mapping[t] = block < 0 ? -1 : (int64_t)block * a.block_size + (pos & (a.block_size - 1));
    if (a.token_request)
        a.token_request[t] = b;
}

// The request of token t: the last b in [lo, hi] with start[b] <= t (empty
// requests share their start with the next one, which the last b skips).
__device__ __forceinline__ int find_request(const int32_t *start, int lo, int hi, int64_t t)
{
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (start[mid] <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// Table entries and the ring's end: a warp to a request. `give` is the first
// given-back block's place behind the ring's end.
__device__ __forceinline__ void fill_blocks(const TablesArgs &a, int b, int4 p, int give, int head, int count, int lane)
{
    int32_t *row = a.block_table + b * a.table_stride;
    for (int j = p.y + lane; j < p.z; j += 32)
        row[j] = ring_at(a, head, p.x + j - p.y);
    for (int j = p.z + lane; j < p.y; j += 32)
        a.free_ring[((long long)head + count + give + j - p.z) % a.ring_size] = row[j];
}

// The scan, by one block. With `fill`, the fill too. The inputs are all read
// before the outputs that may be the same buffers (held counts, ring state)
// are written.
template <bool kFill>
__global__ void __launch_bounds__(kThreads) tables_scan_kernel(const TablesArgs a)
{
    __shared__ Sums warp_sums[32];
    __shared__ int s_state[2];
    const int tid = threadIdx.x;
    if (tid == 0) {
        const int h = a.ring_state[0] % a.ring_size;
        s_state[0] = h < 0 ? h + a.ring_size : h;
        s_state[1] = min(max(a.ring_state[1], 0), a.ring_size);
    }
    Sums all{0, 0, 0};
    long long lacking = 0;
    // first pass: what the batch takes in all (with up to kThreads requests
    // the second pass's numbers are the first's)
    for (int b0 = 0; b0 < a.B; b0 += kThreads) {
        const int b = b0 + tid;
        Sums v{0, 0, 0};
        int wide = 0;
        if (b < a.B) {
            const Request r = request(a, b);
            v = {r.q, max(r.need - r.held, 0), max(r.held - r.need, 0)};
            wide = max(r.need - a.table_width, 0);
        }
        Sums total;
        const Sums x{v.q, v.take, v.give};
        (void)block_exclusive(x, &total, warp_sums);
        all = add(all, total);
        Sums w{wide, 0, 0};
        if (__syncthreads_or(wide)) {
            (void)block_exclusive(w, &total, warp_sums);
            lacking += total.q;
        }
    }
    __syncthreads();
    const int head = s_state[0], count = s_state[1];
    lacking += max(all.take - count, 0ll);
    const bool ok = lacking == 0;
    Sums carry{0, 0, 0};
    for (int b0 = 0; b0 < a.B; b0 += kThreads) {
        const int b = b0 + tid;
        Sums v{0, 0, 0};
        Request r{0, 0, 0, 0};
        if (b < a.B) {
            r = request(a, b);
            v = {r.q, max(r.need - r.held, 0), max(r.held - r.need, 0)};
        }
        Sums total;
        const Sums x = add(carry, block_exclusive(v, &total, warp_sums));
        if (b < a.B) {
            const int after = ok ? r.need : r.held;
            a.query_start[b] = clamp31(x.q);
            a.plan[b] = make_int4(clamp31(x.take), r.held, after, r.len);
            a.give_start[b] = clamp31(x.give);
            a.blocks_held_out[b] = after;
        }
        carry = add(carry, total);
    }
    if (tid == 0) {
        a.query_start[a.B] = clamp31(all.q);
        a.counts[0] = clamp31(all.q);
        a.counts[1] = ok ? clamp31(all.take) : 0;
        a.counts[2] = ok ? clamp31(all.give) : 0;
        a.counts[3] = clamp31(lacking);
        a.ring_state_out[0] = ok ? (int)((head + all.take) % a.ring_size) : head;
        a.ring_state_out[1] = ok ? (int)min(count - all.take + all.give, (long long)a.ring_size) : count;
        if (!kFill) {
            a.state[0] = head;
            a.state[1] = count;
        }
    }
    if (kFill) {
        __syncthreads();
        const int lane = tid & 31, warp = tid >> 5;
        // tokens read old table entries and the ring; blocks that were given
        // back are only written over ring places that hold none
        for (int64_t t = tid; t < a.num_tokens; t += kThreads) {
            if (t < all.q) {
                const int b = find_request(a.query_start, 0, a.B - 1, t);
                const int start = a.query_start[b];
                fill_token(a, t, b, start, a.plan[b], a.query_start[b + 1] - start, head);
            } else {
                a.positions[t] = 0;
                a.slot_mapping[t] = -1;
                if (a.token_request)
                    a.token_request[t] = -1;
            }
        }
        if (all.take + all.give > 0 && ok)
            for (int b = warp; b < a.B; b += kThreads / 32)
                fill_blocks(a, b, a.plan[b], a.give_start[b], head, count, lane);
    }
}

// The fill over the whole GPU: a warp takes 64 consecutive tokens (finds the
// requests of the first and the last, between which its lanes search), then
// one request's blocks.
__global__ void __launch_bounds__(256) tables_fill_kernel(const TablesArgs a)
{
    const int lane = threadIdx.x & 31;
    const int64_t warp = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int64_t warps = ((int64_t)gridDim.x * blockDim.x) >> 5;
    const int head = a.state[0], count = a.state[1];
    const int64_t total = a.counts[0];
    for (int64_t g = warp; g * 64 < a.num_tokens; g += warps) {
        const int64_t t0 = g * 64;
        int lo = 0, hi = 0;
        if (t0 < total) {
            lo = find_request(a.query_start, 0, a.B - 1, t0);
            hi = find_request(a.query_start, lo, min(a.B - 1, lo + 64), min(t0 + 63, total - 1));
            // more than 64 requests further on (empty ones between): search them all
            if (hi == lo + 64)
                hi = a.B - 1;
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int64_t t = t0 + k * 32 + lane;
            if (t >= a.num_tokens)
                break;
            if (t < total) {
                const int b = find_request(a.query_start, lo, hi, t);
                const int start = a.query_start[b];
                fill_token(a, t, b, start, a.plan[b], a.query_start[b + 1] - start, head);
            } else {
                a.positions[t] = 0;
                a.slot_mapping[t] = -1;
                if (a.token_request)
                    a.token_request[t] = -1;
            }
        }
    }
    if (a.counts[3] != 0)
        return;
    for (int64_t b = warp; b < a.B; b += warps)
        fill_blocks(a, (int)b, a.plan[b], a.give_start[b], head, count, lane);
}

} // namespace

cudaError_t launch_block_tables(const TablesArgs &a, int sm_count, cudaStream_t stream)
{
    if (a.num_tokens <= kOneBlockTokens) {
        tables_scan_kernel<true><<<1, kThreads, 0, stream>>>(a);
        return cudaGetLastError();
    }
    tables_scan_kernel<false><<<1, kThreads, 0, stream>>>(a);
    if (const cudaError_t e = cudaGetLastError(); e != cudaSuccess)
        return e;
    const int64_t blocks = (a.num_tokens / 64 + 7) / 8 + 1;
    const int64_t most = (int64_t)(sm_count > 0 ? sm_count : 1) * 8;
    tables_fill_kernel<<<(unsigned)(blocks < most ? blocks : most), 256, 0, stream>>>(a);
    return cudaGetLastError();
}

} // namespace smla

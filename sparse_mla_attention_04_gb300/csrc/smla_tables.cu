// Block tables and slot maps of a serving step, from the requests' lengths
// (sm_103a): two running sums over the requests (new tokens; blocks taken and
// given back), then independent fills of tokens and table entries.
//
// Work and bound: 12 bytes read per request, 20 written per token. A decode
// step is a few kilobytes, so it is one launch of one block (a thread to a
// request, the plan in shared memory); with more than kOneBlockTokens tokens or
// kThreads requests the fill is a second launch over the whole GPU and the plan
// passes through the workspace. No entry that one thread writes is read by
// another within the fill: a token whose block is new takes it from the ring, as
// the table's writer does. Measured on the device: a decode step of 64 requests 5.2
// us, 1000 requests with 1023872 new tokens between them 19 us (21 MB, 1.1 TB/s:
// the scan's one block, then the binary searches); 64-bit remainders of ring places
// alone had taken 10 us of the first.
#include "smla_device.cuh"
#include "smla_step.h"
#include "smla_umma.cuh"

#include <climits>

namespace smla {
namespace {

constexpr int kThreads = 1024;
// Above this many tokens the fill runs on the whole GPU: 4096 tokens of 4 requests 6.8 us
// by one block, 7.6 by two launches; 8192 of one 8.0 and 8.4; 16384 of 16 16.2 and 8.0.
constexpr int kOneBlockTokens = 4096;
// Up to this many requests a block of the whole-GPU fill searches a copy of the starts in shared memory.
constexpr int kSharedStarts = 4096;

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

// Places of the ring, i and head below 2^31 (32-bit remainders: 64-bit ones took most of a step's time).
__device__ __forceinline__ unsigned ring_place(const TablesArgs &a, unsigned head, unsigned i)
{
    return (head + i) % (unsigned)a.ring_size;
}
__device__ __forceinline__ int ring_at(const TablesArgs &a, int head, int i) { return a.free_ring[ring_place(a, head, i)]; }

// One token's position and slot. p: the request's plan {first taken block of the
// batch, held blocks, blocks after the call, length}.
__device__ __forceinline__ void token(const TablesArgs &a, int64_t t, int start, int4 p, int q, int head, int b, int64_t &pos,
                                      int64_t &slot)
{
    const int at = p.w - q + (int)(t - start);
    const int j = at >> a.block_shift;
    int block = -1;
    if (j < p.z)
        block = j < p.y ? a.block_table[b * a.table_stride + j] : ring_at(a, head, p.x + j - p.y);
    pos = at;
    slot = block < 0 ? -1 : (int64_t)block * a.block_size + (at & (a.block_size - 1));
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

// Table entries and the ring's end: a warp to a request, four entries of a lane
// in flight. `give` is the first given-back block's place behind the ring's end.
__device__ __forceinline__ void fill_blocks(const TablesArgs &a, int b, int4 p, int give, int head, int count, int lane)
{
    int32_t *row = a.block_table + b * a.table_stride;
#pragma unroll 4
    for (int j = p.y + lane; j < p.z; j += 32)
        row[j] = ring_at(a, head, p.x + j - p.y);
    const unsigned end = ring_place(a, head, count);
    for (int j = p.z + lane; j < p.y; j += 128) {
        int v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            v[k] = j + 32 * k < p.y ? row[j + 32 * k] : 0;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (j + 32 * k < p.y)
                a.free_ring[ring_place(a, end, give + j + 32 * k - p.z)] = v[k];
    }
}

__device__ __forceinline__ int2 ring_state(const TablesArgs &a)
{
    const int h = a.ring_state[0] % a.ring_size;
    return make_int2(h < 0 ? h + a.ring_size : h, min(max(a.ring_state[1], 0), a.ring_size));
}

__device__ __forceinline__ void finish_scan(const TablesArgs &a, const Sums &all, long long lacking, int head, int count)
{
    const bool ok = lacking == 0;
    a.query_start[a.B] = clamp31(all.q);
    a.counts[0] = clamp31(all.q);
    a.counts[1] = ok ? clamp31(all.take) : 0;
    a.counts[2] = ok ? clamp31(all.give) : 0;
    a.counts[3] = clamp31(lacking);
    a.ring_state_out[0] = ok ? (int)((head + all.take) % a.ring_size) : head;
    a.ring_state_out[1] = ok ? (int)min(count - all.take + all.give, (long long)a.ring_size) : count;
}

// Scan and fill by one block, a thread to a request (B <= kThreads). The
// inputs are all read before the outputs that may be the same buffers (held
// counts, ring state) are written.
__global__ void __launch_bounds__(kThreads) tables_small_kernel(const TablesArgs a)
{
    __shared__ Sums warp_sums[32];
    __shared__ int4 s_plan[kThreads];
    __shared__ int s_start[kThreads + 1], s_give[kThreads];
    __shared__ unsigned long long s_wide; // blocks that rows have no room for
    const int tid = threadIdx.x;
    const int2 ring = ring_state(a);
    const int head = ring.x, count = ring.y;
    Request r{0, 0, 0, 0};
    if (tid < a.B)
        r = request(a, tid);
    if (tid == 0)
        s_wide = 0;
    const Sums v{r.q, max(r.need - r.held, 0), max(r.held - r.need, 0)};
    Sums all;
    const Sums x = block_exclusive(v, &all, warp_sums);
    if (r.need > a.table_width)
        atomicAdd(&s_wide, (unsigned long long)(r.need - a.table_width)); // (whole numbers: any order)
    __syncthreads();
    const long long lacking = (long long)s_wide + max(all.take - count, 0ll);
    const bool ok = lacking == 0;
    if (tid < a.B) {
        const int after = ok ? r.need : r.held;
        s_start[tid] = clamp31(x.q);
        s_plan[tid] = make_int4(clamp31(x.take), r.held, after, r.len);
        s_give[tid] = clamp31(x.give);
        a.query_start[tid] = s_start[tid];
        a.blocks_held_out[tid] = after;
    }
    if (tid == 0) {
        s_start[a.B] = clamp31(all.q);
        finish_scan(a, all, lacking, head, count);
    }
    __syncthreads();
    for (int64_t t = tid; t < a.num_tokens; t += kThreads) {
        if (t < all.q) {
            const int b = find_request(s_start, 0, a.B - 1, t);
            int64_t pos, slot;
            token(a, t, s_start[b], s_plan[b], s_start[b + 1] - s_start[b], head, b, pos, slot);
            a.positions[t] = pos;
            a.slot_mapping[t] = slot;
            if (a.token_request)
                a.token_request[t] = b;
        } else {
            a.positions[t] = 0;
            a.slot_mapping[t] = -1;
            if (a.token_request)
                a.token_request[t] = -1;
        }
    }
    if (!ok)
        return;
    // entries that change, one to a thread: those taken, then those given back
    const unsigned end = ring_place(a, head, count);
    for (int64_t i = tid; i < all.take + all.give; i += kThreads) {
        const bool takes = i < all.take;
        const int x = (int)(takes ? i : i - all.take);
        int lo = 0, hi = a.B - 1; // the last request whose first entry is not behind x
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if ((takes ? s_plan[mid].x : s_give[mid]) <= x)
                lo = mid;
            else
                hi = mid - 1;
        }
        const int4 p = s_plan[lo];
        int32_t *row = a.block_table + lo * a.table_stride;
        if (takes)
            row[p.y + x - p.x] = ring_at(a, head, x);
        else
            a.free_ring[ring_place(a, end, x)] = row[p.z + x - s_give[lo]];
    }
}

// The scan alone, for any number of requests: one block, its plan to the workspace.
__global__ void __launch_bounds__(kThreads) tables_scan_kernel(const TablesArgs a)
{
    __shared__ Sums warp_sums[32];
    const int tid = threadIdx.x;
    const int2 ring = ring_state(a);
    const int head = ring.x, count = ring.y;
    umma::grid_launch_dependents();
    Sums all{0, 0, 0}, mine{0, 0, 0}; // (with one round, the second pass has its sums from the first)
    Request r{0, 0, 0, 0};
    long long lacking = 0;
    for (int b0 = 0; b0 < a.B; b0 += kThreads) {
        const int b = b0 + tid;
        Sums v{0, 0, 0};
        int wide = 0;
        if (b < a.B) {
            r = request(a, b);
            v = {r.q, max(r.need - r.held, 0), max(r.held - r.need, 0)};
            wide = max(r.need - a.table_width, 0);
        }
        Sums total;
        mine = block_exclusive(v, &total, warp_sums);
        all = add(all, total);
        if (__syncthreads_or(wide)) {
            (void)block_exclusive(Sums{wide, 0, 0}, &total, warp_sums);
            lacking += total.q;
        }
    }
    lacking += max(all.take - count, 0ll);
    const bool ok = lacking == 0;
    Sums carry{0, 0, 0};
    for (int b0 = 0; b0 < a.B; b0 += kThreads) {
        const int b = b0 + tid;
        Sums x = mine;
        if (a.B > kThreads) {
            Sums v{0, 0, 0}, total;
            if (b < a.B) {
                r = request(a, b);
                v = {r.q, max(r.need - r.held, 0), max(r.held - r.need, 0)};
            }
            x = add(carry, block_exclusive(v, &total, warp_sums));
            carry = add(carry, total);
        }
        if (b < a.B) {
            const int after = ok ? r.need : r.held;
            a.query_start[b] = clamp31(x.q);
            a.plan[b] = make_int4(clamp31(x.take), r.held, after, r.len);
            a.give_start[b] = clamp31(x.give);
            a.blocks_held_out[b] = after;
        }
    }
    if (tid == 0) {
        a.state[0] = head;
        a.state[1] = count;
        finish_scan(a, all, lacking, head, count);
    }
}

// The fill over the whole GPU: a warp takes 64 consecutive tokens (finds the
// requests of the first and the last, between which its lanes search), then
// one request's blocks.
template <bool kShared>
__global__ void __launch_bounds__(256) tables_fill_kernel(const TablesArgs a)
{
    __shared__ int s_start[kShared ? kSharedStarts + 1 : 1];
    umma::grid_wait(); // the scan is done
    const int32_t *start_of = a.query_start;
    if (kShared) {
        for (int i = threadIdx.x; i <= a.B; i += blockDim.x)
            s_start[i] = a.query_start[i];
        __syncthreads();
        start_of = s_start;
    }
    const int lane = threadIdx.x & 31;
    const int64_t warp = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int64_t warps = ((int64_t)gridDim.x * blockDim.x) >> 5;
    const int head = a.state[0], count = a.state[1];
    const int64_t total = a.counts[0];
    for (int64_t g = warp; g * 64 < a.num_tokens; g += warps) {
        const int64_t t0 = g * 64;
        int lo = 0, hi = 0;
        if (t0 < total) {
            lo = find_request(start_of, 0, a.B - 1, t0);
            hi = find_request(start_of, lo, a.B - 1, min(t0 + 63, total - 1));
        }
        // both of a lane's tokens' loads are in flight before either is written
        int64_t pos[2], slot[2];
        int req[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int64_t t = t0 + k * 32 + lane;
            pos[k] = 0;
            slot[k] = -1;
            req[k] = -1;
            if (t < total && t < a.num_tokens) {
                req[k] = find_request(start_of, lo, hi, t);
                token(a, t, start_of[req[k]], a.plan[req[k]], start_of[req[k] + 1] - start_of[req[k]], head, req[k], pos[k],
                      slot[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int64_t t = t0 + k * 32 + lane;
            if (t < a.num_tokens) {
                a.positions[t] = pos[k];
                a.slot_mapping[t] = slot[k];
                if (a.token_request)
                    a.token_request[t] = req[k];
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
    if (a.num_tokens <= kOneBlockTokens && a.B <= kThreads) {
        tables_small_kernel<<<1, kThreads, 0, stream>>>(a);
        return cudaGetLastError();
    }
    tables_scan_kernel<<<1, kThreads, 0, stream>>>(a);
    if (const cudaError_t e = cudaGetLastError(); e != cudaSuccess)
        return e;
    const int64_t blocks = (a.num_tokens / 64 + 7) / 8 + 1;
    const int64_t most = (int64_t)(sm_count > 0 ? sm_count : 1) * 8;
    // behind the scan, its start overlapped
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(blocks < most ? blocks : most));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, a.B <= kSharedStarts ? tables_fill_kernel<true> : tables_fill_kernel<false>, a);
}

} // namespace smla

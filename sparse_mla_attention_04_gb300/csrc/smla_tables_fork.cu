// Forked block tables (sm_103a): new rows that go on from old ones, the blocks that
// nobody holds any more back to the ring, and a block of its own for every row that
// will write into a block which another row holds too.
//
// Nothing is counted from call to call. A mark for each pool block says, as the
// smallest of what is put there, who keeps it: 0, a new row that has it full; 1 + b,
// new row b, whose last block it is, partly full; 1 + B + place, the first old entry
// that names it. So a row copies its last block if the mark is not its own, and an old
// entry gives its block back if the mark is its own place. Places are then handed out
// by two running sums in the rows' order, so results do not depend on the order of the
// atomics. Phases: marks cleared, set, entries counted (and summed by the block that is
// done last), filled; a warp takes kForkUnit entries of a row, all of a lane's on their way
// at once (one after another 18.6 us for what now takes 12). Bound: latency, of the phases'
// dependent loads and of their launches. Measured on the device: one row to four of 32
// entries 6.4 us, 256 rows to 256 of up to 257 entries 13 us, 1000 to 1000 of 2000 32 us.
#include "smla_device.cuh"
#include "smla_step.h"
#include "smla_umma.cuh"

#include <algorithm>
#include <climits>

namespace smla {
namespace {

constexpr int kThreads = 1024;
constexpr int kLanes = 32, kUnit = kForkUnit, kPer = kUnit / kLanes;

// A new row: the old one that it goes on from (-1: none), what it keeps.
struct NewRow {
    int source, blocks;
    bool tail; // its last block is partly full
    int tokens;
};

__device__ __forceinline__ int held_of(const ForkArgs &a, int r) { return min(max(a.blocks_held[r], 0), a.table_width); }

__device__ __forceinline__ NewRow new_row(const ForkArgs &a, int b)
{
    NewRow x{a.source_rows[b], 0, false, 0};
    if (x.source < 0 || x.source >= a.B_old) {
        x.source = -1;
        return x;
    }
    x.tokens = min(max(a.seq_lens[b], 0), held_of(a, x.source) << a.block_shift);
    x.blocks = (x.tokens + (1 << a.block_shift) - 1) >> a.block_shift;
    x.tail = (x.tokens & ((1 << a.block_shift) - 1)) != 0;
    return x;
}

__device__ __forceinline__ const int32_t *old_row(const ForkArgs &a, int r) { return a.block_table + r * a.table_stride; }
__device__ __forceinline__ bool in_pool(const ForkArgs &a, int e) { return e >= 0 && e < a.num_blocks; }
__device__ __forceinline__ uint32_t place(const ForkArgs &a, int r, int j)
{
    return 1u + (uint32_t)a.B + (uint32_t)((int64_t)r * a.table_width + j); // (B * width below 2^31, B at most 2^30)
}
__device__ __forceinline__ uint32_t mark_of(const ForkArgs &a, int e) { return __ldcg(a.marks + e); }

// Places of the ring, head and i below 2^31.
__device__ __forceinline__ unsigned ring_place(const ForkArgs &a, unsigned head, unsigned i)
{
    return (head + i) % (unsigned)a.ring_size;
}

// The units of rows: row u / units, entries from u % units * kUnit on.
__device__ __forceinline__ int units_of(const ForkArgs &a) { return max(1, (a.table_width + kUnit - 1) / kUnit); }

// A lane's entries of a unit, all on their way at once: -1 where there is none, or none of the pool's.
__device__ __forceinline__ void load_unit(const ForkArgs &a, const int32_t *row, int j0, int end, int lane, int (&e)[kPer])
{
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int j = j0 + k * kLanes + lane;
        e[k] = j < end ? row[j] : -1;
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k)
        e[k] = in_pool(a, e[k]) ? e[k] : -1;
}

// A bit to each of the lane's entries that gives its block back.
__device__ __forceinline__ unsigned giving(const ForkArgs &a, int r, int j0, int lane, const int (&e)[kPer])
{
    uint32_t m[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k)
        m[k] = e[k] >= 0 ? mark_of(a, e[k]) : 0;
    unsigned bits = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k)
        bits |= (unsigned)(e[k] >= 0 && m[k] == place(a, r, j0 + k * kLanes + lane)) << k;
    return bits;
}

__device__ __forceinline__ void clear_marks(const ForkArgs &a, int64_t warp, int64_t warps, int lane)
{
    const int units = units_of(a);
    for (int64_t u = warp; u < (int64_t)a.B_old * units; u += warps) {
        const int r = (int)(u / units), j0 = (int)(u % units) * kUnit, end = min(held_of(a, r), j0 + kUnit);
        if (j0 >= end)
            continue;
        int e[kPer];
        load_unit(a, old_row(a, r), j0, end, lane, e);
#pragma unroll
        for (int k = 0; k < kPer; ++k)
            if (e[k] >= 0)
                a.marks[e[k]] = 0xFFFFFFFFu;
    }
}

__device__ __forceinline__ void set_marks(const ForkArgs &a, int64_t warp, int64_t warps, int lane)
{
    const int units = units_of(a);
    const int64_t old_units = (int64_t)a.B_old * units, all = old_units + (int64_t)a.B * units;
    for (int64_t u = warp; u < all; u += warps) {
        const bool is_new = u >= old_units;
        const int64_t v = is_new ? u - old_units : u;
        const int b = (int)(v / units), j0 = (int)(v % units) * kUnit;
        NewRow x{b, 0, false, 0};
        if (is_new)
            x = new_row(a, b);
        const int end = min(is_new ? x.blocks : held_of(a, b), j0 + kUnit);
        if (j0 >= end)
            continue;
        int e[kPer];
        load_unit(a, old_row(a, x.source), j0, end, lane, e);
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int j = j0 + k * kLanes + lane;
            if (e[k] >= 0)
                atomicMin(a.marks + e[k], !is_new ? place(a, b, j) : x.tail && j == x.blocks - 1 ? 1u + (uint32_t)b : 0u);
        }
    }
}

// What each unit of the old rows gives back.
__device__ __forceinline__ void count_gives(const ForkArgs &a, int64_t warp, int64_t warps, int lane)
{
    const int units = units_of(a);
    for (int64_t u = warp; u < (int64_t)a.B_old * units; u += warps) {
        const int r = (int)(u / units), j0 = (int)(u % units) * kUnit, end = min(held_of(a, r), j0 + kUnit);
        int n = 0;
        if (j0 < end) {
            int e[kPer];
            load_unit(a, old_row(a, r), j0, end, lane, e);
            n = __reduce_add_sync(0xffffffffu, __popc(giving(a, r, j0, lane, e)));
        }
        if (lane == 0)
            a.gives[u] = n;
    }
}

// Exclusive sum over the block's threads; `total` gets the whole sum.
template <typename T> __device__ T block_exclusive(T v, T *total, T *warp_sums)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T inc = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const T o = __shfl_up_sync(0xffffffffu, inc, d);
        inc += lane >= d ? o : 0;
    }
    if (lane == 31)
        warp_sums[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        T w = warp_sums[lane];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const T o = __shfl_up_sync(0xffffffffu, w, d);
            w += lane >= d ? o : 0;
        }
        warp_sums[lane] = w;
    }
    __syncthreads();
    const T base = warp > 0 ? warp_sums[warp - 1] : 0;
    *total = warp_sums[31];
    __syncthreads();
    return base + inc - v;
}

// The running sums, by one block of kThreads: each unit's first place behind the ring's
// end, each new row's plan, the counts and the ring's state.
__device__ __forceinline__ void sum_up(const ForkArgs &a)
{
    __shared__ long long warp_sums[32];
    const int tid = threadIdx.x;
    const int64_t units = (int64_t)a.B_old * units_of(a);
    long long given = 0, taken = 0, tokens = 0, total;
    for (int64_t u0 = 0; u0 < units; u0 += kThreads) {
        const int64_t u = u0 + tid;
        const long long n = u < units ? __ldcg(a.gives + u) : 0; // (other blocks' writes)
        const long long at = given + block_exclusive(n, &total, warp_sums);
        if (u < units)
            a.gives[u] = (int)at;
        given += total;
    }
    for (int64_t b0 = 0; b0 < a.B; b0 += kThreads) {
        const int b = (int)(b0 + tid);
        NewRow x{-1, 0, false, 0};
        bool copies = false;
        if (b0 + tid < a.B) {
            x = new_row(a, b);
            if (x.tail) {
                const int e = old_row(a, x.source)[x.blocks - 1];
                copies = in_pool(a, e) && mark_of(a, e) != 1u + (uint32_t)b;
            }
        }
        // both sums in one: the rows' copies above 2^48 (1024 rows of at most 2^30 tokens stay below)
        const long long mine = ((long long)copies << 48) + x.tokens;
        const long long at = block_exclusive(mine, &total, warp_sums);
        if (b0 + tid < a.B)
            a.plan[b] = make_int4(x.source, x.blocks, copies ? (int)(taken + (at >> 48)) : -1, 0);
        taken += total >> 48;
        tokens += total & ((1ll << 48) - 1);
    }
    if (tid == 0) {
        const int h = a.ring_state[0] % a.ring_size, head = h < 0 ? h + a.ring_size : h;
        const int count = min(max(a.ring_state[1], 0), a.ring_size);
        const long long lacking = max(taken - count, 0ll);
        const bool ok = lacking == 0;
        a.state[0] = head;
        a.state[1] = count;
        a.state[2] = !ok;
        a.counts[0] = (int)min(tokens, (long long)INT_MAX);
        a.counts[1] = ok ? (int)taken : 0;
        a.counts[2] = ok ? (int)given : 0;
        a.counts[3] = (int)lacking;
        a.ring_state_out[0] = ok ? (int)((head + taken) % a.ring_size) : head;
        a.ring_state_out[1] = ok ? (int)min(count - taken + given, (long long)a.ring_size) : count;
    }
}

// New rows and what goes with them; blocks given back.
__device__ __forceinline__ void fill(const ForkArgs &a, int64_t warp, int64_t warps, int lane)
{
    const int units = units_of(a);
    const int head = a.state[0], count = a.state[1];
    const bool ok = a.state[2] == 0;
    const unsigned end_place = ring_place(a, head, count);
    const int64_t new_units = (int64_t)a.B * units, all = new_units + (int64_t)a.B_old * units;
    for (int64_t u = warp; u < all; u += warps) {
        if (u < new_units) {
            const int b = (int)(u / units), j0 = (int)(u % units) * kUnit;
            const int4 p = a.plan[b];
            const int own = ok && p.z >= 0 ? a.free_ring[ring_place(a, head, p.z)] : -1;
            if (j0 == 0 && lane == 0) {
                a.copy_from[b] = own >= 0 ? old_row(a, p.x)[p.y - 1] : -1;
                a.copy_to[b] = own;
                if (ok)
                    a.blocks_held_out[b] = p.y;
            }
            if (!ok || p.x < 0)
                continue;
            const int32_t *row = old_row(a, p.x);
            int32_t *out = a.block_table_out + b * a.out_stride;
            int e[kPer];
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                const int j = j0 + k * kLanes + lane;
                e[k] = j < p.y ? row[j] : 0;
            }
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                const int j = j0 + k * kLanes + lane;
                if (j < p.y)
                    out[j] = p.z >= 0 && j == p.y - 1 ? own : e[k];
            }
        } else if (ok) {
            const int64_t v = u - new_units;
            const int r = (int)(v / units), j0 = (int)(v % units) * kUnit, end = min(held_of(a, r), j0 + kUnit);
            if (j0 >= end)
                continue;
            unsigned at = a.gives[v];
            int e[kPer];
            load_unit(a, old_row(a, r), j0, end, lane, e);
            const unsigned bits = giving(a, r, j0, lane, e);
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                const bool gives = bits >> k & 1;
                const unsigned votes = __ballot_sync(0xffffffffu, gives);
                if (gives)
                    a.free_ring[ring_place(a, end_place, at + __popc(votes & ((1u << lane) - 1)))] = e[k];
                at += __popc(votes);
            }
        }
    }
}

__global__ void __launch_bounds__(kThreads) fork_one_kernel(const ForkArgs a)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int warps = kThreads / 32;
    clear_marks(a, warp, warps, lane);
    __syncthreads();
    set_marks(a, warp, warps, lane);
    __syncthreads();
    count_gives(a, warp, warps, lane);
    __syncthreads();
    sum_up(a);
    __syncthreads();
    fill(a, warp, warps, lane);
}

enum class Phase { kClear, kSet, kFill };
template <Phase kPhase> __global__ void __launch_bounds__(256) fork_phase_kernel(const ForkArgs a)
{
    umma::grid_launch_dependents();
    umma::grid_wait(); // the phase before
    const int lane = threadIdx.x & 31;
    const int64_t warp = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5, warps = ((int64_t)gridDim.x * blockDim.x) >> 5;
    if (kPhase == Phase::kClear) {
        if (warp == 0 && lane == 0)
            a.state[3] = 0; // the counting blocks that are done
        clear_marks(a, warp, warps, lane);
    } else if (kPhase == Phase::kSet) {
        set_marks(a, warp, warps, lane);
    } else {
        fill(a, warp, warps, lane);
    }
}

// Counts, and by the block that is done last the sums.
__global__ void __launch_bounds__(kThreads) fork_count_kernel(const ForkArgs a)
{
    __shared__ bool s_last;
    umma::grid_launch_dependents();
    umma::grid_wait();
    count_gives(a, (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), (int64_t)gridDim.x * (kThreads / 32), threadIdx.x & 31);
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0)
        s_last = atomicAdd(a.state + 3, 1) == (int)gridDim.x - 1;
    __syncthreads();
    if (!s_last)
        return;
    __threadfence();
    sum_up(a);
}

} // namespace

cudaError_t launch_fork_tables(const ForkArgs &a, int sm_count, cudaStream_t stream)
{
    if (fork_by_one_block(a.B_old, a.B, a.table_width)) {
        fork_one_kernel<<<1, kThreads, 0, stream>>>(a);
        return cudaGetLastError();
    }
    const int64_t units = fork_units((int64_t)a.B + a.B_old, a.table_width);
    const unsigned blocks = (unsigned)std::min<int64_t>((units + 7) / 8, (int64_t)std::max(sm_count, 1) * 8);
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const auto go = [&](void (*kernel)(const ForkArgs), unsigned grid, unsigned threads) {
        cfg.gridDim = dim3(grid);
        cfg.blockDim = dim3(threads);
        return cudaLaunchKernelEx(&cfg, kernel, a);
    };
    cudaError_t e = go(fork_phase_kernel<Phase::kClear>, blocks, 256);
    if (e == cudaSuccess)
        e = go(fork_phase_kernel<Phase::kSet>, blocks, 256);
    if (e == cudaSuccess)
        e = go(fork_count_kernel, (blocks + 3) / 4, kThreads);
    if (e == cudaSuccess)
        e = go(fork_phase_kernel<Phase::kFill>, blocks, 256);
    return e;
}

} // namespace smla

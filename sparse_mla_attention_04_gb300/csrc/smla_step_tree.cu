// Masks and positions of drafted trees, from each token's parent (sm_103a).
//
// A token sees itself and the nodes that it descends from, the nearest `window`
// generations of them. A request to a block, a node to a thread: after round k a node
// knows its 2^k nearest generations' nodes and the one behind them, so that twice as
// many follow by joining its own with that one's; a window's generations are joined
// from the rounds of its binary digits. As many rounds as the deepest node's
// generations have digits, each three barriers. (Walks up the parents, a node at a time,
// take as many reads as a tree is deep.) The words go out in order, whole lines at a
// time. Bound: latency, of the parents' read and of the rounds. Measured on the device:
// 1000 requests of up to 200 nodes, a fifth of them chains, in 9.0 us (22 by walks, a
// word at a time to a thread's row), 64 of up to 32 in 2.6 (4.1).
#include "smla_device.cuh"
#include "smla_step.h"

#include <algorithm>

namespace smla {

__device__ int g_tree_error = 0; // bit 16: a parent that does not come before its child, or a tree with too many nodes

namespace {

// kWords words to a mask, 64 kWords threads to a block.
template <int kWords>
__global__ void __launch_bounds__(64 * kWords) tree_mask_kernel(const TreeMaskArgs a, int words)
{
    constexpr int kMost = 64 * kWords;
    extern __shared__ __align__(16) uint64_t s_mask[]; // [kMost][kWords]
    __shared__ int2 s_up[kMost];                       // the node behind those known (-1: none), how many generations those are
    const int b = blockIdx.x, i = threadIdx.x; // (of an empty batch: none of its)
    const int q0 = b < a.B ? min(max(a.query_start[b], 0), a.T) : 0;
    const int q1 = b < a.B ? min(max(a.query_start[b + 1], q0), a.T) : 0;
    const int n = q1 - q0, nodes = min(n, words * 64);
    const int ctx = b < a.B ? max(a.seq_lens[b], 0) - n : 0;
    const int window = a.window < kMost ? a.window : 0; // (as many generations as a tree can have: all)
    bool bad = n > nodes;
    int2 up = make_int2(-1, 1);
    if (i < nodes) {
        const int p = a.parents[q0 + i];
        bad |= p < -1 || p >= i;
        up.x = p < i ? max(p, -1) : -1;
        s_up[i] = up;
#pragma unroll
        for (int w = 0; w < kWords; ++w)
            s_mask[i * kWords + w] = w == i >> 6 ? 1ull << (i & 63) : 0;
    }
    if (__syncthreads_or(bad) && i == 0)
        atomicOr(&g_tree_error, 16);
    uint64_t own[kWords], near[kWords]; // what the node knows; with a window, what of it is seen
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
        own[w] = i < nodes && w == i >> 6 ? 1ull << (i & 63) : 0;
        near[w] = 0;
    }
    int at = i < nodes ? i : -1; // with a window: the node from which on its generations still have to be joined
    for (int k = 0;; ++k) {
        if ((window >> k & 1) && at >= 0) {
#pragma unroll
            for (int w = 0; w < kWords; ++w)
                near[w] |= s_mask[at * kWords + w];
            at = s_up[at].x;
        }
        if (!__syncthreads_or(up.x >= 0 || ((window >> k) > 1 && at >= 0)))
            break;
        if (up.x >= 0) {
#pragma unroll
            for (int w = 0; w < kWords; ++w)
                own[w] |= s_mask[up.x * kWords + w];
            const int2 o = s_up[up.x];
            up = make_int2(o.x, up.y + o.y);
        }
        __syncthreads();
        if (i < nodes) {
            s_up[i] = up;
#pragma unroll
            for (int w = 0; w < kWords; ++w)
                s_mask[i * kWords + w] = own[w];
        }
        __syncthreads();
    }
    if (window > 0) {
        __syncthreads();
        if (i < nodes)
#pragma unroll
            for (int w = 0; w < kWords; ++w)
                s_mask[i * kWords + w] = near[w];
    }
    if (i < nodes)
        a.positions[q0 + i] = max(0, ctx + up.y - 1);
    for (int t = nodes + i; t < n; t += kMost) // nodes that the words have no room for
        a.positions[q0 + t] = max(0, ctx);
    __syncthreads();
    uint64_t *out = a.mask + (int64_t)q0 * words;
    for (int x = i; x < nodes * words; x += kMost)
        out[x] = s_mask[x / words * kWords + x % words];
    for (int64_t x = (int64_t)nodes * words + i; x < (int64_t)n * words; x += kMost)
        out[x] = 0;
    // rows behind the last request
    const int64_t end = a.B > 0 ? min(max(a.query_start[a.B], 0), a.T) : 0;
    for (int64_t t = end + (int64_t)b * kMost + i; t < a.T; t += (int64_t)gridDim.x * kMost) {
        for (int w = 0; w < words; ++w)
            a.mask[t * words + w] = 0;
        a.positions[t] = 0;
    }
}

template <int kWords> cudaError_t launch(const TreeMaskArgs &a, cudaStream_t stream)
{
    constexpr int kBytes = 64 * kWords * kWords * (int)sizeof(uint64_t);
    if (kBytes > 32 * 1024)
        if (const cudaError_t e = cudaFuncSetAttribute(tree_mask_kernel<kWords>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
            e != cudaSuccess)
            return e;
    tree_mask_kernel<kWords><<<(unsigned)std::max(a.B, 1), 64 * kWords, kBytes, stream>>>(a, a.words);
    return cudaGetLastError();
}

} // namespace

cudaError_t launch_tree_masks(const TreeMaskArgs &a, int sm_count, cudaStream_t stream)
{
    (void)sm_count;
    return a.words <= 1   ? launch<1>(a, stream)
           : a.words <= 2 ? launch<2>(a, stream)
           : a.words <= 4 ? launch<4>(a, stream)
           : a.words <= 8 ? launch<8>(a, stream)
                          : launch<16>(a, stream);
}

cudaError_t read_tree_error(int *out, bool reset)
{
    cudaError_t e = cudaMemcpyFromSymbol(out, g_tree_error, sizeof(int));
    if (e == cudaSuccess && reset) {
        const int zero = 0;
        e = cudaMemcpyToSymbol(g_tree_error, &zero, sizeof(int));
    }
    return e;
}

} // namespace smla

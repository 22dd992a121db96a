// Masks and positions of drafted trees, from each token's parent (sm_103a).
//
// A token sees its ancestors among its request's new tokens, and itself:
// mask(i) = {i} + mask(parent(i)); its position is that of the context's end plus its
// depth. A thread to a token walks up its tree's parents in shared memory. Parents
// come before their children, so the bits come in falling order and a word is
// written when the walk leaves it. Bound: the walk's chain of shared-memory reads
// (some 30 cycles a generation) and the words written.
#include "smla_device.cuh"
#include "smla_step.h"

#include <algorithm>

namespace smla {

__device__ int g_tree_error = 0; // bit 16: a parent that does not come before its child, or a tree with too many nodes

namespace {

__global__ void tree_mask_kernel(const TreeMaskArgs a)
{
    __shared__ int16_t s_parent[kMostTreeWords * 64];
    const int b = blockIdx.x; // (of an empty batch: none of its)
    const int q0 = b < a.B ? min(max(a.query_start[b], 0), a.T) : 0;
    const int q1 = b < a.B ? min(max(a.query_start[b + 1], q0), a.T) : 0;
    const int n = q1 - q0, most = a.words * 64;
    const int ctx = b < a.B ? max(a.seq_lens[b], 0) - n : 0;
    bool bad = n > most;
    for (int i = threadIdx.x; i < min(n, most); i += blockDim.x) {
        const int p = a.parents[q0 + i];
        bad |= p < -1 || p >= i;
        s_parent[i] = (int16_t)(p >= 0 && p < i ? p : -1);
    }
    if (__syncthreads_or(bad) && threadIdx.x == 0)
        atomicOr(&g_tree_error, 16);
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        uint64_t *row = a.mask + (int64_t)(q0 + i) * a.words;
        int depth = 0, word = a.words - 1;
        uint64_t bits = 0;
        if (i < most) {
            for (int at = i; at >= 0; at = s_parent[at], ++depth) {
                for (; word > at >> 6; --word) {
                    row[word] = bits;
                    bits = 0;
                }
                if (a.window <= 0 || depth < a.window)
                    bits |= 1ull << (at & 63);
            }
            --depth;
        }
        for (; word >= 0; --word) {
            row[word] = bits;
            bits = 0;
        }
        a.positions[q0 + i] = max(0, ctx + depth);
    }
    // rows behind the last request
    const int64_t end = a.B > 0 ? min(max(a.query_start[a.B], 0), a.T) : 0;
    for (int64_t t = end + (int64_t)blockIdx.x * blockDim.x + threadIdx.x; t < a.T; t += (int64_t)gridDim.x * blockDim.x) {
        for (int w = 0; w < a.words; ++w)
            a.mask[t * a.words + w] = 0;
        a.positions[t] = 0;
    }
}

} // namespace

cudaError_t launch_tree_masks(const TreeMaskArgs &a, int sm_count, cudaStream_t stream)
{
    (void)sm_count;
    // a request to a block, as many threads as the trees may have nodes
    const int threads = std::min(256, a.words * 64);
    tree_mask_kernel<<<(unsigned)std::max(a.B, 1), threads, 0, stream>>>(a);
    return cudaGetLastError();
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

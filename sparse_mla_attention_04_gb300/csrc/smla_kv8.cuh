// What the two attention kernels over the block-scaled cache share (sm_103a).
#pragma once

#include "smla_device.cuh"
#include "smla_internal.h"

namespace smla {
namespace kv8 {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float lg2_approx(float x)
{
    float y;
    asm("lg2.approx.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}

// One request as the kernels see it: every field in range whatever the arrays hold.
struct Request {
    int q0, qlen; // its first flat token and how many
    int len;      // positions [0, len) exist
    int begin;    // positions below it (a multiple of 32) are seen by none of its tokens
    __device__ int pos(int i) const { return len - qlen + i; } // may be negative: sees nothing
};

__device__ __forceinline__ Request request(const Kv8AttnArgs &a, int b)
{
    Request r;
    const int q0 = min(max(a.query_start[b], 0), a.T);
    const int q1 = min(max(a.query_start[b + 1], q0), a.T);
    r.q0 = q0;
    r.qlen = q1 - q0;
    r.len = (int)min((long long)max(a.seq_lens[b], 0), (long long)a.table_width << a.block_shift);
    r.begin = 0;
    if (a.window > 0)
        r.begin = (int)max(0ll, (long long)r.len - r.qlen - a.window + 1) & ~31;
    return r;
}

// The final values of a row from its sums: m the reference (log2 units), l the
// softmax denominator relative to it. Returns the factor for the value sums.
__device__ __forceinline__ float finish_row(float m, float l, const float *sinks, int head, float *lse)
{
    float f = 1.0f;
    if (sinks) {
        const float s = sinks[head] * kLog2e;
        const float top = fmaxf(m, s);
        if (top == -INFINITY) { // nothing seen and a sink of -inf
            *lse = -INFINITY;
            return 0.0f;
        }
        f = ex2_approx(m - top); // m = -inf: 0
        l = l * f + ex2_approx(s - top);
        m = top;
    }
    if (l == 0.0f) {
        *lse = -INFINITY;
        return 0.0f;
    }
    *lse = (m + lg2_approx(l)) * kLn2;
    return __fdividef(f, l);
}

} // namespace kv8
} // namespace smla

// Root-mean-square norms of each query and key head and the rotary positions
// behind them, in one pass (sm_103a).
//
// y = x r (w + offset), r = (mean of x^2 over the head's D columns + eps)^-1/2, then the
// rotated columns turned, all in binary32, and one rounding at the end: the split
// chain (norm, store, rotation) rounds twice and moves every element twice.
// Bound: the bytes in and out. Two lanes' worth of a row never meet in memory: a
// row is a group of up to 32 lanes, each with two 16-byte chunks of it (with
// halves, those that a rotation pairs), so a row is read once, its sum goes through
// shuffles, and it may be written where it was.
#include "smla_device.cuh"
#include "smla_rope.cuh"
#include "smla_step.h"

#include <algorithm>
#include <cfloat>
#include <climits>

namespace smla {

__device__ int g_norm_rope_error = 0; // bit 4: a position out of range

namespace {

using namespace rope;

constexpr int kBatch = 2;    // heads of a group on their way at a time
constexpr int kThreads = 256;

// r of a row from the sum of its squares. Where that passes binary32 the row's
// elements are to be taken 2^-70 times (`small`), and the sum is one of those: finite
// for every finite row of up to 2^17 columns.
constexpr float kSmall = 0x1p-70f;
__device__ __forceinline__ float inverse_rms(float sum, int D, float eps, bool small)
{
    const float mean = __fdiv_rn(sum, (float)D);
    return __frsqrt_rn(mean + (small ? eps * kSmall * kSmall : eps));
}

template <typename Wt>
__device__ __forceinline__ float weight_at(const void *w, int64_t i)
{
    return to_f(static_cast<const Wt *>(w)[i]);
}

// Where a group's lane stands: its two chunks' columns (-1: none) and whether they turn.
template <int kVec, bool kNeox> struct Place {
    int ca, cb;
    bool ta, tb;
    int pair_a, pair_b; // the angles' first pairs
    __device__ __forceinline__ Place(const NormRopeArgs &a, int u)
    {
        const int n = a.rot_dim / 2;
        ta = tb = false;
        ca = cb = -1;
        pair_a = pair_b = 0;
        if (kNeox) {
            const int turned = n / kVec, plain = (a.D - a.rot_dim) / kVec, half = (plain + 1) / 2;
            if (u < turned) {
                ca = a.rot_offset + u * kVec;
                cb = ca + n;
                ta = tb = true;
                pair_a = u * kVec;
            } else if (u < turned + half) {
                const int m = u - turned;
                ca = m * kVec;
                ca += ca >= a.rot_offset ? a.rot_dim : 0;
                if (m + half < plain) {
                    cb = (m + half) * kVec;
                    cb += cb >= a.rot_offset ? a.rot_dim : 0;
                }
            }
        } else {
            const int chunks = a.D / kVec, half = (chunks + 1) / 2;
            const auto turns = [&](int c) { return c >= a.rot_offset && c < a.rot_offset + a.rot_dim; };
            if (u < half) {
                ca = u * kVec;
                ta = turns(ca);
                pair_a = (ca - a.rot_offset) / 2;
                if (u + half < chunks) {
                    cb = (u + half) * kVec;
                    tb = turns(cb);
                    pair_b = (cb - a.rot_offset) / 2;
                }
            }
        }
    }
};

// A group of blockDim.x lanes takes heads y, y + spread, ... of a token's queries, then of its keys.
template <typename E, typename Wt, bool kNeox>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const NormRopeArgs a, int spread)
{
    constexpr int kVec = 16 / sizeof(E);
    using P = Pack<E, kVec>;
    const int64_t item = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const int64_t t = item / spread;
    const int y = (int)(item - t * spread);
    const bool live = t < a.T;
    const int64_t pos = live ? a.positions[t] : 0;
    const Place<kVec, kNeox> at(a, threadIdx.x);
    bool first = true, ok = live;
    float c[kVec], s[kVec]; // halves: of the pairs; interleaved: of chunk A's pairs, then of B's
#pragma unroll
    for (int e = 0; e < kVec; ++e)
        c[e] = 1.f, s[e] = 0.f;
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
        const int count = side ? a.H_k : a.H;
        if (count == 0)
            continue;
        const int64_t sh = side ? a.k_sh : a.q_sh, oh = side ? a.ko_sh : a.qo_sh, wh = side ? a.kw_sh : a.qw_sh;
        const E *src = static_cast<const E *>(side ? a.k : a.q) + t * (side ? a.k_st : a.q_st);
        E *dst = static_cast<E *>(side ? a.k_out : a.q_out) + t * (side ? a.ko_st : a.qo_st);
        const void *w = side ? a.k_weight : a.q_weight;
        float wa[kVec], wb[kVec];
        const auto weights = [&](int h) {
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
                wa[e] = w && at.ca >= 0 ? weight_at<Wt>(w, h * wh + at.ca + e) + a.weight_offset : 1.f;
                wb[e] = w && at.cb >= 0 ? weight_at<Wt>(w, h * wh + at.cb + e) + a.weight_offset : 1.f;
            }
        };
#pragma unroll 1
        for (int h0 = y; h0 - y < count; h0 += kBatch * spread) { // (the same rounds for all groups of a warp)
            P xa[kBatch], xb[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int h = h0 + i * spread;
                xa[i].w = xb[i].w = make_uint4(0, 0, 0, 0);
                if (live && h < count && at.ca >= 0)
                    xa[i].load(src + h * sh + at.ca);
                if (live && h < count && at.cb >= 0)
                    xb[i].load(src + h * sh + at.cb);
            }
            if (wh == 0 && h0 == y)
                weights(0);
            if (first) {
                first = false;
                if (live && (pos < 0 || pos >= a.max_position)) {
                    if (threadIdx.x == 0 && y == 0)
                        atomicOr(&g_norm_rope_error, 4);
                    ok = false;
                }
                if (ok) {
                    const float *row = a.cos_sin + pos * a.rot_dim;
                    const int n = a.rot_dim / 2;
                    if (kNeox) {
                        if (at.ta) {
                            load_angles<kVec>(row + at.pair_a, c);
                            load_angles<kVec>(row + n + at.pair_a, s);
                        }
                    } else {
                        float(&ca)[kVec / 2] = *reinterpret_cast<float(*)[kVec / 2]>(c);
                        float(&sa)[kVec / 2] = *reinterpret_cast<float(*)[kVec / 2]>(s);
                        float(&cb)[kVec / 2] = *reinterpret_cast<float(*)[kVec / 2]>(c + kVec / 2);
                        float(&sb)[kVec / 2] = *reinterpret_cast<float(*)[kVec / 2]>(s + kVec / 2);
                        if (at.ta) {
                            load_angles<kVec / 2>(row + at.pair_a, ca);
                            load_angles<kVec / 2>(row + n + at.pair_a, sa);
                        }
                        if (at.tb) {
                            load_angles<kVec / 2>(row + at.pair_b, cb);
                            load_angles<kVec / 2>(row + n + at.pair_b, sb);
                        }
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int h = h0 + i * spread;
                float va[kVec], vb[kVec];
                float sum = 0.f;
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    va[e] = to_f(xa[i].at(e));
                    vb[e] = to_f(xb[i].at(e));
                    sum = fmaf(va[e], va[e], sum);
                    sum = fmaf(vb[e], vb[e], sum);
                }
                for (int d = 1; d < (int)blockDim.x; d <<= 1)
                    sum += __shfl_xor_sync(0xffffffffu, sum, d);
                const bool small = !(sum <= FLT_MAX);
                if (__any_sync(0xffffffffu, small)) { // (seldom)
                    float again = 0.f;
#pragma unroll
                    for (int e = 0; e < kVec; ++e) {
                        va[e] *= small ? kSmall : 1.f;
                        vb[e] *= small ? kSmall : 1.f;
                        again = fmaf(va[e], va[e], again);
                        again = fmaf(vb[e], vb[e], again);
                    }
                    for (int d = 1; d < (int)blockDim.x; d <<= 1)
                        again += __shfl_xor_sync(0xffffffffu, again, d);
                    sum = small ? again : sum;
                }
                const float r = inverse_rms(sum, a.D, a.eps, small);
                if (!ok || h >= count)
                    continue; // (no shuffles below)
                if (wh != 0)
                    weights(h);
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    va[e] = va[e] * r * wa[e];
                    vb[e] = vb[e] * r * wb[e];
                }
                if (kNeox) {
                    if (at.ta) {
#pragma unroll
                        for (int e = 0; e < kVec; ++e) {
                            const float p = va[e], q = vb[e];
                            va[e] = rot_a(p, q, c[e], s[e]);
                            vb[e] = rot_b(p, q, c[e], s[e]);
                        }
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < kVec / 2; ++e) {
                        float p = va[2 * e], q = va[2 * e + 1];
                        if (at.ta) {
                            va[2 * e] = rot_a(p, q, c[e], s[e]);
                            va[2 * e + 1] = rot_b(p, q, c[e], s[e]);
                        }
                        p = vb[2 * e], q = vb[2 * e + 1];
                        if (at.tb) {
                            vb[2 * e] = rot_a(p, q, c[kVec / 2 + e], s[kVec / 2 + e]);
                            vb[2 * e + 1] = rot_b(p, q, c[kVec / 2 + e], s[kVec / 2 + e]);
                        }
                    }
                }
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    xa[i].at(e) = from_f<E>(va[e]);
                    xb[i].at(e) = from_f<E>(vb[e]);
                }
                if (at.ca >= 0)
                    xa[i].store(dst + h * oh + at.ca);
                if (at.cb >= 0)
                    xb[i].store(dst + h * oh + at.cb);
            }
        }
    }
}

// Any width, offset and alignment: a warp to a row, by single elements, which are read
// for the sum and again (from L1) for the values. A pair is one lane's, and the sum's
// shuffles part the two passes, so a row may be written where it was.
template <typename E, typename Wt>
__global__ void __launch_bounds__(kThreads) norm_rope_any_kernel(const NormRopeArgs a)
{
    const int lane = threadIdx.x & 31;
    const int heads = a.H + a.H_k, n = a.rot_dim / 2;
    const int64_t row = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5;
    const int64_t t = row / heads;
    if (t >= a.T)
        return;
    int h = (int)(row - t * heads);
    const bool side = h >= a.H;
    h -= side ? a.H : 0;
    const int64_t pos = a.positions[t];
    if (pos < 0 || pos >= a.max_position) {
        if (lane == 0)
            atomicOr(&g_norm_rope_error, 4);
        return;
    }
    const E *src = static_cast<const E *>(side ? a.k : a.q) + t * (side ? a.k_st : a.q_st) + h * (side ? a.k_sh : a.q_sh);
    E *dst = static_cast<E *>(side ? a.k_out : a.q_out) + t * (side ? a.ko_st : a.qo_st) + h * (side ? a.ko_sh : a.qo_sh);
    const void *w = side ? a.k_weight : a.q_weight;
    const int64_t w0 = h * (side ? a.kw_sh : a.qw_sh);
    float f = 1.f, sum = 0.f;
    for (int pass = 0; pass < 2; ++pass) {
        sum = 0.f;
        for (int i = lane; i < a.D; i += 32) {
            const float x = to_f(src[i]) * f;
            sum = fmaf(x, x, sum);
        }
#pragma unroll
        for (int d = 1; d < 32; d <<= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (sum <= FLT_MAX || f != 1.f)
            break;
        f = kSmall;
    }
    const float r = inverse_rms(sum, a.D, a.eps, f != 1.f);
    const auto value = [&](int i) {
        return to_f(src[i]) * f * r * (w ? weight_at<Wt>(w, w0 + i) + a.weight_offset : 1.f);
    };
    for (int i = lane; i < a.D - a.rot_dim; i += 32) {
        const int col = i < a.rot_offset ? i : i + a.rot_dim;
        dst[col] = from_f<E>(value(col));
    }
    const float *angles = a.cos_sin + pos * a.rot_dim;
    for (int i = lane; i < n; i += 32) {
        const int p = a.rot_offset + (a.neox ? i : 2 * i), q = p + (a.neox ? n : 1);
        const float x = value(p), y = value(q), c = angles[i], s = angles[n + i];
        dst[p] = from_f<E>(rot_a(x, y, c, s));
        dst[q] = from_f<E>(rot_b(x, y, c, s));
    }
}

template <typename E, typename Wt>
cudaError_t launch(const NormRopeArgs &a, int sm_count, cudaStream_t stream)
{
    constexpr int kVec = 16 / sizeof(E);
    const int heads = a.H + a.H_k;
    // 16-byte accesses where every row, the rotated part and its halves allow them, and a row fits a group of lanes
    const uintptr_t bits = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.q_out) |
                           reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.k_out);
    const int64_t odd = a.q_st | a.q_sh | a.qo_st | a.qo_sh | a.k_st | a.k_sh | a.ko_st | a.ko_sh | a.D | a.rot_offset |
                        (a.neox ? a.rot_dim / 2 : a.rot_dim);
    const int units = a.neox ? a.rot_dim / 2 / kVec + ((a.D - a.rot_dim) / kVec + 1) / 2 : (a.D / kVec + 1) / 2;
    if (bits % 16 != 0 || odd % kVec != 0 || units > 32) {
        const int64_t blocks = ((int64_t)a.T * heads + kThreads / 32 - 1) / (kThreads / 32);
        if (blocks > INT_MAX)
            return cudaErrorInvalidValue;
        norm_rope_any_kernel<E, Wt><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
        return cudaGetLastError();
    }
    int lanes = 1;
    while (lanes < units)
        lanes *= 2;
    // Few tokens: a head to a group, so that all SMs have some. Many: as many groups to a token as leave each at least
    // three rounds of heads (positions and angles are read once for them) and waste least of the rounds.
    int spread = heads;
    if ((int64_t)a.T * heads * lanes > (int64_t)sm_count * 2048) {
        const auto rounds = [&](int y) {
            return (a.H + kBatch * y - 1) / (kBatch * y) + (a.H_k + kBatch * y - 1) / (kBatch * y);
        };
        spread = 1;
        for (int y = 2; y <= heads && rounds(y) >= 3; ++y)
            if (rounds(y) * y <= rounds(spread) * spread)
                spread = y;
    }
    const int groups = kThreads / lanes;
    const int64_t blocks = ((int64_t)a.T * spread + groups - 1) / groups;
    if (blocks > INT_MAX)
        return cudaErrorInvalidValue;
    const dim3 block(lanes, groups);
    if (a.neox)
        norm_rope_kernel<E, Wt, true><<<(unsigned)blocks, block, 0, stream>>>(a, spread);
    else
        norm_rope_kernel<E, Wt, false><<<(unsigned)blocks, block, 0, stream>>>(a, spread);
    return cudaGetLastError();
}

template <typename E>
cudaError_t launch_type(const NormRopeArgs &a, bool weight_f32, int sm_count, cudaStream_t stream)
{
    return weight_f32 ? launch<E, float>(a, sm_count, stream) : launch<E, E>(a, sm_count, stream);
}

} // namespace

cudaError_t launch_norm_rope(const NormRopeArgs &a, int dtype, bool weight_f32, int sm_count, cudaStream_t stream)
{
    switch (dtype) {
    case SMLA_BF16:
        return launch_type<__nv_bfloat16>(a, weight_f32, sm_count, stream);
    case SMLA_F16:
        return launch_type<__half>(a, weight_f32, sm_count, stream);
    default:
        return launch<float, float>(a, sm_count, stream);
    }
}

cudaError_t read_norm_rope_error(int *out, bool reset)
{
    cudaError_t e = cudaMemcpyFromSymbol(out, g_norm_rope_error, sizeof(int));
    if (e == cudaSuccess && reset) {
        const int zero = 0;
        e = cudaMemcpyToSymbol(g_norm_rope_error, &zero, sizeof(int));
    }
    return e;
}

} // namespace smla

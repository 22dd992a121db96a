// Root-mean-square norms of each query and key head and the rotary positions
// behind them, in one pass (sm_103a).
//
// y = x r (w + offset), r = (mean of x^2 over the head's D columns + eps)^-1/2, then the
// rotated columns turned, all in binary32, and one rounding at the end: the split
// chain (norm, store, rotation) rounds twice and moves every element twice.
// A row is a group of up to 32 lanes, each with two 16-byte chunks of it (with halves,
// those that a rotation pairs): it is read once, its sum goes through shuffles, and it
// may be written where it was. A group takes up to eight rows and keeps what they share:
// a token's angles, or a head's weights where each head has its own. Bound: the bytes in
// and out. Measured on the device: 8192 tokens, 32 + 8 heads of 128 columns in bf16 (168
// MB) in 29.0 us, 5.8 TB/s (the device's own copy of as many bytes: 31), in 32.7 with
// binary32 weights for each head (40.5 with the weights read for each row); 64 tokens 2.7
// us. What counted: arithmetic on pairs of elements and weights by 16 bytes (60 us by single
// ones), more warps (two rows at a time in registers 45, one and the next 36), three rows
// on their way in shared memory (29), eight rows to a group (four 32, sixteen 31).
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

constexpr int kMostPer = 8; // rows that a group takes
constexpr int kDepth = 4;   // and that are on their way at a time, with the one in hand (a power of two)
constexpr int kThreads = 128;

// r of a row from the sum of its squares. Where that passes binary32 (`small`) the sum is
// one of the row taken 2^-74 times: below 2^(2 (128 - 74)) 2^16 = 2^124 for every finite
// row of up to 65536 columns. The row's elements themselves are not scaled: those of less
// than 2^-52 would lose bits. r may then be below the normals, where its rounding is at
// most 2^-22 of it (r > 2^-128). (rsqrtf: 2 units in the last place.)
constexpr float kSmall = 0x1p-74f;
__device__ __forceinline__ float inverse_rms(float sum, float inv_D, float eps, bool small)
{
    const float r = rsqrtf(fmaf(sum, inv_D, small ? eps * kSmall * kSmall : eps));
    return small ? r * kSmall : r;
}

// Two binary32 operations in one instruction.
__device__ __forceinline__ uint64_t pair(float x, float y)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 unpair(uint64_t r)
{
    float2 v;
    asm("mov.b64 {%0, %1}, %2;\n" : "=f"(v.x), "=f"(v.y) : "l"(r));
    return v;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// The values of a chunk in pairs, and pairs as a chunk.
template <typename E> struct Chunk;
template <> struct Chunk<__nv_bfloat16> {
    static __device__ __forceinline__ void open(const uint4 &w, uint64_t (&v)[4])
    {
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = pair(__uint_as_float(x[i] << 16), __uint_as_float(x[i] & 0xFFFF0000u));
    }
    static __device__ __forceinline__ uint32_t word(uint64_t v)
    {
        const float2 f = unpair(v);
        const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
        return *reinterpret_cast<const uint32_t *>(&b);
    }
    static __device__ __forceinline__ uint4 close(const uint64_t (&v)[4])
    {
        return make_uint4(word(v[0]), word(v[1]), word(v[2]), word(v[3]));
    }
};
template <> struct Chunk<__half> {
    static __device__ __forceinline__ void open(const uint4 &w, uint64_t (&v)[4])
    {
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&x[i]));
            v[i] = pair(f.x, f.y);
        }
    }
    static __device__ __forceinline__ uint32_t word(uint64_t v)
    {
        const float2 f = unpair(v);
        const __half2 b = __floats2half2_rn(f.x, f.y);
        return *reinterpret_cast<const uint32_t *>(&b);
    }
    static __device__ __forceinline__ uint4 close(const uint64_t (&v)[4])
    {
        return make_uint4(word(v[0]), word(v[1]), word(v[2]), word(v[3]));
    }
};
template <> struct Chunk<float> {
    static __device__ __forceinline__ void open(const uint4 &w, uint64_t (&v)[2])
    {
        v[0] = pair(__uint_as_float(w.x), __uint_as_float(w.y));
        v[1] = pair(__uint_as_float(w.z), __uint_as_float(w.w));
    }
    static __device__ __forceinline__ uint4 close(const uint64_t (&v)[2])
    {
        const float2 a = unpair(v[0]), b = unpair(v[1]);
        return make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
    }
};

// kVec weights from column col on, by 16 bytes where they are aligned (`whole`).
template <typename Wt, int kVec>
__device__ __forceinline__ void load_weights(const Wt *w, bool whole, float offset, float (&v)[kVec])
{
    if (whole) {
        constexpr int kPer = 16 / sizeof(Wt);
#pragma unroll
        for (int i = 0; i < kVec / kPer; ++i) {
            Pack<Wt, kPer> p;
            p.w = __ldg(reinterpret_cast<const uint4 *>(w) + i);
#pragma unroll
            for (int e = 0; e < kPer; ++e)
                v[i * kPer + e] = to_f(p.at(e)) + offset;
        }
    } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e)
            v[e] = to_f(w[e]) + offset;
    }
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

// Sixteen bytes to shared memory, without waiting.
__device__ __forceinline__ void copy16(void *dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// A group of blockDim.x lanes takes `per` rows one after another, the next ones on their way meanwhile: heads of one
// token's queries or keys, whose angles it keeps, or (kHeads: weights of their own for each head) one head of as many
// tokens, whose weights it keeps; the groups of a block are then heads of the same tokens, which find the angles in L1.
template <typename E, typename Wt, bool kNeox, bool kHeads>
__global__ void __launch_bounds__(kThreads, 6) norm_rope_kernel(const NormRopeArgs a, int per, int q_groups, int groups)
{
    constexpr int kVec = 16 / sizeof(E), kPairs = kVec / 2;
    using C = Chunk<E>;
    const int64_t item = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const int64_t t = item / groups * (kHeads ? per : 1); // the (first) token
    int y = (int)(item % groups);
    const bool live = t < a.T;
    int64_t pos = live ? a.positions[t] : 0;
    const bool side = y >= q_groups, reports = threadIdx.x == 0 && y == 0;
    y -= side ? q_groups : 0;
    const Place<kVec, kNeox> at(a, threadIdx.x);
    const int h0 = kHeads ? y : y * per;
    const int count = !live ? 0 : (int)(kHeads ? min((int64_t)per, a.T - t) : (int64_t)min(per, (side ? a.H_k : a.H) - h0));
    const int64_t sh = side ? a.k_sh : a.q_sh, oh = side ? a.ko_sh : a.qo_sh;
    const int64_t st = side ? a.k_st : a.q_st, ot = side ? a.ko_st : a.qo_st;
    const int64_t src_step = kHeads ? st : sh, dst_step = kHeads ? ot : oh; // from row to row
    const E *src = static_cast<const E *>(side ? a.k : a.q) + t * st + h0 * sh;
    E *dst = static_cast<E *>(side ? a.k_out : a.q_out) + t * ot + h0 * oh;
    // the next rows' chunks come to the thread's own places in shared memory, which hold no registers meanwhile
    __shared__ uint4 s_ring[kDepth][2][kThreads];
    const int tid = threadIdx.y * blockDim.x + threadIdx.x;
    const uint4 none = make_uint4(0, 0, 0, 0);
    const auto ask = [&](int i) {
        if (i < count) {
            const E *row = src + i * src_step;
            if (at.ca >= 0)
                copy16(&s_ring[i % kDepth][0][tid], row + at.ca);
            if (at.cb >= 0)
                copy16(&s_ring[i % kDepth][1][tid], row + at.cb);
        }
        asm volatile("cp.async.commit_group;\n" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i)
        ask(i);
    float wa[kVec], wb[kVec];
#pragma unroll
    for (int e = 0; e < kVec; ++e)
        wa[e] = wb[e] = 1.f;
    if (const Wt *w = static_cast<const Wt *>(side ? a.k_weight : a.q_weight)) {
        const int64_t wh = side ? a.kw_sh : a.qw_sh;
        const bool whole = ((reinterpret_cast<uintptr_t>(w) | (uintptr_t)(wh * sizeof(Wt))) & 15) == 0;
        w += kHeads ? h0 * wh : 0;
        if (at.ca >= 0)
            load_weights<Wt, kVec>(w + at.ca, whole, a.weight_offset, wa);
        if (at.cb >= 0)
            load_weights<Wt, kVec>(w + at.cb, whole, a.weight_offset, wb);
    }
    bool ok = false; // the token's position is one
    float c[kVec], s[kVec]; // halves: of the pairs; interleaved: of chunk A's pairs, then of B's
    const auto angles = [&](bool there) {
#pragma unroll
        for (int e = 0; e < kVec; ++e)
            c[e] = 1.f, s[e] = 0.f;
        ok = there && pos >= 0 && pos < a.max_position;
        if (there && !ok && reports)
            atomicOr(&g_norm_rope_error, 4);
        if (ok) {
            const float *row = a.cos_sin + pos * a.rot_dim;
            const int n = a.rot_dim / 2;
            if (kNeox) {
                if (at.ta) {
                    load_angles<kVec>(row + at.pair_a, c);
                    load_angles<kVec>(row + n + at.pair_a, s);
                }
            } else {
                if (at.ta) {
                    load_angles<kPairs>(row + at.pair_a, *reinterpret_cast<float(*)[kPairs]>(c));
                    load_angles<kPairs>(row + n + at.pair_a, *reinterpret_cast<float(*)[kPairs]>(s));
                }
                if (at.tb) {
                    load_angles<kPairs>(row + at.pair_b, *reinterpret_cast<float(*)[kPairs]>(c + kPairs));
                    load_angles<kPairs>(row + n + at.pair_b, *reinterpret_cast<float(*)[kPairs]>(s + kPairs));
                }
            }
        }
    };
    if (!kHeads)
        angles(live);
#pragma unroll 1
    for (int i = 0; i < per; ++i) { // (the same rounds for all groups of a warp)
        if (kHeads) { // asked for before the row is waited for
            angles(i < count);
            pos = i + 1 < count ? a.positions[t + i + 1] : 0;
        }
        ask(i + kDepth - 1);
        asm volatile("cp.async.wait_group %0;\n" ::"n"(kDepth - 1) : "memory");
        uint64_t va[kPairs], vb[kPairs], sums = 0;
        C::open(at.ca >= 0 && i < count ? s_ring[i % kDepth][0][tid] : none, va);
        C::open(at.cb >= 0 && i < count ? s_ring[i % kDepth][1][tid] : none, vb);
#pragma unroll
        for (int e = 0; e < kPairs; ++e)
            sums = fma2(vb[e], vb[e], fma2(va[e], va[e], sums));
        const float2 both = unpair(sums);
        float sum = both.x + both.y;
        for (int d = 1; d < (int)blockDim.x; d <<= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, d);
        const bool small = !(sum <= FLT_MAX);
        if (__any_sync(0xffffffffu, small)) { // (seldom)
            const uint64_t f = pair(small ? kSmall : 1.f, small ? kSmall : 1.f);
            sums = 0;
#pragma unroll
            for (int e = 0; e < kPairs; ++e) {
                const uint64_t p = mul2(va[e], f), q = mul2(vb[e], f);
                sums = fma2(q, q, fma2(p, p, sums));
            }
            const float2 again = unpair(sums);
            float x = again.x + again.y;
            for (int d = 1; d < (int)blockDim.x; d <<= 1)
                x += __shfl_xor_sync(0xffffffffu, x, d);
            sum = small ? x : sum;
        }
        if (!ok || i >= count)
            continue; // (no shuffles below)
        const float r = inverse_rms(sum, a.inv_D, a.eps, small);
        const uint64_t rr = pair(r, r);
#pragma unroll
        for (int e = 0; e < kPairs; ++e) {
            va[e] = mul2(mul2(va[e], rr), pair(wa[2 * e], wa[2 * e + 1]));
            vb[e] = mul2(mul2(vb[e], rr), pair(wb[2 * e], wb[2 * e + 1]));
        }
        if (kNeox) {
            if (at.ta) {
#pragma unroll
                for (int e = 0; e < kPairs; ++e) {
                    const uint64_t p = va[e], q = vb[e], cc = pair(c[2 * e], c[2 * e + 1]);
                    va[e] = fma2(p, cc, mul2(q, pair(-s[2 * e], -s[2 * e + 1])));
                    vb[e] = fma2(q, cc, mul2(p, pair(s[2 * e], s[2 * e + 1])));
                }
            }
        } else {
            const auto turn = [](uint64_t v, float c, float s) {
                const float2 x = unpair(v);
                return pair(fmaf(x.x, c, -(x.y * s)), fmaf(x.y, c, x.x * s));
            };
            if (at.ta)
#pragma unroll
                for (int e = 0; e < kPairs; ++e)
                    va[e] = turn(va[e], c[e], s[e]);
            if (at.tb)
#pragma unroll
                for (int e = 0; e < kPairs; ++e)
                    vb[e] = turn(vb[e], c[kPairs + e], s[kPairs + e]);
        }
        E *row = dst + i * dst_step;
        if (at.ca >= 0)
            __stcs(reinterpret_cast<uint4 *>(row + at.ca), C::close(va));
        if (at.cb >= 0)
            __stcs(reinterpret_cast<uint4 *>(row + at.cb), C::close(vb));
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
    const Wt *w = static_cast<const Wt *>(side ? a.k_weight : a.q_weight);
    if (w)
        w += h * (side ? a.kw_sh : a.qw_sh);
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
    const float r = inverse_rms(sum, a.inv_D, a.eps, f != 1.f);
    const auto value = [&](int i) {
        return to_f(src[i]) * r * (w ? to_f(w[i]) + a.weight_offset : 1.f);
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
    // Few tokens: a row to a group, so that all SMs have some. Many: up to eight, so that positions and angles (or
    // weights) are read once for them.
    const bool many = (int64_t)a.T * heads * lanes > (int64_t)sm_count * 2048;
    const bool each = a.qw_sh != 0 || a.kw_sh != 0; // weights of their own for each head
    const int per = !many ? 1 : std::min(kMostPer, each ? a.T : std::max(a.H, a.H_k));
    const int q_groups = each ? a.H : (a.H + per - 1) / per;
    const int token_groups = q_groups + (each ? a.H_k : (a.H_k + per - 1) / per); // of one token, or of `per` tokens
    const int groups = kThreads / lanes;
    const int64_t blocks = ((each ? ((int64_t)a.T + per - 1) / per : (int64_t)a.T) * token_groups + groups - 1) / groups;
    if (blocks > INT_MAX)
        return cudaErrorInvalidValue;
    const dim3 block(lanes, groups);
    const auto kernel = a.neox ? (each ? norm_rope_kernel<E, Wt, true, true> : norm_rope_kernel<E, Wt, true, false>)
                               : (each ? norm_rope_kernel<E, Wt, false, true> : norm_rope_kernel<E, Wt, false, false>);
    kernel<<<(unsigned)blocks, block, 0, stream>>>(a, per, q_groups, token_groups);
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

// Rotary positions (sm_103a): the cos/sin table of a scaled frequency set, and
// the rotation of part of each head.
#include "smla_device.cuh"
#include "smla_internal.h"

#include <algorithm>
#include <climits>

namespace smla {

__device__ int g_rope_error = 0; // bit 4: a position out of range

namespace {

// Sine and cosine of a 64-bit fraction of a turn (its high 32 bits: 2^-32 of a
// turn is 1.5e-9 radians, a fortieth of binary32's step at 1). The nearest
// quarter turn leaves an angle of at most pi/4, for which the Taylor series to
// x^9 and x^10 are off by less than 2e-9; the quarter then swaps and negates.
__device__ __forceinline__ void sincos_turn(unsigned hi, float &s, float &c)
{
    const unsigned q = (hi + 0x20000000u) >> 30;
    const float x = (float)(int)(hi - (q << 30)) * 1.4629180792671596e-9f; // 2 pi 2^-32
    const float y = x * x;
    float sn = fmaf(y, 2.7557319e-6f, -1.9841270e-4f);
    sn = fmaf(sn, y, 8.3333333e-3f);
    sn = fmaf(sn, y, -1.6666667e-1f);
    sn = fmaf(sn * y, x, x);
    float cs = fmaf(y, -2.7557319e-7f, 2.4801587e-5f);
    cs = fmaf(cs, y, -1.3888889e-3f);
    cs = fmaf(cs, y, 4.1666667e-2f);
    cs = fmaf(cs, y, -0.5f);
    cs = fmaf(cs, y, 1.0f);
    const float a = q & 1 ? cs : sn, b = q & 1 ? sn : cs;
    s = q & 2 ? -a : a;
    c = (q + 1) & 2 ? -b : b;
}

// The table. frac[i] is pair i's frequency as a fraction of a turn, times 2^64:
// position * frac modulo 2^64 is then the angle modulo one turn, with no
// rounding at all however far the position, in integer arithmetic (binary64
// would run at 1/64 of the binary32 rate here). A thread keeps its kVec pairs
// and walks down the rows, adding a constant to each angle. Bound: 4 bytes
// written per value.
template <int kVec>
__global__ void __launch_bounds__(256) rope_table_kernel(float *__restrict__ table, int64_t rows, int64_t first,
                                                         const RopeFrequencies f)
{
    const int n = f.pairs, lanes = n / kVec;
    const int per = blockDim.x / lanes; // rows a block writes at a time
    const int i = threadIdx.x % lanes * kVec, r0 = threadIdx.x / lanes;
    if (r0 >= per)
        return;
    const int64_t stride = (int64_t)gridDim.x * per;
    int64_t r = (int64_t)blockIdx.x * per + r0;
    unsigned long long at[kVec], step[kVec];
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
        at[e] = (unsigned long long)(first + r) * f.frac[i + e];
        step[e] = (unsigned long long)stride * f.frac[i + e];
    }
#pragma unroll 2
    for (; r < rows; r += stride) {
        struct alignas(4 * kVec) {
            float v[kVec];
        } c, s;
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            sincos_turn((unsigned)(at[e] >> 32), s.v[e], c.v[e]);
            c.v[e] *= f.factor;
            s.v[e] *= f.factor;
            at[e] += step[e];
        }
        float *row = table + r * 2 * n + i;
        *reinterpret_cast<decltype(c) *>(row) = c;
        *reinterpret_cast<decltype(s) *>(row + n) = s;
    }
}

__device__ __forceinline__ float rot_a(float a, float b, float c, float s)
{
    return __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
}
__device__ __forceinline__ float rot_b(float a, float b, float c, float s)
{
    return __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}

__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(float x) { return x; }
template <typename E> __device__ __forceinline__ E from_f(float x);
template <> __device__ __forceinline__ __nv_bfloat16 from_f(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half from_f(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ float from_f(float x) { return x; }

// kVec elements moved as one access.
template <typename E, int kVec> struct alignas(sizeof(E) * kVec) Pack {
    E e[kVec];
};

// A unit is what one thread turns or copies of one head: with halves, kVec
// elements of each half (kVec pairs); interleaved, kVec elements (kVec / 2
// pairs; two for kVec = 1); or kVec plain columns. A thread keeps its unit, so
// its cosines and sines are loaded once, and walks over the heads of q, then k.
// threadIdx.x is the unit, threadIdx.y the first head, blockIdx.x the token.
// Both elements of a pair are read before either is written, by the one thread
// that has them: in-place calls are safe. Bound: bytes in and out.
constexpr int kBatch = 4;
template <typename E, int kVec, bool kNeox>
__global__ void __launch_bounds__(256) rope_kernel(const RopeArgs a)
{
    constexpr int kV = kNeox || kVec > 1 ? kVec : 2; // elements of a rotated unit (of each half with kNeox)
    const int64_t t = blockIdx.x;
    const int64_t pos = a.positions[t];
    if (pos < 0 || pos >= a.max_position) {
        if (threadIdx.x == 0 && threadIdx.y == 0 && blockIdx.y == 0)
            atomicOr(&g_rope_error, 4);
        return;
    }
    const int n = a.rot_dim / 2;
    const int turned = kNeox ? n / kV : a.rot_dim / kV;
    const int units = turned + (a.D - a.rot_dim) / kVec;
    const float *row = a.cos_sin + pos * a.rot_dim;
    const int heads = a.H + a.H_k;
    const int hstep = blockDim.y * gridDim.y;
    for (int u = threadIdx.x; u < units; u += blockDim.x) {
        if (u >= turned) {
            int col = (u - turned) * kVec; // plain column, the rotated ones left out
            if (col >= a.rot_offset)
                col += a.rot_dim;
            for (int h = blockIdx.y * blockDim.y + threadIdx.y; h < heads; h += hstep) {
                const bool isq = h < a.H;
                const E *src = static_cast<const E *>(isq ? a.q : a.k) + (isq ? t * a.q_st + h * a.q_sh : t * a.k_st + (h - a.H) * a.k_sh);
                E *dst = static_cast<E *>(isq ? a.q_out : a.k_out) + (isq ? t * a.qo_st + h * a.qo_sh : t * a.ko_st + (h - a.H) * a.ko_sh);
                if (src != dst)
                    *reinterpret_cast<Pack<E, kVec> *>(dst + col) = *reinterpret_cast<const Pack<E, kVec> *>(src + col);
            }
            continue;
        }
        constexpr int kPairs = kNeox ? kV : kV / 2;
        float c[kPairs], s[kPairs];
        const int p0 = u * kPairs;
#pragma unroll
        for (int e = 0; e < kPairs; ++e) {
            c[e] = __ldg(row + p0 + e);
            s[e] = __ldg(row + n + p0 + e);
            s[e] = a.inverse ? -s[e] : s[e];
        }
        // kBatch heads at a time: their loads are in flight together
        for (int h0 = blockIdx.y * blockDim.y + threadIdx.y; h0 < heads; h0 += kBatch * hstep) {
            Pack<E, kVec> x[kBatch], y[kBatch];
            E *out[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int h = h0 + k * hstep;
                if (h < heads) {
                    const bool isq = h < a.H;
                    const E *src = static_cast<const E *>(isq ? a.q : a.k) + (isq ? t * a.q_st + h * a.q_sh : t * a.k_st + (h - a.H) * a.k_sh) + a.rot_offset;
                    out[k] = static_cast<E *>(isq ? a.q_out : a.k_out) + (isq ? t * a.qo_st + h * a.qo_sh : t * a.ko_st + (h - a.H) * a.ko_sh) + a.rot_offset;
                    if (kNeox) {
                        x[k] = *reinterpret_cast<const Pack<E, kVec> *>(src + p0);
                        y[k] = *reinterpret_cast<const Pack<E, kVec> *>(src + n + p0);
                    } else {
                        x[k] = *reinterpret_cast<const Pack<E, kVec> *>(src + 2 * p0);
                        if (kVec == 1)
                            y[k] = *reinterpret_cast<const Pack<E, kVec> *>(src + 2 * p0 + 1);
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                if (h0 + k * hstep >= heads)
                    break;
                E *dst = out[k];
                Pack<E, kVec> xo, yo;
                if (kNeox || kVec == 1) {
#pragma unroll
                    for (int e = 0; e < kVec; ++e) {
                        xo.e[e] = from_f<E>(rot_a(to_f(x[k].e[e]), to_f(y[k].e[e]), c[e % kPairs], s[e % kPairs]));
                        yo.e[e] = from_f<E>(rot_b(to_f(x[k].e[e]), to_f(y[k].e[e]), c[e % kPairs], s[e % kPairs]));
                    }
                    *reinterpret_cast<Pack<E, kVec> *>(dst + (kNeox ? p0 : 2 * p0)) = xo;
                    *reinterpret_cast<Pack<E, kVec> *>(dst + (kNeox ? n + p0 : 2 * p0 + 1)) = yo;
                } else {
#pragma unroll
                    for (int e = 0; e < kPairs; ++e) {
                        const float xa = to_f(x[k].e[(2 * e) % kVec]), xb = to_f(x[k].e[(2 * e + 1) % kVec]);
                        xo.e[(2 * e) % kVec] = from_f<E>(rot_a(xa, xb, c[e], s[e]));
                        xo.e[(2 * e + 1) % kVec] = from_f<E>(rot_b(xa, xb, c[e], s[e]));
                    }
                    *reinterpret_cast<Pack<E, kVec> *>(dst + 2 * p0) = xo;
                }
            }
        }
    }
}

template <typename E, int kVec>
cudaError_t launch_vec(const RopeArgs &a, int sm_count, cudaStream_t stream)
{
    const int n = a.rot_dim / 2;
    const int kV = a.neox || kVec > 1 ? kVec : 2;
    const int units = (a.neox ? n : a.rot_dim) / kV + (a.D - a.rot_dim) / kVec;
    const int x = std::min(units, 256);
    const int heads = a.H + a.H_k;
    // a thread's batches should come out even: 40 heads over 16 threads' rows would leave the last half idle
    int y = std::max(1, std::min(128 / x, heads));
    const int64_t rounds = (heads + (int64_t)y * kBatch - 1) / ((int64_t)y * kBatch);
    if (rounds == 1)
        y = std::max(1, std::min(y, (heads + kBatch - 1) / kBatch));
    // few tokens: their heads are spread over blocks until the SMs have two each
    int64_t groups = (heads + y - 1) / y;
    groups = std::min<int64_t>(groups, std::max<int64_t>(1, (int64_t)2 * sm_count / a.T));
    const dim3 grid((unsigned)a.T, (unsigned)std::min<int64_t>(groups, 65535)), block(x, y);
    if (a.neox)
        rope_kernel<E, kVec, true><<<grid, block, 0, stream>>>(a);
    else
        rope_kernel<E, kVec, false><<<grid, block, 0, stream>>>(a);
    return cudaGetLastError();
}

template <typename E>
cudaError_t launch_type(const RopeArgs &a, int sm_count, cudaStream_t stream)
{
    // 16-byte accesses where every row, the rotated part, its halves and the
    // plain part allow them, single elements otherwise
    constexpr int kVec = 16 / sizeof(E);
    uintptr_t bits = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.q_out) |
                     reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.k_out);
    int64_t odd = a.q_st | a.q_sh | a.qo_st | a.qo_sh | a.k_st | a.k_sh | a.ko_st | a.ko_sh | a.D | a.rot_offset |
                  (a.neox ? a.rot_dim / 2 : a.rot_dim);
    if (bits % 16 == 0 && odd % kVec == 0)
        return launch_vec<E, kVec>(a, sm_count, stream);
    return launch_vec<E, 1>(a, sm_count, stream);
}

} // namespace

cudaError_t launch_rope_table(float *table, int64_t rows, int64_t first, const RopeFrequencies &f, int sm_count,
                              cudaStream_t stream)
{
    if (rows == 0)
        return cudaSuccess;
    // four pairs to a thread (16-byte stores) where the rows allow it
    const bool vec = f.pairs % 4 == 0 && reinterpret_cast<uintptr_t>(table) % 16 == 0;
    const int per = 256 / (vec ? f.pairs / 4 : f.pairs);
    const int64_t blocks = std::min<int64_t>((rows + per - 1) / per, (int64_t)std::max(sm_count, 1) * 8);
    if (vec)
        rope_table_kernel<4><<<(unsigned)blocks, 256, 0, stream>>>(table, rows, first, f);
    else
        rope_table_kernel<1><<<(unsigned)blocks, 256, 0, stream>>>(table, rows, first, f);
    return cudaGetLastError();
}

cudaError_t launch_rope(const RopeArgs &a, int dtype, int sm_count, cudaStream_t stream)
{
    switch (dtype) {
    case SMLA_BF16:
        return launch_type<__nv_bfloat16>(a, sm_count, stream);
    case SMLA_F16:
        return launch_type<__half>(a, sm_count, stream);
    default:
        return launch_type<float>(a, sm_count, stream);
    }
}

cudaError_t read_rope_error(int *out, bool reset)
{
    cudaError_t e = cudaMemcpyFromSymbol(out, g_rope_error, sizeof(int));
    if (e == cudaSuccess && reset) {
        const int zero = 0;
        e = cudaMemcpyToSymbol(g_rope_error, &zero, sizeof(int));
    }
    return e;
}

} // namespace smla

// Rotary positions (sm_103a): the cos/sin table of a scaled frequency set, and
// the rotation of part of each head.
#include "smla_device.cuh"
#include "smla_internal.h"

#include <algorithm>
#include <climits>

namespace smla {

__device__ int g_rope_error = 0; // bit 4: a position out of range

namespace {

// The table. frac[i] is pair i's frequency as a fraction of a turn, times 2^64:
// position * frac modulo 2^64 is then the angle modulo one turn, with no
// rounding at all however far the position, in integer arithmetic (binary64
// would run at 1/64 of the binary32 rate here). The signed high part, times
// 2^-63, is the angle in half turns in [-1, 1), which sinpi / cospi take.
// Bound: 4 bytes written per value.
__global__ void __launch_bounds__(256) rope_table_kernel(float *__restrict__ table, int64_t rows, int64_t first,
                                                         const RopeFrequencies f)
{
    // a thread keeps its pair and walks down the rows
    const int n = f.pairs;
    const int per = blockDim.x / n; // rows a block writes at a time
    const int i = threadIdx.x % n, r0 = threadIdx.x / n;
    if (r0 >= per)
        return;
    const unsigned long long step = f.frac[i];
    for (int64_t r = (int64_t)blockIdx.x * per + r0; r < rows; r += (int64_t)gridDim.x * per) {
        const long long a = (long long)((unsigned long long)(first + r) * step);
        float s, c;
        sincospif((float)a * 0x1p-63f, &s, &c);
        float *row = table + r * 2 * n;
        row[i] = c * f.factor;
        row[n + i] = s * f.factor;
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
        for (int h = blockIdx.y * blockDim.y + threadIdx.y; h < heads; h += hstep) {
            const bool isq = h < a.H;
            const E *src = static_cast<const E *>(isq ? a.q : a.k) + (isq ? t * a.q_st + h * a.q_sh : t * a.k_st + (h - a.H) * a.k_sh) + a.rot_offset;
            E *dst = static_cast<E *>(isq ? a.q_out : a.k_out) + (isq ? t * a.qo_st + h * a.qo_sh : t * a.ko_st + (h - a.H) * a.ko_sh) + a.rot_offset;
            if (kNeox) {
                const Pack<E, kVec> x = *reinterpret_cast<const Pack<E, kVec> *>(src + p0);
                const Pack<E, kVec> y = *reinterpret_cast<const Pack<E, kVec> *>(src + n + p0);
                Pack<E, kVec> xo, yo;
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    xo.e[e] = from_f<E>(rot_a(to_f(x.e[e]), to_f(y.e[e]), c[e], s[e]));
                    yo.e[e] = from_f<E>(rot_b(to_f(x.e[e]), to_f(y.e[e]), c[e], s[e]));
                }
                *reinterpret_cast<Pack<E, kVec> *>(dst + p0) = xo;
                *reinterpret_cast<Pack<E, kVec> *>(dst + n + p0) = yo;
            } else if (kVec > 1) {
                const Pack<E, kVec> x = *reinterpret_cast<const Pack<E, kVec> *>(src + 2 * p0);
                Pack<E, kVec> o;
#pragma unroll
                for (int e = 0; e < kPairs; ++e) {
                    const float xa = to_f(x.e[(2 * e) % kVec]), xb = to_f(x.e[(2 * e + 1) % kVec]);
                    o.e[(2 * e) % kVec] = from_f<E>(rot_a(xa, xb, c[e], s[e]));
                    o.e[(2 * e + 1) % kVec] = from_f<E>(rot_b(xa, xb, c[e], s[e]));
                }
                *reinterpret_cast<Pack<E, kVec> *>(dst + 2 * p0) = o;
            } else {
                const float xa = to_f(src[2 * p0]), xb = to_f(src[2 * p0 + 1]);
                dst[2 * p0] = from_f<E>(rot_a(xa, xb, c[0], s[0]));
                dst[2 * p0 + 1] = from_f<E>(rot_b(xa, xb, c[0], s[0]));
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
    const int y = std::max(1, std::min(256 / x, heads));
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
    const int per = 256 / f.pairs;
    const int64_t blocks = std::min<int64_t>((rows + per - 1) / per, (int64_t)std::max(sm_count, 1) * 8);
    rope_table_kernel<<<(unsigned)blocks, 256, 0, stream>>>(table, rows, first, f);
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

// Rotary positions (sm_103a): the cos/sin table of a scaled frequency set, and
// the rotation of part of each head.
#include "smla_device.cuh"
#include "smla_step.h"

#include <algorithm>
#include <climits>

namespace smla {

__device__ int g_rope_error = 0; // bit 4: a position out of range

namespace {

// Sine and cosine of a 64-bit fraction of a turn, times `factor`. The nearest quarter
// turn leaves an angle of at most pi/4, all of whose bits go into its rounding to
// binary32 (the sines of the first positions of a slow pair are as small as the
// angles), and for which the Taylor series to x^9 and x^10 are off by less than 2e-9
// of the value; the quarter then swaps and negates. In all below 6 * 2^-24 of each
// value. `at` is the fraction plus kHalves: half a quarter, so that bits 63 and 62 are
// the nearest quarter, and half of bit 32, so that the word above is rounded and the
// word below is what is left of it, with its sign.
constexpr unsigned long long kHalves = 0x2000000080000000ull;
__device__ __forceinline__ void sincos_turn(unsigned long long at, float factor, float &s, float &c)
{
    const unsigned hi = (unsigned)(at >> 32), lo = (unsigned)at;
    const float x = fmaf((float)(int)(lo ^ 0x80000000u), 0x1p-32f, (float)((int)(hi & 0x3FFFFFFFu) - 0x20000000)) *
                    1.4629180792671596e-9f; // 2 pi 2^-32
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
    const bool odd = hi & 0x40000000u;
    const unsigned f = __float_as_uint(factor);
    s = (odd ? cs : sn) * __uint_as_float(f ^ (hi & 0x80000000u));                 // quarters 2 and 3: negative
    c = (odd ? sn : cs) * __uint_as_float(f ^ ((hi + 0x40000000u) & 0x80000000u)); // quarters 1 and 2
}

// The table. frac[i] is pair i's frequency as a fraction of a turn, times 2^64:
// position * frac modulo 2^64 is then the angle modulo one turn, with no
// rounding at all however far the position, in integer arithmetic (binary64
// would run at 1/64 of the binary32 rate here). A thread keeps its kVec pairs
// and walks down the rows, adding a constant to each angle. Bound: 4 bytes
// written per value; the instructions come close to it. Measured: 1048576 rows of 64
// values (268 MB) in 40.3 us, 6.67 TB/s, 98% of the copy bandwidth (39.8 with the
// angle cut to 32 bits, 43.0 with the signs chosen instead of set, 59.4 with the
// angle converted from 64 bits at once, 63.5 with CUDA's sincospif and 4-byte stores).
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
        at[e] = (unsigned long long)(first + r) * f.frac[i + e] + kHalves;
        step[e] = (unsigned long long)stride * f.frac[i + e];
    }
#pragma unroll 2
    for (; r < rows; r += stride) {
        struct alignas(4 * kVec) {
            float v[kVec];
        } c, s;
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            sincos_turn(at[e], f.factor, s.v[e], c.v[e]);
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

// kVec elements moved as one access: as one word, whose elements are looked at in
// place (a structure of elements would be copied element by element).
template <int kBytes> struct Word;
template <> struct Word<16> { using type = uint4; };
template <> struct Word<4> { using type = uint32_t; };
template <> struct Word<2> { using type = uint16_t; };
template <typename E, int kVec> struct Pack {
    typename Word<sizeof(E) * kVec>::type w;
    __device__ __forceinline__ void load(const E *p) { w = *reinterpret_cast<const decltype(w) *>(p); }
    __device__ __forceinline__ void store(E *p) const { *reinterpret_cast<decltype(w) *>(p) = w; }
    __device__ __forceinline__ E &at(int i) { return reinterpret_cast<E *>(&w)[i]; }
};

// A unit is what one thread turns or copies of one head: with halves, kVec
// elements of each half (kVec pairs); interleaved, kVec elements (kVec / 2
// pairs; two for kVec = 1); or kVec plain columns. A thread keeps its unit, so
// its cosines and sines are loaded once, and walks over the heads of q, then k,
// a batch (64 bytes) at a time. threadIdx.x is the unit, threadIdx.y the first
// head, blockIdx.x and threadIdx.z the token. The first batch's elements are
// asked for before the position is known. Both elements of a pair are read before
// either is written, by the one thread that has them: in-place calls are safe. Bound: bytes in and
// out. Measured: 8192 tokens, 32 + 8 heads of 128 columns in bf16 (168 MB) in 30.5 us on
// the device, 5.5 TB/s (the device's own copy of as many bytes: 31 us); 64 tokens in a
// 10 us call.
template <int kVec, bool kNeox> constexpr int kBatch = kNeox || kVec == 1 ? 2 : 4;

// kPairs consecutive floats of a table row, by 16 bytes where they are aligned.
template <int kPairs>
__device__ __forceinline__ void load_angles(const float *p, float (&v)[kPairs])
{
    if (kPairs % 4 == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
#pragma unroll
        for (int e = 0; e < kPairs / 4; ++e) {
            const float4 f = __ldg(reinterpret_cast<const float4 *>(p) + e);
            v[4 * e] = f.x;
            v[(4 * e + 1) % kPairs] = f.y;
            v[(4 * e + 2) % kPairs] = f.z;
            v[(4 * e + 3) % kPairs] = f.w;
        }
    } else {
#pragma unroll
        for (int e = 0; e < kPairs; ++e)
            v[e] = __ldg(p + e);
    }
}

template <typename E, int kVec, bool kNeox>
__global__ void __launch_bounds__(256, 4) rope_kernel(const RopeArgs a)
{
    using P = Pack<E, kVec>;
    constexpr int kB = kBatch<kVec, kNeox>;
    constexpr bool kTwo = kNeox || kVec == 1;          // a unit's pairs lie in two accesses
    constexpr int kPairs = kTwo ? kVec : kVec / 2;
    const int64_t t = (int64_t)blockIdx.x * blockDim.z + threadIdx.z;
    if (t >= a.T)
        return;
    const int64_t pos = a.positions[t];
    const int n = a.rot_dim / 2;
    const int turned = n / kPairs;
    const int units = turned + (a.D - a.rot_dim) / kVec;
    const int h_first = blockIdx.y * blockDim.y + threadIdx.y, hstep = blockDim.y * gridDim.y;
    for (int u = threadIdx.x; u < units; u += blockDim.x) {
        const bool turns = u < turned;
        // the unit's columns: c0 and, of pairs in two accesses, c0 + apart
        const int apart = kNeox ? n : 1;
        int c0;
        if (!turns) {
            c0 = (u - turned) * kVec;
            c0 += c0 >= a.rot_offset ? a.rot_dim : 0;
        } else {
            c0 = a.rot_offset + u * (kNeox || !kTwo ? kVec : 2);
        }
        float c[kPairs], s[kPairs];
        bool first = true;
        // q's heads, then k's, as one row of heads
        int h = h_first;
#pragma unroll 1
        for (int side = 0; side < 2; ++side) {
            const int count = side ? a.H_k : a.H;
            const int64_t sh = side ? a.k_sh : a.q_sh, oh = side ? a.ko_sh : a.qo_sh;
            const E *src = static_cast<const E *>(side ? a.k : a.q) + t * (side ? a.k_st : a.q_st) + c0 + h * sh;
            E *dst = static_cast<E *>(side ? a.k_out : a.q_out) + t * (side ? a.ko_st : a.qo_st) + c0 + h * oh;
            const int64_t src_step = hstep * sh, dst_step = hstep * oh;
#pragma unroll 1
            for (; h < count; h += kB * hstep, src += kB * src_step, dst += kB * dst_step) {
                P x[kB], y[kTwo ? kB : 1];
#pragma unroll
                for (int i = 0; i < kB; ++i)
                    if (h + i * hstep < count) {
                        x[i].load(src + i * src_step);
                        if (kTwo && turns)
                            y[kTwo ? i : 0].load(src + i * src_step + apart);
                    }
                if (first) {
                    first = false;
                    if (pos < 0 || pos >= a.max_position) {
                        if (threadIdx.x == 0 && threadIdx.y == 0 && blockIdx.y == 0)
                            atomicOr(&g_rope_error, 4);
                        return;
                    }
                    if (turns) {
                        const float *row = a.cos_sin + pos * a.rot_dim + u * kPairs;
                        load_angles<kPairs>(row, c);
                        load_angles<kPairs>(row + n, s);
                        if (a.inverse)
#pragma unroll
                            for (int e = 0; e < kPairs; ++e)
                                s[e] = -s[e];
                    }
                }
#pragma unroll
                for (int i = 0; i < kB; ++i) {
                    if (h + i * hstep >= count)
                        break;
                    if (turns && kTwo) {
                        P yo;
#pragma unroll
                        for (int e = 0; e < kVec; ++e) {
                            const float xa = to_f(x[i].at(e)), xb = to_f(y[kTwo ? i : 0].at(e));
                            x[i].at(e) = from_f<E>(rot_a(xa, xb, c[e % kPairs], s[e % kPairs]));
                            yo.at(e) = from_f<E>(rot_b(xa, xb, c[e % kPairs], s[e % kPairs]));
                        }
                        yo.store(dst + i * dst_step + apart);
                    } else if (turns) {
#pragma unroll
                        for (int e = 0; e < kPairs; ++e) {
                            const float xa = to_f(x[i].at((2 * e) % kVec)), xb = to_f(x[i].at((2 * e + 1) % kVec));
                            x[i].at((2 * e) % kVec) = from_f<E>(rot_a(xa, xb, c[e], s[e]));
                            x[i].at((2 * e + 1) % kVec) = from_f<E>(rot_b(xa, xb, c[e], s[e]));
                        }
                    }
                    x[i].store(dst + i * dst_step);
                }
            }
            // the next side's first head of this thread: the batches above pass heads beyond the end
            if (side == 0)
                h = h_first >= a.H ? h_first - a.H : (hstep - (a.H - h_first) % hstep) % hstep;
        }
    }
}

template <typename E, int kVec>
cudaError_t launch_vec(const RopeArgs &a, int sm_count, cudaStream_t stream)
{
    const int batch = a.neox || kVec == 1 ? 2 : 4;
    const int units = a.rot_dim / 2 / (a.neox || kVec == 1 ? kVec : kVec / 2) + (a.D - a.rot_dim) / kVec;
    const int x = std::min(units, 256);
    const int heads = a.H + a.H_k;
    // Many tokens: three batches of heads to a thread, so that the positions' and angles' latency is paid once for
    // them, and as many tokens as fill a block. Few tokens: their heads are spread over threads and blocks until the
    // SMs have eight blocks each.
    int y = std::max(1, std::min(256 / x, (heads + 3 * batch - 1) / (3 * batch)));
    int z = std::min(64, 256 / (x * y));
    int64_t groups = 1;
    if ((int64_t)a.T * x * y < (int64_t)sm_count * 2048) {
        z = 1;
        y = std::max(1, std::min(std::min(128 / x, 64), (heads + batch - 1) / batch));
        groups = std::min<int64_t>((heads + y - 1) / y, std::max<int64_t>(1, (int64_t)8 * sm_count / a.T));
    }
    const dim3 grid((unsigned)(((int64_t)a.T + z - 1) / z), (unsigned)std::min<int64_t>(groups, 65535)), block(x, y, z);
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

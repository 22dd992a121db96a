// What the rotation kernels share: element types, words of elements, angles (sm_103a).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace smla {
namespace rope {

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

} // namespace rope
} // namespace smla

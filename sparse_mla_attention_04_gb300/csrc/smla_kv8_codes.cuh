// Codes of the block-scaled cache under another scale (sm_103a).
#pragma once

#include "smla_device.cuh"

namespace smla {

// Four older codes under a grown scale: E4M3(code * old / now), each operation rounded in binary32.
static __device__ __noinline__ uint32_t requant4(uint32_t w, float old, float now)
{
    uint32_t lo, hi;
    e4m3x4_to_f16x4(w, lo, hi);
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    const float2 qa = make_float2(__fdiv_rn(__fmul_rn(a.x, old), now), __fdiv_rn(__fmul_rn(a.y, old), now));
    const float2 qb = make_float2(__fdiv_rn(__fmul_rn(b.x, old), now), __fdiv_rn(__fmul_rn(b.y, old), now));
    const uint32_t ca = __nv_cvt_float2_to_fp8x2(qa, __NV_SATFINITE, __NV_E4M3);
    const uint32_t cb = __nv_cvt_float2_to_fp8x2(qb, __NV_SATFINITE, __NV_E4M3);
    return (ca & 0xFFFFu) | (cb << 16);
}

} // namespace smla

// What the two attention kernels over the block-scaled cache share (sm_103a).
#pragma once

#include "smla_device.cuh"
#include "smla_step.h"
#include "smla_umma.cuh"

namespace smla {
namespace kv8 {

// The 64-byte swizzled layout (CU_TENSOR_MAP_SWIZZLE_64B), K-major: rows of
// 64 B in atoms of 8 rows (512 B), the 16-byte chunk index (0..3) XORed with
// half the row index in the atom; SBO = distance between atoms.
__device__ __forceinline__ uint64_t desc_sw64(uint32_t saddr, uint32_t lbo, uint32_t sbo)
{
    return umma::desc(saddr, lbo, sbo) | (4ull << 61);
}

// True in one lane of a converged warp. With it the code around stays uniform, so
// that descriptors are computed in uniform registers, which tcgen05 instructions
// take; under a branch on the lane each operand is moved there first.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}

// Ends an mbarrier's use: its place may be set up anew.
__device__ __forceinline__ void mbar_inval(uint32_t mbar)
{
    asm volatile("mbarrier.inval.shared::cta.b64 [%0];\n" ::"r"(mbar) : "memory");
}

// A bounded wait of a whole converged warp (as umma::mbar_wait). The warp votes
// on what it saw, so the control flow stays uniform: where lanes branch on their
// own, coming together again costs 100 to 200 cycles a wait.
__device__ __forceinline__ bool mbar_wait_warp(uint32_t mbar, uint32_t parity)
{
    const auto look = [&] {
        uint32_t done;
        asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
                     : "=r"(done)
                     : "r"(mbar), "r"(parity)
                     : "memory");
        return __all_sync(0xffffffffu, done);
    };
    if (look())
        return true;
    const long long c0 = clock64();
    while (!look())
        if (__any_sync(0xffffffffu, clock64() - c0 > (1ll << 32)))
            return false;
    return true;
}

// TMA tile load of the box at (x, y, z) of a 3-D tensor map into shared memory at
// dst (in the map's swizzle), bytes counted on mbar; out-of-range parts of the box
// are filled with zeros.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void *tmap, int x, int y, int z, uint32_t mbar)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(dst),
                 "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(mbar)
                 : "memory");
}

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

// q's rows as two E4M3 parts: the power of two that brings a row below 2^8, and
// its inverse (NaN for a row with an infinity, which has no finite logit).
__device__ __forceinline__ void split_scale(float amax, float &up, float &down)
{
    const int e = min(max((int)(__float_as_uint(amax) >> 23) - 127, -100), 127);
    up = __uint_as_float((uint32_t)(127 + 7 - e) << 23);
    down = isinf(amax) ? NAN : __uint_as_float((uint32_t)(127 + e - 7) << 23);
}

// The largest |x| of eight bf16 values (NaN loses).
__device__ __forceinline__ float amax8(const uint4 &v)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i]));
        m = fmaxf(m, fmaxf(fabsf(f.x), fabsf(f.y)));
    }
    return m;
}

// Eight bf16 values times `up` as E4M3 codes: hi = E4M3(x) and lo = E4M3(x - hi).
// Below 2^8 the scaled values are exact in binary16 down to 2^-17, far below lo's
// smallest step.
__device__ __forceinline__ void split8(const uint4 &v, float up, uint32_t (&hi)[2], uint32_t (&lo)[2])
{
    const __nv_bfloat162 u = __float2bfloat162_rn(up);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __bfloat1622float2(__hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i]), u));
        const __half2 x = __floats2half2_rn(f.x, f.y);
        h[i] = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(x), __NV_SATFINITE, __NV_E4M3);
        const __half2 back = static_cast<__half2>(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)h[i], __NV_E4M3));
        l[i] = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(__hsub2(x, back)), __NV_SATFINITE, __NV_E4M3);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        hi[i] = __byte_perm(h[2 * i], h[2 * i + 1], 0x5410);
        lo[i] = __byte_perm(l[2 * i], l[2 * i + 1], 0x5410);
    }
}

// Tensor maps of the two caches as blocks of [block_size, D] codes, copied
// min(block_size, most_rows) rows at a time into swizzled rows of D bytes. False
// where the driver has no encoder or refuses. (Of an empty pool nothing is read:
// any aligned address will do.)
inline bool kv8_tensor_maps(const Kv8AttnArgs &a, int D, int most_rows, CUtensorMap (&maps)[2])
{
    const PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (encode == nullptr)
        return false;
    const int64_t blocks = a.num_blocks * a.H_kv;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a.block_size, (cuuint64_t)(blocks > 0 ? blocks : 1)};
    const cuuint64_t strides[2] = {(cuuint64_t)D, (cuuint64_t)D * a.block_size};
    const cuuint32_t rows = (cuuint32_t)(a.block_size < most_rows ? a.block_size : most_rows);
    const cuuint32_t box[3] = {(cuuint32_t)D, rows, 1}, step[3] = {1, 1, 1};
    for (int i = 0; i < 2; ++i) {
        void *pool = blocks > 0 ? const_cast<uint8_t *>(i ? a.v_cache : a.k_cache) : const_cast<void *>(a.q);
        if (encode(&maps[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, pool, dims, strides, box, step,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return false;
    }
    return true;
}

// The final values of a row from its sums: m the reference (log2 units), l the
// softmax denominator relative to it. Returns the factor for the value sums.
__device__ __forceinline__ float finish_row(float m, float l, const float *sinks, int head, float *lse)
{
    float f = 1.0f;
    if (sinks) {
        const float s = sinks[head] * kLog2e;
        const float top = fmaxf(m, s);
        if (fabsf(top) == INFINITY) { // a sink beside which nothing is left, or nothing seen and a sink of -inf
            *lse = sinks[head] + l;   // (a NaN among the sums stays)
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

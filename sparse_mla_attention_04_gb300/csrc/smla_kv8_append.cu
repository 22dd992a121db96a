// The write of the block-scaled 8-bit cache (sm_103a): E4M3 codes with one
// scale per (block, kv head), kept right as blocks fill.
//
// A team of one or four warps takes one run (the new tokens of one block) of one
// head of K or V: it finds the run's largest |x|, settles the block's scale,
// requantizes the block's older codes when the scale grew, and writes the run's
// codes. Nothing is shared between teams, so there are no atomics on data. What a
// lane reads of a run (kHeld 16-byte pieces) stays in registers between the two
// passes; what is beyond is read again (from L2). Bound: 2 bytes read and 1
// written per element. Measured: a prompt of 8192 tokens, 8 kv heads of 128 columns
// (50 MB) in 20.5 us on the device, 2.4 TB/s: 2048 blocks in 2.7 waves, each with its
// slots' scan, loads, two meetings, quotients and stores one after another (0.6 of the
// issue slots: four values take some ten, two conversions to bracket each quotient among
// them); one token for each of 64 requests in 4.5 us on the device, in a 17 us call.
#include "smla_device.cuh"
#include "smla_step.h"

#include <algorithm>

namespace smla {

__device__ int g_append_error = 0; // bit 8: a slot out of range

namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;
constexpr int kAlone = 2; // runs that begin in 32 tokens, above which each warp takes runs of its own
constexpr int kMinWindow = 4;
constexpr float kMinScale = 0x1p-60f;

__device__ __forceinline__ uint32_t amax2(uint32_t a, uint32_t b)
{
    const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162 *>(&a),
                                     *reinterpret_cast<const __nv_bfloat162 *>(&b)); // a NaN loses
    return *reinterpret_cast<const uint32_t *>(&m);
}

// max(m, |x|) over a vector, pairwise. kFinite: infinities left out.
template <bool kFinite>
__device__ __forceinline__ uint32_t amax8(uint32_t m, const uint4 &v)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t a = w[i] & 0x7FFF7FFFu;
        if (kFinite) {
            if ((a & 0x7FFFu) >= 0x7F80u)
                a &= 0x7FFF0000u;
            if ((a >> 16) >= 0x7F80u)
                a &= 0xFFFFu;
        }
        m = amax2(m, a);
    }
    return m;
}

// The codes of eight quotients by division: out of line, for the few vectors
// that need it (its code would be most of the kernel's).
__device__ __noinline__ uint2 divide8(const uint4 v, float s)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i]));
        c[i] = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(f.x, s), __fdiv_rn(f.y, s)), __NV_SATFINITE, __NV_E4M3);
    }
    return make_uint2((c[0] & 0xFFFFu) | (c[1] << 16), (c[2] & 0xFFFFu) | (c[3] << 16));
}

// Two products in one instruction.
__device__ __forceinline__ float2 mul2(float x, float y, float f)
{
    uint64_t a, b, r;
    asm("mov.b64 %0, {%1, %2};\n" : "=l"(a) : "f"(x), "f"(y));
    asm("mov.b64 %0, {%1, %1};\n" : "=l"(b) : "f"(f));
    asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
    float2 v;
    asm("mov.b64 {%0, %1}, %2;\n" : "=f"(v.x), "=f"(v.y) : "l"(r));
    return v;
}

// Eight bf16 values as codes of x / s (binary32 division): found by the two
// products that bracket each quotient (see quant4_e4m3), divided where they differ.
__device__ __forceinline__ uint2 quant8(const uint4 v, float s, const E4m3Recip &r)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t lo[4], hi[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float x = __uint_as_float(w[i] << 16), y = __uint_as_float(w[i] & 0xFFFF0000u);
        lo[i] = __nv_cvt_float2_to_fp8x2(mul2(x, y, r.lo), __NV_SATFINITE, __NV_E4M3);
        hi[i] = __nv_cvt_float2_to_fp8x2(mul2(x, y, r.hi), __NV_SATFINITE, __NV_E4M3);
    }
    const uint2 a = make_uint2(__byte_perm(lo[0], lo[1], 0x5410), __byte_perm(lo[2], lo[3], 0x5410));
    const uint2 b = make_uint2(__byte_perm(hi[0], hi[1], 0x5410), __byte_perm(hi[2], hi[3], 0x5410));
    if (!r.ok || a.x != b.x || a.y != b.y)
        return divide8(v, s);
    return a;
}

// Four older codes under a grown scale: E4M3(code * old / now), each operation rounded in binary32.
__device__ __noinline__ uint32_t requant4(uint32_t w, float old, float now)
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

__device__ __forceinline__ float warp_amax(uint32_t m)
{
    const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&m));
    return warp_max(fmaxf(f.x, f.y));
}

// A run's place: its first token, its block, its head (twice, plus 1 for V).
struct Run {
    int first, block, which;
};

// Writes a run, by a team of kTeam warps (four: the block); tid: the thread's number
// in it. kHeld: 16-byte pieces of a lane that stay in registers between the passes.
template <int D, int kTeam, int kHeld>
__device__ __forceinline__ void write_run(const Kv8AppendArgs &a, const Run &run, int tid, uint32_t *s_amax)
{
    constexpr int kLanes = D / 8;                  // lanes of one row
    constexpr int kRows = 32 * kTeam / kLanes;     // rows of one team-wide access
    const int lane = threadIdx.x & 31;
    const int bs = 1 << a.block_shift, h = run.which >> 1;
    const bool isv = run.which & 1;
    const int64_t st = isv ? a.v_st : a.k_st;
    // the largest over the team
    auto team_max = [&](uint32_t m) {
        float f = warp_amax(m);
        if (kTeam > 1) {
            __syncthreads();
            if (lane == 0)
                s_amax[threadIdx.x >> 5] = __float_as_uint(f);
            __syncthreads();
#pragma unroll
            for (int w = 0; w < kTeam; ++w)
                f = fmaxf(f, __uint_as_float(s_amax[w]));
        }
        return f;
    };
    float *cell = (isv ? a.v_scale : a.k_scale) + (int64_t)run.block * a.H_kv + h;
    const float old = *cell;
    const int64_t first_slot = (int64_t)run.block << a.block_shift;
    const int64_t *run_slots = a.slot_mapping + run.first;
    const int off0 = (int)(run_slots[0] - first_slot);
    const int sub = tid / kLanes, col = (tid % kLanes) * 8;
    const __nv_bfloat16 *rows = (isv ? a.v + h * a.v_sh : a.k + h * a.k_sh) + (run.first + sub) * st + col;
    const int64_t step = kRows * st;
    // A team of four asks for what a run that fills its block has before the run's
    // length is known: mostly it does.
    const int room = min(bs - off0, a.T - run.first);
    uint4 held[kHeld];
    if (kTeam > 1) {
        const __nv_bfloat16 *p = rows;
#pragma unroll
        for (int i = 0; i < kHeld; ++i, p += step)
            held[i] = i * kRows + sub < room ? *reinterpret_cast<const uint4 *>(p) : make_uint4(0, 0, 0, 0);
    }
    // the run's length, its smallest offset, and whether its slots follow one another
    int n = 0, low = bs;
    bool dense = true;
    while (true) {
        int off[4], took = 0; // offsets in the block: outside [0, bs) for another block's slots
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = n + 32 * k + lane;
            const int64_t d = i < a.T - run.first ? run_slots[i] - first_slot : -1;
            off[k] = d >= 0 && d < bs ? (int)d : -1;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const unsigned out = __ballot_sync(0xffffffffu, off[k] < 0);
            const int take = took < 32 * k ? 0 : out ? __ffs(out) - 1 : 32;
            if (lane < take) {
                low = min(low, off[k]);
                dense = dense && off[k] == off0 + n + 32 * k + lane;
            }
            took += take;
        }
        n += took;
        if (took < 128)
            break;
    }
    low = __reduce_min_sync(0xffffffffu, low);
    dense = __all_sync(0xffffffffu, dense);

    uint32_t m = 0;
    if (kTeam == 1 || n > room) {
        const __nv_bfloat16 *p = rows;
#pragma unroll
        for (int i = 0; i < kHeld; ++i, p += step)
            held[i] = i * kRows + sub < n ? *reinterpret_cast<const uint4 *>(p) : make_uint4(0, 0, 0, 0);
    } else if (n < room) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            held[i] = i * kRows + sub < n ? held[i] : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
        m = amax8<false>(m, held[i]);
    for (int r = kHeld * kRows + sub; r < n; r += kRows)
        m = amax8<false>(m, *reinterpret_cast<const uint4 *>(rows + (int64_t)(r - sub) * st));
    float amax = team_max(m);
    if (isinf(amax)) { // an infinity among the rows: the largest finite value counts
        m = 0;
        for (int r = sub; r < n; r += kRows)
            m = amax8<true>(m, *reinterpret_cast<const uint4 *>(rows + (int64_t)(r - sub) * st));
        amax = team_max(m);
    }
    // (rows of zeros, which any scale holds, ask for the smallest: they change no block that has other rows)
    float now = fmaxf(__fdiv_rn(amax, 448.0f), kMinScale);
    uint8_t *dst = (isv ? a.v_cache : a.k_cache) + (((int64_t)run.block * a.H_kv + h) << a.block_shift) * D;
    if (low > 0) {
        if (now > old) {
            for (int i = tid * 16; i < low * D; i += 512 * kTeam) {
                uint4 w = *reinterpret_cast<const uint4 *>(dst + i);
                w.x = requant4(w.x, old, now);
                w.y = requant4(w.y, old, now);
                w.z = requant4(w.z, old, now);
                w.w = requant4(w.w, old, now);
                *reinterpret_cast<uint4 *>(dst + i) = w;
            }
        } else {
            now = old;
        }
    }
    // (every thread of the team has read the old scale: it passed the team's maximum, or is in the one warp)
    __syncwarp();
    if (tid == 0)
        *cell = now;
    const E4m3Recip inv = e4m3_recip(now);
    dst += col;
    if (dense) {
        uint8_t *p = dst + (off0 + sub) * D;
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            if (i * kRows + sub < n)
                *reinterpret_cast<uint2 *>(p + i * kRows * D) = quant8(held[i], now, inv);
    } else {
#pragma unroll 1
        for (int r = sub; r < min(n, kHeld * kRows); r += kRows)
            *reinterpret_cast<uint2 *>(dst + (int)(run_slots[r] - first_slot) * D) =
                quant8(*reinterpret_cast<const uint4 *>(rows + (int64_t)(r - sub) * st), now, inv);
    }
    for (int r = kHeld * kRows + sub; r < n; r += kRows)
        *reinterpret_cast<uint2 *>(dst + (int)(run_slots[r] - first_slot) * D) =
            quant8(*reinterpret_cast<const uint4 *>(rows + (int64_t)(r - sub) * st), now, inv);
}

// A block takes the runs that begin in a window of tokens, for one head of K or V.
// Where few begin in 32 tokens, its four warps work on one run together (a prompt's
// fill their blocks); where many do, each warp takes runs of its own (a decode
// step's are one token long). The host cannot know which, since the slots are on the
// device. With 8 kv heads of 128 columns, on the device: 1024 tokens of one request 9.5
// us (24 by single warps, 7.6 by teams alone), 1400 tokens of as many requests 20 us
// (26 and 121).
template <int D> __global__ void __launch_bounds__(kThreads, 5) kv8_append_kernel(const __grid_constant__ Kv8AppendArgs a)
{
    __shared__ uint32_t s_amax[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int which = (int)(blockIdx.x % (2 * a.H_kv));
    const int t0 = (int)(blockIdx.x / (2 * a.H_kv)) * a.window;
    const int64_t slots = a.num_blocks << a.block_shift;

    // a run begins where the block changes; lane l looks at tokens t0 + l, t0 + 32 + l, ... of the window
    auto block_of = [&](int t, bool report) -> int {
        if (t < 0 || t >= a.T)
            return -1;
        const int64_t s = a.slot_mapping[t];
        if (s >= slots && report)
            atomicOr(&g_append_error, 8);
        return s >= 0 && s < slots ? (int)(s >> a.block_shift) : -1;
    };
    int last = block_of(t0 - 1, false); // of the token before
    for (int w0 = 0; w0 < a.window; w0 += 32) {
        const int blk = w0 + lane < a.window ? block_of(t0 + w0 + lane, which == 0 && warp == 0) : -1;
        int before = __shfl_up_sync(0xffffffffu, blk, 1);
        before = lane == 0 ? last : before;
        last = __shfl_sync(0xffffffffu, blk, 31);
        unsigned begins = __ballot_sync(0xffffffffu, blk >= 0 && blk != before);
        const bool alone = __popc(begins) > kAlone; // (all warps see the same)
        for (int i = 0; begins; ++i) {
            const int l0 = __ffs(begins) - 1;
            begins &= begins - 1;
            const int block = __shfl_sync(0xffffffffu, blk, l0);
            if (!alone)
                write_run<D, kWarps, 8>(a, Run{t0 + w0 + l0, block, which}, tid, s_amax);
            else if (i % kWarps == warp)
                write_run<D, 1, 2>(a, Run{t0 + w0 + l0, block, which}, lane, s_amax);
        }
    }
}

template <int D>
cudaError_t launch(const Kv8AppendArgs &a, cudaStream_t stream)
{
    const int64_t blocks = ((int64_t)a.T + a.window - 1) / a.window * a.H_kv * 2;
    if (blocks > 0x7FFFFFFF)
        return cudaErrorInvalidValue;
    kv8_append_kernel<D><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

} // namespace

cudaError_t launch_kv8_append(const Kv8AppendArgs &args, int D, int sm_count, cudaStream_t stream)
{
    Kv8AppendArgs a = args;
    // windows as large as leave eight blocks to an SM, at most a cache block: what a block looks at
    // in vain costs least then, and there is still enough to run at a time
    a.window = kMinWindow;
    while (a.window < 1 << a.block_shift && (int64_t)a.T / (2 * a.window) * a.H_kv * 2 >= (int64_t)sm_count * 8)
        a.window *= 2;
    return D == 128 ? launch<128>(a, stream) : launch<64>(a, stream);
}

cudaError_t read_append_error(int *out, bool reset)
{
    cudaError_t e = cudaMemcpyFromSymbol(out, g_append_error, sizeof(int));
    if (e == cudaSuccess && reset) {
        const int zero = 0;
        e = cudaMemcpyToSymbol(g_append_error, &zero, sizeof(int));
    }
    return e;
}

} // namespace smla

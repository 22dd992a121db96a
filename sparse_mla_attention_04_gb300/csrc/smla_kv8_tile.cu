// Attention over the block-scaled 8-bit cache for many query rows (prompts and
// chunks of prompts, sm_103a): 128 query rows to a tile, both products on the
// tensor cores (tcgen05), scores and sums in tensor memory.
//
// A CTA takes 128 rows (token, head of the kv head's group) of one request and
// kv head and walks over the visible positions in tiles of 128. Two CTAs share
// an SM: one's softmax runs while the other's products do, so each CTA's own
// chain stays simple: scores, softmax, values, scores, ... Its warps:
//   0-3  softmax, a row to a thread; the epilogue
//   4-5  V: codes to registers and, expanded to binary16, to shared memory
//   6    K: the blocks' codes by TMA as they lie in the cache; the blocks' scales
//   7    one thread issues the tensor-core products
// (eight warps, so that both CTAs' threads have 128 registers).
//
// S = Q K^T runs on the cache's codes as they are. q's bf16 values are carried
// exactly by two E4M3 parts: scaled by a power of two to below 2^8, hi = E4M3(q)
// and lo = E4M3(q - hi) hold the 8 significant bits of every element down to
// 2^-9 of the row's largest (smaller ones to 2^-17 of it); two fp8 products
// take the time of one in 16 bits and need no expansion of K.
// O += P V takes P in binary16 from tensor memory (where it overlays S) and V
// expanded exactly to binary16: 8-bit weights would lose half of their bits.
// The block scales enter as in the streaming kernel: K's multiplies the logits,
// V's is folded into the exponent, p' = 2^(s + log2(vs) - m), and the
// denominator adds p' / vs. A row's reference m moves, and its O is rescaled,
// only when a logit passes it by 8 (p' <= 2^8 is far inside binary16).
//
// Shared memory: K in TMA's swizzled rows; Q and V in 8-row x 16-byte core
// matrices, written so that eight lanes fill one (no bank conflict). Blocks
// outside the pool and V beyond the visible positions are zero-filled and not
// read.
#include "smla_kv8.cuh"
#include "smla_umma.cuh"

#include <algorithm>

namespace smla {

__device__ int g_kv8_error = 0; // 1: a bounded wait gave up; 2: products in flight did not drain

namespace {

using namespace kv8;
using namespace umma;

constexpr int kRows = 128;
constexpr int kTile = 128;
constexpr int kSoftmaxThreads = 128, kVThreads = 64;
constexpr int kThreads = 256;
constexpr float kSlack = 8.0f;
constexpr int kMaxSplits = 8;

template <int D> struct Shape {
    static constexpr int kQBytes = kRows * D;       // one part of Q, or one tile of K codes
    static constexpr int kVBytes = kTile * D * 2;   // a tile of V in binary16
    static constexpr int kQAtoms = D / 16 * 128;    // 8 rows of Q: D / 16 core matrices
    static constexpr int kVAtoms = D / 8 * 128;     // 8 rows of V
    static constexpr int kK = 0;                    // two stages
    static constexpr int kQ = 2 * kQBytes;          // hi, lo
    static constexpr int kV = kQ + 2 * kQBytes;
    static constexpr int kScales = kV + kVBytes;    // 4 stages x 8 groups x {c, log2 vs, 1 / vs}
    static constexpr int kBars = kScales + 4 * 8 * 12;
    static constexpr int kMisc = kBars + 10 * 8;
    static constexpr int kNan = kMisc + 16;         // a bit for each (row, column)
    static constexpr int kNanWords = kRows * D / 32;
    static constexpr int kSmem = kNan + kNanWords * 4 + 1024; // the base is rounded up to 1024
    static constexpr uint32_t kTmem = 256;          // S (P over its first half) and O
    static constexpr uint32_t kO = 128;
    static constexpr uint32_t kIdescS = idesc(128, kTile, 0, 0, 0, 0);
    static constexpr uint32_t kIdescO = idesc(128, D, 0, 0, 0, 1);
};

struct Part {
    float2 *ml; // [items][splits][128]
    float *o;   // [items][splits][128][D]
    int splits;
};

// A tile's item: request, chunk of rows, kv head.
struct Item {
    int b, chunk, h;
};

// Items are numbered request by request; request b's first number is
// floor(q0 G / 128) + b, which leaves room for its ceil(rows / 128) chunks
// without a running sum. Returns false for a number that no chunk has.
__device__ __forceinline__ bool find_item(const Kv8AttnArgs &a, int n, Item *it)
{
    int lo = 0, hi = a.B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        const int q0 = min(max(a.query_start[mid], 0), a.T);
        if ((int)((long long)q0 * a.G / kRows) + mid <= n)
            lo = mid;
        else
            hi = mid - 1;
    }
    const Request r = request(a, lo);
    it->b = lo;
    it->chunk = n - ((int)((long long)r.q0 * a.G / kRows) + lo);
    return it->chunk >= 0 && (long long)it->chunk * kRows < (long long)r.qlen * a.G;
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w)
{
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// Four floats below 2^8 as E4M3 codes of hi and of the rest lo.
__device__ __forceinline__ void split4(float a, float b, float c, float d, uint32_t &hi, uint32_t &lo)
{
    const uint32_t h0 = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t h1 = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    hi = (h0 & 0xFFFFu) | (h1 << 16);
    uint32_t f0, f1;
    e4m3x4_to_f16x4(hi, f0, f1);
    const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&f0));
    const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&f1));
    const uint32_t l0 = __nv_cvt_float2_to_fp8x2(make_float2(a - x.x, b - x.y), __NV_SATFINITE, __NV_E4M3);
    const uint32_t l1 = __nv_cvt_float2_to_fp8x2(make_float2(c - y.x, d - y.y), __NV_SATFINITE, __NV_E4M3);
    lo = (l0 & 0xFFFFu) | (l1 << 16);
}

// Two binary32 operations in one instruction.
__device__ __forceinline__ uint64_t pair(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t r, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;\n" : "=f"(a), "=f"(b) : "l"(r)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c)); // a NaN loses, as with fmaxf
    return r;
}

// Waits for this thread's tensor-memory loads; x holds what they brought only after it.
__device__ __forceinline__ void wait_ld16(uint32_t (&x)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;\n"
                 : "+r"(x[0]), "+r"(x[1]), "+r"(x[2]), "+r"(x[3]), "+r"(x[4]), "+r"(x[5]), "+r"(x[6]), "+r"(x[7]),
                   "+r"(x[8]), "+r"(x[9]), "+r"(x[10]), "+r"(x[11]), "+r"(x[12]), "+r"(x[13]), "+r"(x[14]), "+r"(x[15])::"memory");
}

// The largest logit of 16 scores of one row. sc: the group's factor of K,
// sc[8]: log2 of its value scale. kClear: every position is seen; else position
// t + i is when pos_lo <= t + i <= pos.
template <bool kClear>
__device__ __forceinline__ float group_max(const uint32_t (&x)[16], const float *sc, float qs, int t, int pos, int pos_lo)
{
    float b0 = -INFINITY, b1 = -INFINITY;
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            y[e] = __uint_as_float(x[i + e]);
            if (!kClear)
                y[e] = (t + i + e <= pos && t + i + e >= pos_lo) ? y[e] : -INFINITY;
        }
        b0 = max3(b0, y[0], y[1]);
        b1 = max3(b1, y[2], y[3]);
    }
    b0 = fmaxf(b0, b1);
    const float s = fmaf(b0, sc[0] * qs, sc[8]);
    // (a masked group has no logit; -inf times a factor of 0 would be NaN)
    return !kClear && b0 == -INFINITY ? b0 : s;
}

// The largest logit of a row's 128 scores (the thread's lane of tensor memory);
// a group's load is in flight while the one before is looked at.
template <bool kClear>
__device__ __forceinline__ float row_max(uint32_t my, const float *sc, float qs, int t0, int pos, int pos_lo)
{
    float top = -INFINITY;
    uint32_t a[16], b[16];
    ld16(my, a);
    wait_ld16(a);
#pragma unroll 1
    for (int g = 0; g < 8; g += 2) {
        ld16(my + g * 16 + 16, b);
        top = fmaxf(top, group_max<kClear>(a, sc + g, qs, t0 + g * 16, pos, pos_lo));
        wait_ld16(b);
        if (g < 6)
            ld16(my + g * 16 + 32, a);
        top = fmaxf(top, group_max<kClear>(b, sc + g + 1, qs, t0 + g * 16 + 16, pos, pos_lo));
        wait_ld16(a);
    }
    return top;
}

// The weights 2^(s + log2(vs) - ref) of 16 scores, in binary16, written over
// scores that were read before; their sum divided by vs is added to l. sc[16]:
// 1 / vs. kPlain: every position is seen and |ref| is small.
template <bool kPlain>
__device__ __forceinline__ float group_weights(const uint32_t (&x)[16], uint32_t dst, const float *sc, float qs, float ref,
                                               float l, int t, int pos, int pos_lo)
{
    uint32_t p[8];
    const float k0 = sc[0] * qs, b0 = sc[8] - ref;
    const uint64_t kk = pair(k0, k0), bb = pair(b0, b0);
    uint64_t sum = 0;
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
        const float x0 = __uint_as_float(x[i]), x1 = __uint_as_float(x[i + 1]);
        float p0, p1;
        if (kPlain) {
            unpair(fma2(pair(x0, x1), kk, bb), p0, p1);
            p0 = ex2_approx(p0);
            p1 = ex2_approx(p1);
        } else {
            p0 = ex2_approx(fmaf(x0, k0, sc[8]) - ref);
            p1 = ex2_approx(fmaf(x1, k0, sc[8]) - ref);
            p0 = (t + i <= pos && t + i >= pos_lo) ? p0 : 0.f;
            p1 = (t + i + 1 <= pos && t + i + 1 >= pos_lo) ? p1 : 0.f;
        }
        sum = add2(sum, pair(p0, p1));
        p[i / 2] = pack_f16x2(p0, p1);
    }
    st8(dst, p);
    float s0, s1;
    unpair(sum, s0, s1);
    return fmaf(s0 + s1, sc[16], l);
}

template <bool kPlain>
__device__ __forceinline__ float row_weights(uint32_t my, const float *sc, float qs, float ref, float l, int t0, int pos,
                                             int pos_lo)
{
    uint32_t a[16], b[16];
    ld16(my, a);
    wait_ld16(a);
#pragma unroll 1
    for (int g = 0; g < 8; g += 2) {
        ld16(my + g * 16 + 16, b);
        l = group_weights<kPlain>(a, my + g * 8, sc + g, qs, ref, l, t0 + g * 16, pos, pos_lo);
        wait_ld16(b);
        if (g < 6)
            ld16(my + g * 16 + 32, a);
        l = group_weights<kPlain>(b, my + g * 8 + 8, sc + g + 1, qs, ref, l, t0 + g * 16 + 16, pos, pos_lo);
        wait_ld16(a);
    }
    return l;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2) kv8_tile_kernel(const __grid_constant__ CUtensorMap k_map, const Kv8AttnArgs a,
                                                               const Part part)
{
    using S = Shape<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
    uint32_t *s_nan = reinterpret_cast<uint32_t *>(smem + S::kNan);
    int *s_any_nan = reinterpret_cast<int *>(smem + S::kMisc + 8);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t base = smem_u32(smem);
    const uint32_t bars = base + S::kBars;
    // K landed / free (two stages), scores ready, P ready, V ready, values done, drained
    const uint32_t k_full = bars, k_empty = bars + 16, s_full = bars + 32, p_full = bars + 40, v_full = bars + 48,
                   v_empty = bars + 56, drained = bars + 64;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + S::kMisc);

    // the longest rows first: a causal prompt's last chunks
    Item it;
    const int n_item = (int)((gridDim.x - 1 - blockIdx.x) / a.H_kv);
    it.h = (int)((gridDim.x - 1 - blockIdx.x) % a.H_kv);
    if (!find_item(a, n_item, &it))
        return;
    const Request rq = request(a, it.b);
    const int row0 = it.chunk * kRows;
    const int rows = min(kRows, rq.qlen * a.G - row0);
    const int p_first = rq.pos(row0 / a.G), p_last = rq.pos((row0 + rows - 1) / a.G);
    const int kv_end = min(rq.len, p_last + 1);                                       // beyond: seen by none
    const int kv_begin = a.window > 0 ? max(0, p_first - a.window + 1) : 0;
    const int all_from = a.window > 0 ? p_last - a.window + 1 : 0;                    // [all_from, p_first]: seen by all
    const int tb0 = kv_begin & ~(kTile - 1); // so that the blocks lie whole in the tiles
    const int tiles_all = kv_end > tb0 ? (kv_end - tb0 + kTile - 1) / kTile : 0;
    const int split = blockIdx.y;
    const int t_begin = (int)((long long)tiles_all * split / part.splits);
    const int t_end = (int)((long long)tiles_all * (split + 1) / part.splits);
    const int n = t_end - t_begin;
    const bool many = p_first != p_last;

    if (n <= 0) { // nothing to see here
        if (tid < rows) {
            const int64_t t = rq.q0 + (row0 + tid) / a.G;
            const int head = it.h * a.G + (row0 + tid) % a.G;
            if (part.splits > 1) {
                part.ml[(((int64_t)n_item * a.H_kv + it.h) * part.splits + split) * kRows + tid] = make_float2(-INFINITY, 0.f);
            } else {
                float lse;
                finish_row(-INFINITY, 0.f, a.sinks, head, &lse);
                uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + (t * a.H + head) * D);
                for (int i = 0; i < D / 8; ++i)
                    dst[i] = make_uint4(0, 0, 0, 0);
                if (a.lse)
                    a.lse[t * a.H + head] = lse;
            }
        }
        return;
    }

    if (tid == 0) {
        *s_any_nan = 0;
        mbar_init(k_full, 2); // the copies' bytes; the scales
        mbar_init(k_full + 8, 2);
        mbar_init(k_empty, 1);
        mbar_init(k_empty + 8, 1);
        mbar_init(s_full, 1);
        mbar_init(p_full, kSoftmaxThreads);
        mbar_init(v_full, kVThreads);
        mbar_init(v_empty, 1);
        mbar_init(drained, 1);
        mbar_init_fence();
    }
    if (many)
        for (int i = tid; i < S::kNanWords; i += kThreads)
            s_nan[i] = 0;
    if (warp == 7)
        alloc(smem_u32(tmem_slot), S::kTmem);
    const float scale_log2 = fabsf(a.scale) * kLog2e; // the sign goes into q

    float qs = 0.f;
    if (tid < kSoftmaxThreads) {
        // this thread's row of Q, in two E4M3 parts
        const int r = tid;
        const bool live = r < rows;
        const int rr = row0 + (live ? r : 0);
        const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.q) +
                                                           (int64_t)(rq.q0 + rr / a.G) * a.q_st +
                                                           (int64_t)(it.h * a.G + rr % a.G) * a.q_sh);
        float amax = 0.f;
#pragma unroll 4
        for (int i = 0; i < D / 8; ++i) {
            const uint4 v = live ? src[i] : make_uint4(0, 0, 0, 0);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[e]));
                amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
        }
        const int e = min(max((int)(__float_as_uint(amax) >> 23) - 127, -100), 127);
        float up = __uint_as_float((uint32_t)(127 + 7 - e) << 23);
        qs = isinf(amax) ? NAN : __uint_as_float((uint32_t)(127 + e - 7) << 23); // an infinite q has no finite logit
        up = a.scale < 0.f ? -up : up;
        const uint32_t dst = base + S::kQ + (r >> 3) * S::kQAtoms + (r & 7) * 16;
#pragma unroll 2
        for (int i = 0; i < D / 16; ++i) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e2 = 0; e2 < 2; ++e2) {
                const uint4 v = live ? src[2 * i + e2] : make_uint4(0, 0, 0, 0);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float2 f0 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[2 * x]));
                    const float2 f1 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[2 * x + 1]));
                    split4(f0.x * up, f0.y * up, f1.x * up, f1.y * up, hi[2 * e2 + x], lo[2 * e2 + x]);
                }
            }
            sts128(dst + i * 128, hi[0], hi[1], hi[2], hi[3]);
            sts128(dst + S::kQBytes + i * 128, lo[0], lo[1], lo[2], lo[3]);
        }
        fence_async_smem();
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    bool ok = true;
    // a bounded wait, by whole warps (or by the one thread of warp 7)
    auto wait_warp = [&](uint32_t bar, uint32_t parity) {
        ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, parity));
        if (!ok && lane == 0)
            atomicOr(&g_kv8_error, 1);
        return ok;
    };

    if (warp < 4) {
        // ---------------------------------------------------------------- softmax
        const int r = tid;
        const int pos = r < rows ? rq.pos((row0 + r) / a.G) : -1;
        const int pos_lo = a.window > 0 ? pos - a.window + 1 : 0;
        const uint32_t my = tmem + ((uint32_t)(warp * 32) << 16);
        const float *scales = reinterpret_cast<const float *>(smem + S::kScales);
        float m = -INFINITY, l = 0.f;
        for (int j = 0; j < n; ++j) {
            // the scales of this tile's blocks come with its K; then its scores
            if (!wait_warp(k_full + (j & 1) * 8, (j >> 1) & 1) || !wait_warp(s_full, j & 1))
                break;
            fence_after_sync();
            const int tb = tb0 + (t_begin + j) * kTile;
            const float *sc = scales + (j & 3) * 24;
            const bool clear = tb + kTile - 1 <= p_first && tb >= all_from;
            const float top = clear ? row_max<true>(my, sc, qs, 0, 0, 0) : row_max<false>(my, sc, qs, tb, pos, pos_lo);
            const bool raise = top > m + kSlack;
            if (__any_sync(0xffffffffu, raise)) {
                // O is at rest: the scores just read were issued after its last product was done
                const float f = !raise ? 1.f : (m == -INFINITY ? 0.f : ex2_approx(m - top));
                m = raise ? top : m;
                l *= f;
                if (j > 0) {
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t x[32];
                        ld32(my + S::kO + c * 32, x);
                        wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            x[i] = __float_as_uint(__uint_as_float(x[i]) * f);
                        st32(my + S::kO + c * 32, x);
                    }
                }
            }
            const float ref = m == -INFINITY ? 0.f : m;
            // beyond 2^20, s - m is taken from the rounded logit, as m was, or the rounding
            // of m alone could pass any bound of p'
            const bool plain = clear && !__any_sync(0xffffffffu, fabsf(ref) > 0x1p20f);
            l = plain ? row_weights<true>(my, sc, qs, ref, l, 0, 0, 0) : row_weights<false>(my, sc, qs, ref, l, tb, pos, pos_lo);
            wait_st();
            fence_before_sync();
            mbar_arrive(p_full);
        }
        // (V's last arrival carries the notes of NaN codes)
        if (ok && wait_warp(v_full, (n - 1) & 1) && wait_warp(v_empty, (n - 1) & 1)) {
            fence_after_sync();
            const bool live = r < rows;
            const int rr = row0 + (live ? r : 0);
            const int64_t t = rq.q0 + rr / a.G;
            const int head = it.h * a.G + rr % a.G;
            const int64_t slot = (((int64_t)n_item * a.H_kv + it.h) * part.splits + split) * kRows + r;
            const bool nans = many && *s_any_nan;
            float lse = 0.f, f = 1.f;
            if (part.splits == 1)
                f = finish_row(m, l, a.sinks, head, &lse);
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                uint32_t x[32];
                ld32(my + S::kO + c * 32, x);
                wait_ld();
                if (nans) {
                    const uint32_t bits = s_nan[(r * D + c * 32) >> 5];
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        x[i] = (bits >> i & 1) ? 0x7FC00000u : x[i];
                }
                if (!live)
                    continue;
                if (part.splits == 1) {
                    uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + (t * a.H + head) * D + c * 32);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            w[e] = pack_bf16x2(__uint_as_float(x[i * 8 + 2 * e]) * f, __uint_as_float(x[i * 8 + 2 * e + 1]) * f);
                        dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                } else {
                    uint4 *dst = reinterpret_cast<uint4 *>(part.o + slot * D + c * 32);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        dst[i] = make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
                }
            }
            if (live) {
                if (part.splits > 1)
                    part.ml[slot] = make_float2(m, l);
                else if (a.lse)
                    a.lse[t * a.H + head] = lse;
            }
        }
    } else if (warp < 6) {
        // ---------------------------------------------------------------- V
        constexpr int kC = D / 64;                   // 16-byte pieces of a row to a lane
        const int vw = warp - 4;
        const int sub = lane & 7, piece = lane >> 3; // rows vw * 64 + sub + 8 k, pieces piece + 4 c
        const int32_t *table = a.block_table + it.b * a.table_stride;
        int raw[4]; // table entries of the warp's four groups of 16 positions
        uint4 vr[8][kC];
        auto load_blocks = [&](int j) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int t = tb0 + (t_begin + j) * kTile + vw * 64 + 16 * x;
                const int e = t >> a.block_shift;
                raw[x] = t < kv_end && e < a.table_width ? __ldg(table + e) : -1;
            }
        };
        auto load_v = [&](int j) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int t = tb0 + (t_begin + j) * kTile + vw * 64 + sub + 8 * k;
                const int v = raw[k >> 1];
                const bool in = v >= 0 && v < a.num_blocks && t < kv_end && t >= kv_begin;
                const uint8_t *src = a.v_cache + piece * 16 +
                                     ((((int64_t)v * a.H_kv + it.h) << a.block_shift) + (t & (a.block_size - 1))) * D;
#pragma unroll
                for (int c = 0; c < kC; ++c)
                    vr[k][c] = in ? __ldg(reinterpret_cast<const uint4 *>(src + c * 64)) : make_uint4(0, 0, 0, 0);
            }
        };
        load_blocks(0);
        load_v(0);
        if (n > 1)
            load_blocks(1);
        for (int j = 0; j < n; ++j) {
            if (j > 0 && !wait_warp(v_empty, (j - 1) & 1))
                break;
            const int tb = tb0 + (t_begin + j) * kTile;
            if (many && !(tb + kTile - 1 <= p_first && tb >= all_from)) {
                // A NaN code at a position that some rows see and others do not must not
                // reach the others through 0 * NaN: it is taken out and noted for the
                // rows that see it.
#pragma unroll
                for (int k = 0; k < 8; ++k)
#pragma unroll
                    for (int c = 0; c < kC; ++c) {
                        uint32_t w[4] = {vr[k][c].x, vr[k][c].y, vr[k][c].z, vr[k][c].w};
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const uint32_t bad = nan_bytes(w[y]);
                            if (bad) {
                                const int t = tb + vw * 64 + sub + 8 * k;
                                for (int z = 0; z < 4; ++z)
                                    if (bad >> (8 * z + 7) & 1) {
                                        const int d = (piece + 4 * c) * 16 + 4 * y + z;
                                        for (int r = 0; r < rows; ++r) {
                                            const int p = rq.pos((row0 + r) / a.G);
                                            if (t <= p && (a.window <= 0 || t > p - a.window))
                                                atomicOr(&s_nan[(r * D + d) >> 5], 1u << (d & 31));
                                        }
                                    }
                                *s_any_nan = 1;
                                w[y] &= ~((bad >> 7) * 0xFFu);
                            }
                        }
                        vr[k][c] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
            }
            const uint32_t dst = base + S::kV + vw * 8 * S::kVAtoms + sub * 16 + piece * 256;
#pragma unroll
            for (int k = 0; k < 8; ++k)
#pragma unroll
                for (int c = 0; c < kC; ++c) {
                    uint32_t f[8];
                    e4m3x4_to_f16x4(vr[k][c].x, f[0], f[1]);
                    e4m3x4_to_f16x4(vr[k][c].y, f[2], f[3]);
                    e4m3x4_to_f16x4(vr[k][c].z, f[4], f[5]);
                    e4m3x4_to_f16x4(vr[k][c].w, f[6], f[7]);
                    sts128(dst + k * S::kVAtoms + c * 1024, f[0], f[1], f[2], f[3]);
                    sts128(dst + k * S::kVAtoms + c * 1024 + 128, f[4], f[5], f[6], f[7]);
                }
            fence_async_smem();
            mbar_arrive(v_full);
            if (j + 1 < n)
                load_v(j + 1);
            if (j + 2 < n)
                load_blocks(j + 2);
        }
    } else if (warp == 6) {
        // ---------------------------------------------------------------- K and the scales
        const int32_t *table = a.block_table + it.b * a.table_stride;
        const int pages = kTile >> a.block_shift;
        float *scales = reinterpret_cast<float *>(smem + S::kScales);
        auto entry = [&](int j) { // lane g < 8: the table entry of group g
            const int t = tb0 + (t_begin + j) * kTile + 16 * (lane & 7);
            const int e = t >> a.block_shift;
            return t < kv_end && e < a.table_width ? __ldg(table + e) : -1;
        };
        int raw = entry(0), issued = 0;
        for (int j = 0; j < n; ++j) {
            const int v = raw >= 0 && raw < a.num_blocks ? raw : -1;
            if (j + 1 < n)
                raw = entry(j + 1);
            if (j > 1 && !wait_warp(k_empty + (j & 1) * 8, ((j >> 1) - 1) & 1))
                break;
            const uint32_t full = k_full + (j & 1) * 8;
            if (lane == 0)
                mbar_arrive_expect_tx(full, S::kQBytes);
            __syncwarp();
            const int page = __shfl_sync(0xffffffffu, v, (lane << a.block_shift >> 4) & 7);
            if (lane < pages) // a block outside the pool: rows outside the map, which fills zeros and reads nothing
                tma_load_3d(base + S::kK + (j & 1) * S::kQBytes + (lane << a.block_shift) * D, &k_map, 0,
                            page >= 0 ? 0 : a.block_size, page >= 0 ? page * a.H_kv + it.h : 0, full);
            issued = j + 1;
            if (lane < 8) {
                // a group outside the pool (or past the end): logits of -inf
                const float ks = v >= 0 ? __ldg(a.k_scale + (int64_t)v * a.H_kv + it.h) : 0.f;
                const float vs = v >= 0 ? __ldg(a.v_scale + (int64_t)v * a.H_kv + it.h) : 0.f;
                float *sc = scales + (j & 3) * 24 + lane;
                sc[0] = ks * scale_log2;
                sc[8] = v >= 0 ? lg2_approx(vs) : -INFINITY;
                sc[16] = v >= 0 ? __frcp_rn(vs) : 1.f;
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(full);
        }
        // no copy outlives the block, also where a wait gave up
        for (int j = max(0, issued - 2); j < issued; ++j)
            if (!mbar_wait(k_full + (j & 1) * 8, (j >> 1) & 1) && lane == 0)
                atomicOr(&g_kv8_error, 2);
    } else if (lane == 0) {
        // ---------------------------------------------------------------- products
        auto wait = [&](uint32_t bar, uint32_t parity) {
            ok = ok && mbar_wait(bar, parity);
            if (!ok)
                atomicOr(&g_kv8_error, 1);
            return ok;
        };
        const uint64_t q_hi = desc(base + S::kQ, 128, S::kQAtoms);
        const uint64_t q_lo = desc(base + S::kQ + S::kQBytes, 128, S::kQAtoms);
        const uint64_t v_d = desc(base + S::kV, S::kVAtoms, 128);
        for (int j = 0; j < n; ++j) {
            // P overlays S: the last product of P is done before scores are written there
            if (!wait(k_full + (j & 1) * 8, (j >> 1) & 1) || (j > 0 && !wait(v_empty, (j - 1) & 1)))
                break;
            fence_after_sync();
            const uint32_t k_s = base + S::kK + (j & 1) * S::kQBytes;
            const uint64_t k_d = D == 128 ? desc_sw128(k_s, 16, 1024) : desc_sw64(k_s, 16, 512);
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk) // 32 columns: two core matrices of Q, 32 bytes of a row of K
                mma_f8(tmem, q_hi + kk * 16, k_d + kk * 2, S::kIdescS, kk > 0);
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk)
                mma_f8(tmem, q_lo + kk * 16, k_d + kk * 2, S::kIdescS, 1);
            commit(s_full);
            commit(k_empty + (j & 1) * 8);
            if (!wait(v_full, j & 1) || !wait(p_full, j & 1))
                break;
            fence_after_sync();
#pragma unroll
            for (int kk = 0; kk < kTile / 16; ++kk) // 16 positions: 8 columns of P, two atoms of V
                mma_f16_ts(tmem + S::kO, tmem + kk * 8, v_d + (uint64_t)(kk * 2 * S::kVAtoms / 16), S::kIdescO, j > 0 || kk > 0);
            commit(v_empty);
        }
        if (!ok) { // what was issued ends before its memory is given back
            commit(drained);
            if (!mbar_wait(drained, 0))
                atomicOr(&g_kv8_error, 2);
        }
    }
    __syncwarp();
    fence_before_sync();
    __syncthreads();
    if (warp == 7)
        dealloc(tmem, S::kTmem);
}

// Joins the splits of each item's rows, a warp to a row.
template <int D>
__global__ void __launch_bounds__(256) kv8_tile_join_kernel(const Kv8AttnArgs a, const Part part)
{
    constexpr int kD = D / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Item it;
    const int n_item = (int)(blockIdx.x / a.H_kv);
    it.h = (int)(blockIdx.x % a.H_kv);
    if (!find_item(a, n_item, &it))
        return;
    const Request rq = request(a, it.b);
    const int row0 = it.chunk * kRows;
    const int rows = min(kRows, rq.qlen * a.G - row0);
    const int64_t slot0 = ((int64_t)n_item * a.H_kv + it.h) * part.splits * kRows;
    for (int r = warp + 8 * blockIdx.y; r < rows; r += 8 * gridDim.y) {
        float2 ml[kMaxSplits];
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int s = 0; s < kMaxSplits; ++s)
            if (s < part.splits) {
                ml[s] = part.ml[slot0 + s * kRows + r];
                m = fmaxf(m, ml[s].x);
            }
        float acc[kD];
#pragma unroll
        for (int i = 0; i < kD; ++i)
            acc[i] = 0.f;
#pragma unroll
        for (int s = 0; s < kMaxSplits; ++s)
            if (s < part.splits && !(ml[s].x == -INFINITY && ml[s].y == 0.f)) { // nothing seen: no sums were written
                const float f = ml[s].x == -INFINITY ? 1.f : ex2_approx(ml[s].x - m);
                l += ml[s].y * f;
                const float *src = part.o + (slot0 + s * kRows + r) * D + lane * kD;
#pragma unroll
                for (int i = 0; i < kD; i += 2) {
                    const float2 v = *reinterpret_cast<const float2 *>(src + i);
                    acc[i] += v.x * f;
                    acc[i + 1] += v.y * f;
                }
            }
        const int64_t t = rq.q0 + (row0 + r) / a.G;
        const int head = it.h * a.G + (row0 + r) % a.G;
        float lse;
        const float f = finish_row(m, l, a.sinks, head, &lse);
        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.out) + (t * a.H + head) * D + lane * kD;
#pragma unroll
        for (int i = 0; i < kD; i += 2)
            *reinterpret_cast<uint32_t *>(dst + i) = pack_bf16x2(acc[i] * f, acc[i + 1] * f);
        if (a.lse && lane == 0)
            a.lse[t * a.H + head] = lse;
    }
}

int64_t items_of(int B, int T, int G) { return (int64_t)T * G / kRows + B; }

// Splits of a request's positions: while the items are fewer than three to
// each CTA slot, so that ragged lengths even out.
int splits_of(int B, int T, int H, int H_kv, int sm_count)
{
    const int64_t items = items_of(B, T, H / H_kv) * H_kv, slots = 2 * (int64_t)std::max(sm_count, 1);
    return (int)std::min<int64_t>(kMaxSplits, std::max<int64_t>(1, 3 * slots / std::max<int64_t>(items, 1)));
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

template <int D>
cudaError_t launch(const Kv8AttnArgs &a, void *workspace, int sm_count, cudaStream_t stream)
{
    const int64_t items = items_of(a.B, a.T, a.G) * a.H_kv;
    Part part;
    part.splits = splits_of(a.B, a.T, a.G * a.H_kv, a.H_kv, sm_count);
    const size_t slots = (size_t)items * part.splits * kRows;
    part.ml = static_cast<float2 *>(workspace);
    part.o = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + up256(slots * sizeof(float2)));
    cudaError_t e = cudaFuncSetAttribute(kv8_tile_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<D>::kSmem);
    if (e != cudaSuccess)
        return e;
    // K as blocks of [block_size, D] bytes, the rows swizzled as they land
    const PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (encode == nullptr)
        return cudaErrorNotSupported;
    CUtensorMap k_map;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a.block_size, (cuuint64_t)std::max<int64_t>(1, a.num_blocks * a.H_kv)};
    const cuuint64_t strides[2] = {(cuuint64_t)D, (cuuint64_t)D * a.block_size};
    const cuuint32_t box[3] = {(cuuint32_t)D, (cuuint32_t)a.block_size, 1}, step[3] = {1, 1, 1};
    // (of an empty pool nothing is read: any aligned address will do)
    void *pool = a.num_blocks > 0 ? const_cast<uint8_t *>(a.k_cache) : const_cast<void *>(a.q);
    if (encode(&k_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, pool, dims, strides, box, step,
               CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    kv8_tile_kernel<D><<<dim3((unsigned)items, part.splits), kThreads, Shape<D>::kSmem, stream>>>(k_map, a, part);
    if ((e = cudaGetLastError()) != cudaSuccess || part.splits == 1)
        return e;
    kv8_tile_join_kernel<D><<<dim3((unsigned)items, 4), 256, 0, stream>>>(a, part);
    return cudaGetLastError();
}

} // namespace

size_t kv8_tile_workspace(int B, int T, int H, int H_kv, int D, int sm_count)
{
    const int splits = splits_of(B, T, H, H_kv, sm_count);
    if (splits == 1)
        return 256;
    const size_t slots = (size_t)items_of(B, T, H / H_kv) * H_kv * splits * kRows;
    return up256(slots * sizeof(float2)) + slots * D * sizeof(float);
}

cudaError_t launch_kv8_tile(const Kv8AttnArgs &a, int D, void *workspace, int sm_count, cudaStream_t stream)
{
    return D == 128 ? launch<128>(a, workspace, sm_count, stream) : launch<64>(a, workspace, sm_count, stream);
}

cudaError_t read_kv8_error(int *out, bool reset)
{
    cudaError_t e = cudaMemcpyFromSymbol(out, g_kv8_error, sizeof(int));
    if (e == cudaSuccess && reset) {
        const int zero = 0;
        e = cudaMemcpyToSymbol(g_kv8_error, &zero, sizeof(int));
    }
    return e;
}

} // namespace smla

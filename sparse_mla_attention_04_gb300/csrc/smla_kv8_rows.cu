// Attention over the block-scaled 8-bit cache for some dozens of query rows (drafted
// trees, sm_103a): up to 64 rows (token, head of the kv head's group) of a request to
// a unit, both products transposed on the tensor cores (tcgen05), so that positions
// and value columns fill their 128 rows and the query rows the columns, of which a
// unit has as many as it needs. (The tile kernel has query rows on the 128 and pays
// for all of them.)
//
// A CTA stays on its SM and takes its part of the work, which is cut evenly as in the
// streaming kernel: units laid end to end, each as long as its tiles of 128 positions
// and a constant; a unit that several CTAs share leaves partial sums that a second
// kernel joins in a fixed order. Nothing is planned before, nothing depends on the host
// knowing the lengths. Warps:
//   8  softmax: a position to a thread (four warps), half of the columns each. Q before,
//      the epilogue behind
//   4  V's codes, expanded to binary16
//   3  K's copies (TMA) and scales, V's copies, the products
// Each role walks the units by itself; between them stand barriers that count through
// all units, so that the next unit's copies come while the last one ends.
//
// S^T = K Q^T runs on the cache's codes as they are, q in two E4M3 parts (as in the
// tile kernel). P^T goes to shared memory in binary16, O^T = V^T P^T accumulates in
// tensor memory. p' = 2^(s + log2(vs) - m) with V's block scale in the exponent, and the
// denominator, which every thread keeps for its position and columns in binary32, adds
// p' / vs. The reference m of a row moves (to 2^10 below the largest) only when a weight
// would pass 2^15.9: each tile's threads vote on that before the exponentials, in one
// barrier; a row that has seen nothing has a reference so low that what it sees moves it.
#include "smla_kv8.cuh"
#include "smla_umma.cuh"

#include <algorithm>

namespace smla {

__device__ int g_kv8_rows_error = 0; // 1: a bounded wait gave up; 2: copies or products in flight did not drain

namespace {

using namespace kv8;
using namespace umma;

constexpr int R = 64;      // rows of a unit
constexpr int kTile = 128; // positions
constexpr int kGroups = kTile / 16;
constexpr float kTop = 10.0f;   // (log2) the largest weight where the reference is set,
constexpr float kSlack = 15.9f; // and what none may pass: binary16 ends at 65504
constexpr float kUnseen = -1e38f; // the reference of a row that has seen nothing
constexpr float kNoRow = 1e30f;   // that of columns without a row: all their weights are 0
constexpr int kUnitCost = 4;    // a unit's start and end, in tiles
constexpr int kMinPart = 3;     // a CTA's part of the work, in tiles, before more CTAs share it

constexpr int kSoftmax = 8, kV0 = 8, kVWarps = 4, kLoadK = 12, kLoadV = 13, kMma = 14, kWarps = 15;
constexpr int kThreads = kWarps * 32;
constexpr int kKStages = 4, kScaleSlots = 8, kBatch = 4; // scales come for four tiles at a time

// What the softmax warps share of a unit's rows.
struct Rows {
    float qs[R], m[R]; // factor of the logits, reference
    float g[R];        // by which sums are scaled when it moves; at the end the factor of the values
    float top[4][R], l[4][R];
};

// Where the CTA is in the work: every role has its own.
struct Walk {
    long long at, hi, base; // cost: here, the part's end, before request b
    int b;
};

struct Misc {
    Walk start;
    long long total;
    int parts;
    uint32_t tmem;
    int any_nan;
    long long warp_cost[kWarps];
};

template <int D> struct Shape {
    static constexpr int kTileBytes = kTile * D;
    static constexpr int kQBytes = R * D;        // one part of Q
    static constexpr int kQAtoms = D / 16 * 128; // 8 rows of Q: D / 16 core matrices
    static constexpr int kVAtoms = D / 8 * 128;  // 8 positions of V
    static constexpr int kPAtoms = R / 8 * 128;  // 8 positions of P
    static constexpr int kPBytes = kTile / 8 * kPAtoms, kVBytes = kTile / 8 * kVAtoms;
    static constexpr int kK = 0;
    static constexpr int kCodes = kK + kKStages * kTileBytes; // V as it comes, two stages
    static constexpr int kV = kCodes + 2 * kTileBytes;        // two stages
    static constexpr int kP = kV + 2 * kVBytes;               // two stages
    static constexpr int kQ = kP + 2 * kPBytes;               // hi, lo
    static constexpr int kScales = kQ + 2 * kQBytes;          // slots x 4 tiles x 8 groups x {c, log2 vs, 1 / vs, -}
    static constexpr int kRows = kScales + kScaleSlots * kBatch * kGroups * 16;
    static constexpr int kBars = kRows + (int)sizeof(Rows);
    // K landed / free; V's codes landed / free; scales of four tiles written; Q written; scores ready / read; P ready; V
    // ready; values done; the unit's values read; drained
    static constexpr int kKFull = 0, kKEmpty = kKFull + kKStages, kCFull = kKEmpty + kKStages, kCEmpty = kCFull + 2,
                         kScFull = kCEmpty + 2, kQFull = kScFull + kScaleSlots, kSFull = kQFull + 1, kSEmpty = kSFull + 2,
                         kPFull = kSEmpty + 2, kVFull = kPFull + 2, kDone = kVFull + 2, kOFree = kDone + 2, kDrained = kOFree + 1,
                         kBarriers = kDrained + 1;
    static constexpr int kMisc = kBars + (kBarriers + 1) / 2 * 16;
    static constexpr int kSmem = kMisc + (int)sizeof(Misc);
    static constexpr uint32_t kO = 2 * R, kTmem = 256; // two S, then O
    static_assert(kSmem <= 227 * 1024, "one CTA to an SM");
};

// The units of one request and the cost of each.
struct Units {
    int tb0, tiles; // from position tb0 (a multiple of kTile)
    long long count, cost;
};

__device__ __forceinline__ Units units_of(const Kv8AttnArgs &a, const Request &r)
{
    Units u;
    u.tb0 = r.begin & ~(kTile - 1);
    u.tiles = max(1, (r.len - u.tb0 + kTile - 1) / kTile);
    u.count = (((long long)r.qlen * a.G + R - 1) / R) * a.H_kv;
    u.cost = u.tiles + kUnitCost;
    return u;
}

// Equal parts of the total cost.
__device__ __forceinline__ long long part_begin(long long total, int parts, int i) { return total * i / parts; }
__device__ __forceinline__ int part_of(long long total, int parts, long long x) { return (int)(((x + 1) * parts - 1) / total); }

// The workspace: for each CTA the unit that it begins and others end, {last CTA (-1: none), request, index in the
// request}; then a head and a tail partial of each CTA.
struct Part {
    int4 *dir;
    float2 *ml; // [2 CTAs][R]
    float *o;   // [2 CTAs][R][D]
};

// A piece of a unit: tiles [t0, t1) of it.
struct Piece {
    Request rq;
    int b, index, h, row0, rows, columns; // columns: rows up to a multiple of 16
    int tb0, t0, t1;
    bool whole, first; // first: it begins the unit
    int p_first, all_from, kv_begin, kv_end; // [all_from, p_first] is seen by all rows; what is outside [kv_begin, kv_end) by none
    long long end_cost; // of the unit, for what begins it

    __device__ bool clear(int tb) const { return tb + kTile - 1 <= p_first && tb >= all_from; }
};

// The next piece; false when the part is done. (Pieces in a unit's constant cost have no tiles and are passed over.)
__device__ __forceinline__ bool next_piece(const Kv8AttnArgs &a, Walk &w, Piece &p)
{
    while (w.at < w.hi) {
        Request rq = request(a, w.b);
        Units un = units_of(a, rq);
        while (w.at >= w.base + un.count * un.cost) { // requests without tokens have no units
            w.base += un.count * un.cost;
            rq = request(a, ++w.b);
            un = units_of(a, rq);
        }
        const long long ui = (w.at - w.base) / un.cost;
        const long long ubase = w.base + ui * un.cost;
        const long long uend = min(w.hi, ubase + un.cost);
        p.t0 = (int)max(0ll, w.at - ubase - kUnitCost);
        p.t1 = (int)max(0ll, uend - ubase - kUnitCost);
        w.at = uend;
        if (p.t0 >= p.t1)
            continue;
        p.rq = rq;
        p.b = w.b;
        p.index = (int)ui;
        p.h = (int)(ui % a.H_kv);
        p.row0 = (int)(ui / a.H_kv) * R;
        p.rows = min(R, rq.qlen * a.G - p.row0);
        p.columns = (p.rows + 15) & ~15;
        p.tb0 = un.tb0;
        p.first = p.t0 == 0;
        p.whole = p.first && p.t1 == un.tiles;
        p.p_first = rq.pos(-1);
        p.kv_end = rq.len;
        p.kv_begin = a.window > 0 ? max(0, p.p_first - a.window + 2) : 0;
        p.all_from = a.window > 0 ? rq.len - a.window : 0;
        p.end_cost = ubase + un.cost;
        return true;
    }
    return false;
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w)
{
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ void sts64(uint32_t addr, uint32_t x, uint32_t y)
{
    asm volatile("st.shared.v2.b32 [%0], {%1,%2};\n" ::"r"(addr), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

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
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// The softmax warps' barrier, with a vote: whether any thread says yes.
__device__ __forceinline__ bool any_of_softmax(bool yes)
{
    uint32_t r;
    asm volatile("{\n.reg .pred p, q;\nsetp.ne.u32 p, %1, 0;\nbarrier.cta.red.or.pred q, 1, 256, p;\nselp.u32 %0, 1, 0, q;\n}\n"
                 : "=r"(r)
                 : "r"((uint32_t)yes)
                 : "memory");
    return r != 0;
}
__device__ __forceinline__ void softmax_sync() { named_bar(1, kSoftmax * 32); }

// Waits for this thread's tensor-memory loads; x holds what they brought only after it.
__device__ __forceinline__ void wait_ld8(uint32_t (&x)[8])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;\n"
                 : "+r"(x[0]), "+r"(x[1]), "+r"(x[2]), "+r"(x[3]), "+r"(x[4]), "+r"(x[5]), "+r"(x[6]), "+r"(x[7])::"memory");
}

// Which of the thread's columns see position j: bit c for column c0 + c. (Seldom: a unit has one or two such tiles.)
__device__ __noinline__ uint32_t sight_of(const Kv8AttnArgs &a, const Piece &p, int c0, int n, int j)
{
    uint32_t see = 0;
#pragma unroll 1
    for (int c = 0; c < n; ++c) {
        const int r = c0 + c;
        const TreeRow row(a, p.rq, p.rq.q0 + (p.row0 + r) / a.G, r < p.rows);
        see |= (uint32_t)row.sees(j) << c;
    }
    return see;
}

// V's codes of a position in a tile that not every row sees whole: nothing where no row sees it (the block holds
// anything there), and a NaN code that some rows see and others do not must not reach the others through 0 * NaN: it is
// taken out, and the rows that see it look for it at their end.
__device__ __noinline__ uint4 visible_codes(uint4 v, bool in, int *any_nan)
{
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int y = 0; y < 4; ++y) {
        w[y] = in ? w[y] : 0;
        const uint32_t bad = nan_bytes(w[y]);
        if (bad) {
            *any_nan = 1;
            w[y] &= ~((bad >> 7) * 0xFFu);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Which of the thread's columns see a NaN code in value column d, in the tiles where some rows see positions that
// others do not (there the codes were taken out).
template <int D>
__device__ __noinline__ uint32_t nan_rows(const Kv8AttnArgs &a, const Piece &p, int c0, int n, int d)
{
    uint32_t bits = 0;
    for (int t = p.t0; t < p.t1; ++t) {
        const int tb = p.tb0 + t * kTile;
        if (p.clear(tb))
            continue;
        for (int j = max(tb, p.kv_begin); j < min(tb + kTile, p.kv_end); ++j) {
            const int e = j >> a.block_shift;
            const int v = e < a.table_width ? a.block_table[p.b * a.table_stride + e] : -1;
            if (v < 0 || v >= a.num_blocks)
                continue;
            const uint8_t code =
                a.v_cache[((((int64_t)v * a.H_kv + p.h) << a.block_shift) + (j & (a.block_size - 1))) * D + d];
            if ((code & 0x7F) == 0x7F)
                bits |= sight_of(a, p, c0, n, j);
        }
    }
    return bits;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv8_rows_kernel(const __grid_constant__ CUtensorMap k_map,
                                                               const __grid_constant__ CUtensorMap v_map,
                                                               const __grid_constant__ Kv8AttnArgs a, const Part part)
{
    using S = Shape<D>;
    extern __shared__ __align__(1024) uint8_t smem[]; // (the swizzle goes by address)
    Misc *misc = reinterpret_cast<Misc *>(smem + S::kMisc);
    Rows *rows = reinterpret_cast<Rows *>(smem + S::kRows);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t base = smem_u32(smem), bars = base + S::kBars;
    const auto bar = [&](int first, int i) { return bars + 8 * (first + i); };
    grid_launch_dependents();

    const bool fits = (base & 1023u) == 0; // otherwise a layout that the swizzle does not fit
    if (!fits && tid == 0)
        atomicOr(&g_kv8_rows_error, 1);
    if (tid == 0)
        part.dir[blockIdx.x] = make_int4(-1, 0, 0, 0);
    const int rows_in = min(kTile, a.block_size), pages = kTile / rows_in; // of a block in a tile; blocks of a tile
    if (tid < S::kBarriers) { // a barrier to a thread
        const int count = tid < S::kKEmpty    ? pages
                          : tid < S::kCFull   ? 1
                          : tid < S::kCEmpty  ? pages
                          : tid < S::kScFull  ? kVWarps
                          : tid < S::kQFull   ? 1
                          : tid < S::kSFull   ? kSoftmax
                          : tid < S::kSEmpty  ? 1
                          : tid < S::kVFull   ? kSoftmax // scores read, P ready
                          : tid < S::kDone    ? kVWarps
                          : tid < S::kOFree   ? 1
                          : tid < S::kDrained ? kSoftmax
                                              : 1;
        mbar_init(bar(tid, 0), count);
        mbar_init_fence();
    }
    if (warp == kMma)
        alloc(smem_u32(&misc->tmem), S::kTmem);
    // The total cost and this CTA's part of it: each thread adds up its requests, the block scans the sums, and the
    // thread whose requests hold the part's begin finds the request.
    {
        const int per = (a.B + kThreads - 1) / kThreads;
        long long cost = 0;
        for (int i = 0; i < per; ++i) {
            const int b = tid * per + i;
            if (b < a.B) {
                const Units u = units_of(a, request(a, b));
                cost += u.count * u.cost;
            }
        }
        long long cost_to = cost; // inclusive
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, cost_to, d);
            cost_to += lane >= d ? x : 0;
        }
        if (lane == 31)
            misc->warp_cost[warp] = cost_to;
        if (tid == 0)
            misc->start = Walk{0, 0, 0, 0};
        __syncthreads();
        long long total = 0, cost0 = cost_to - cost;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            cost0 += w < warp ? misc->warp_cost[w] : 0;
            total += misc->warp_cost[w];
        }
        const int parts = (int)min((long long)gridDim.x, max(1ll, (total + kMinPart - 1) / kMinPart));
        if (fits && (int)blockIdx.x < parts && total > 0) {
            const long long lo = part_begin(total, parts, blockIdx.x), hi = part_begin(total, parts, blockIdx.x + 1);
            if (lo < hi && lo >= cost0 && lo < cost0 + cost) {
                int b = tid * per;
                Units u = units_of(a, request(a, b));
                while (lo >= cost0 + u.count * u.cost) {
                    cost0 += u.count * u.cost;
                    u = units_of(a, request(a, ++b));
                }
                misc->start = Walk{lo, hi, cost0, b};
                misc->total = total;
                misc->parts = parts;
            }
        }
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = misc->tmem;
    Walk walk = misc->start;
    Piece p;
    bool ok = true;
    // a bounded wait, by whole warps; after one that gave up, none waits
    const auto wait_warp = [&](uint32_t b, uint32_t parity) {
        ok = ok && mbar_wait_warp(b, parity);
        if (!ok && lane == 0)
            atomicOr(&g_kv8_rows_error, 1);
        return ok;
    };
    uint32_t it = 0; // tiles so far, of all pieces: the same in every role

    if (warp < kSoftmax) {
        // ---------------------------------------------------------------- softmax
        const int quad = warp & 3, half = warp >> 2;
        const uint32_t my = tmem + ((uint32_t)(quad * 32) << 16);
        const int place = quad * 32 + lane; // the thread's position in a tile
        uint32_t batch = 0, unit = 0;
        for (; next_piece(a, walk, p); ++unit) {
            if (p.first && !p.whole && tid == 0)
                part.dir[blockIdx.x] = make_int4(part_of(misc->total, misc->parts, p.end_cost - 1), p.b, p.index, 0);
            const int mine = p.columns / 2, c0 = half * mine; // the thread's columns
            if (tid == 0)
                misc->any_nan = 0; // (V's warps write it in this piece's tiles only: they wait for Q)
            // Q in two E4M3 parts: four lanes to a row, eight rows to a warp
            {
                const int r = warp * 8 + (lane >> 2);
                const bool live = r < p.rows;
                const int row = p.row0 + (live ? r : 0);
                const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.q) +
                                                                   (int64_t)(p.rq.q0 + row / a.G) * a.q_st +
                                                                   (int64_t)(p.h * a.G + row % a.G) * a.q_sh) + (lane & 3);
                uint4 x[D / 32];
                float amax = 0.f;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    x[c] = live ? src[4 * c] : make_uint4(0, 0, 0, 0);
                    amax = fmaxf(amax, amax8(x[c]));
                }
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                float up, down;
                split_scale(amax, up, down);
                up = a.scale < 0.f ? -up : up;
                const uint32_t dst = base + S::kQ + warp * S::kQAtoms + (lane >> 2) * 16 + (lane >> 1 & 1) * 128 + (lane & 1) * 8;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t hi[2], lo[2];
                    split8(x[c], up, hi, lo);
                    sts64(dst + c * 256, hi[0], hi[1]);
                    sts64(dst + c * 256 + S::kQBytes, lo[0], lo[1]);
                }
                if ((lane & 3) == 0) {
                    rows->qs[r] = live ? down : 0.f;
                    rows->m[r] = live ? kUnseen : kNoRow;
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar(S::kQFull, 0));
            }
            softmax_sync();
            float l[32];
#pragma unroll
            for (int c = 0; c < 32; ++c)
                l[c] = 0.f;
            const float *scales = reinterpret_cast<const float *>(smem + S::kScales);
            for (int t = p.t0; t < p.t1; ++t, ++it) {
                const int tb = p.tb0 + t * kTile, j = t - p.t0;
                if ((j & (kBatch - 1)) == 0) {
                    wait_warp(bar(S::kScFull, batch & (kScaleSlots - 1)), batch / kScaleSlots & 1);
                    ++batch;
                }
                wait_warp(bar(S::kSFull, it & 1), it >> 1 & 1);
                fence_after_sync();
                const float4 f = reinterpret_cast<const float4 *>(
                    scales)[(((batch - 1) & (kScaleSlots - 1)) * kBatch + (j & (kBatch - 1))) * kGroups + (place >> 4)];
                const uint32_t my_s = my + (it & 1) * R + c0;
                const uint32_t see = p.clear(tb) ? 0xffffffffu : sight_of(a, p, c0, mine, tb + place);
                const uint64_t kk = pair(f.x, f.x), vs = pair(f.y, f.y);
                float y[32]; // logits relative to the reference
                const auto logits = [&](bool relative) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (8 * c < mine) {
                            uint32_t x[8];
                            ld8(my_s + 8 * c, x);
                            const float4 q0 = *reinterpret_cast<const float4 *>(rows->qs + c0 + 8 * c),
                                         q1 = *reinterpret_cast<const float4 *>(rows->qs + c0 + 8 * c + 4);
                            const float4 m0 = *reinterpret_cast<const float4 *>(rows->m + c0 + 8 * c),
                                         m1 = *reinterpret_cast<const float4 *>(rows->m + c0 + 8 * c + 4);
                            const float q[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
                            const float m[8] = {m0.x, m0.y, m0.z, m0.w, m1.x, m1.y, m1.z, m1.w};
                            wait_ld8(x);
#pragma unroll
                            for (int i = 0; i < 8; i += 2) {
                                uint64_t s = fma2(pair(__uint_as_float(x[i]), __uint_as_float(x[i + 1])),
                                                  mul2(kk, pair(q[i], q[i + 1])), vs);
                                if (relative)
                                    s = add2(s, pair(-m[i], -m[i + 1]));
                                unpair(s, y[8 * c + i], y[8 * c + i + 1]);
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                y[8 * c + i] = -INFINITY;
                        }
                    if (see != 0xffffffffu)
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            y[c] = see >> c & 1 ? y[c] : -INFINITY;
                };
                logits(true);
                float top = -INFINITY;
#pragma unroll
                for (int c = 0; c < 32; ++c)
                    top = fmaxf(top, y[c]); // (a NaN loses)
                if (any_of_softmax(top > kSlack)) {
                    // references move: the rows' largest logits, by lane, warp and block
                    logits(false);
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        float x = y[c];
#pragma unroll
                        for (int d = 16; d > 0; d >>= 1)
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
                        if (lane == c && c < mine)
                            rows->top[quad][c0 + c] = x;
                    }
                    softmax_sync();
                    if (tid < p.columns) {
                        const float m = rows->m[tid];
                        const float x = fmaxf(fmaxf(rows->top[0][tid], rows->top[1][tid]), fmaxf(rows->top[2][tid], rows->top[3][tid]));
                        const bool moves = m == kUnseen ? x > -INFINITY : __fadd_ru(x, -m) > kSlack;
                        // (rounded up, so that far out, where kTop is less than the logits' step, no weight passes 1)
                        const float now = moves ? __fadd_ru(x, -kTop) : m;
                        rows->g[tid] = moves ? (m == kUnseen ? 0.f : ex2_approx(m - now)) : 1.f;
                        rows->m[tid] = now;
                    }
                    softmax_sync();
                    // O is at rest once the last tile's product is done: the next one waits for this tile's weights
                    if (j > 0)
                        wait_warp(bar(S::kDone, (it - 1) & 1), (it - 1) >> 1 & 1);
                    fence_after_sync();
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (8 * c < mine) {
                            float g[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                g[i] = rows->g[c0 + 8 * c + i];
                                l[8 * c + i] *= g[i];
                            }
                            if (j > 0) {
                                uint32_t o[8];
                                ld8(my + S::kO + c0 + 8 * c, o);
                                wait_ld8(o);
#pragma unroll
                                for (int i = 0; i < 8; ++i)
                                    o[i] = __float_as_uint(__uint_as_float(o[i]) * g[i]);
                                st8(my + S::kO + c0 + 8 * c, o);
                            }
                        }
                    wait_st();
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        if (c < mine)
                            y[c] -= rows->m[c0 + c];
                }
                fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar(S::kSEmpty, it & 1));
                if (it > 1) // P's stage is free
                    wait_warp(bar(S::kDone, it & 1), ((it >> 1) - 1) & 1);
                const uint64_t iv = pair(f.z, f.z);
                const uint32_t dst = base + S::kP + (it & 1) * S::kPBytes + (place >> 3) * S::kPAtoms + (place & 7) * 16 + c0 / 8 * 128;
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (8 * c < mine) {
                        uint32_t w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float p0 = ex2_approx(y[8 * c + 2 * i]), p1 = ex2_approx(y[8 * c + 2 * i + 1]);
                            unpair(fma2(pair(p0, p1), iv, pair(l[8 * c + 2 * i], l[8 * c + 2 * i + 1])), l[8 * c + 2 * i],
                                   l[8 * c + 2 * i + 1]);
                            w[i] = pack_f16x2(p0, p1);
                        }
                        sts128(dst + c * 128, w[0], w[1], w[2], w[3]);
                    }
                fence_async_smem();
                fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar(S::kPFull, it & 1));
            }
            // the piece's end: the denominators of the columns, over positions, lanes (column c to lane c) and warps
#pragma unroll
            for (int d = 16; d > 0; d >>= 1)
#pragma unroll
                for (int i = 0; i < d; ++i) {
                    const bool up = lane & d;
                    const float keep = up ? l[i + d] : l[i], give = up ? l[i] : l[i + d];
                    l[i] = keep + __shfl_xor_sync(0xffffffffu, give, d);
                }
            if (lane < mine)
                rows->l[quad][c0 + lane] = l[0];
            wait_warp(bar(S::kVFull, (it - 1) & 1), (it - 1) >> 1 & 1); // (carries the notes of NaN codes)
            wait_warp(bar(S::kDone, (it - 1) & 1), (it - 1) >> 1 & 1);
            fence_after_sync();
            softmax_sync();
            const int64_t slot = (2 * (int64_t)blockIdx.x + (p.first ? 1 : 0)) * R;
            if (ok && tid < p.rows) {
                const float m = rows->m[tid] == kUnseen ? -INFINITY : rows->m[tid];
                const float sum = (rows->l[0][tid] + rows->l[1][tid]) + (rows->l[2][tid] + rows->l[3][tid]);
                if (p.whole) {
                    const int64_t t = p.rq.q0 + (p.row0 + tid) / a.G;
                    const int head = p.h * a.G + (p.row0 + tid) % a.G;
                    float lse;
                    rows->g[tid] = finish_row(m, sum, a.sinks, head, &lse);
                    if (a.lse)
                        a.lse[t * a.H + head] = lse;
                } else {
                    part.ml[slot + tid] = make_float2(m, sum);
                }
            }
            softmax_sync();
            // value column d of the thread's lane (of 64: sixteen lanes of each warp)
            const int d = D == 128 ? place : quad * 16 + (lane & 15);
            const bool live = ok && (D == 128 || lane < 16);
            uint32_t bad = 0;
            if (misc->any_nan)
                bad = nan_rows<D>(a, p, c0, mine, d);
#pragma unroll 1
            for (int c = 0; c < mine; c += 8) {
                uint32_t x[8];
                ld8(my + S::kO + c0 + c, x);
                wait_ld8(x);
                if (live) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int r = c0 + c + i;
                        float v = __uint_as_float(x[i]);
                        v = bad >> (c + i) & 1 ? NAN : v;
                        if (r < p.rows) {
                            if (p.whole) {
                                const int64_t t = p.rq.q0 + (p.row0 + r) / a.G;
                                const int head = p.h * a.G + (p.row0 + r) % a.G;
                                static_cast<__nv_bfloat16 *>(a.out)[(t * a.H + head) * D + d] = __float2bfloat16_rn(v * rows->g[r]);
                            } else {
                                part.o[(slot + r) * D + d] = v;
                            }
                        }
                    }
                }
            }
            fence_before_sync();
            softmax_sync(); // every warp is done with the rows' values, and with O
            if (lane == 0)
                mbar_arrive(bar(S::kOFree, 0));
        }
    } else if (warp < kLoadK) {
        // ---------------------------------------------------------------- V
        constexpr int kTurns = kTile / kVWarps / 8;
        const int row_in = (warp - kV0) * kTurns * 8 + (lane & 7), piece = lane >> 3; // rows row_in + 8 k, pieces piece + 4 c
        const int turn = D == 128 ? lane & 7 : (lane >> 1) & 3;                      // the swizzle of the lane's rows
        uint32_t unit = 0;
        for (; next_piece(a, walk, p); ++unit) {
            wait_warp(bar(S::kQFull, 0), unit & 1); // (the notes of NaN codes are this piece's)
            for (int t = p.t0; t < p.t1; ++t, ++it) {
                const int stage = it & 1, tb = p.tb0 + t * kTile;
                wait_warp(bar(S::kCFull, stage), it >> 1 & 1);
                if (it > 1)
                    wait_warp(bar(S::kDone, stage), ((it >> 1) - 1) & 1);
                const bool clear = p.clear(tb);
                const uint32_t src = base + S::kCodes + stage * S::kTileBytes + row_in * D;
                const uint32_t dst = base + S::kV + stage * S::kVBytes + (row_in >> 3) * S::kVAtoms + (lane & 7) * 16 + piece * 256;
                uint4 q[kTurns][D / 64]; // all of them on their way before the first is used
#pragma unroll
                for (int k = 0; k < kTurns; ++k)
#pragma unroll
                    for (int c = 0; c < D / 64; ++c)
                        q[k][c] = lds128(src + k * 8 * D + (((piece + 4 * c) ^ turn) << 4));
#pragma unroll
                for (int k = 0; k < kTurns; ++k)
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) {
                        const int pos = tb + row_in + 8 * k;
                        if (!clear)
                            q[k][c] = visible_codes(q[k][c], pos < p.kv_end && pos >= p.kv_begin, &misc->any_nan);
                        const uint32_t w[4] = {q[k][c].x, q[k][c].y, q[k][c].z, q[k][c].w};
                        uint32_t f[8];
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            e4m3x4_to_f16x4(w[y], f[2 * y], f[2 * y + 1]);
                        sts128(dst + k * S::kVAtoms + c * 1024, f[0], f[1], f[2], f[3]);
                        sts128(dst + k * S::kVAtoms + c * 1024 + 128, f[4], f[5], f[6], f[7]);
                    }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(S::kCEmpty, stage));
                    mbar_arrive(bar(S::kVFull, stage));
                }
            }
        }
    } else if (warp <= kLoadV) {
        // ---------------------------------------------------------------- the cache's codes and scales
        // Lane l looks after group l % 8 (16 positions) of tile l / 8 of four: the table is read two fours ahead, the
        // scales one, so that no latency is waited for.
        const bool keys = warp == kLoadK;
        const float scale_log2 = fabsf(a.scale) * kLog2e; // the sign goes into q
        float4 *scales = reinterpret_cast<float4 *>(smem + S::kScales);
        uint32_t batch = 0;
        while (next_piece(a, walk, p)) {
            const int32_t *table = a.block_table + p.b * a.table_stride;
            const auto entry = [&](int four) {
                const int x = p.tb0 + (p.t0 + kBatch * four + (lane >> 3)) * kTile + 16 * (lane & 7);
                const int e = x >> a.block_shift;
                return x < p.kv_end && e < a.table_width ? __ldg(table + e) : -1;
            };
            const auto in_pool = [&](int e) { return e >= 0 && e < a.num_blocks ? e : -1; };
            const auto scale_of = [&](const float *s, int v) { return keys && v >= 0 ? __ldg(s + (int64_t)v * a.H_kv + p.h) : 0.f; };
            int v = -1, v_next = in_pool(entry(0)), raw = entry(1);
            float ks = 0.f, vs = 0.f, ks_next = scale_of(a.k_scale, v_next), vs_next = scale_of(a.v_scale, v_next);
            for (int t = p.t0; t < p.t1; ++t, ++it) {
                const int j = t - p.t0;
                if ((j & (kBatch - 1)) == 0) {
                    v = v_next;
                    ks = ks_next;
                    vs = vs_next;
                    v_next = in_pool(raw);
                    ks_next = scale_of(a.k_scale, v_next);
                    vs_next = scale_of(a.v_scale, v_next);
                    raw = entry(j / kBatch + 2);
                }
                // lane i: block i of the tile. A block outside the pool: rows outside the map, which fills zeros and
                // reads nothing
                const int page = __shfl_sync(0xffffffffu, v, (j & (kBatch - 1)) * 8 + ((lane * rows_in >> 4) & 7));
                const int y = page >= 0 ? (p.tb0 + t * kTile + lane * rows_in) & (a.block_size - 1) : a.block_size;
                const int z = page >= 0 ? page * a.H_kv + p.h : 0;
                const uint32_t at = lane * rows_in * D;
                if (keys) {
                    const int stage = it & (kKStages - 1);
                    if (it >= kKStages)
                        wait_warp(bar(S::kKEmpty, stage), (it / kKStages - 1) & 1);
                    if (ok && lane < pages) {
                        mbar_arrive_expect_tx(bar(S::kKFull, stage), rows_in * D);
                        tma_load_3d(base + S::kK + stage * S::kTileBytes + at, &k_map, 0, y, z, bar(S::kKFull, stage));
                    }
                    if ((j & (kBatch - 1)) == 0) {
                        // the scales of four tiles, a group to a lane. A group outside the pool, past the end, or below
                        // what any row sees (where the block may have gone to another request: a bad scale would reach
                        // the sums as 0 * NaN): logits of -inf. (Of the batch eight before all is read: K's stage was
                        // waited for above, which four tiles, so at most four batches, back was free.)
                        const bool seen = v >= 0 && p.tb0 + (t + (lane >> 3)) * kTile + 16 * (lane & 7) + 15 >= p.kv_begin;
                        scales[((batch & (kScaleSlots - 1)) * kBatch + (lane >> 3)) * kGroups + (lane & 7)] =
                            seen ? make_float4(ks * scale_log2, lg2_approx(vs), __frcp_rn(vs), 0.f) : make_float4(0.f, -INFINITY, 1.f, 0.f);
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(bar(S::kScFull, batch & (kScaleSlots - 1)));
                        ++batch;
                    }
                } else {
                    const int stage = it & 1;
                    if (it > 1)
                        wait_warp(bar(S::kCEmpty, stage), ((it >> 1) - 1) & 1);
                    if (ok && lane < pages) {
                        mbar_arrive_expect_tx(bar(S::kCFull, stage), rows_in * D);
                        tma_load_3d(base + S::kCodes + stage * S::kTileBytes + at, &v_map, 0, y, z, bar(S::kCFull, stage));
                    }
                }
                if (!ok)
                    break;
            }
            if (!ok)
                break;
        }
        // no copy outlives the block, also where a wait gave up (`it`: tiles issued)
        const uint32_t depth = keys ? kKStages : 2;
        for (uint32_t x = it > depth ? it - depth : 0; x < it; ++x) {
            const uint32_t b = keys ? bar(S::kKFull, x & (kKStages - 1)) : bar(S::kCFull, x & 1);
            if (!mbar_wait(b, x / depth & 1) && lane == 0)
                atomicOr(&g_kv8_rows_error, 2);
        }
    } else {
        // ---------------------------------------------------------------- the products
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint64_t q_hi = desc(base + S::kQ, 128, S::kQAtoms), q_lo = desc(base + S::kQ + S::kQBytes, 128, S::kQAtoms);
        uint32_t unit = 0;
        for (; ok && next_piece(a, walk, p); ++unit) {
            const int n = p.t1 - p.t0;
            const uint32_t idesc_s = idesc(128, p.columns, 0, 0, 0, 0), idesc_o = idesc(D, p.columns, 0, 0, 1, 1);
            const auto scores = [&](uint32_t x) { // of the x-th tile
                const int stage = x & (kKStages - 1);
                if (!wait_warp(bar(S::kKFull, stage), x / kKStages & 1) ||
                    (x > 1 && !wait_warp(bar(S::kSEmpty, x & 1), ((x >> 1) - 1) & 1)))
                    return false;
                fence_after_sync();
                const uint32_t k_s = base + S::kK + stage * S::kTileBytes;
                const uint64_t k_d = D == 128 ? desc_sw128(k_s, 16, 1024) : desc_sw64(k_s, 16, 512);
                const uint32_t dst = tm + (x & 1) * R;
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < D / 32; ++kk) // 32 columns: 32 bytes of a row of K, two core matrices of Q
                        mma_f8(dst, k_d + kk * 2, q_hi + kk * 16, idesc_s, kk > 0);
#pragma unroll
                    for (int kk = 0; kk < D / 32; ++kk)
                        mma_f8(dst, k_d + kk * 2, q_lo + kk * 16, idesc_s, 1);
                    commit(bar(S::kSFull, x & 1));
                    commit(bar(S::kKEmpty, stage));
                }
                __syncwarp();
                return true;
            };
            bool go = wait_warp(bar(S::kQFull, 0), unit & 1);
            fence_after_sync();
            go = go && scores(it) && (n == 1 || scores(it + 1));
            for (int j = 0; go && j < n; ++j) {
                const uint32_t x = it + j;
                const int stage = x & 1, phase = x >> 1 & 1;
                if (!wait_warp(bar(S::kPFull, stage), phase) || !wait_warp(bar(S::kVFull, stage), phase) ||
                    (j == 0 && unit > 0 && !wait_warp(bar(S::kOFree, 0), (unit - 1) & 1)))
                    break;
                fence_after_sync();
                const uint64_t v_d = desc(base + S::kV + stage * S::kVBytes, S::kVAtoms, 128);
                const uint64_t p_d = desc(base + S::kP + stage * S::kPBytes, S::kPAtoms, 128);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < kTile / 16; ++kk) // 16 positions: two atoms of V and of P
                        mma_f16(tm + S::kO, v_d + (uint64_t)(kk * 2 * S::kVAtoms / 16), p_d + (uint64_t)(kk * 2 * S::kPAtoms / 16),
                                idesc_o, j > 0 || kk > 0);
                    commit(bar(S::kDone, stage));
                }
                __syncwarp();
                if (j + 2 < n && !scores(x + 2))
                    break;
            }
            it += n;
        }
        if (!ok) { // what was issued ends before its memory is given back
            if (elect_one())
                commit(bar(S::kDrained, 0));
            if (!mbar_wait(bar(S::kDrained, 0), 0) && lane == 0)
                atomicOr(&g_kv8_rows_error, 2);
        }
    }
    __syncwarp();
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (warp == kMma)
        dealloc(tmem, S::kTmem);
}

// Joins the partial sums of the units that several CTAs share: a warp to a row, D / 32 columns to a lane.
constexpr int kJoinWarps = 8;
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) kv8_rows_join_kernel(const Kv8AttnArgs a, const Part part)
{
    constexpr int kD = D / 32;
    grid_wait();
    const int lane = threadIdx.x & 31, c0 = blockIdx.x, r = blockIdx.y * kJoinWarps + (threadIdx.x >> 5);
    const int4 u = part.dir[c0];
    if (u.x <= c0)
        return;
    const Request rq = request(a, u.y);
    const int h = u.z % a.H_kv, row0 = u.z / a.H_kv * R;
    if (r >= min(R, rq.qlen * a.G - row0))
        return;
    const auto slot = [&](int c) { return (2 * (int64_t)c + (c == c0)) * R + r; };
    float m = -INFINITY, l = 0.f;
    for (int c = c0 + lane; c <= u.x; c += 32)
        m = fmaxf(m, part.ml[slot(c)].x);
    m = warp_max(m);
    float acc[kD];
#pragma unroll
    for (int i = 0; i < kD; ++i)
        acc[i] = 0.f;
#pragma unroll 4
    for (int c = c0; c <= u.x; ++c) {
        const float2 ml = part.ml[slot(c)];
        // one that saw nothing has m = -inf; its sums are 0, or NaN from a NaN logit
        const float f = ml.x == -INFINITY ? 1.f : ex2_approx(ml.x - m);
        l += ml.y * f;
        const float *src = part.o + slot(c) * D + lane * kD;
        if (D == 128) {
            const float4 v = *reinterpret_cast<const float4 *>(src);
            acc[0] += v.x * f;
            acc[1] += v.y * f;
            acc[kD - 2] += v.z * f;
            acc[kD - 1] += v.w * f;
        } else {
            const float2 v = *reinterpret_cast<const float2 *>(src);
            acc[0] += v.x * f;
            acc[1] += v.y * f;
        }
    }
    const int64_t t = rq.q0 + (row0 + r) / a.G;
    const int head = h * a.G + (row0 + r) % a.G;
    float lse;
    const float f = finish_row(m, l, a.sinks, head, &lse);
    __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.out) + (t * a.H + head) * D + lane * kD;
#pragma unroll
    for (int i = 0; i < kD; i += 2)
        *reinterpret_cast<uint32_t *>(dst + i) = pack_bf16x2(acc[i] * f, acc[i + 1] * f);
    if (a.lse && lane == 0)
        a.lse[t * a.H + head] = lse;
}

// The most work that there can be decides the CTAs: one without a part ends at once, but not for nothing.
int grid_of(const Kv8AttnArgs &a, int sm_count)
{
    const double units = ((double)a.T * a.G / R + a.B) * a.H_kv; // each request's last chunk may be short
    const double most = units * ((double)((int64_t)a.table_width << a.block_shift) / kTile + 1 + kUnitCost);
    return (int)std::min((double)std::max(sm_count, 1), most / kMinPart + 1);
}

struct Sizes {
    size_t ml, o, total;
};

Sizes sizes(int D, size_t blocks)
{
    Sizes s;
    s.ml = up256(blocks * sizeof(int4));
    s.o = up256(s.ml + 2 * blocks * R * sizeof(float2));
    s.total = s.o + 2 * blocks * R * D * sizeof(float);
    return s;
}

template <int D>
cudaError_t launch(const Kv8AttnArgs &a, void *workspace, int sm_count, cudaStream_t stream)
{
    const int grid = grid_of(a, sm_count);
    const Sizes sz = sizes(D, grid);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const Part part{reinterpret_cast<int4 *>(ws), reinterpret_cast<float2 *>(ws + sz.ml), reinterpret_cast<float *>(ws + sz.o)};
    cudaError_t e = cudaFuncSetAttribute(kv8_rows_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<D>::kSmem);
    if (e != cudaSuccess)
        return e;
    CUtensorMap maps[2];
    if (!kv8_tensor_maps(a, D, kTile, maps))
        return cudaErrorInvalidValue;
    kv8_rows_kernel<D><<<grid, kThreads, Shape<D>::kSmem, stream>>>(maps[0], maps[1], a, part);
    if ((e = cudaGetLastError()) != cudaSuccess)
        return e;
    if (grid == 1)
        return cudaSuccess; // (every unit is whole)
    // behind it, its start overlapped (it waits for the first kernel's end)
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, R / kJoinWarps);
    cfg.blockDim = dim3(kJoinWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv8_rows_join_kernel<D>, a, part);
}

} // namespace

size_t kv8_rows_workspace(int D, int sm_count) { return sizes(D, std::max(sm_count, 1)).total; }

cudaError_t launch_kv8_rows(const Kv8AttnArgs &a, int D, void *workspace, int sm_count, cudaStream_t stream)
{
    return D == 128 ? launch<128>(a, workspace, sm_count, stream) : launch<64>(a, workspace, sm_count, stream);
}

cudaError_t read_kv8_rows_error(int *out, bool reset)
{
    cudaError_t e = cudaMemcpyFromSymbol(out, g_kv8_rows_error, sizeof(int));
    if (e == cudaSuccess && reset) {
        const int zero = 0;
        e = cudaMemcpyToSymbol(g_kv8_rows_error, &zero, sizeof(int));
    }
    return e;
}

} // namespace smla

// Attention over the block-scaled 8-bit cache for many query rows (prompts and
// chunks of prompts, sm_103a): 128 query rows to a row tile, both products on the
// tensor cores (tcgen05), scores and sums in tensor memory.
//
// A unit of work is up to 128 or 256 rows (token, head of the kv head's group) of
// one request and kv head. A CTA walks over its visible positions in tiles of 64.
// Scores have two buffers in tensor memory for each row tile: while a tile's softmax
// runs, the next one's scores are computed. Where a request's rows may fill more than
// one row tile, a CTA has two and an SM one CTA: the row tiles share the copies of K
// and V and V's expansion. With fewer rows a CTA has one and an SM two CTAs, so that
// the tensor cores have the other's products meanwhile (with 40 rows to a request
// the second row tile would have nothing). Warps of a CTA with NR row tiles:
//   4 NR   softmax, a row to a thread; Q before and the epilogue behind it
//   2 NR   V's codes, expanded to binary16
//   NR     the blocks' codes by TMA as they lie in the cache (K and V by a warp each
//          with two row tiles), the blocks' scales
//   NR     the tensor-core products of a row tile each
// The CTAs stay and take unit after unit; a kernel before lays out the work (see
// Plan), one behind joins the units that several CTAs shared.
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
// denominator adds p' / vs. A row's reference m is set so that the largest p' of the
// first tile that it sees is 2^5. The weights of a tile are taken without looking for
// its maximum; their sum (at most 65504, so that each is inside binary16) says whether
// m must move, and only then, which is seldom, the tile is gone through again and what
// was added up so far is rescaled. Binary16 holds p' to 2^-11 of itself down to 2^-14,
// 2^-19 of the largest: with the largest at 1 the values of blocks whose scale is 2^-16
// of another's, which may hold nothing of its size, lost bits. A larger first weight
// leaves the sums less to grow: a prompt of 8192 tokens takes 440 us with 2^0 or 2^5,
// 444 with 2^6, 448 with 2^7.
//
// Shared memory: the codes in TMA's swizzled rows; Q and the expanded V in 8-row
// x 16-byte core matrices, written so that eight lanes fill one (no bank
// conflict). Blocks outside the pool are zero-filled and not read.
//
// Bound and measured. A prompt of 8192 tokens, 32 heads on 8 kv heads of 128
// columns: 0.442 ms, 1.24 PFLOP/s (65% of the measured bf16 rate; the products alone
// keep the tensor pipe busy for 55% of it, S being bound by what its operands
// take from shared memory: 49 cycles for 64 columns against 32). Six chunks of 45 to
// 701 tokens behind 2114 to 32001 positions, 16 heads on 2 kv heads of 64 columns,
// blocks of 16: 238 us, 0.76 PFLOP/s; there a tile has half the products for the same
// softmax, whose instructions (some 300 a tile and warp, with four exponentials a
// cycle of a sub-core) take over half of the issue slots. What counted on the way:
// short loops (eight to sixteen warps run five different pieces of code, and what is
// not in the instruction cache costs some 12 cycles an instruction); products issued
// under uniform control; the table and scales read and handed over eight tiles at a
// time; K and V copied by a warp each; whole rows of Q and out to an access.
#include "smla_kv8.cuh"
#include "smla_umma.cuh"

#include <algorithm>
#include <climits>

namespace smla {

__device__ int g_kv8_error = 0; // 1: a bounded wait gave up; 2: products in flight did not drain

namespace {

using namespace kv8;
using namespace umma;

constexpr int kRows = 128;  // of a row tile
constexpr int kTile = 64;
constexpr float kTop = 5.0f;     // (log2) the largest weight where the reference is set
constexpr float kSlack = 9.9f;  // (log2) the largest weight that does not move it, when it is looked at
constexpr float kMostSum = 65504.0f; // of 64 weights that are not looked at: 64 of 2^kSlack stay below
constexpr int kPieceCost = 13; // a unit's start and end, in tiles (measured: 14000 to 19000 cycles, a tile 1450 to 1550)
constexpr int kMinPart = 22;  // a CTA's part of the work, in tiles, before more CTAs share it

// The CTA's place in the work, and what else its warps share.
struct Misc {
    long long at, hi, total; // cost: where it is, where its part ends, all
    long long base;          // without a plan: before the request `item`,
    int q0, qlen, len;       // that request,
    int tiles, count;        // and its units
    int item, parts;
    int units, next;         // units taken whole (0: the work is cut into parts), the next one
    uint32_t tmem;
    int any_nan;
};

template <int D, int NR> struct Shape {
    static constexpr int kItemRows = NR * kRows;
    static constexpr int kVWarps = 2 * NR;
    static constexpr int kV0 = 4 * NR, kLoader = kV0 + kVWarps, kMma = kLoader + NR; // the roles' first warps
    static constexpr int kThreads = (kMma + NR) * 32;
    static constexpr int kQBytes = kRows * D;       // one part of a row tile's Q
    static constexpr int kTileBytes = kTile * D;    // one tile of codes
    static constexpr int kVBytes = kTile * D * 2;   // a tile of V in binary16
    static constexpr int kQAtoms = D / 16 * 128;    // 8 rows of Q: D / 16 core matrices
    static constexpr int kVAtoms = D / 8 * 128;     // 8 rows of V
    static constexpr int kKStages = 2 * NR;         // of two tiles (a power of two)
    static constexpr int kK = 0;
    static constexpr int kCodes = 2 * kKStages * kTileBytes; // V as it comes, two stages
    static constexpr int kQ = kCodes + 2 * kTileBytes; // of each row tile: hi, lo
    static constexpr int kV = kQ + NR * 2 * kQBytes; // two stages
    static constexpr int kScales = kV + 2 * kVBytes; // 2 stages x 8 tiles x {c, log2 vs, 1 / vs} x 4 groups
    static constexpr int kBars = kScales + 2 * 8 * 4 * 12;
    // K landed / free (each stage); V's codes landed / free (two stages); scales of eight tiles written (two stages);
    // drained (each row tile); Q written; of each row tile, two stages: scores ready, P and V ready, values done
    static constexpr int kKFull = 0, kKEmpty = kKFull + kKStages, kCFull = kKEmpty + kKStages, kCEmpty = kCFull + 2,
                         kScFull = kCEmpty + 2, kDrained = kScFull + 2, kQFull = kDrained + NR, kSFull = kQFull + 1,
                         kPFull = kSFull + 2 * NR, kVEmpty = kPFull + 2 * NR, kBarriers = kVEmpty + 2 * NR;
    static_assert(kBarriers <= 32, "a lane sets each up");
    static constexpr int kMisc = kBars + (kBarriers + 1) / 2 * 16;
    static constexpr int kSmem = kMisc + (int)sizeof(Misc);
    static constexpr uint32_t kTmem = 256;          // of a row tile: two S (P over each one's first half) and O
    static constexpr uint32_t kO = 2 * kTile;
    static constexpr uint32_t kIdescS = idesc(128, kTile, 0, 0, 0, 0);
    static constexpr uint32_t kIdescO = idesc(128, D, 0, 0, 0, 1);
    static_assert(NR == 2 || 2 * (kSmem + 1024) <= 228 * 1024, "two CTAs to an SM");
};

// The plan of a call, in the workspace. A unit is an item's kv head. Where the
// longest unit is at most a third of a CTA's share, the CTAs take whole units, the
// longest first, as they are free (a prompt of 8192 tokens with 8 kv heads: 440 us,
// cut into equal parts 460); otherwise the units laid end to end are cut into equal
// parts, one for each CTA, wherever in a unit that falls (ragged chunks: 236 us, in
// pieces of at most half of a share, the longest first, 276).
struct PlannedItem {
    int b, chunk, tiles, none;
    int q0, qlen, len, none2; // the request
};
struct Plan {
    int *head;       // units taken whole (0: cut); how many are taken
    long long *cost; // [items + 1]: of the items before, for one kv head, in tiles
    PlannedItem *items;
    int *order;      // [items]: the longest first
    int4 *dir;       // [CTAs]: the unit that it begins and others end, {last CTA (-1: none), request, chunk, head}
    float2 *ml; // [2 CTAs][item_rows]
    float *o;   // [2 CTAs][item_rows][D]
    int n_items, item_rows;
};

// Drafted trees of few requests go without that kernel and its launch: all rows of a request see the same tiles, so
// the CTAs find their parts by the requests alone (as the streaming kernel does), where units are too few to be taken
// whole (`items` is NULL). 16 requests of 8192 positions with 16 nodes 75.6 us, planned 79.5; one of 509 with 8 17.8 and
// 19.6.

// The units of a request with drafted trees and the cost of each.
struct Units {
    int tiles, count, cost;
    __device__ long long all() const { return (long long)count * cost; }
};

// A tile's item: request, chunk of rows, kv head.
struct Item {
    int b, chunk, h;
};

// Items are numbered request by request; request b's first number is
// floor(q0 G / item_rows) + b, which leaves room for its ceil(rows / item_rows)
// chunks without a running sum. Returns false for a number that no chunk has.
__device__ __forceinline__ bool find_item(const Kv8AttnArgs &a, int item_rows, int n, Item *it)
{
    int lo = 0, hi = a.B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        const int q0 = min(max(a.query_start[mid], 0), a.T);
        if ((int)((long long)q0 * a.G / item_rows) + mid <= n)
            lo = mid;
        else
            hi = mid - 1;
    }
    const Request r = request(a, lo);
    it->b = lo;
    it->chunk = n - ((int)((long long)r.q0 * a.G / item_rows) + lo);
    return it->chunk >= 0 && (long long)it->chunk * item_rows < (long long)r.qlen * a.G;
}

// What an item's rows see.
struct Span {
    int row0, rows, p_first, p_last;
    int kv_begin, kv_end; // beyond: seen by none
    int all_from;         // [all_from, p_first]: seen by all
    int tb0, tiles;       // tiles of kTile positions from tb0 on (a multiple of kTile: blocks lie whole in the tiles)
};

__device__ __forceinline__ Span span_of(const Kv8AttnArgs &a, int item_rows, const Request &rq, int chunk)
{
    Span s;
    s.row0 = chunk * item_rows;
    s.rows = min(item_rows, rq.qlen * a.G - s.row0);
    const bool tree = a.tree_mask != nullptr; // the context's positions are seen by all rows, those behind by some
    s.p_first = tree ? rq.pos(-1) : rq.pos(s.row0 / a.G);
    s.p_last = tree ? rq.len - 1 : rq.pos((s.row0 + s.rows - 1) / a.G);
    s.kv_end = min(rq.len, s.p_last + 1);
    s.kv_begin = a.window > 0 ? max(0, s.p_first - a.window + (tree ? 2 : 1)) : 0;
    s.all_from = a.window > 0 ? s.p_last - a.window + 1 : 0;
    s.tb0 = s.kv_begin & ~(kTile - 1);
    s.tiles = s.kv_end > s.tb0 ? (s.kv_end - s.tb0 + kTile - 1) / kTile : 0;
    return s;
}

__device__ __forceinline__ Units units_of(const Kv8AttnArgs &a, int item_rows, const Request &rq)
{
    Units u;
    u.tiles = rq.qlen > 0 ? span_of(a, item_rows, rq, 0).tiles : 0;
    u.count = (int)(((long long)rq.qlen * a.G + item_rows - 1) / item_rows * a.H_kv); // (checked on the host)
    u.cost = max(1, u.tiles) + kPieceCost;
    return u;
}

// This CTA's part of the work without a plan, by the whole block: each thread adds up its requests, the block scans the
// sums, and the thread whose requests hold the part's begin finds the request. `sums`: two words to a warp, free by now.
template <int kThreads>
__device__ __forceinline__ void find_part(const Kv8AttnArgs &a, int item_rows, bool fits, Misc *misc, long long *sums)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.B + kThreads - 1) / kThreads;
    long long cost = 0;
    int count = 0; // (fewer than three to a CTA)
    for (int i = 0; i < per; ++i) {
        const int b = tid * per + i;
        if (b < a.B) {
            const Units u = units_of(a, item_rows, request(a, b));
            cost += u.all();
            count += u.count;
        }
    }
    long long to = cost; // inclusive
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, to, d);
        to += lane >= d ? x : 0;
    }
    count = __reduce_add_sync(0xffffffffu, count);
    if (lane == 31) {
        sums[2 * warp] = to;
        sums[2 * warp + 1] = count;
    }
    if (tid == 0)
        misc->at = misc->hi = 0;
    __syncthreads();
    long long total = 0, before = to - cost, units = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        before += w < warp ? sums[2 * w] : 0;
        total += sums[2 * w];
        units += sums[2 * w + 1];
    }
    // (at least a CTA to a unit: eight units of one tile 16 us, in five parts 20)
    const int parts = (int)min((long long)gridDim.x, max(max(1ll, units), (total + kMinPart - 1) / kMinPart));
    if (fits && (int)blockIdx.x < parts) {
        const long long lo = total * blockIdx.x / parts, hi = total * (blockIdx.x + 1) / parts;
        if (lo < hi && lo >= before && lo < before + cost) {
            int b = tid * per;
            Request rq = request(a, b);
            Units u = units_of(a, item_rows, rq);
            while (lo >= before + u.all()) {
                before += u.all();
                rq = request(a, ++b);
                u = units_of(a, item_rows, rq);
            }
            misc->at = lo;
            misc->hi = hi;
            misc->base = before;
            misc->q0 = rq.q0;
            misc->qlen = rq.qlen;
            misc->len = rq.len;
            misc->tiles = u.tiles;
            misc->count = u.count;
            misc->item = b;
            misc->total = total;
            misc->parts = parts;
        }
    }
}

// Plans a call, by one block. Where a unit stands in the order, and which CTA takes
// it, does not change what is computed from it.
constexpr int kPlanThreads = 1024;
__global__ void __launch_bounds__(kPlanThreads) kv8_tile_plan_kernel(const Kv8AttnArgs a, const Plan plan, int ctas)
{
    __shared__ long long s_warp[kPlanThreads / 32];
    __shared__ int s_most, s_real, s_class[64];
    grid_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid < 64)
        s_class[tid] = 0;
    if (tid == 0)
        s_most = s_real = 0;
    __syncthreads();
    long long before = 0;
    for (int n0 = 0; n0 < plan.n_items; n0 += kPlanThreads) {
        const int n = n0 + tid;
        Item it;
        long long cost = 0;
        if (n < plan.n_items && find_item(a, plan.item_rows, n, &it)) {
            const Request rq = request(a, it.b);
            const int tiles = span_of(a, plan.item_rows, rq, it.chunk).tiles;
            cost = max(1, tiles) + kPieceCost;
            plan.items[n] = PlannedItem{it.b, it.chunk, tiles, 0, rq.q0, rq.qlen, rq.len, 0};
        }
        long long to = cost;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, to, d);
            to += lane >= d ? x : 0;
        }
        if (lane == 31)
            s_warp[warp] = to;
        __syncthreads();
        long long all = 0;
        for (int w = 0; w < kPlanThreads / 32; ++w) {
            const long long x = s_warp[w];
            to += w < warp ? x : 0;
            all += x;
        }
        if (n < plan.n_items)
            plan.cost[n] = before + to - cost;
        const int most = __reduce_max_sync(0xffffffffu, (int)cost), real = __popc(__ballot_sync(0xffffffffu, cost > 0));
        if (lane == 0 && real > 0) {
            atomicMax(&s_most, most);
            atomicAdd(&s_real, real);
        }
        before += all;
        __syncthreads();
    }
    const int most = s_most;
    const bool whole = 3ll * most * ctas <= before * a.H_kv && (long long)s_real * a.H_kv < INT_MAX / 2;
    if (tid == 0) {
        plan.cost[plan.n_items] = before;
        plan.head[0] = whole ? s_real * a.H_kv : 0;
        plan.head[1] = 0;
    }
    if (!whole)
        return;
    // sorted by length, in 64 classes (a thread reads what it wrote)
    const auto class_of = [&](int n) {
        const int tiles = plan.items[n].tiles;
        return 63 - (int)((max(1, tiles) + kPieceCost) * 63ll / most);
    };
    const auto real = [&](int n) {
        Item it;
        return find_item(a, plan.item_rows, n, &it);
    };
    for (int n = tid; n < plan.n_items; n += kPlanThreads)
        if (real(n))
            atomicAdd(&s_class[class_of(n)], 1);
    __syncthreads();
    if (tid < 32) { // the classes' first places
        const int x0 = s_class[2 * lane], x1 = s_class[2 * lane + 1];
        int to = x0 + x1;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, to, d);
            to += lane >= d ? y : 0;
        }
        s_class[2 * lane] = to - x0 - x1;
        s_class[2 * lane + 1] = to - x1;
    }
    __syncthreads();
    for (int n = tid; n < plan.n_items; n += kPlanThreads)
        if (real(n))
            plan.order[atomicAdd(&s_class[class_of(n)], 1)] = n;
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
// Waits for this thread's tensor-memory loads; x holds what they brought only after it.
__device__ __forceinline__ void wait_ld32(uint32_t (&x)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;\n"
                 : "+r"(x[0]), "+r"(x[1]), "+r"(x[2]), "+r"(x[3]), "+r"(x[4]), "+r"(x[5]), "+r"(x[6]), "+r"(x[7]),
                   "+r"(x[8]), "+r"(x[9]), "+r"(x[10]), "+r"(x[11]), "+r"(x[12]), "+r"(x[13]), "+r"(x[14]), "+r"(x[15]),
                   "+r"(x[16]), "+r"(x[17]), "+r"(x[18]), "+r"(x[19]), "+r"(x[20]), "+r"(x[21]), "+r"(x[22]), "+r"(x[23]),
                   "+r"(x[24]), "+r"(x[25]), "+r"(x[26]), "+r"(x[27])::"memory");
    asm volatile("" : "+r"(x[28]), "+r"(x[29]), "+r"(x[30]), "+r"(x[31])::"memory");
}

__device__ __forceinline__ void wait_ld16(uint32_t (&x)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;\n"
                 : "+r"(x[0]), "+r"(x[1]), "+r"(x[2]), "+r"(x[3]), "+r"(x[4]), "+r"(x[5]), "+r"(x[6]), "+r"(x[7]),
                   "+r"(x[8]), "+r"(x[9]), "+r"(x[10]), "+r"(x[11]), "+r"(x[12]), "+r"(x[13]), "+r"(x[14]), "+r"(x[15])::"memory");
}

// What the rows of a tile see of 32 positions.
template <bool kTree> struct Sight;
template <> struct Sight<false> {
    int p_first, all_from; // the tile's: see Span
    int pos, pos_lo;       // this row: pos_lo <= t <= pos
    __device__ __forceinline__ Sight(const Kv8AttnArgs &a, const Span &sp, const Request &rq, int r)
        : p_first(sp.p_first), all_from(sp.all_from), pos(r < sp.rows ? rq.pos((sp.row0 + r) / a.G) : -1),
          pos_lo(a.window > 0 ? pos - a.window + 1 : 0)
    {
    }
    __device__ bool all(int t) const { return t + 31 <= p_first && t >= all_from; }
    __device__ bool sees(int t) const { return t <= pos && t >= pos_lo; }
    __device__ int first() const { return pos_lo; }
    __device__ int last() const { return pos; }
};
template <> struct Sight<true> {
    int p_first, all_from;
    TreeRow row;
    __device__ __forceinline__ Sight(const Kv8AttnArgs &a, const Span &sp, const Request &rq, int r)
        : p_first(sp.p_first), all_from(sp.all_from), row(a, rq, rq.q0 + (sp.row0 + r) / a.G, r < sp.rows)
    {
    }
    __device__ bool all(int t) const { return t + 31 <= p_first && t >= all_from; }
    __device__ bool sees(int t) const { return row.sees(t); }
    __device__ int first() const { return max(row.lo, 0); }
    __device__ int last() const { return row.len - 1; }
};

// A row's running sums.
struct Row {
    float m, l; // reference (log2 units), denominator relative to it
};

// The factors of a tile's 4 groups of 16 positions: of their logits, log2 of
// their value scales, and its inverse.
struct Factors {
    float k[4], vs[4], iv[4];
    __device__ __forceinline__ Factors(const float *sc, float qs)
    {
        const float4 f = *reinterpret_cast<const float4 *>(sc), v = *reinterpret_cast<const float4 *>(sc + 4),
                     w = *reinterpret_cast<const float4 *>(sc + 8);
        k[0] = f.x * qs, k[1] = f.y * qs, k[2] = f.z * qs, k[3] = f.w * qs;
        vs[0] = v.x, vs[1] = v.y, vs[2] = v.z, vs[3] = v.w;
        iv[0] = w.x, iv[1] = w.y, iv[2] = w.z, iv[3] = w.w;
    }
};

// Sixteen logits relative to the reference become weights in binary16; their sum.
__device__ __forceinline__ float weigh(const uint32_t *x, uint32_t *p)
{
    uint64_t sum = 0;
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
        const float p0 = ex2_approx(__uint_as_float(x[i])), p1 = ex2_approx(__uint_as_float(x[i + 1]));
        sum = add2(sum, pair(p0, p1));
        p[i / 2] = pack_f16x2(p0, p1);
    }
    float s0, s1;
    unpair(sum, s0, s1);
    return s0 + s1;
}

// One row's 64 scores (the thread's lane of tensor memory at my) become weights
// 2^(s + log2(vs) - m) in binary16, over the scores they come from; their sum,
// each group's divided by vs, joins l. False where the reference may have to move
// (the sum passes what binary16 holds, so a weight may) for some row of
// the warp: then nothing is changed. For tiles that all rows see.
__device__ __forceinline__ bool row_tile(uint32_t my, const float *sc, float qs, Row &row)
{
    uint32_t x[64];
    ld32(my, *reinterpret_cast<uint32_t(*)[32]>(x));
    ld32(my + 32, *reinterpret_cast<uint32_t(*)[32]>(x + 32));
    const Factors f(sc, qs);
    wait_ld32(*reinterpret_cast<uint32_t(*)[32]>(x));
    wait_ld32(*reinterpret_cast<uint32_t(*)[32]>(x + 32));
    uint32_t p[32];
    float l = row.l, all = 0.f;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const float b = f.vs[c] - row.m;
#pragma unroll
        for (int i = c * 16; i < c * 16 + 16; i += 2) {
            float e0, e1;
            unpair(fma2(pair(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), pair(f.k[c], f.k[c]), pair(b, b)), e0, e1);
            x[i] = __float_as_uint(e0);
            x[i + 1] = __float_as_uint(e1);
        }
        const float s = weigh(x + c * 16, p + c * 8);
        all += s;
        l = fmaf(s, f.iv[c], l);
    }
    // beyond 2^20 the rounding of m alone could pass any bound of the weights
    if (__any_sync(0xffffffffu, all > kMostSum || !(fabsf(row.m) <= 0x1p20f)))
        return false;
    row.l = l;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        st16(my + 16 * i, *reinterpret_cast<uint32_t(*)[16]>(p + 16 * i));
    return true;
}

// Sixteen of the row's logits, -inf where it does not see the position.
template <bool kTree>
__device__ __forceinline__ void logits(uint32_t my, const float *sc, float qs, int t0, const Sight<kTree> &see, int c,
                                       uint32_t (&x)[16])
{
    ld16(my + c * 16, x);
    const float k = sc[c] * qs, vs = sc[4 + c];
    const int t = t0 + c * 16;
    uint32_t bits = 0;
    if constexpr (kTree)
        bits = see.row.sees16(t);
    wait_ld16(x);
#pragma unroll
    for (int i = 0; i < 16; ++i)
        x[i] = __float_as_uint((kTree ? bits >> i & 1 : see.sees(t + i)) ? fmaf(__uint_as_float(x[i]), k, vs) : -INFINITY);
}

// The largest of the row's 64 logits that it sees.
template <bool kTree>
__device__ __forceinline__ float largest(uint32_t my, const float *sc, float qs, int t0, const Sight<kTree> &see)
{
    float top = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
        uint32_t x[16];
        logits(my, sc, qs, t0, see, c, x);
#pragma unroll
        for (int i = 0; i < 16; ++i)
            top = fmaxf(top, __uint_as_float(x[i])); // (a NaN loses)
    }
    return top;
}

// The next two run seldom, so they are short loops: code that is not in the
// instruction cache costs some 12 cycles an instruction.

// The reference of a row whose largest logit is `top` (rounded up, so that far out,
// where kTop is less than the logits' step, no weight passes 1).
__device__ __forceinline__ float reference(float top) { return __fadd_ru(top, -kTop); }

// The row's first reference.
template <bool kTree>
__device__ __noinline__ float row_first(uint32_t my, const float *sc, float qs, int t0, const Sight<kTree> see)
{
    if (!see.all(t0) || !see.all(t0 + 32))
        return reference(largest(my, sc, qs, t0, see));
    float top = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
        uint32_t x[16];
        ld16(my + c * 16, x);
        const float k = sc[c] * qs, vs = sc[4 + c];
        wait_ld16(x);
#pragma unroll
        for (int i = 0; i < 16; ++i)
            top = fmaxf(top, fmaf(__uint_as_float(x[i]), k, vs));
    }
    return reference(top);
}

// row_tile for any tile and any reference: the reference moves where a weight passes
// 2^kSlack (to 2^kTop), and what was added up is rescaled (O is at
// rest; o_cols: its columns, 0 before the first product); positions that the row
// does not see are left out; the difference is taken from the rounded logit, as the
// reference is.
template <bool kTree>
__device__ __noinline__ Row row_tile_moving(uint32_t my, uint32_t my_o, int o_cols, const float *sc, float qs, Row row, int t0,
                                            const Sight<kTree> see)
{
    const float top = largest(my, sc, qs, t0, see);
    const bool raise = row.m == -INFINITY ? top > -INFINITY : top - row.m > kSlack;
    if (__any_sync(0xffffffffu, raise)) {
        const float ref = reference(top);
        const float g = raise ? (row.m == -INFINITY ? 0.f : ex2_approx(row.m - ref)) : 1.f;
        row.m = raise ? ref : row.m;
        row.l *= g;
#pragma unroll 1
        for (int o = 0; o < o_cols; o += 16) {
            uint32_t p[16];
            ld16(my_o + o, p);
            wait_ld16(p);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                p[i] = __float_as_uint(__uint_as_float(p[i]) * g);
            st16(my_o + o, p);
        }
    }
    const float ref = row.m == -INFINITY ? 0.f : row.m;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) { // (the weights lie over scores of groups before)
        uint32_t x[16], p[8];
        logits(my, sc, qs, t0, see, c, x);
#pragma unroll
        for (int i = 0; i < 16; ++i)
            x[i] = __float_as_uint(__uint_as_float(x[i]) - ref);
        row.l = fmaf(weigh(x, p), sc[8 + c], row.l);
        st8(my + c * 8, p);
    }
    return row;
}

// V's codes of a position in a tile that not every row sees whole: nothing where
// no row sees it (the block holds anything there); and a NaN code that some rows
// see and others do not must not reach the others through 0 * NaN: it is taken
// out, and the rows that see it look for it at their end.
__device__ __noinline__ void visible_codes(uint32_t (&w)[4], bool in, bool many, int *any_nan)
{
#pragma unroll
    for (int y = 0; y < 4; ++y) {
        w[y] = in ? w[y] : 0;
        const uint32_t bad = many ? nan_bytes(w[y]) : 0;
        if (bad) {
            *any_nan = 1;
            w[y] &= ~((bad >> 7) * 0xFFu);
        }
    }
}

// Which of the 32 value columns from 32 c on hold a NaN code at a position that
// the row sees, in the tiles where some rows see positions that others do not
// (there the codes were taken out, so that 0 * NaN does not reach the others).
template <int D, bool kTree>
__device__ __noinline__ uint32_t nan_columns(const Kv8AttnArgs &a, const Item &it, const Sight<kTree> &see, int tb0, int t_begin,
                                             int n, int c)
{
    uint32_t bits = 0;
    for (int t = max(see.first(), tb0 + t_begin * kTile); t <= see.last() && t < tb0 + (t_begin + n) * kTile; ++t) {
        const int tile = t & ~(kTile - 1); // (tb0 is a multiple of it)
        if ((tile + kTile - 1 <= see.p_first && tile >= see.all_from) || (kTree && !see.sees(t)))
            continue;
        const int e = t >> a.block_shift;
        const int v = e < a.table_width ? a.block_table[it.b * a.table_stride + e] : -1;
        if (v < 0 || v >= a.num_blocks)
            continue;
        const uint8_t *row = a.v_cache + ((((int64_t)v * a.H_kv + it.h) << a.block_shift) + (t & (a.block_size - 1))) * D + c * 32;
        for (int i = 0; i < 32; ++i)
            bits |= (row[i] & 0x7F) == 0x7F ? 1u << i : 0u;
    }
    return bits;
}

// A part of a unit, as much of it as a CTA's part of the work holds.
struct Piece {
    Item it;
    Request rq;
    int t_begin, t_end; // tiles
    bool whole;
    int64_t slot0;      // where the partial sums of its rows go
};

// Works on a piece, by the whole block; false where a wait gave up. The barriers
// were last used for a piece before (not the first time).
template <int D, int NR, bool kTree>
__device__ __forceinline__ bool work_on(const CUtensorMap &k_map, const CUtensorMap &v_map, const Kv8AttnArgs &a, const Plan &plan,
                                        uint8_t *smem, const Piece &piece, bool first)
{
    using S = Shape<D, NR>;
    Misc *misc = reinterpret_cast<Misc *>(smem + S::kMisc);
    int *s_any_nan = &misc->any_nan;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t base = smem_u32(smem), bars = base + S::kBars;
    const uint32_t k_full = bars + 8 * S::kKFull, k_empty = bars + 8 * S::kKEmpty, c_full = bars + 8 * S::kCFull,
                   c_empty = bars + 8 * S::kCEmpty, sc_full = bars + 8 * S::kScFull, drained = bars + 8 * S::kDrained,
                   q_full = bars + 8 * S::kQFull, s_full = bars + 8 * S::kSFull, p_full = bars + 8 * S::kPFull,
                   v_empty = bars + 8 * S::kVEmpty;
    const Item it = piece.it;
    const Request rq = piece.rq;
    const int64_t slot0 = piece.slot0;
    const Span sp = span_of(a, S::kItemRows, rq, it.chunk);
    const int row0 = sp.row0, rows = sp.rows, p_first = sp.p_first, p_last = sp.p_last, kv_begin = sp.kv_begin,
              kv_end = sp.kv_end, all_from = sp.all_from, tb0 = sp.tb0;
    const int t_begin = piece.t_begin, n = piece.t_end - t_begin;
    const bool many = p_first != p_last;
    const int live_tiles = NR == 1 || rows <= kRows ? 1 : 2; // (a row tile without rows does nothing)

    if (n <= 0) { // nothing to see (a whole unit)
        if (tid < rows) {
            const int64_t t = rq.q0 + (row0 + tid) / a.G;
            const int head = it.h * a.G + (row0 + tid) % a.G;
            uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + (t * a.H + head) * D);
            for (int i = 0; i < D / 8; ++i)
                dst[i] = make_uint4(0, 0, 0, 0);
            if (a.lse)
                a.lse[t * a.H + head] = a.sinks ? a.sinks[head] : -INFINITY;
        }
        return true;
    }

    if (tid < S::kBarriers) { // a barrier to a lane
        const int pages = kTile / min(kTile, a.block_size);
        const int count = tid < S::kKEmpty    ? 2 * pages
                          : tid < S::kCFull   ? live_tiles
                          : tid < S::kCEmpty  ? pages
                          : tid < S::kScFull  ? S::kVWarps
                          : tid == S::kQFull  ? live_tiles * kRows
                          : tid < S::kPFull   ? 1
                          : tid < S::kVEmpty  ? kRows + S::kVWarps
                                              : 1;
        if (!first)
            mbar_inval(bars + 8 * tid);
        mbar_init(bars + 8 * tid, count);
        mbar_init_fence();
        if (tid == 0)
            *s_any_nan = 0;
    }
    const float scale_log2 = fabsf(a.scale) * kLog2e; // the sign goes into q

    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = misc->tmem;
    bool ok = true;
    // a bounded wait, by whole warps
    auto wait_warp = [&](uint32_t bar, uint32_t parity) {
        ok = ok && mbar_wait_warp(bar, parity);
        if (!ok && lane == 0)
            atomicOr(&g_kv8_error, 1);
        return ok;
    };

    if (warp < 4 * live_tiles) {
        // ---------------------------------------------------------------- softmax
        const int tile = warp >> 2; // of rows
        // Q in two E4M3 parts; meanwhile the first codes come. Four lanes to a row, eight rows to an access (a row to a
        // lane took 11000 cycles of a 128-column item: 32 cache lines an access).
        const int r = tid;
        float qs = 0.f;
        {
            const uint32_t dst = base + S::kQ + tile * 2 * S::kQBytes + (warp & 3) * 4 * S::kQAtoms + (lane >> 2) * 16 +
                                 (lane >> 1 & 1) * 128 + (lane & 1) * 8;
            const auto load = [&](int g, uint4(&x)[D / 32]) {
                const int rr = warp * 32 + g * 8 + (lane >> 2);
                const bool live = rr < rows;
                const int row = row0 + (live ? rr : 0);
                const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.q) +
                                                                   (int64_t)(rq.q0 + row / a.G) * a.q_st +
                                                                   (int64_t)(it.h * a.G + row % a.G) * a.q_sh) + (lane & 3);
#pragma unroll
                for (int c = 0; c < D / 32; ++c)
                    x[c] = live ? src[4 * c] : make_uint4(0, 0, 0, 0);
            };
            uint4 x[D / 32], next[D / 32];
            load(0, next);
#pragma unroll 1
            for (int g = 0; g < 4; ++g) {
#pragma unroll
                for (int c = 0; c < D / 32; ++c)
                    x[c] = next[c];
                if (g < 3)
                    load(g + 1, next);
                float amax = 0.f;
#pragma unroll
                for (int c = 0; c < D / 32; ++c)
                    amax = fmaxf(amax, amax8(x[c]));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                float up, down;
                split_scale(amax, up, down);
                up = a.scale < 0.f ? -up : up;
                // the row's factor for its own thread
                down = __shfl_sync(0xffffffffu, down, (lane & 7) * 4);
                qs = (lane >> 3) == g ? down : qs;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t hi[2], lo[2];
                    split8(x[c], up, hi, lo);
                    sts64(dst + g * S::kQAtoms + c * 256, hi[0], hi[1]);
                    sts64(dst + g * S::kQAtoms + c * 256 + S::kQBytes, lo[0], lo[1]);
                }
            }
            fence_async_smem();
            mbar_arrive(q_full);
        }
        const Sight<kTree> see(a, sp, rq, r);
        const uint32_t my = tmem + tile * S::kTmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t s_ready = s_full + tile * 16, p_ready = p_full + tile * 16, o_done = v_empty + tile * 16;
        const float *scales = reinterpret_cast<const float *>(smem + S::kScales);
        Row sums{r < rows ? -INFINITY : 0.f, 0.f}; // (a row that is not there, all zeros, moves no reference)
        if (wait_warp(sc_full, 0) && wait_warp(s_ready, 0)) {
            fence_after_sync();
            sums.m = fmaxf(sums.m, row_first(my, scales, qs, tb0 + t_begin * kTile, see));
        }
#pragma unroll 1
        for (int j = 0; j < n; ++j) {
            // the scales of the next eight tiles' blocks, this tile's scores
            if (((j & 7) == 0 && !wait_warp(sc_full + (j >> 3 & 1) * 8, (j >> 4) & 1)) || !wait_warp(s_ready + (j & 1) * 8, (j >> 1) & 1))
                break;
            fence_after_sync();
            const int t0 = tb0 + (t_begin + j) * kTile;
            const float *sc = scales + (j & 15) * 12;
            const uint32_t my_s = my + (j & 1) * kTile;
            const bool all = see.all(t0) && see.all(t0 + 32);
            if (!(all && row_tile(my_s, sc, qs, sums))) {
                // O is at rest once the last tile's product is done: the next one waits for this tile's weights
                if (j > 0 && !wait_warp(o_done + ((j - 1) & 1) * 8, ((j - 1) >> 1) & 1))
                    break;
                fence_after_sync();
                sums = row_tile_moving(my_s, my + S::kO, j > 0 ? D : 0, sc, qs, sums, t0, see);
            }
            wait_st();
            fence_before_sync();
            mbar_arrive(p_ready + (j & 1) * 8);
        }
        const float m = sums.m, l = sums.l;
        // (V's last arrival carries the notes of NaN codes)
        if (ok && wait_warp(p_ready + ((n - 1) & 1) * 8, ((n - 1) >> 1) & 1) &&
            wait_warp(o_done + ((n - 1) & 1) * 8, ((n - 1) >> 1) & 1)) {
            fence_after_sync();
            const bool live = r < rows;
            const int rr = row0 + (live ? r : 0);
            const int64_t t = rq.q0 + rr / a.G;
            const int head = it.h * a.G + rr % a.G;
            const int64_t slot = slot0 + r;
            const bool nans = many && *s_any_nan;
            float lse = 0.f, f = 1.f;
            if (piece.whole)
                f = finish_row(m, l, a.sinks, head, &lse);
            // 32 columns of the warp's 32 rows at a time, through what was Q: written a row to a lane, read and stored
            // in whole rows (16-byte pieces XORed with the row, so that neither meets a bank twice)
            const uint32_t room = base + S::kQ + tile * 2 * S::kQBytes + (warp & 3) * (2 * S::kQBytes / 4);
            __nv_bfloat16 *dst[4]; // of the four rows that the lane stores pieces of
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = row0 + warp * 32 + i * 8 + (lane >> 2);
                dst[i] = static_cast<__nv_bfloat16 *>(a.out) + ((int64_t)(rq.q0 + row / a.G) * a.H + it.h * a.G + row % a.G) * D +
                         (lane & 3) * 8;
            }
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t x[32];
                ld32(my + S::kO + c * 32, x);
                wait_ld32(x);
                if (nans) {
                    const uint32_t bits = live ? nan_columns<D, kTree>(a, it, see, tb0, t_begin, n, c) : 0;
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        x[i] = (bits >> i & 1) ? 0x7FC00000u : x[i];
                }
                if (piece.whole) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            w[e] = pack_bf16x2(__uint_as_float(x[i * 8 + 2 * e]) * f, __uint_as_float(x[i * 8 + 2 * e + 1]) * f);
                        sts128(room + lane * 64 + ((i ^ (lane >> 1 & 3)) << 4), w[0], w[1], w[2], w[3]);
                    }
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int wr = i * 8 + (lane >> 2), rr = warp * 32 + wr; // four lanes to a row
                        const uint4 v = lds128(room + wr * 64 + (((lane & 3) ^ (wr >> 1 & 3)) << 4));
                        if (rr < rows)
                            *reinterpret_cast<uint4 *>(dst[i] + c * 32) = v;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        sts128(room + lane * 128 + ((i ^ (lane & 7)) << 4), x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int wr = i * 4 + (lane >> 3), rr = warp * 32 + wr; // eight lanes to a row
                        const uint4 v = lds128(room + wr * 128 + (((lane & 7) ^ (wr & 7)) << 4));
                        if (rr < rows)
                            *reinterpret_cast<uint4 *>(plan.o + (slot0 + rr) * D + c * 32 + (lane & 7) * 4) = v;
                    }
                }
                __syncwarp();
            }
            if (live) {
                if (!piece.whole)
                    plan.ml[slot] = make_float2(m, l);
                else if (a.lse)
                    a.lse[t * a.H + head] = lse;
            }
        }
    } else if (warp < S::kV0) {
        // a row tile without rows
    } else if (warp < S::kLoader) {
        // ---------------------------------------------------------------- V
        constexpr int kTurns = kTile / S::kVWarps / 8;
        const int row_in = (warp - S::kV0) * kTurns * 8 + (lane & 7), piece = lane >> 3; // rows row_in + 8 k, pieces piece + 4 c
        const int turn = D == 128 ? lane & 7 : (lane >> 1) & 3;                      // the swizzle of the lane's rows
#pragma unroll 1
        for (int j = 0; j < n; ++j) {
            const int stage = j & 1;
            if (!wait_warp(c_full + stage * 8, (j >> 1) & 1) ||
                (j > 1 && (!wait_warp(v_empty + stage * 8, ((j >> 1) - 1) & 1) ||
                           (live_tiles > 1 && !wait_warp(v_empty + 16 + stage * 8, ((j >> 1) - 1) & 1)))))
                break;
            const int tb = tb0 + (t_begin + j) * kTile;
            const bool clear = tb + kTile - 1 <= p_first && tb >= all_from;
            const uint32_t src = base + S::kCodes + stage * S::kTileBytes + row_in * D;
            const uint32_t dst = base + S::kV + stage * S::kVBytes + (row_in >> 3) * S::kVAtoms + (lane & 7) * 16 + piece * 256;
            uint4 q[kTurns][D / 64]; // all of them on their way before the first is used
#pragma unroll
            for (int k = 0; k < kTurns; ++k)
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
                    q[k][c] = lds128(src + k * 8 * D + (((piece + 4 * c) ^ turn) << 4));
#pragma unroll
            for (int k = 0; k < kTurns; ++k) {
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    uint32_t w[4] = {q[k][c].x, q[k][c].y, q[k][c].z, q[k][c].w};
                    if (!clear)
                        visible_codes(w, tb + row_in + 8 * k < kv_end && tb + row_in + 8 * k >= kv_begin, many, s_any_nan);
                    uint32_t f[8];
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        e4m3x4_to_f16x4(w[y], f[2 * y], f[2 * y + 1]);
                    sts128(dst + k * S::kVAtoms + c * 1024, f[0], f[1], f[2], f[3]);
                    sts128(dst + k * S::kVAtoms + c * 1024 + 128, f[4], f[5], f[6], f[7]);
                }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(c_empty + stage * 8);
            if (lane < live_tiles)
                mbar_arrive(p_full + lane * 16 + stage * 8);
        }
    } else if (warp < S::kMma) {
        // ---------------------------------------------------------------- the cache's codes and scales
        // One row tile: one warp for K and V; two: a warp for each (one alone held up the rest with small blocks).
        const bool with_k = NR == 1 || warp == S::kLoader, with_v = NR == 1 || warp != S::kLoader;
        const int32_t *table = a.block_table + it.b * a.table_stride;
        const int rows_in = min(kTile, a.block_size); // of a block in a tile
        const int pages = kTile / rows_in;
        float *scales = reinterpret_cast<float *>(smem + S::kScales);
        // Lane l looks after group l % 4 (16 positions) of tile l / 4 of eight: the table is read two eights
        // ahead, the scales one, so that no latency is waited for (tile by tile this warp held up the rest).
        auto entry = [&](int eight) {
            const int t = tb0 + (t_begin + 8 * eight + (lane >> 2)) * kTile + 16 * (lane & 3);
            const int e = t >> a.block_shift;
            return t < kv_end && e < a.table_width ? __ldg(table + e) : -1;
        };
        auto in_pool = [&](int e) { return e >= 0 && e < a.num_blocks ? e : -1; };
        auto scale_of = [&](const float *p, int v) { return v >= 0 ? __ldg(p + (int64_t)v * a.H_kv + it.h) : 0.f; };
        int v = in_pool(entry(0)), v_next = in_pool(entry(1)), raw = entry(2), issued = 0, v_issued = 0;
        float ks = scale_of(a.k_scale, v), vs = scale_of(a.v_scale, v), ks_next = scale_of(a.k_scale, v_next),
              vs_next = scale_of(a.v_scale, v_next);
#pragma unroll 1
        for (int j = 0; j < n; ++j) {
            if ((j & 7) == 0 && j > 0) {
                v = v_next;
                ks = ks_next;
                vs = vs_next;
                v_next = in_pool(raw);
                ks_next = scale_of(a.k_scale, v_next);
                vs_next = scale_of(a.v_scale, v_next);
                raw = entry((j >> 3) + 2);
            }
            // lane p: block p of the tile and (of K) of the next one. A block outside the pool: rows outside the map,
            // which fills zeros and reads nothing
            const int page = __shfl_sync(0xffffffffu, v, ((j & 7) * 4 + (lane * rows_in >> 4)) & 31);
            const int y = page >= 0 ? (tb0 + (t_begin + j) * kTile + lane * rows_in) & (a.block_size - 1) : a.block_size;
            const int z = page >= 0 ? page * a.H_kv + it.h : 0;
            const uint32_t at = lane * rows_in * D;
            if (with_k && !(j & 1)) {
                const int two = j >> 1;
                const int stage = two & (S::kKStages - 1);
                const uint32_t full = k_full + stage * 8;
                if (two >= S::kKStages && !wait_warp(k_empty + stage * 8, (two / S::kKStages - 1) & 1))
                    break;
                if (lane < 2 * pages) {
                    mbar_arrive_expect_tx(full, rows_in * D);
                    tma_load_3d(base + S::kK + stage * 2 * S::kTileBytes + at, &k_map, 0, y, z, full);
                }
                issued = two + 1;
            }
            if (with_k && (j & 7) == 0) {
                // the scales of eight tiles, a group to a lane. A group outside the pool, past the end, or below
                // what any row sees (where the block may have gone to another request: a bad scale would reach
                // the sums as 0 * NaN): logits of -inf. (The place was last read for tiles up to j - 9; the scores
                // of j - 7 are there, which waited for the values of j - 9.)
                float *sc = scales + ((j & 15) + (lane >> 2)) * 12 + (lane & 3);
                const bool seen = v >= 0 && tb0 + (t_begin + j + (lane >> 2)) * kTile + 16 * (lane & 3) + 15 >= kv_begin;
                sc[0] = seen ? ks * scale_log2 : 0.f;
                sc[4] = seen ? lg2_approx(vs) : -INFINITY;
                sc[8] = seen ? __frcp_rn(vs) : 1.f;
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(sc_full + (j >> 3 & 1) * 8);
            }
            if (with_v) {
                const uint32_t full = c_full + (j & 1) * 8;
                if (j > 1 && !wait_warp(c_empty + (j & 1) * 8, ((j >> 1) - 1) & 1))
                    break;
                if (lane < pages) {
                    mbar_arrive_expect_tx(full, rows_in * D);
                    tma_load_3d(base + S::kCodes + (j & 1) * S::kTileBytes + at, &v_map, 0, y, z, full);
                }
                v_issued = j + 1;
            }
        }
        // no copy outlives the block, also where a wait gave up
        for (int j = max(0, issued - S::kKStages); j < issued; ++j)
            if (!mbar_wait(k_full + (j & (S::kKStages - 1)) * 8, (j / S::kKStages) & 1) && lane == 0)
                atomicOr(&g_kv8_error, 2);
        // nor does the news that K is free, which comes from the tensor core and which nobody waits for
        for (int j = max(0, issued - S::kKStages); ok && j < issued; ++j)
            (void)wait_warp(k_empty + (j & (S::kKStages - 1)) * 8, (j / S::kKStages) & 1);
        for (int j = max(0, v_issued - 2); j < v_issued; ++j)
            if (!mbar_wait(c_full + (j & 1) * 8, (j >> 1) & 1) && lane == 0)
                atomicOr(&g_kv8_error, 2);
    } else if (warp - S::kMma < live_tiles) {
        // ---------------------------------------------------------------- products of a row tile
        const int tile = __shfl_sync(0xffffffffu, warp - S::kMma, 0);
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0) + tile * S::kTmem;
        const uint32_t s_ready = s_full + tile * 16, p_ready = p_full + tile * 16, o_done = v_empty + tile * 16;
        const uint64_t q_hi = desc(base + S::kQ + tile * 2 * S::kQBytes, 128, S::kQAtoms);
        const uint64_t q_lo = desc(base + S::kQ + (tile * 2 + 1) * S::kQBytes, 128, S::kQAtoms);
        const auto scores = [&](int j) {
            const int stage = (j >> 1) & (S::kKStages - 1);
            if (!(j & 1) && !wait_warp(k_full + stage * 8, (j >> 1) / S::kKStages & 1))
                return false;
            fence_after_sync();
            const uint32_t k_s = base + S::kK + (stage * 2 + (j & 1)) * S::kTileBytes;
            const uint64_t k_d = D == 128 ? desc_sw128(k_s, 16, 1024) : desc_sw64(k_s, 16, 512);
            const uint32_t dst = tm + (j & 1) * kTile;
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < D / 32; ++kk) // 32 columns: two core matrices of Q, 32 bytes of a row of K
                    mma_f8(dst, q_hi + kk * 16, k_d + kk * 2, S::kIdescS, kk > 0);
#pragma unroll
                for (int kk = 0; kk < D / 32; ++kk)
                    mma_f8(dst, q_lo + kk * 16, k_d + kk * 2, S::kIdescS, 1);
                commit(s_ready + (j & 1) * 8);
                if ((j & 1) || j == n - 1)
                    commit(k_empty + stage * 8);
            }
            __syncwarp();
            return true;
        };
        bool go = wait_warp(q_full, 0) && scores(0) && (n == 1 || scores(1));
#pragma unroll 1
        for (int j = 0; go && j < n; ++j) {
            const int stage = j & 1, phase = (j >> 1) & 1;
            if (!wait_warp(p_ready + stage * 8, phase))
                break;
            fence_after_sync();
            const uint64_t v_d = desc(base + S::kV + stage * S::kVBytes, S::kVAtoms, 128);
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < kTile / 16; ++kk) // 16 positions: 8 columns of P, two atoms of V
                    mma_f16_ts(tm + S::kO, tm + stage * kTile + kk * 8, v_d + (uint64_t)(kk * 2 * S::kVAtoms / 16), S::kIdescO,
                               j > 0 || kk > 0);
                commit(o_done + stage * 8);
            }
            __syncwarp();
            // P lies over its scores: those of two tiles on go there when its product is done
            if (j + 2 < n && (!wait_warp(o_done + stage * 8, phase) || !scores(j + 2)))
                break;
        }
        if (!ok) { // what was issued ends before its memory is given back
            if (elect_one())
                commit(drained + tile * 8);
            if (!mbar_wait(drained + tile * 8, 0) && lane == 0)
                atomicOr(&g_kv8_error, 2);
        }
    }
    __syncwarp();
    fence_before_sync();
    return ok;
}

template <int D, int NR, bool kTree>
__global__ void __launch_bounds__((Shape<D, NR>::kThreads), NR == 1 ? 2 : 1) kv8_tile_kernel(const __grid_constant__ CUtensorMap k_map,
                                                                                             const __grid_constant__ CUtensorMap v_map,
                                                                                             const Kv8AttnArgs a, const Plan plan)
{
    using S = Shape<D, NR>;
    extern __shared__ __align__(1024) uint8_t smem[]; // (the swizzle goes by address)
    Misc *misc = reinterpret_cast<Misc *>(smem + S::kMisc);
    const int tid = threadIdx.x, warp = tid >> 5;
    const bool fits = (smem_u32(smem) & 1023u) == 0; // otherwise a layout that the swizzle does not fit
    if (!fits && tid == 0)
        atomicOr(&g_kv8_error, 1);
    if (warp == S::kMma)
        alloc(smem_u32(&misc->tmem), NR * S::kTmem);
    const bool planned = !kTree || plan.items != nullptr;
    if (planned)
        grid_wait(); // the plan
    if (tid == 0)
        plan.dir[blockIdx.x] = make_int4(-1, 0, 0, 0);
    if (!planned)
        find_part<S::kThreads>(a, S::kItemRows, fits, misc, reinterpret_cast<long long *>(smem + S::kQ));
    else if (tid == 0) {
        const long long total = plan.cost[plan.n_items] * a.H_kv;
        const int parts = (int)min((long long)gridDim.x, max(1ll, (total + kMinPart - 1) / kMinPart));
        const bool mine = fits && (int)blockIdx.x < parts;
        misc->total = total;
        misc->units = fits ? plan.head[0] : 0;
        misc->next = misc->units > 0 ? atomicAdd(plan.head + 1, 1) : 0;
        misc->parts = parts;
        misc->at = mine ? total * blockIdx.x / parts : 0;
        misc->hi = mine ? total * (blockIdx.x + 1) / parts : 0;
        int lo = 0, hi = plan.n_items - 1; // the last item that begins at or before: items that are none cost nothing
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (plan.cost[mid] * a.H_kv <= misc->at)
                lo = mid;
            else
                hi = mid - 1;
        }
        misc->item = lo;
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    bool first = true;
    const int units = planned ? misc->units : 0;
    while (units > 0 ? misc->next < units : misc->at < misc->hi) {
        Piece piece;
        int s0 = 0, s1 = 1, item;
        int last = -1; // the CTA that ends the unit
        long long end = 0;
        int tiles;
        long long base = 0;
        Units un{0, 0, 0};
        if (!planned) {
            const long long at = misc->at;
            base = misc->base;
            item = misc->item; // (the request)
            piece.rq = Request{misc->q0, misc->qlen, misc->len, 0};
            un.tiles = misc->tiles;
            un.count = misc->count;
            un.cost = max(1, un.tiles) + kPieceCost;
            while (at >= base + un.all()) { // requests without tokens have no units
                base += un.all();
                piece.rq = request(a, ++item);
                un = units_of(a, S::kItemRows, piece.rq);
            }
            const long long x = at - base;
            const int u = x < INT_MAX ? (int)x / un.cost : (int)(x / un.cost);
            const long long unit = base + (long long)u * un.cost;
            end = min(misc->hi, unit + un.cost);
            s0 = (int)max(0ll, at - unit - kPieceCost);
            s1 = (int)max(0ll, end - unit - kPieceCost);
            last = (int)(((unit + un.cost) * misc->parts - 1) / misc->total);
            piece.it = Item{item, u / a.H_kv, u % a.H_kv};
            tiles = un.tiles;
        } else if (units > 0) {
            const int u = misc->next;
            item = plan.order[u / a.H_kv];
            piece.it.h = u % a.H_kv;
        } else {
            const long long at = misc->at;
            item = misc->item;
            base = plan.cost[item] * a.H_kv;
            long long next = plan.cost[item + 1] * a.H_kv;
            while (at >= next) {
                base = next;
                next = plan.cost[++item + 1] * a.H_kv;
            }
            const int cost = (int)((next - base) / a.H_kv);
            piece.it.h = (int)((at - base) / cost);
            const long long unit = base + (long long)piece.it.h * cost;
            end = min(misc->hi, unit + cost);
            s0 = (int)max(0ll, at - unit - kPieceCost);
            s1 = (int)max(0ll, end - unit - kPieceCost);
            last = (int)(((unit + cost) * misc->parts - 1) / misc->total);
        }
        if (planned) {
            const int4 *in = reinterpret_cast<const int4 *>(plan.items + item);
            const int4 i0 = in[0], i1 = in[1];
            tiles = i0.z;
            piece.it.b = i0.x;
            piece.it.chunk = i0.y;
            piece.rq = Request{i1.x, i1.y, i1.z, 0};
        }
        if (units > 0)
            s1 = max(1, tiles);
        piece.t_begin = s0;
        piece.t_end = min(s1, tiles);
        piece.whole = s0 == 0 && s1 == max(1, tiles);
        piece.slot0 = (2 * (int64_t)blockIdx.x + (s0 == 0 ? 1 : 0)) * S::kItemRows;
        __syncthreads(); // all have read the place
        if (tid == 0) {
            misc->at = end;
            misc->item = item;
            if (!planned) {
                misc->base = base;
                misc->q0 = piece.rq.q0;
                misc->qlen = piece.rq.qlen;
                misc->len = piece.rq.len;
                misc->tiles = un.tiles;
                misc->count = un.count;
            }
            if (s0 == 0 && s0 < s1 && !piece.whole) // (the thread that wrote it above)
                plan.dir[blockIdx.x] = make_int4(last, piece.it.b, piece.it.chunk, piece.it.h);
        }
        if (units > 0 && tid == S::kV0 * 32)
            misc->next = atomicAdd(plan.head + 1, 1);
        if (s0 < s1) {
            const bool ok = work_on<D, NR, kTree>(k_map, v_map, a, plan, smem, piece, first);
            first = first && piece.t_end <= s0;
            if (!ok) { // (every warp that waited on that gives up, too)
                misc->hi = 0;
                misc->next = INT_MAX;
            }
        }
        fence_async_smem(); // what was written or read here, before copies land there again
        __syncthreads();
        fence_after_sync();
    }
    if (warp == S::kMma)
        dealloc(misc->tmem, NR * S::kTmem);
}

// Joins the partial sums of the units that several CTAs share: a row to D / 4
// lanes, four rows of a lane at a time, whose loads are on their way together.
constexpr int kJoinWarps = 8, kJoinRows = 4;
template <int D, int NR>
__global__ void __launch_bounds__(kJoinWarps * 32) kv8_tile_join_kernel(const Kv8AttnArgs a, const Plan plan)
{
    constexpr int kItemRows = NR * kRows, kLanes = D / 4, kPer = 32 / kLanes; // lanes to a row, rows to a warp's access
    grid_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c0 = blockIdx.x;
    const int4 u = plan.dir[c0];
    if (u.x <= c0)
        return;
    const Request rq = request(a, u.y);
    const int row0 = u.z * kItemRows, rows = min(kItemRows, rq.qlen * a.G - row0);
    const int first = (blockIdx.y * kJoinWarps + warp) * kPer * kJoinRows + lane / kLanes, part = lane % kLanes;
    const auto slot = [&](int c, int k) { // (rows that are not there: another one's, not stored)
        return (2 * (int64_t)c + (c == c0)) * kItemRows + min(first + k * kPer, rows - 1);
    };
    float m[kJoinRows], l[kJoinRows];
    float4 acc[kJoinRows];
#pragma unroll
    for (int k = 0; k < kJoinRows; ++k) {
        m[k] = -INFINITY;
        l[k] = 0.f;
        acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int c = c0; c <= u.x; ++c)
#pragma unroll
        for (int k = 0; k < kJoinRows; ++k)
            m[k] = fmaxf(m[k], plan.ml[slot(c, k)].x);
    for (int c = c0; c <= u.x; ++c) {
        float2 ml[kJoinRows];
        float4 v[kJoinRows];
#pragma unroll
        for (int k = 0; k < kJoinRows; ++k) {
            ml[k] = plan.ml[slot(c, k)];
            v[k] = *reinterpret_cast<const float4 *>(plan.o + slot(c, k) * D + part * 4);
        }
#pragma unroll
        for (int k = 0; k < kJoinRows; ++k) {
            // one that saw nothing has m = -inf; its sums are 0, or NaN from a NaN logit
            const float f = ml[k].x == -INFINITY ? 1.f : ex2_approx(ml[k].x - m[k]);
            l[k] += ml[k].y * f;
            acc[k].x += v[k].x * f;
            acc[k].y += v[k].y * f;
            acc[k].z += v[k].z * f;
            acc[k].w += v[k].w * f;
        }
    }
#pragma unroll
    for (int k = 0; k < kJoinRows; ++k) {
        const int r = first + k * kPer;
        if (r >= rows)
            break;
        const int64_t t = rq.q0 + (row0 + r) / a.G;
        const int head = u.w * a.G + (row0 + r) % a.G;
        float lse;
        const float f = finish_row(m[k], l[k], a.sinks, head, &lse);
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + (t * a.H + head) * D + part * 4) =
            make_uint2(pack_bf16x2(acc[k].x * f, acc[k].y * f), pack_bf16x2(acc[k].z * f, acc[k].w * f));
        if (a.lse && part == 0)
            a.lse[t * a.H + head] = lse;
    }
}

struct Sizes {
    int64_t items;
    size_t cost_at, items_at, order_at, dir_at, ml_at, o_at, total;
};

int slots_of(int NR, int sm_count) { return (NR == 1 ? 2 : 1) * std::max(sm_count, 1); } // CTAs at a time

Sizes sizes_of(int64_t B, int64_t T, int G, int D, int NR, int sm_count)
{
    Sizes z;
    const size_t rows = NR * kRows, partials = 2 * (size_t)slots_of(NR, sm_count);
    z.items = T * G / (int64_t)rows + B; // each request's last chunk may be short
    z.cost_at = 256;
    z.items_at = up256(z.cost_at + (size_t)(z.items + 1) * sizeof(long long));
    z.order_at = up256(z.items_at + (size_t)z.items * sizeof(PlannedItem));
    z.dir_at = up256(z.order_at + (size_t)z.items * sizeof(int));
    z.ml_at = up256(z.dir_at + (size_t)slots_of(NR, sm_count) * sizeof(int4));
    z.o_at = up256(z.ml_at + partials * rows * sizeof(float2));
    z.total = z.o_at + partials * rows * D * sizeof(float);
    return z;
}

// A launch behind the last one, its start overlapped (the kernel waits for the last one's end itself).
template <typename... Args, typename... Given>
cudaError_t launch_behind(void (*kernel)(Args...), dim3 grid, int threads, int smem, cudaStream_t stream, const Given &...given)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, given...);
}

template <int D, int NR, bool kTree>
cudaError_t launch(const Kv8AttnArgs &a, void *workspace, int sm_count, cudaStream_t stream)
{
    using S = Shape<D, NR>;
    const Sizes z = sizes_of(a.B, a.T, a.G, D, NR, sm_count);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    Plan plan{reinterpret_cast<int *>(ws),
                    reinterpret_cast<long long *>(ws + z.cost_at),
                    reinterpret_cast<PlannedItem *>(ws + z.items_at),
                    reinterpret_cast<int *>(ws + z.order_at),
                    reinterpret_cast<int4 *>(ws + z.dir_at),
                    reinterpret_cast<float2 *>(ws + z.ml_at),
                    reinterpret_cast<float *>(ws + z.o_at),
                    (int)z.items,
                    S::kItemRows};
    const int grid = slots_of(NR, sm_count);
    cudaError_t e = cudaFuncSetAttribute(kv8_tile_kernel<D, NR, kTree>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess)
        return e;
    CUtensorMap maps[2];
    if (!kv8_tensor_maps(a, D, kTile, maps))
        return cudaErrorInvalidValue;
    // (units that are taken whole are at least three to a CTA)
    if (kTree && z.items * a.H_kv < 3ll * grid) {
        plan.items = nullptr;
        kv8_tile_kernel<D, NR, kTree><<<grid, S::kThreads, S::kSmem, stream>>>(maps[0], maps[1], a, plan);
        e = cudaGetLastError();
    } else {
        kv8_tile_plan_kernel<<<1, kPlanThreads, 0, stream>>>(a, plan, grid);
        if ((e = cudaGetLastError()) != cudaSuccess)
            return e;
        e = launch_behind(kv8_tile_kernel<D, NR, kTree>, dim3((unsigned)grid), S::kThreads, S::kSmem, stream, maps[0], maps[1], a, plan);
    }
    if (e != cudaSuccess)
        return e;
    constexpr int kRowsOfBlock = kJoinWarps * 32 / (D / 4) * kJoinRows;
    return launch_behind(kv8_tile_join_kernel<D, NR>, dim3((unsigned)grid, S::kItemRows / kRowsOfBlock), kJoinWarps * 32, 0, stream, a,
                         plan);
}

// Row tiles of a CTA: two where a request's rows may fill more than one. 16 requests of
// 8192 positions, 8 kv heads of 128 columns: 132 rows 129 us (one row tile: 145), 256
// rows 134 (150); 128 rows 120 (92), 40 rows 118 (90).
int row_tiles(int G, int max_query_len) { return (int64_t)G * max_query_len > kRows ? 2 : 1; }

template <bool kTree>
cudaError_t launch_rows(const Kv8AttnArgs &a, int D, int max_query_len, void *workspace, int sm_count, cudaStream_t stream)
{
    if (row_tiles(a.G, max_query_len) == 2)
        return D == 128 ? launch<128, 2, kTree>(a, workspace, sm_count, stream) : launch<64, 2, kTree>(a, workspace, sm_count, stream);
    return D == 128 ? launch<128, 1, kTree>(a, workspace, sm_count, stream) : launch<64, 1, kTree>(a, workspace, sm_count, stream);
}

} // namespace

size_t kv8_tile_workspace(int B, int T, int H, int H_kv, int D, int max_query_len, int sm_count)
{
    return sizes_of(B, T, H / H_kv, D, row_tiles(H / H_kv, max_query_len), sm_count).total;
}

cudaError_t launch_kv8_tile(const Kv8AttnArgs &a, int D, int max_query_len, void *workspace, int sm_count, cudaStream_t stream)
{
    return a.tree_mask ? launch_rows<true>(a, D, max_query_len, workspace, sm_count, stream)
                       : launch_rows<false>(a, D, max_query_len, workspace, sm_count, stream);
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

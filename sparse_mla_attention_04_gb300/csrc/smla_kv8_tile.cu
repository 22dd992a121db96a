// Attention over the block-scaled 8-bit cache for many query rows (prompts and
// chunks of prompts, sm_103a): 128 query rows to a tile, both products on the
// tensor cores (tcgen05), scores and sums in tensor memory.
//
// A CTA takes 128 rows (token, head of the kv head's group) of one request and
// kv head and walks over the visible positions in tiles of 64. Scores have two
// buffers in tensor memory: while a tile's softmax runs, the next one's scores
// are computed; two CTAs share an SM, so that the tensor cores have the other's
// products meanwhile. Warps of a CTA:
//   0-3  softmax, a row to a thread; the epilogue
//   4-5  V's codes, expanded to binary16
//   6    the blocks' codes by TMA as they lie in the cache; the blocks' scales
//   7    issues the tensor-core products
// (eight warps, so that both CTAs' threads have 128 registers). Their loops are
// kept short, not unrolled: all run at once, and with long straight code each
// instruction was fetched again every tile (8 to 20 cycles an instruction).
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
// denominator adds p' / vs. A row's reference m moves, and what was added up
// so far is rescaled, only when a logit passes it by 15 (p' <= 2^15 is inside
// binary16, whose precision is relative): the scores are read once, with no
// pass for the maximum before.
//
// Shared memory: the codes in TMA's swizzled rows; Q and the expanded V in 8-row
// x 16-byte core matrices, written so that eight lanes fill one (no bank
// conflict). Blocks outside the pool are zero-filled and not read.
#include "smla_kv8.cuh"
#include "smla_umma.cuh"

#include <algorithm>

namespace smla {

__device__ int g_kv8_error = 0; // 1: a bounded wait gave up; 2: products in flight did not drain

namespace {

using namespace kv8;
using namespace umma;

constexpr int kRows = 128;  // of a row tile
constexpr int kTile = 64;
constexpr float kSlack = 8.0f;
constexpr int kMaxSplits = 16; // of an item's positions
constexpr int kWaves = 2;      // an item is split where it is more than this part of a CTA slot's share
constexpr int kMinSplit = 16;  // tiles of a split, at least

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
    static constexpr int kMisc = kBars + 31 * 8;    // the tensor memory's address, a flag
    static constexpr int kSmem = kMisc + 8;
    static constexpr uint32_t kTmem = 256;          // of a row tile: two S (P over each one's first half) and O
    static constexpr uint32_t kO = 2 * kTile;
    static constexpr uint32_t kIdescS = idesc(128, kTile, 0, 0, 0, 0);
    static constexpr uint32_t kIdescO = idesc(128, D, 0, 0, 0, 1);
    static_assert(NR == 2 || 2 * (kSmem + 1024) <= 228 * 1024, "two CTAs to an SM");
};

// The plan of a call, in the workspace: how many entries and how many split items
// there are; the entries, the longest first; the split items {request, chunk,
// splits, first partial}; their partial sums.
struct Entry {
    int b, chunk, split, first;   // split | splits << 16; first partial
    int q0, qlen, len, none;      // the request
};
struct Plan {
    int *header;
    Entry *entries;
    int4 *splits;
    float2 *ml; // [partials][H_kv][item_rows]
    float *o;   // [partials][H_kv][item_rows][D]
    int n_items, item_rows;
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
    s.p_first = rq.pos(s.row0 / a.G);
    s.p_last = rq.pos((s.row0 + s.rows - 1) / a.G);
    s.kv_end = min(rq.len, s.p_last + 1);
    s.kv_begin = a.window > 0 ? max(0, s.p_first - a.window + 1) : 0;
    s.all_from = a.window > 0 ? s.p_last - a.window + 1 : 0;
    s.tb0 = s.kv_begin & ~(kTile - 1);
    s.tiles = s.kv_end > s.tb0 ? (s.kv_end - s.tb0 + kTile - 1) / kTile : 0;
    return s;
}

// Plans a call, by one block: items that are longer than their part of a CTA
// slot's share are split, and the entries are sorted by length (64 classes), so
// that ragged requests fill the GPU evenly whatever their order. Where an entry
// or a partial stands does not change what is computed from it. The first
// kPlanned items of a thread stay in registers.
constexpr int kPlanThreads = 1024, kPlanned = 4;
__global__ void __launch_bounds__(kPlanThreads) kv8_tile_plan_kernel(const Kv8AttnArgs a, const Plan plan, int slots)
{
    __shared__ long long s_total;
    __shared__ int s_most, s_hist[64], s_parts, s_split_items;
    grid_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31;
    if (tid == 0) {
        s_total = 0;
        s_most = 0;
        s_parts = 0;
        s_split_items = 0;
    }
    if (tid < 64)
        s_hist[tid] = 0;
    __syncthreads();
    auto tiles_of = [&](int n) { // -1: no such item
        Item it;
        return find_item(a, plan.item_rows, n, &it) ? span_of(a, plan.item_rows, request(a, it.b), it.chunk).tiles : -1;
    };
    int kept[kPlanned];
    long long sum = 0;
    int most = 0;
#pragma unroll
    for (int i = 0; i < kPlanned; ++i) {
        const int n = tid + i * kPlanThreads;
        kept[i] = n < plan.n_items ? tiles_of(n) : -1;
        sum += max(kept[i], 0);
        most = max(most, kept[i]);
    }
    for (int n = tid + kPlanned * kPlanThreads; n < plan.n_items; n += kPlanThreads) {
        const int tiles = tiles_of(n);
        sum += max(tiles, 0);
        most = max(most, tiles);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, d);
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) {
        atomicAdd(reinterpret_cast<unsigned long long *>(&s_total), (unsigned long long)sum);
        atomicMax(&s_most, most);
    }
    __syncthreads();
    const int target = (int)max((long long)kMinSplit, (s_total * a.H_kv + (long long)kWaves * slots - 1) / ((long long)kWaves * slots));
    const int longest = max(1, min(s_most, target));
    auto splits = [&](int tiles) { return min(kMaxSplits, max(1, (tiles + target - 1) / target)); };
    auto bucket = [&](int tiles) { return 63 - min(63, (int)((long long)(tiles / splits(tiles)) * 63 / longest)); };
    auto count = [&](int tiles) {
        if (tiles >= 0)
            atomicAdd(&s_hist[bucket(tiles)], splits(tiles));
    };
#pragma unroll
    for (int i = 0; i < kPlanned; ++i)
        count(kept[i]);
    for (int n = tid + kPlanned * kPlanThreads; n < plan.n_items; n += kPlanThreads)
        count(tiles_of(n));
    __syncthreads();
    if (tid < 32) { // the classes' first places
        const int x0 = s_hist[2 * lane], x1 = s_hist[2 * lane + 1];
        int to = x0 + x1;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, to, d);
            to += lane >= d ? y : 0;
        }
        s_hist[2 * lane] = to - x0 - x1;
        s_hist[2 * lane + 1] = to - x1;
        if (lane == 31)
            plan.header[0] = to;
    }
    __syncthreads();
    auto place = [&](int n, int tiles) {
        if (tiles < 0)
            return;
        const int ns = splits(tiles);
        const int at = atomicAdd(&s_hist[bucket(tiles)], ns);
        int first = 0;
        Item it;
        (void)find_item(a, plan.item_rows, n, &it);
        if (ns > 1) {
            first = atomicAdd(&s_parts, ns);
            plan.splits[atomicAdd(&s_split_items, 1)] = make_int4(it.b, it.chunk, ns, first);
        }
        const Request rq = request(a, it.b);
        for (int i = 0; i < ns; ++i)
            plan.entries[at + i] = Entry{it.b, it.chunk, i | ns << 16, first, rq.q0, rq.qlen, rq.len, 0};
    };
#pragma unroll
    for (int i = 0; i < kPlanned; ++i)
        place(tid + i * kPlanThreads, kept[i]);
    for (int n = tid + kPlanned * kPlanThreads; n < plan.n_items; n += kPlanThreads)
        place(n, tiles_of(n));
    __syncthreads();
    if (tid == 0)
        plan.header[1] = s_split_items;
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
struct Sight {
    int p_first, all_from; // the tile's: see Span
    int pos, pos_lo;       // this row: pos_lo <= t <= pos
    __device__ bool all(int t) const { return t + 31 <= p_first && t >= all_from; }
    __device__ bool sees(int t) const { return t <= pos && t >= pos_lo; }
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
// (the sum passes 2^15, so a weight may pass what binary16 holds) for some row of
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
    if (__any_sync(0xffffffffu, all > 0x1p15f || !(fabsf(row.m) <= 0x1p20f)))
        return false;
    row.l = l;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        st16(my + 16 * i, *reinterpret_cast<uint32_t(*)[16]>(p + 16 * i));
    return true;
}

// Sixteen of the row's logits, -inf where it does not see the position.
__device__ __forceinline__ void logits(uint32_t my, const float *sc, float qs, int t0, const Sight &see, int c, uint32_t (&x)[16])
{
    ld16(my + c * 16, x);
    const float k = sc[c] * qs, vs = sc[4 + c];
    const int t = t0 + c * 16;
    wait_ld16(x);
#pragma unroll
    for (int i = 0; i < 16; ++i)
        x[i] = __float_as_uint(see.sees(t + i) ? fmaf(__uint_as_float(x[i]), k, vs) : -INFINITY);
}

// The largest of the row's 64 logits that it sees.
__device__ __forceinline__ float largest(uint32_t my, const float *sc, float qs, int t0, const Sight &see)
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

// The row's first reference.
__device__ __noinline__ float row_first(uint32_t my, const float *sc, float qs, int t0, const Sight see)
{
    return largest(my, sc, qs, t0, see);
}

// row_tile for any tile and any reference: the reference moves to the tile's largest
// logit where that passes it by kSlack, and what was added up is rescaled (O is at
// rest; o_cols: its columns, 0 before the first product); positions that the row
// does not see are left out; the difference is taken from the rounded logit, as the
// reference is.
__device__ __noinline__ Row row_tile_moving(uint32_t my, uint32_t my_o, int o_cols, const float *sc, float qs, Row row, int t0,
                                            const Sight see)
{
    const float top = largest(my, sc, qs, t0, see);
    const bool raise = row.m == -INFINITY ? top > -INFINITY : top - row.m > kSlack;
    if (__any_sync(0xffffffffu, raise)) {
        const float g = raise ? (row.m == -INFINITY ? 0.f : ex2_approx(row.m - top)) : 1.f;
        row.m = raise ? top : row.m;
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
template <int D>
__device__ __noinline__ uint32_t nan_columns(const Kv8AttnArgs &a, const Item &it, const Sight &see, int tb0, int t_begin, int n,
                                             int c)
{
    uint32_t bits = 0;
    for (int t = max(see.pos_lo, tb0 + t_begin * kTile); t <= see.pos && t < tb0 + (t_begin + n) * kTile; ++t) {
        const int tile = t & ~(kTile - 1); // (tb0 is a multiple of it)
        if (tile + kTile - 1 <= see.p_first && tile >= see.all_from)
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

template <int D, int NR>
__global__ void __launch_bounds__((Shape<D, NR>::kThreads), NR == 1 ? 2 : 1) kv8_tile_kernel(const __grid_constant__ CUtensorMap k_map,
                                                               const __grid_constant__ CUtensorMap v_map,
                                                               const Kv8AttnArgs a, const Plan plan)
{
    using S = Shape<D, NR>;
    extern __shared__ __align__(1024) uint8_t smem[]; // (the swizzle goes by address)
    int *s_any_nan = reinterpret_cast<int *>(smem + S::kMisc + 4);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t base = smem_u32(smem);
    if (base & 1023u) { // a layout that the swizzle does not fit
        if (tid == 0)
            atomicOr(&g_kv8_error, 1);
        return;
    }
    const uint32_t bars = base + S::kBars;
    // K landed / free (up to four stages of two tiles); V's codes landed / free (two stages); scales of eight tiles written
    // (two stages); drained (each row tile); Q written; of each row tile, two stages: scores ready, P and V ready,
    // values done
    const uint32_t k_full = bars, k_empty = bars + 32, c_full = bars + 64, c_empty = bars + 80, sc_full = bars + 96,
                   drained = bars + 112, q_full = bars + 128, s_full = bars + 136, p_full = bars + 168, v_empty = bars + 200;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + S::kMisc);

    grid_wait(); // the plan
    const int n_entry = (int)(blockIdx.x / a.H_kv);
    const int4 *at = reinterpret_cast<const int4 *>(plan.entries + n_entry); // (inside the workspace, whatever it holds)
    const int4 e0 = at[0], e1 = at[1];
    if (n_entry >= plan.header[0])
        return;
    const int split = e0.z & 0xFFFF, splits = e0.z >> 16;
    const Item it{e0.x, e0.y, (int)(blockIdx.x % a.H_kv)};
    const int64_t slot0 = ((int64_t)(e0.w + split) * a.H_kv + it.h) * S::kItemRows; // (of a split item)
    const Request rq{e1.x, e1.y, e1.z, 0};
    const Span sp = span_of(a, S::kItemRows, rq, it.chunk);
    const int row0 = sp.row0, rows = sp.rows, p_first = sp.p_first, p_last = sp.p_last, kv_begin = sp.kv_begin,
              kv_end = sp.kv_end, all_from = sp.all_from, tb0 = sp.tb0;
    const int t_begin = sp.tiles * split / splits, t_end = sp.tiles * (split + 1) / splits; // (tiles < 2^25, splits <= 16)
    const int n = t_end - t_begin;
    const bool many = p_first != p_last;
    const int live_tiles = NR == 1 || rows <= kRows ? 1 : 2; // (a row tile without rows does nothing)

    if (n <= 0) { // nothing to see here
        if (tid < rows) {
            const int64_t t = rq.q0 + (row0 + tid) / a.G;
            const int head = it.h * a.G + (row0 + tid) % a.G;
            if (splits > 1) {
                plan.ml[slot0 + tid] = make_float2(-INFINITY, 0.f);
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
        const int pages = kTile / min(kTile, a.block_size);
        for (int i = 0; i < S::kKStages; ++i) {
            mbar_init(k_full + 8 * i, 2 * pages);
            mbar_init(k_empty + 8 * i, live_tiles);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(c_full + 8 * i, pages);
            mbar_init(c_empty + 8 * i, S::kVWarps);
            mbar_init(sc_full + 8 * i, 1);
            mbar_init(drained + 8 * i, 1);
        }
        for (int i = 0; i < 2 * NR; ++i) {
            mbar_init(s_full + 8 * i, 1);
            mbar_init(p_full + 8 * i, kRows + S::kVWarps);
            mbar_init(v_empty + 8 * i, 1);
        }
        mbar_init(q_full, live_tiles * kRows);
        mbar_init_fence();
    }
    if (warp == S::kMma)
        alloc(smem_u32(tmem_slot), NR * S::kTmem);
    const float scale_log2 = fabsf(a.scale) * kLog2e; // the sign goes into q

    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    bool ok = true;
    // a bounded wait, by whole warps
    auto wait_warp = [&](uint32_t bar, uint32_t parity) {
        ok = ok && mbar_wait_warp(bar, parity);
        if (!ok && lane == 0)
            atomicOr(&g_kv8_error, 1);
        return ok;
    };

    if (warp < S::kV0) {
        const int tile = warp >> 2; // of rows
        if (tile < live_tiles) {
        // ---------------------------------------------------------------- softmax
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
        const int pos = r < rows ? rq.pos((row0 + r) / a.G) : -1;
        const Sight see{p_first, all_from, pos, a.window > 0 ? pos - a.window + 1 : 0};
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
            if (splits == 1)
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
                    const uint32_t bits = live ? nan_columns<D>(a, it, see, tb0, t_begin, n, c) : 0;
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        x[i] = (bits >> i & 1) ? 0x7FC00000u : x[i];
                }
                if (splits == 1) {
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
                if (splits > 1)
                    plan.ml[slot] = make_float2(m, l);
                else if (a.lse)
                    a.lse[t * a.H + head] = lse;
            }
        }
        }
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
    __syncthreads();
    if (warp == S::kMma)
        dealloc(tmem, NR * S::kTmem);
}

// Joins the splits of the split items' rows, a warp to a row; the blocks share
// out the items by eight rows.
template <int D, int NR>
__global__ void __launch_bounds__(256) kv8_tile_join_kernel(const Kv8AttnArgs a, const Plan plan)
{
    constexpr int kD = D / 32;
    constexpr int kItemRows = NR * kRows, kEights = kItemRows / 8;
    grid_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int work = plan.header[1] * a.H_kv * kEights; // (partials are fewer than 2^31 / 256)
    for (int x = blockIdx.x; x < work; x += gridDim.x) {
        const int4 info = plan.splits[x / kEights / a.H_kv];
        const int splits = info.z, h = x / kEights % a.H_kv;
        const Request rq = request(a, info.x);
        const int row0 = info.y * kItemRows;
        const int rows = min(kItemRows, rq.qlen * a.G - row0);
        const int r = warp + 8 * (int)(x % kEights);
        if (r < rows) {
            auto slot = [&](int s) { return ((int64_t)(info.w + s) * a.H_kv + h) * kItemRows + r; };
            const float2 mine = lane < splits ? plan.ml[slot(lane)] : make_float2(-INFINITY, 0.f);
            const float m = warp_max(mine.x);
            const float f_mine = mine.x == -INFINITY ? 1.f : ex2_approx(mine.x - m);
            // nothing seen: no sums were written
            const unsigned seen = __ballot_sync(0xffffffffu, lane < splits && !(mine.x == -INFINITY && mine.y == 0.f));
            float acc[kD], l = 0.f;
#pragma unroll
            for (int i = 0; i < kD; ++i)
                acc[i] = 0.f;
#pragma unroll 8
            for (int s = 0; s < splits; ++s) {
                float2 v[kD / 2];
                const float2 *src = reinterpret_cast<const float2 *>(plan.o + slot(s) * D + lane * kD);
#pragma unroll
                for (int i = 0; i < kD / 2; ++i)
                    v[i] = seen >> s & 1 ? src[i] : make_float2(0.f, 0.f);
                const float sl = __shfl_sync(0xffffffffu, mine.y, s), f = __shfl_sync(0xffffffffu, f_mine, s);
                l += sl * f;
#pragma unroll
                for (int i = 0; i < kD / 2; ++i) {
                    acc[2 * i] += v[i].x * f;
                    acc[2 * i + 1] += v[i].y * f;
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
    }
}

struct Sizes {
    int64_t items, entries, partials; // entries and partials: for each kv head
    size_t entries_at, splits_at, ml_at, o_at, total;
};

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

int slots_of(int NR, int sm_count) { return (NR == 1 ? 2 : 1) * std::max(sm_count, 1); } // CTAs at a time

// Items: each request's last chunk may be short. Entries: an item, and one more
// for each whole part of the shares that its length holds. Split items: no more
// than there are parts; their partials at most twice as many.
Sizes sizes_of(int64_t B, int64_t T, int G, int H_kv, int D, int NR, int sm_count)
{
    Sizes z;
    const int64_t parts = (int64_t)kWaves * slots_of(NR, sm_count) / H_kv + 1;
    const int64_t item_rows = NR * kRows;
    z.items = T * G / item_rows + B;
    z.entries = z.items + parts;
    z.partials = 2 * parts;
    z.entries_at = 256;
    z.splits_at = up256(z.entries_at + (size_t)z.entries * sizeof(Entry));
    z.ml_at = up256(z.splits_at + (size_t)parts * sizeof(int4));
    z.o_at = up256(z.ml_at + (size_t)z.partials * H_kv * item_rows * sizeof(float2));
    z.total = z.o_at + (size_t)z.partials * H_kv * item_rows * D * sizeof(float);
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

template <int D, int NR>
cudaError_t launch(const Kv8AttnArgs &a, void *workspace, int sm_count, cudaStream_t stream)
{
    using S = Shape<D, NR>;
    const Sizes z = sizes_of(a.B, a.T, a.G, a.H_kv, D, NR, sm_count);
    if (z.entries * a.H_kv > 0x7FFFFFFF)
        return cudaErrorInvalidValue;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const Plan plan{reinterpret_cast<int *>(ws), reinterpret_cast<Entry *>(ws + z.entries_at), reinterpret_cast<int4 *>(ws + z.splits_at),
                    reinterpret_cast<float2 *>(ws + z.ml_at), reinterpret_cast<float *>(ws + z.o_at), (int)z.items,
                    S::kItemRows};
    cudaError_t e = cudaFuncSetAttribute(kv8_tile_kernel<D, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess)
        return e;
    CUtensorMap maps[2];
    if (!kv8_tensor_maps(a, D, kTile, maps))
        return cudaErrorInvalidValue;
    kv8_tile_plan_kernel<<<1, kPlanThreads, 0, stream>>>(a, plan, slots_of(NR, sm_count));
    if ((e = cudaGetLastError()) != cudaSuccess)
        return e;
    e = launch_behind(kv8_tile_kernel<D, NR>, dim3((unsigned)(z.entries * a.H_kv)), S::kThreads, S::kSmem, stream, maps[0],
                      maps[1], a, plan);
    if (e != cudaSuccess)
        return e;
    return launch_behind(kv8_tile_join_kernel<D, NR>, dim3((unsigned)(16 * sm_count)), 256, 0, stream, a, plan);
}

// Row tiles of a CTA: two where a request's rows may fill more than one.
int row_tiles(int G, int max_query_len) { return (int64_t)G * max_query_len > kRows ? 2 : 1; }

} // namespace

size_t kv8_tile_workspace(int B, int T, int H, int H_kv, int D, int max_query_len, int sm_count)
{
    return sizes_of(B, T, H / H_kv, H_kv, D, row_tiles(H / H_kv, max_query_len), sm_count).total;
}

cudaError_t launch_kv8_tile(const Kv8AttnArgs &a, int D, int max_query_len, void *workspace, int sm_count, cudaStream_t stream)
{
    if (row_tiles(a.G, max_query_len) == 2)
        return D == 128 ? launch<128, 2>(a, workspace, sm_count, stream) : launch<64, 2>(a, workspace, sm_count, stream);
    return D == 128 ? launch<128, 1>(a, workspace, sm_count, stream) : launch<64, 1>(a, workspace, sm_count, stream);
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

// Attention over the block-scaled 8-bit cache for few query rows (decode,
// sm_103a): every code of K and V crosses the bus once, at HBM's rate.
//
// The work is cut evenly, whatever the lengths: a unit is (request, chunk of
// R = 8 kTiles query rows, kv head), its length in steps of 32 positions plus a
// constant for its start and end; the units laid end to end are cut into parts,
// one per block: equal ones that fill the GPU once with eleven twelfths of the
// work, then as many small ones for the blocks that are done first (SMs differ by
// 15% in what they get through). A block walks its part; a unit that lies in
// it whole is finished there, one that several blocks share leaves partial sums
// that a second kernel (launched behind, its start overlapped) joins in a fixed
// order. Nothing depends on the host knowing the lengths, so a captured call
// follows them; the division depends on nothing else, so results do not vary.
//
// In a block the four warps take a unit's steps in turn, each with its own
// softmax state and its own ring of TMA copies: nothing is waited for between
// warps until a unit ends. Copies land in TMA's swizzled rows, and the order of
// a step's positions in the products is chosen so that eight lanes' 16-byte
// reads of K and of V both fall on different banks.
//
// Arithmetic: S^T = K Q^T and O^T = V^T P^T by warp-level products with binary32
// sums: the tokens (for S) and the value columns (for O) fill the 16 rows, 8
// query rows the columns, which wastes nothing for the 4 to 16 query heads of a
// kv head. S runs on the cache's codes as they are (m16n8k32): q's bf16 values
// are carried by two E4M3 parts, exactly down to 2^-9 of the row's largest
// (smaller ones to 2^-17 of it), and two such products take the time of one in
// binary16 (4.4 against 8.7 cycles each) without expanding K. V's codes are
// expanded to binary16, exactly, as are not the weights: 8-bit parts of a weight
// lose those far below the largest, of which a long context has many. The order
// of a product's inner index is free, so it is chosen for the loads: a lane's 16
// bytes of a K row are two k-steps of its fragment, and its 16 bytes of four V
// rows are its whole V^T fragment.
// The block scales: K's multiplies the logits, V's is folded into the exponent,
// p' = 2^(s + log2(vs) - m), and the denominator adds p' / vs. The reference m is
// set so that the largest p' is 2^11 and moves only when one would pass 2^15: one
// vote a step instead of a reduction. Binary16 holds p' to 2^-11 of itself down
// to 2^-14, a 2^-25th of the largest: with the largest at 1 a value scale 2^-20 of
// another's, whose block may hold nothing of that size, lost all but a few bits.
//
// Measured: 64 requests of up to 32768 positions (1.08 GB of codes, 32 heads on 8 kv
// heads of 128 columns) in 189 us, 5.7 TB/s, 84% of the copy bandwidth; one request of
// 509 positions in 23 us a call, of which the two kernels take about 10. Steps of 64
// positions, cp.async copies and binary16 products for S took 253 us; equal parts
// without the small ones 196.
#include "smla_kv8.cuh"
#include "smla_umma.cuh"

#include <algorithm>

namespace smla {

__device__ int g_kv8_stream_error = 0; // 1: a bounded wait gave up; 2: copies in flight did not land

namespace {

using namespace kv8;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStep = 32;     // positions a warp takes at a time
constexpr int kStages = 2;
constexpr int kUnitCost = 2;  // a unit's start and end, in steps
constexpr int kMinPart = 6;   // a block's part, in steps, before more blocks share the work
constexpr float kTop = 11.0f;   // (log2) the largest weight where the reference is set,
constexpr float kSlack = 15.0f; // and what none may pass: binary16 ends at 65504

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint4 lds128(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr));
    return v;
}

__device__ __forceinline__ uint2 lds64(uint32_t addr)
{
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];\n" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}

// Bytes of the NaN code (0x7F or 0xFF) as 0x80 in the same byte.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// The units of one request and the cost of each.
struct Units {
    int steps; // of kStep positions
    long long count, cost;
};

template <int R>
__device__ __forceinline__ Units units_of(const Kv8AttnArgs &a, const Request &r)
{
    Units u;
    u.steps = max(1, (r.len - r.begin + kStep - 1) / kStep);
    u.count = (((long long)r.qlen * a.G + R - 1) / R) * a.H_kv;
    u.cost = u.steps + kUnitCost;
    return u;
}

// How the total cost is cut: `big` equal parts of the first big_total, then
// `small` equal ones.
constexpr int kSmallPerBig = 1;
struct Division {
    long long total, big_total;
    int big, small;

    // fill: the blocks that the GPU holds; grid: those launched (fill, or with the small parts too)
    __device__ static Division of(long long total, int fill, int grid)
    {
        Division d{total, total, 0, 0};
        const long long parts = max(1ll, (total + kMinPart - 1) / kMinPart);
        d.big = (int)min((long long)min(fill, grid), parts); // (never more than there are, whatever the starts hold)
        // small parts of a twelfth of a block's share, where that is work enough for one
        if (grid > fill && total / 12 >= (long long)2 * kMinPart * fill) {
            d.small = grid - fill;
            d.big_total = total - total / 12 * kSmallPerBig;
        }
        return d;
    }
    __device__ long long begin(int i) const
    {
        return i <= big ? big_total * i / big : big_total + (total - big_total) * (i - big) / small;
    }
    // the part that holds cost x
    __device__ int part(long long x) const
    {
        return x < big_total ? (int)(((x + 1) * big - 1) / big_total)
                             : big + (int)(((x - big_total + 1) * small - 1) / (total - big_total));
    }
};

template <int D, int NT> struct Layout {
    static constexpr int R = 8 * NT;
    static constexpr int kSide = kStep * D;                     // K (or V) of one step
    static constexpr int kStageBytes = 2 * kSide;
    static constexpr int kRing = kWarps * kStages * kStageBytes;
    static constexpr int kMerge = kWarps * R * D * 4;           // the warps' value sums at a unit's end
    static constexpr int kBig = kRing > kMerge ? kRing : kMerge;
    static constexpr int kNanWords = R * D / 32;
    static constexpr int kSmem = kBig + kWarps * R * 8 + kWarps * kStages * 32 + kNanWords * 4 + kWarps * kStages * 8;
};

// The workspace: for each block the unit that it begins and others end, {last
// block (-1: none), request, index in the request}; then a head and a tail
// partial of each block. Its size follows from the blocks launched, so nothing that
// the lengths hold leads outside it.
struct Part {
    int4 *dir;
    float2 *ml;   // [2 blocks][R]
    float *o;     // [2 blocks][R][D]
    int fill;     // blocks that the GPU holds at a time
};

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 3 : 2) kv8_stream_kernel(const __grid_constant__ CUtensorMap k_map,
                                                                                const __grid_constant__ CUtensorMap v_map,
                                                                                const Kv8AttnArgs a, const Part part)
{
    using L = Layout<D, NT>;
    constexpr int R = L::R;
    constexpr int kH = D / 64;      // 16-byte pieces of a lane's K row
    constexpr int kV = D / 8;       // bytes of a lane's V row
    constexpr int kM = D / 16;      // 16-row tiles of the value columns
    extern __shared__ __align__(1024) uint8_t smem[];
    float2 *s_ml = reinterpret_cast<float2 *>(smem + L::kBig);
    float4 *s_meta = reinterpret_cast<float4 *>(smem + L::kBig + kWarps * R * 8);
    uint32_t *s_nan = reinterpret_cast<uint32_t *>(smem + L::kBig + kWarps * R * 8 + kWarps * kStages * 32);
    // The block's place in the work, kept here and not in registers while a unit is worked on.
    __shared__ struct {
        long long at, hi;      // cost: where the block is, where its part ends
        long long base;        // cost before request b
        int b;
        Division cut;
        long long warp_cost[kWarps];
    } s_walk;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t4 = lane & 3;
    umma::grid_launch_dependents();

    if (tid == 0)
        part.dir[blockIdx.x] = make_int4(-1, 0, 0, 0);
    // The total cost and this block's part of it: each thread adds up its requests, the block scans the sums, and
    // the thread whose requests hold the part's begin finds the request.
    {
        const int per = (a.B + kThreads - 1) / kThreads;
        long long cost = 0;
        for (int i = 0; i < per; ++i) {
            const int b = tid * per + i;
            if (b < a.B) {
                const Units u = units_of<R>(a, request(a, b));
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
            s_walk.warp_cost[warp] = cost_to;
        __syncthreads();
        long long total = 0, cost0 = cost_to - cost;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            cost0 += w < warp ? s_walk.warp_cost[w] : 0;
            total += s_walk.warp_cost[w];
        }
        const Division cut = Division::of(total, part.fill, gridDim.x);
        if ((int)blockIdx.x >= cut.big + cut.small)
            return;
        const long long lo = cut.begin(blockIdx.x), hi = cut.begin(blockIdx.x + 1);
        if (lo >= hi)
            return;
        if (lo >= cost0 && lo < cost0 + cost) {
            int b = tid * per;
            Units u = units_of<R>(a, request(a, b));
            while (lo >= cost0 + u.count * u.cost) {
                cost0 += u.count * u.cost;
                u = units_of<R>(a, request(a, ++b));
            }
            s_walk.at = lo;
            s_walk.hi = hi;
            s_walk.base = cost0;
            s_walk.b = b;
            s_walk.cut = cut;
        }
    }
    const float scale_log2 = a.scale * kLog2e;
    const uint32_t full = smem_u32(smem + L::kBig + kWarps * R * 8 + kWarps * kStages * 32 + L::kNanWords * 4) + warp * kStages * 8;
    if (lane == 0) {
        for (int i = 0; i < kStages; ++i)
            umma::mbar_init(full + 8 * i, 1);
        umma::mbar_init_fence();
    }
    __syncwarp();
    uint32_t phases = 0; // bit i: the parity that stage i's next copies complete
    bool ok = (smem_u32(smem) & 1023u) == 0; // (the swizzle goes by address)
    if (!ok && tid == 0)
        atomicOr(&g_kv8_stream_error, 1);
    const int rows_in = min(kStep, a.block_size), pages = kStep / rows_in; // of a block in a step; blocks of a step
    const uint32_t ring = smem_u32(smem) + warp * kStages * L::kStageBytes;
    float4 *meta = s_meta + warp * kStages * 2;

    __syncthreads();
    while (s_walk.at < s_walk.hi) {
        long long at = s_walk.at, base = s_walk.base;
        int b = s_walk.b;
        Request rq = request(a, b);
        Units un = units_of<R>(a, rq);
        while (at >= base + un.count * un.cost) { // requests without tokens have no units
            base += un.count * un.cost;
            ++b;
            rq = request(a, b);
            un = units_of<R>(a, rq);
        }
        const long long ui = (at - base) / un.cost;
        const long long ubase = base + ui * un.cost;
        const long long uend = min(s_walk.hi, ubase + un.cost);
        const int s0 = (int)max(0ll, at - ubase - kUnitCost), s1 = (int)max(0ll, uend - ubase - kUnitCost);
        __syncthreads(); // all have read the place
        if (tid == 0) {
            s_walk.at = uend;
            s_walk.base = base;
            s_walk.b = b;
        }
        if (s0 >= s1) {
            __syncthreads();
            continue;
        }
        const bool whole = s0 == 0 && s1 == un.steps;
        if (s0 == 0 && !whole && tid == 0) // (the same thread as above)
            part.dir[blockIdx.x] = make_int4(s_walk.cut.part(ubase + un.cost - 1), b, (int)ui, 0);
        const int h = (int)(ui % a.H_kv);
        const int row0 = (int)(ui / a.H_kv) * R;
        const int rows = min(R, rq.qlen * a.G - row0);
        // the chunk's tokens and what its rows see
        const int p_first = rq.pos(row0 / a.G), p_last = rq.pos((row0 + rows - 1) / a.G);
        const int kv_end = min(rq.len, p_last + 1);                                    // beyond: seen by none
        const int kv_begin = a.window > 0 ? max(0, p_first - a.window + 1) : 0;
        const int all_from = a.window > 0 ? p_last - a.window + 1 : 0;                 // [all_from, p_first]: seen by all
        const bool many = p_first != p_last;

        // the lane's table entry, first + lane: its block (-1: none), the factor of its logits, log2 and
        // inverse of its value scale (a block outside the pool: logits of -inf, nothing is read)
        const int32_t *row = a.block_table + b * a.table_stride;
        int first = -(1 << 30);
        int e_blk = -1;
        float e_c = 0.f, e_lv = -INFINITY, e_iv = 1.f;
        // Position 8 i + tau(j) of a step is number j of its i-th eight: tau(2 t + e) = (2 t ^ 4 e) | e. The
        // rows of lanes g = 2 t and 2 t + 1 (K) then differ in bit 2, those of the four t (V) in bits 1 and
        // 2, so that with the swizzle eight lanes read eight different 16-byte columns.
        const int tau_g = ((g & 6) ^ (4 * (g & 1))) | (g & 1);
        const int tau_t[2] = {2 * t4, (2 * t4 ^ 4) | 1};

        auto issue = [&](int s, int stage) {
            if (s < s1) {
                const int tb = rq.begin + s * kStep;
                const int e = tb >> a.block_shift;
                if (e - first >= 31 || e < first) {
                    first = e;
                    const int x = e + lane;
                    e_blk = x < a.table_width && ((long long)x << a.block_shift) < rq.len ? row[x] : -1;
                    e_c = 0.f;
                    e_lv = -INFINITY;
                    e_iv = 1.f;
                    if (e_blk >= 0 && e_blk < a.num_blocks) {
                        const float vs = a.v_scale[(int64_t)e_blk * a.H_kv + h];
                        e_c = a.k_scale[(int64_t)e_blk * a.H_kv + h] * scale_log2;
                        e_lv = lg2_approx(vs);
                        e_iv = __frcp_rn(vs);
                    } else {
                        e_blk = -1;
                    }
                }
                if (lane == 0)
                    umma::mbar_arrive_expect_tx(full + 8 * stage, L::kStageBytes);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int ex = ((tb + 16 * x) >> a.block_shift) - first;
                    const float c = __shfl_sync(0xffffffffu, e_c, ex), lv = __shfl_sync(0xffffffffu, e_lv, ex),
                                iv = __shfl_sync(0xffffffffu, e_iv, ex);
                    // of 16 positions that no row sees (below the window, where a block may have gone to
                    // another request) the scales are not used: a bad one would reach the sums as 0 * NaN
                    const bool seen = tb + 16 * x + 15 >= kv_begin;
                    if (lane == 0)
                        meta[stage * 2 + x] = seen ? make_float4(c, lv, iv, 0.f) : make_float4(0.f, -INFINITY, 1.f, 0.f);
                }
                __syncwarp();
                // lanes p and 16 + p: block p of the step, for K and for V. A block outside the pool: rows
                // outside the map, which fills zeros and reads nothing.
                const int p = lane & 15;
                const int blk = __shfl_sync(0xffffffffu, e_blk, ((tb + (p < pages ? p : 0) * rows_in) >> a.block_shift) - first);
                if (p < pages)
                    tma_load_3d(ring + stage * L::kStageBytes + (lane >> 4) * L::kSide + p * rows_in * D,
                                      lane < 16 ? &k_map : &v_map, 0, blk >= 0 ? tb & (a.block_size - 1) : a.block_size,
                                      blk >= 0 ? blk * a.H_kv + h : 0, full + 8 * stage);
            }
        };

        for (int k = 0; ok && k < kStages; ++k)
            issue(s0 + warp + k * kWarps, k);

        // this lane's part of Q: fragment column g of each tile, and the factors of its columns 2 t4, 2 t4 + 1
        uint32_t qf[NT][2 * kH][2][2]; // k-step, part (hi, lo), register
        float qscale[NT];
        int pos[NT][2];
        float cscale[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = nt * 8 + g;
            uint4 v[kH][2];
            float amax = 0.f;
            const int rr = row0 + r;
            const __nv_bfloat16 *qr = static_cast<const __nv_bfloat16 *>(a.q) +
                                      (int64_t)(rq.q0 + (r < rows ? rr / a.G : 0)) * a.q_st +
                                      (int64_t)(h * a.G + (r < rows ? rr % a.G : 0)) * a.q_sh;
#pragma unroll
            for (int hh = 0; hh < kH; ++hh)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    v[hh][e] = r < rows ? *reinterpret_cast<const uint4 *>(qr + hh * 64 + t4 * 16 + e * 8)
                                        : make_uint4(0, 0, 0, 0);
                    amax = fmaxf(amax, amax8(v[hh][e]));
                }
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            float up;
            split_scale(amax, up, qscale[nt]);
#pragma unroll
            for (int hh = 0; hh < kH; ++hh)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    split8(v[hh][e], up, qf[nt][hh * 2 + e][0], qf[nt][hh * 2 + e][1]);
#pragma unroll
            for (int e2 = 0; e2 < 2; ++e2) {
                cscale[nt][e2] = __shfl_sync(0xffffffffu, qscale[nt], 4 * (2 * t4 + e2));
                const int rc = nt * 8 + 2 * t4 + e2;
                pos[nt][e2] = rc < rows ? rq.pos((row0 + rc) / a.G) : -1;
            }
        }

        float o[kM][NT][4];
        float m[NT][2], l[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int i = 0; i < kM; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o[i][nt][e] = 0.f;
        }
        if (many) {
            for (int i = tid; i < L::kNanWords; i += kThreads)
                s_nan[i] = 0;
            __syncthreads();
        }

        const int n_mine = (s1 - s0 - warp + kWarps - 1) / kWarps; // steps s0 + warp + 4 k
        for (int k = 0; ok && k < n_mine; ++k) {
            const int stage = k % kStages;
            ok = __all_sync(0xffffffffu, umma::mbar_wait(full + 8 * stage, phases >> stage & 1));
            if (!ok) {
                if (lane == 0)
                    atomicOr(&g_kv8_stream_error, 1);
                break;
            }
            phases ^= 1u << stage;
            const int s = s0 + warp + k * kWarps;
            const int tb = rq.begin + s * kStep;
            const uint32_t src = ring + stage * L::kStageBytes;

            float sc[2][NT][4];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float odd[NT][4]; // the low parts: two chains of products
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        sc[x][nt][e] = odd[nt][e] = 0.f;
                const int ra = 16 * x + tau_g; // the lane's rows: ra, ra + 8
#pragma unroll
                for (int hh = 0; hh < kH; ++hh) {
                    const uint32_t col = D == 128 ? ((t4 + 4 * hh) ^ (ra & 7)) * 16 : (t4 ^ ((ra >> 1) & 3)) * 16;
                    const uint4 ka = lds128(src + ra * D + col), kb = lds128(src + (ra + 8) * D + col);
                    const uint32_t f0[4] = {ka.x, kb.x, ka.y, kb.y}, f1[4] = {ka.z, kb.z, ka.w, kb.w};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma_e4m3_16832(sc[x][nt], f0, qf[nt][2 * hh][0][0], qf[nt][2 * hh][0][1]);
                        mma_e4m3_16832(odd[nt], f0, qf[nt][2 * hh][1][0], qf[nt][2 * hh][1][1]);
                        mma_e4m3_16832(sc[x][nt], f1, qf[nt][2 * hh + 1][0][0], qf[nt][2 * hh + 1][0][1]);
                        mma_e4m3_16832(odd[nt], f1, qf[nt][2 * hh + 1][1][0], qf[nt][2 * hh + 1][1][1]);
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        sc[x][nt][e] += odd[nt][e];
            }
            const float4 mt[2] = {meta[stage * 2], meta[stage * 2 + 1]};
            const bool clear = tb + kStep - 1 <= p_first && tb >= all_from && rows == R;
            bool raise = false;
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float y = fmaf(sc[x][nt][e], mt[x].x * cscale[nt][e & 1], mt[x].y);
                        if (!clear) {
                            const int j = tb + 16 * x + tau_g + 4 * (e & 2);
                            const int p = pos[nt][e & 1];
                            if (!(j <= p && (a.window <= 0 || j > p - a.window)))
                                y = -INFINITY;
                        }
                        sc[x][nt][e] = y;
                        raise |= y > __fadd_rd(m[nt][e & 1], kSlack); // (rounded so that no weight passes it, far out too)
                    }
            if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = fmaxf(fmaxf(sc[0][nt][e], sc[0][nt][e + 2]), fmaxf(sc[1][nt][e], sc[1][nt][e + 2]));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                        const float now = fmaxf(m[nt][e], __fadd_ru(x, -kTop));
                        const float f = m[nt][e] == -INFINITY ? 0.f : ex2_approx(m[nt][e] - now);
                        m[nt][e] = now;
                        l[nt][e] *= f;
#pragma unroll
                        for (int i = 0; i < kM; ++i) {
                            o[i][nt][e] *= f;
                            o[i][nt][e + 2] *= f;
                        }
                    }
            }
            uint32_t pf[2][NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float m0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0], m1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float p0 = ex2_approx(sc[x][nt][0] - m0), p1 = ex2_approx(sc[x][nt][1] - m1);
                    const float p2 = ex2_approx(sc[x][nt][2] - m0), p3 = ex2_approx(sc[x][nt][3] - m1);
                    l[nt][0] += (p0 + p2) * mt[x].z;
                    l[nt][1] += (p1 + p3) * mt[x].z;
                    pf[x][nt][0] = movmatrix_trans(pack_f16x2(p0, p1));
                    pf[x][nt][1] = movmatrix_trans(pack_f16x2(p2, p3));
                }
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                uint32_t vw[4][kV / 4];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const int r = 16 * x + 8 * (y >> 1) + tau_t[y & 1];
                    if (D == 128) {
                        const uint4 v = lds128(src + L::kSide + r * D + ((g ^ (r & 7)) << 4));
                        vw[y][0] = v.x;
                        vw[y][1] = v.y;
                        vw[y][(kV / 4) - 2] = v.z;
                        vw[y][(kV / 4) - 1] = v.w;
                    } else {
                        const uint2 v = lds64(src + L::kSide + r * D + (((g >> 1) ^ ((r >> 1) & 3)) << 4) + (g & 1) * 8);
                        vw[y][0] = v.x;
                        vw[y][1] = v.y;
                    }
                    // where no row sees the position the block may hold anything
                    if (!clear && !(tb + r < kv_end && tb + r >= kv_begin))
#pragma unroll
                        for (int w = 0; w < kV / 4; ++w)
                            vw[y][w] = 0;
                }
                // A NaN code of V at a position that some rows see and others do not
                // must not reach the others through 0 * NaN: it is taken out and
                // noted for the rows that see it.
                if (many && !clear) {
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const int j = tb + 16 * x + 8 * (y >> 1) + tau_t[y & 1];
#pragma unroll
                        for (int w = 0; w < kV / 4; ++w) {
                            const uint32_t bad = nan_bytes(vw[y][w]);
                            if (bad) {
                                for (int z = 0; z < 4; ++z)
                                    if (bad >> (8 * z + 7) & 1) {
                                        const int d = kV * g + 4 * w + z;
                                        for (int r = 0; r < rows; ++r) {
                                            const int p = rq.pos((row0 + r) / a.G);
                                            if (j <= p && (a.window <= 0 || j > p - a.window))
                                                atomicOr(&s_nan[(r * D + d) >> 5], 1u << (d & 31));
                                        }
                                    }
                                vw[y][w] &= ~((bad >> 7) * 0xFFu);
                            }
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < kM; ++i) {
                    // value columns kV g + 2 i (row g of the tile) and + 1 (row g + 8)
                    const int w = i >> 1;
                    uint32_t f[4];
                    const uint32_t sel = (i & 1) ? 0x7362 : 0x5140;
                    e4m3x4_to_f16x4(__byte_perm(vw[0][w], vw[1][w], sel), f[0], f[1]);
                    e4m3x4_to_f16x4(__byte_perm(vw[2][w], vw[3][w], sel), f[2], f[3]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma_f16_16816(o[i][nt], f, pf[x][nt][0], pf[x][nt][1]);
                }
            }
            // the stage is free: every lane has used what it read of it
            __syncwarp();
            issue(s0 + warp + (k + kStages) * kWarps, stage);
        }
        // the unit's end: the four warps' sums are joined through shared memory
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1)
                    l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], d);
                if (g == 0)
                    s_ml[warp * R + nt * 8 + 2 * t4 + e] = make_float2(m[nt][e], l[nt][e]);
            }
        __syncthreads(); // every warp is done with the ring
        float *so = reinterpret_cast<float *>(smem);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float *dst = so + (warp * R + nt * 8 + 2 * t4 + e) * D + kV * g;
#pragma unroll
                for (int i = 0; i < kM; i += 2)
                    *reinterpret_cast<float4 *>(dst + 2 * i) =
                        make_float4(o[i][nt][e], o[i][nt][e + 2], o[i + 1][nt][e], o[i + 1][nt][e + 2]);
            }
        __syncthreads();
        for (int x = tid; x < rows * (D / 4); x += kThreads) {
            const int r = x / (D / 4), d = (x % (D / 4)) * 4;
            float2 ml[kWarps];
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                ml[w] = s_ml[w * R + r];
                top = fmaxf(top, ml[w].x);
            }
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                // a warp that saw nothing has m = -inf; its sums are 0, or NaN from a NaN logit
                const float f = ml[w].x == -INFINITY ? 1.f : ex2_approx(ml[w].x - top);
                const float4 v = *reinterpret_cast<const float4 *>(so + (w * R + r) * D + d);
                sum += ml[w].y * f;
                acc.x += v.x * f;
                acc.y += v.y * f;
                acc.z += v.z * f;
                acc.w += v.w * f;
            }
            if (many) {
                const uint32_t bits = s_nan[(r * D + d) >> 5] >> (d & 31);
                acc.x = (bits & 1) ? NAN : acc.x;
                acc.y = (bits & 2) ? NAN : acc.y;
                acc.z = (bits & 4) ? NAN : acc.z;
                acc.w = (bits & 8) ? NAN : acc.w;
            }
            if (whole) {
                const int64_t t = rq.q0 + (row0 + r) / a.G;
                const int head = h * a.G + (row0 + r) % a.G;
                float lse;
                const float f = finish_row(top, sum, a.sinks, head, &lse);
                uint2 out2 = make_uint2(pack_bf16x2(acc.x * f, acc.y * f), pack_bf16x2(acc.z * f, acc.w * f));
                *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + (t * a.H + head) * D + d) = out2;
                if (a.lse && d == 0)
                    a.lse[t * a.H + head] = lse;
            } else {
                const int64_t slot = 2 * (int64_t)blockIdx.x + (s0 == 0 ? 1 : 0);
                *reinterpret_cast<float4 *>(part.o + (slot * R + r) * D + d) = acc;
                if (d == 0)
                    part.ml[slot * R + r] = make_float2(top, sum);
            }
        }
        // the ring and the sums are free again; what was written there is done before the next copies land
        umma::fence_async_smem();
        __syncthreads();
    }
    // no copy outlives the block, also where a wait gave up
    if (!ok)
        for (int i = 0; i < kStages; ++i)
            if (!umma::mbar_wait(full + 8 * i, phases >> i & 1) && lane == 0)
                atomicOr(&g_kv8_stream_error, 2);
}

// Joins the partial sums of the units that several blocks share: a block to a
// row, its warps take the parts in turn, and their sums are added in order.
constexpr int kJoinWarps = 4;
template <int D, int NT>
__global__ void __launch_bounds__(kJoinWarps * 32) kv8_join_kernel(const Kv8AttnArgs a, const Part part)
{
    constexpr int R = 8 * NT;
    constexpr int kD = D / 32; // columns of a lane
    __shared__ float s_acc[kJoinWarps][D];
    __shared__ float s_m[kJoinWarps], s_l[kJoinWarps];
    umma::grid_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int4 u = part.dir[blockIdx.x];
    const int c0 = blockIdx.x, c1 = u.x;
    if (c1 <= c0)
        return;
    const Request rq = request(a, u.y);
    const int h = u.z % a.H_kv, row0 = u.z / a.H_kv * R, r = blockIdx.y;
    if (r >= min(R, rq.qlen * a.G - row0))
        return;
    float m = -INFINITY, l = 0.f;
    for (int c = c0 + threadIdx.x; c <= c1; c += kJoinWarps * 32)
        m = fmaxf(m, part.ml[(2 * (int64_t)c + (c == c0)) * R + r].x);
    m = warp_max(m);
    if (lane == 0)
        s_m[warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w)
        m = fmaxf(m, s_m[w]);
    float acc[kD];
#pragma unroll
    for (int i = 0; i < kD; ++i)
        acc[i] = 0.f;
#pragma unroll 4
    for (int c = c0 + warp; c <= c1; c += kJoinWarps) {
        const int64_t slot = (2 * (int64_t)c + (c == c0)) * R + r;
        const float2 ml = part.ml[slot];
        const float f = ml.x == -INFINITY ? 1.f : ex2_approx(ml.x - m);
        l += ml.y * f;
        const float *src = part.o + slot * D + lane * kD;
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
#pragma unroll
    for (int i = 0; i < kD; ++i)
        s_acc[warp][lane * kD + i] = acc[i];
    if (lane == 0)
        s_l[warp] = l;
    __syncthreads();
    if (warp != 0)
        return;
#pragma unroll
    for (int w = 1; w < kJoinWarps; ++w) {
        l += s_l[w];
#pragma unroll
        for (int i = 0; i < kD; ++i)
            acc[i] += s_acc[w][lane * kD + i];
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

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

int fill_of(int NT, int sm_count) { return sm_count * (NT == 1 ? 3 : 2); }

struct Sizes {
    size_t ml, o, total;
};

// The most work that there can be decides the blocks: one without a part ends at once, but not for nothing.
int grid_of(int B, int T, int G, int H_kv, int NT, int64_t positions, int sm_count)
{
    const double units = ((double)T * G / (8 * NT) + B) * H_kv; // each request's last chunk may be short
    const double most = units * ((double)positions / kStep + kUnitCost + 1);
    const int fill = fill_of(NT, sm_count);
    if (most < (double)fill * kMinPart)
        return std::max(1, (int)(most / kMinPart) + 1);
    return most < 24.0 * kMinPart * fill ? fill : fill * (1 + kSmallPerBig); // (small parts only where they are work enough)
}

Sizes sizes(int D, int NT, size_t blocks)
{
    const int R = 8 * NT;
    Sizes s;
    s.ml = up256(blocks * sizeof(int4));
    s.o = up256(s.ml + 2 * blocks * R * sizeof(float2));
    s.total = s.o + 2 * blocks * R * D * sizeof(float);
    return s;
}

template <int D, int NT>
cudaError_t launch(const Kv8AttnArgs &a, void *workspace, int sm_count, cudaStream_t stream)
{
    using L = Layout<D, NT>;
    const int grid = grid_of(a.B, a.T, a.G, a.H_kv, NT, (int64_t)a.table_width << a.block_shift, sm_count);
    const Sizes sz = sizes(D, NT, grid);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const Part part{reinterpret_cast<int4 *>(ws), reinterpret_cast<float2 *>(ws + sz.ml), reinterpret_cast<float *>(ws + sz.o),
                    fill_of(NT, sm_count)};
    cudaError_t e = cudaFuncSetAttribute(kv8_stream_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
    if (e != cudaSuccess)
        return e;
    CUtensorMap maps[2];
    if (!kv8_tensor_maps(a, D, kStep, maps))
        return cudaErrorInvalidValue;
    kv8_stream_kernel<D, NT><<<grid, kThreads, L::kSmem, stream>>>(maps[0], maps[1], a, part);
    if ((e = cudaGetLastError()) != cudaSuccess)
        return e;
    if (grid == 1)
        return cudaSuccess; // (every unit is whole)
    // behind it, its start overlapped (it waits for the first kernel's end)
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 8 * NT);
    cfg.blockDim = dim3(kJoinWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv8_join_kernel<D, NT>, a, part);
}

// Query rows to a unit: 8, or 16 where the requests' rows fill more than 8.
int tiles_for(int G, int max_query_len) { return (int64_t)G * max_query_len > 8 ? 2 : 1; }

} // namespace

size_t kv8_stream_workspace(int B, int T, int G, int H_kv, int D, int max_query_len, int64_t positions, int sm_count)
{
    const int nt = tiles_for(G, max_query_len);
    return sizes(D, nt, grid_of(B, T, G, H_kv, nt, positions, sm_count)).total;
}

cudaError_t launch_kv8_stream(const Kv8AttnArgs &a, int D, int max_query_len, void *workspace, int sm_count,
                              cudaStream_t stream)
{
    const int nt = tiles_for(a.G, max_query_len);
    if (D == 128)
        return nt == 1 ? launch<128, 1>(a, workspace, sm_count, stream) : launch<128, 2>(a, workspace, sm_count, stream);
    return nt == 1 ? launch<64, 1>(a, workspace, sm_count, stream) : launch<64, 2>(a, workspace, sm_count, stream);
}

cudaError_t read_kv8_stream_error(int *out, bool reset)
{
    cudaError_t e = cudaMemcpyFromSymbol(out, g_kv8_stream_error, sizeof(int));
    if (e == cudaSuccess && reset) {
        const int zero = 0;
        e = cudaMemcpyToSymbol(g_kv8_stream_error, &zero, sizeof(int));
    }
    return e;
}

} // namespace smla

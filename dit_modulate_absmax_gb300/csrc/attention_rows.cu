// attention_rows.cu -- attention of few queries (decoding): a tile of 8 or 16
// rows against a part of the keys, joined afterwards where there are several
// parts.
//
// Reads every visible code once (2 * dim bytes a token and cache head) for each
// 16 rows, of which there are 32 at most, so it is bound by HBM.  What it takes to stay there:
//  - The keys are spread evenly over as many CTAs as fit; each of a CTA's 4
//    warps runs its own online softmax over units of 32 tokens, fed by its own
//    ring of TMA copies (one lane issues two a unit), with no barrier between
//    warps in the loop.
//  - Codes go from shared memory to registers as they lie and are converted to
//    FP16 there (exact) for mma.sync m16n8k16 with FP32 accumulation.  The
//    order of the contraction index is free, so a lane takes 4 adjacent
//    channels where the instruction wants (2t, 2t+1, 2t+8, 2t+9): S = Q K^T
//    reads each token's row in 16-byte pieces, and in O^T = V^T P^T a lane
//    reads 16 channels of its 4 tokens and pairs up tokens with byte
//    permutes.  S's accumulator layout is that product's B operand.
//  - The copies XOR-swizzle rows in 16-byte pieces (dim 128: no bank conflicts;
//    dim 64: two-way for the values).
// Measured: one sequence of 262,143 keys, 8 cache heads of 128 channels, 96 us
// (5.6 TB/s; 1,048,576 keys 6.6 TB/s), 32 ragged ones of up to 8,190 keys 75 us
// (4.6 TB/s): beyond the copying, a CTA's start, the copies that run dry where
// a CTA goes from one sequence to the next, and the join.
// The tensor work is small next to the memory's (24 instructions per 4 KB of
// codes at dim 128 and 8 rows), so the older warp-level instruction serves; a
// 128-row tcgen05 tile would be 8-16 times padding.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cstring>
#include <mutex>

#include "attention.cuh"
#include "ptx_attention.cuh"

namespace h3fp4 {
namespace {

__device__ uint32_t g_error;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kUnit = 32;                 // tokens a warp takes at a time
constexpr int kStages = 2;
constexpr int kMaxEntries = 512;          // pages of one part
// Weights are FP16 and stand against the row's maximum less this (log2): the largest is 2^15, below FP16's limit of nearly
// 2^16, one 2^-29 as large is still a normal number, one 2^-40 as large not yet nothing.
constexpr float kLift = 15.0f;

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Byte offset of 16-byte piece c of row r of a [32][kDim] tile as the tensor map's swizzle lays it.
template <int kDim>
__device__ __forceinline__ uint32_t piece(int r, int c)
{
    if (kDim == 128)
        return static_cast<uint32_t>(r * 128 + ((c ^ (r & 7)) << 4));
    return static_cast<uint32_t>(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

constexpr uint64_t kWaitNs = 2000000000ull;

// Adds a part's mean v times its share of the row's sum, half^2 inv: the square alone may be below the smallest number where
// v is very large.
__device__ __forceinline__ void join(float4 &mean, const float4 &v, float half, float inv)
{
    const float rest = half * inv;
    mean.x = fmaf(v.x * half, rest, mean.x);
    mean.y = fmaf(v.y * half, rest, mean.y);
    mean.z = fmaf(v.z * half, rest, mean.z);
    mean.w = fmaf(v.w * half, rest, mean.w);
}

// CTAs that fit an SM: shared memory at 128 channels, registers at 64.
template <int kDim, int kRows>
constexpr int resident()
{
    return kDim == 128 ? (kRows == 8 ? 3 : 2) : (kRows == 8 ? 4 : 3);
}

// Units of 128 tokens, one for each warp's 32, that a sequence's rows take: its
// share of the work for each cache head and row tile.  0: nothing to do.
struct Units {
    int begin, count, tiles;   // first token (a multiple of 32), units, row tiles
};

template <int kRows>
__device__ __forceinline__ Units units_of(const AttnArgs &a, const KvSequence &s)
{
    if (!s.ok || s.n == 0 || s.len > a.max_kv ||
        (s.len > 0 && ((s.len - 1) / a.cache.page_size >= a.batch.ld_table || a.cache.num_pages == 0)))
        return Units{0, 0, 0};   // (a cache without pages has no arrays either: nothing of it may be read)
    const Span first = seen_by(a, s, 0), last = seen_by(a, s, s.n - 1);
    const int begin = min(first.lo, last.lo) & ~(kUnit - 1), end = max(first.hi, last.hi);
    constexpr int kTokens = kWarps * kUnit;
    return Units{begin, max(1, (end - begin + kTokens - 1) / kTokens),   // rows that see nothing are written all the same
                 (s.n * (a.heads / a.cache.heads) + kRows - 1) / kRows};
}

// a / b of numbers that mostly fit 32 bits, where a division is several times shorter.
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b)
{
    if (((a | b) >> 32) == 0)
        return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// CTA i of g (g <= T) takes the units [i T / g, (i + 1) T / g) of T, the
// sequences one after another, within each its row tiles and cache heads.  The
// CTA of unit x:
__device__ __forceinline__ int64_t cta_of(int64_t x, int64_t g, int64_t total) { return divide((x + 1) * g - 1, total); }

// kWithhold: for a check that waits end.  Each copy is announced larger than it is, so that none completes.
template <int kDim, int kRows, bool kWithhold = false>
__global__ void __launch_bounds__(kThreads, resident<kDim, kRows>())
    rows_kernel(AttnArgs a, SplitPlan plan, float *ws_log, float *ws_out, const __grid_constant__ CUtensorMap k_map,
                const __grid_constant__ CUtensorMap v_map, uint64_t wait_ns)
{
    constexpr int kSteps = kDim / 16;            // k16 steps of Q K^T = 16-channel tiles of O^T
    constexpr int kHalf = kRows / 8;             // groups of 8 rows
    constexpr int kTile = kUnit * kDim;          // bytes of a unit's keys
    constexpr int kTokens = kWarps * kUnit;
    extern __shared__ __align__(1024) uint8_t dyn[];
    __shared__ PageEntry entry[kMaxEntries];
    __shared__ uint64_t full[kWarps][kStages];
    __shared__ float part_log[kWarps][16];       // a warp's log2 of the sum of each row
    __shared__ float sum_ref[kWarps][16];        // with far scales: what a warp's sum of a row is kept against
    __shared__ int64_t warp_units[kWarps], found_rest;
    __shared__ int found_b;

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int page = a.cache.page_size, group = a.heads / a.cache.heads, heads = a.cache.heads;
    const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(dyn)) + warp * (kStages * 2 * kTile);
    const int box = min(page, kUnit), shift = 31 - __clz(page);
    if (lane == 0)
        for (int i = 0; i < kStages; ++i)
            mbar_init(smem_u32(&full[warp][i]), 1);
    fence_mbar_init();
    if (threadIdx.x == 0 && a.cache.num_pages > 0) {   // (without pages there are no maps)
        prefetch_tmap(&k_map);
        prefetch_tmap(&v_map);
    }
    // The join's CTAs may come as places fall free; they wait for this grid's end before they read its parts.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    int64_t x = 0, x_end = 1;                    // units to do
    // Each thread counts the units of a share of the sequences (one, mostly), [mine_lo, mine_hi) of all.
    const int share = (a.batch.batch + kThreads - 1) / kThreads;
    int64_t mine_lo = 0, mine_hi = 0;
    if (!plan.cluster) {
        int64_t mine = 0;
        for (int b = threadIdx.x * share; b < min(a.batch.batch, (static_cast<int>(threadIdx.x) + 1) * share); ++b) {
            const KvSequence s = kv_sequence(a.batch, b, a.tokens);
            const Units u = units_of<kRows>(a, s);
            mine += static_cast<int64_t>(u.count) * u.tiles * heads;
            if (u.count == 0 && s.n != 0 && blockIdx.x == 0)
                atomicOr(&g_error, ERR_KV_RANGE);
        }
        mine_hi = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xFFFFFFFFu, mine_hi, o);
            mine_hi += lane >= o ? y : 0;
        }
        if (lane == 31)
            warp_units[warp] = mine_hi;
        __syncthreads();
        int64_t total = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            mine_hi += w < warp ? warp_units[w] : 0;
            total += warp_units[w];
        }
        mine_lo = mine_hi - mine;
        const int64_t takers = min(static_cast<int64_t>(gridDim.x), total);   // every one of them has a unit
        x_end = 0;
        if (blockIdx.x < takers) {
            x = divide(blockIdx.x * total, takers);
            x_end = divide((blockIdx.x + 1) * total, takers);
        }
    }
    int stage = 0;
    uint32_t parity = 0;
    bool ok = true;   // of a warp: no wait has given up
    const int64_t x_first = x;
    while (x < x_end) {   // the same in every thread
    // The segment that unit x begins: a sequence, a row tile, a cache head and tokens [seg_begin, seg_end).
    int b, tile, kh, seg_begin, seg_end;
    bool whole = true;
    int64_t next = x_end;
    KvSequence s;
    if (plan.cluster) {   // one unit a CTA, a cluster for the rows of a sequence and cache head
        b = blockIdx.y;
        tile = 0;
        kh = blockIdx.x / plan.splits;
        s = kv_sequence(a.batch, b, a.tokens);
        const Units u = units_of<kRows>(a, s);
        if (u.count == 0) {   // the same in the whole cluster
            if (s.n != 0 && threadIdx.x == 0)
                atomicOr(&g_error, ERR_KV_RANGE);
            return;
        }
        __syncthreads();      // barriers initialised
        seg_begin = u.begin + blockIdx.x % plan.splits * kTokens;
        seg_end = seg_begin + kTokens;
    } else {
        if (mine_lo <= x && x < mine_hi) {   // one thread: in its share, which sequence
            int64_t rest = x - mine_lo;
            int at = threadIdx.x * share;
            if (share > 1)
                for (;; ++at) {
                    const Units v = units_of<kRows>(a, kv_sequence(a.batch, at, a.tokens));
                    const int64_t n = static_cast<int64_t>(v.count) * v.tiles * heads;
                    if (rest < n)
                        break;
                    rest -= n;
                }
            found_b = at;
            found_rest = rest;
        }
        __syncthreads();
        b = found_b;
        const int64_t rest = found_rest;
        s = kv_sequence(a.batch, b, a.tokens);
        const Units u = units_of<kRows>(a, s);
        const int item = static_cast<int>(divide(rest, u.count)), u0 = static_cast<int>(rest - static_cast<int64_t>(item) * u.count);
        const int u1 = static_cast<int>(min(static_cast<int64_t>(u.count), u0 + (x_end - x)));
        kh = item % heads;
        tile = item / heads;
        seg_begin = u.begin + u0 * kTokens;
        seg_end = u.begin + u1 * kTokens;
        whole = u0 == 0 && u1 == u.count;
        next = x + (u1 - u0);
    }
    const int rows = s.n * group, row0 = tile * kRows;   // rows of this kernel are few: no overflow
    // what the tile's first and last rows see bounds what all of them see
    const Span first = seen_by(a, s, row0 / group), last = seen_by(a, s, min(rows - 1, row0 + kRows - 1) / group);
    const int in_lo = max(first.lo, last.lo), in_hi = min(first.hi, last.hi);   // seen by every row
    const int out_lo = min(first.lo, last.lo), out_hi = max(first.hi, last.hi); // seen by any
    seg_begin = max(seg_begin, out_lo & ~(kUnit - 1));
    seg_end = min(seg_end, out_hi);
    // The first pages' numbers are on their way while the queries are read.
    const int first_page = (seg_begin >> shift) + threadIdx.x;
    const int32_t first_id = seg_begin < seg_end && first_page <= (seg_end - 1) >> shift
                                 ? a.batch.page_table[b * a.batch.ld_table + first_page] : 0;

    // Q: rows g and g + 8; this lane's channels kDim/4 * t ...
    uint32_t q[kSteps][4];
    float c_row[kHalf];
    Span see[kHalf];
#pragma unroll
    for (int hf = 0; hf < kHalf; ++hf) {
        const int r = row0 + g + 8 * hf;
        const bool live = r < rows;
        const uint16_t *src = a.q + (s.row + (live ? r / group : 0)) * a.qt + (kh * group + (live ? r % group : 0)) * a.qh +
                              (kDim / 4) * t;
        uint32_t w[kDim / 8], m2 = 0;
#pragma unroll
        for (int i = 0; i < kDim / 32; ++i) {
            const uint4 v = live ? *reinterpret_cast<const uint4 *>(src + 8 * i) : make_uint4(0, 0, 0, 0);
            w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
        }
#pragma unroll
        for (int i = 0; i < kDim / 8; ++i)
            m2 = bf16x2_absmax(m2, w[i]);
        uint32_t amax = max(m2 & 0xFFFFu, m2 >> 16);
        amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
        const float2 p = row_power(amax);
        const float f = a.scale < 0.0f ? -p.x : p.x;
#pragma unroll
        for (int st = 0; st < kSteps; ++st) {
            q[st][hf] = bf16x2_to_half2(w[2 * st], f);
            q[st][hf + 2] = bf16x2_to_half2(w[2 * st + 1], f);
            if (kHalf == 1)
                q[st][1] = q[st][3] = 0u;
        }
        c_row[hf] = fabsf(a.scale) * kLog2e * p.y;
        see[hf] = live ? seen_by(a, s, r / group) : Span{0, 0};
    }
    float o[kHalf][kSteps][4];
    float m[kHalf], l[kHalf];
#pragma unroll
    for (int hf = 0; hf < kHalf; ++hf) {
        m[hf] = -INFINITY;
        l[hf] = 0.0f;
#pragma unroll
        for (int j = 0; j < kSteps; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o[hf][j][e] = 0.0f;
    }


    // In parts whose pages fit the table: their entries, the first copies, then the scales.
    bool far_scales = false;   // the same in the whole CTA
    constexpr int kCap = (kMaxEntries - 2) * 16 / kTokens * kTokens;
    for (int begin = seg_begin; begin < seg_end; begin += kCap) {
    const int end = min(seg_end, begin + kCap);
    const int page0 = begin >> shift, pages = ((end - 1) >> shift) - page0 + 1;
    if (__syncthreads_or(!ok))   // the last part's readers are done
        break;
    for (int i = threadIdx.x; i < pages; i += kThreads) {
        int32_t id = begin == seg_begin && i < kThreads ? first_id : a.batch.page_table[b * a.batch.ld_table + page0 + i];
        // Units begin at multiples of 32 tokens, so that a page of 16 may lie before all that the rows see: whatever the
        // table holds for it (it may be given up under a window), it is not copied.
        if ((page0 + i + 1) << shift <= out_lo) {
            id = -1;
        } else if (id < 0 || id >= a.cache.num_pages) {
            atomicOr(&g_error, ERR_KV_RANGE);
            id = -1;
        }
        entry[i].id = id;
    }
    __syncthreads();
    const auto fetch = [&](int unit, int stage) {   // one lane; unit: first token, below end
        const uint32_t bar = smem_u32(&full[warp][stage]), dst = ring + stage * (2 * kTile);
        const int at = (unit >> shift) - page0;
        const int32_t id0 = entry[at].id, id1 = page < kUnit && unit + page < end ? entry[at + 1].id : -1;
        mbar_arrive_expect_tx(bar, ((id0 >= 0) + (id1 >= 0)) * 2 * box * kDim + (kWithhold ? 16 : 0));
        if (id0 >= 0) {
            tma_load_3d(dst, &k_map, 0, unit & (page - 1), id0 * heads + kh, bar);
            tma_load_3d(dst + kTile, &v_map, 0, unit & (page - 1), id0 * heads + kh, bar);
        }
        if (id1 >= 0) {
            tma_load_3d(dst + kTile / 2, &k_map, 0, 0, id1 * heads + kh, bar);
            tma_load_3d(dst + kTile + kTile / 2, &v_map, 0, 0, id1 * heads + kh, bar);
        }
    };
    const int unit0 = begin + warp * kUnit;
    if (lane == 0)
        for (int i = 0; i < kStages; ++i)
            if (unit0 + i * kTokens < end)
                fetch(unit0 + i * kTokens, (stage + i) % kStages);
    bool far = false;
    for (int i = threadIdx.x; i < pages; i += kThreads) {
        const int32_t id = entry[i].id;
        const int64_t bh = static_cast<int64_t>(id) * heads + kh;
        const float vs = id >= 0 ? a.cache.v_scale[bh] : 1.0f;
        entry[i].ks = id >= 0 ? a.cache.k_scale[bh] : 1.0f;
        const float lv = lg2(vs);
        entry[i].lv = lv;
        entry[i].inv_vs = ex2(-lv);
        far = far || far_scale(vs);
    }
    if (__syncthreads_or(far) && !far_scales) {   // scales are there
        far_scales = true;
#pragma unroll
        for (int hf = 0; hf < kHalf; ++hf) {   // the sum so far, kept against m, becomes 1 against its logarithm
            l[hf] += __shfl_xor_sync(0xFFFFFFFFu, l[hf], 1);
            l[hf] += __shfl_xor_sync(0xFFFFFFFFu, l[hf], 2);
            if (t == 0)
                sum_ref[warp][g + 8 * hf] = log_of_sum(m[hf], l[hf]);
            l[hf] = t == 0 ? own_sum(l[hf]) : 0.0f;
        }
        __syncwarp();
    }
    for (int unit = unit0; unit < end; unit += kTokens) {
        if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded(smem_u32(&full[warp][stage]), parity, wait_ns))) {
            // The copies have not come: the CTA ends, once those of this warp that are on their way had as long again.
            ok = false;
            const int other = (stage + 1) % kStages;
            mbar_wait_bounded(smem_u32(&full[warp][stage]), parity, wait_ns);
            if (unit + kTokens < end)
                mbar_wait_bounded(smem_u32(&full[warp][other]), parity ^ (other == 0), wait_ns);
            break;
        }
        const uint8_t *kt = dyn + warp * (kStages * 2 * kTile) + stage * (2 * kTile), *vt = kt + kTile;

        float sc[4][4];   // S of the unit's four groups of 8 tokens
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            uint32_t w[kDim / 16];
#pragma unroll
            for (int i = 0; i < kDim / 64; ++i) {
                const uint4 v = *reinterpret_cast<const uint4 *>(kt + piece<kDim>(8 * n + g, (kDim / 64) * t + i));
                w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
            }
            sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.0f;
#pragma unroll
            for (int st = 0; st < kSteps; ++st)
            {
                const uint2 kb = e4m3x4_to_f16x4(w[st]);
                mma_f16(sc[n], q[st], kb.x, kb.y);
            }
        }

        const bool edge = unit < in_lo || unit + kUnit > in_hi;
        float top[kHalf];
#pragma unroll
        for (int hf = 0; hf < kHalf; ++hf)
            top[hf] = -INFINITY;
        const int e0 = (unit >> shift) - page0, e1 = min(pages - 1, ((unit + 16) >> shift) - page0);
        const PageEntry pe[2] = {entry[e0], entry[e1]};
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int hf = 0; hf < kHalf; ++hf)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float &v = sc[n][2 * hf + e];
                    v = fmaf(v, c_row[hf] * pe[n >> 1].ks, pe[n >> 1].lv);
                    if (edge) {
                        const int tok = unit + 8 * n + 2 * t + e;
                        if (tok < see[hf].lo || tok >= see[hf].hi)
                            v = -INFINITY;
                    }
                    top[hf] = fmaxf(top[hf], v);
                }
        bool grew = false;
        float keep[kHalf], ref[kHalf];
#pragma unroll
        for (int hf = 0; hf < kHalf; ++hf) {
            top[hf] = fmaxf(top[hf], __shfl_xor_sync(0xFFFFFFFFu, top[hf], 1));
            top[hf] = fmaxf(top[hf], __shfl_xor_sync(0xFFFFFFFFu, top[hf], 2));
            const float mm = fmaxf(m[hf], fabsf(top[hf]) < 0x1p22f ? top[hf] - kLift : top[hf]);   // (exact, or not at all)
            ref[hf] = mm == -INFINITY ? 0.0f : mm;
            keep[hf] = ex2(m[hf] - ref[hf]);
            grew |= mm > m[hf];
            m[hf] = mm;
        }
        if (__any_sync(0xFFFFFFFFu, grew)) {
#pragma unroll
            for (int hf = 0; hf < kHalf; ++hf) {
                l[hf] *= far_scales ? 1.0f : keep[hf];
                // the accumulator holds rows 2t and 2t + 1, whose factors are in lanes 8t and 8t + 4
                const float f0 = __shfl_sync(0xFFFFFFFFu, keep[hf], 8 * t), f1 = __shfl_sync(0xFFFFFFFFu, keep[hf], 8 * t + 4);
#pragma unroll
                for (int j = 0; j < kSteps; ++j) {
                    o[hf][j][0] *= f0;
                    o[hf][j][1] *= f1;
                    o[hf][j][2] *= f0;
                    o[hf][j][3] *= f1;
                }
            }
        }
        if (far_scales) {
#pragma unroll
            for (int hf = 0; hf < kHalf; ++hf) {
                float u = -INFINITY, sum = 0.0f;
#pragma unroll
                for (int n = 0; n < 4; ++n)
                    u = fmaxf(u, fmaxf(sc[n][2 * hf], sc[n][2 * hf + 1]) - pe[n >> 1].lv);
                u = fmaxf(u, __shfl_xor_sync(0xFFFFFFFFu, u, 1));
                u = fmaxf(u, __shfl_xor_sync(0xFFFFFFFFu, u, 2));
                float &kept = sum_ref[warp][g + 8 * hf];
                const float was = kept, next = fmaxf(was, u), base = next == -INFINITY ? 0.0f : next;
#pragma unroll
                for (int n = 0; n < 4; ++n)
                    sum += ex2(sc[n][2 * hf] - pe[n >> 1].lv - base) + ex2(sc[n][2 * hf + 1] - pe[n >> 1].lv - base);
                l[hf] = fmaf(l[hf], ex2(was - base), sum);
                __syncwarp();
                if (t == 0)
                    kept = next;
                __syncwarp();
            }
        }
        uint32_t pb[kHalf][4];   // weights of the four token groups, FP16 pairs
#pragma unroll
        for (int hf = 0; hf < kHalf; ++hf) {
#pragma unroll
            for (int n2 = 0; n2 < 2; ++n2) {
                float sum = 0.0f;
#pragma unroll
                for (int n = 2 * n2; n < 2 * n2 + 2; ++n) {
                    const float p0 = ex2(sc[n][2 * hf] - ref[hf]), p1 = ex2(sc[n][2 * hf + 1] - ref[hf]);
                    sum += p0 + p1;
                    pb[hf][n] = pack_half2(p0, p1);
                }
                if (!far_scales)
                    l[hf] = fmaf(sum, pe[n2].inv_vs, l[hf]);
            }
        }

#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {   // 16 tokens at a time
            constexpr int kW = kDim / 32;  // words of 4 channels per token: this lane's kDim/8 channels
            uint32_t w[4][kW];
            uint32_t odd = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 16 * hh + 2 * t + (i & 1) + 8 * (i >> 1);
                if constexpr (kDim == 128) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(vt + piece<kDim>(r, g));
                    w[i][0] = v.x; w[i][1] = v.y; w[i][2] = v.z; w[i][3] = v.w;
                } else {
                    const uint2 v = *reinterpret_cast<const uint2 *>(vt + piece<kDim>(r, g >> 1) + 8 * (g & 1));
                    w[i][0] = v.x; w[i][1] = v.y;
                }
                if (edge) {   // codes that no row sees may be anything: zeros
                    const int tok = unit + r;
                    const uint32_t mask = tok >= out_lo && tok < out_hi ? 0xFFFFFFFFu : 0u;
#pragma unroll
                    for (int x = 0; x < kW; ++x) {
                        w[i][x] &= mask;
                        odd |= nan_bytes(w[i][x]);
                    }
                }
            }
            // NaN among tokens that some rows see and others do not: a zero weight would not keep it out.  The NaN
            // codes leave the product, and a product of two masks counts the NaNs that each row and channel sees.
            const bool slow = edge && __any_sync(0xFFFFFFFFu, odd != 0);
#pragma unroll
            for (int x = 0; x < kW; ++x) {
                // bytes of 4 tokens per channel: a 4 x 4 byte transpose
                const uint32_t a01 = __byte_perm(w[0][x], w[1][x], 0x5140), b01 = __byte_perm(w[0][x], w[1][x], 0x7362);
                const uint32_t a23 = __byte_perm(w[2][x], w[3][x], 0x5140), b23 = __byte_perm(w[2][x], w[3][x], 0x7362);
                const uint32_t ch[4] = {__byte_perm(a01, a23, 0x5410), __byte_perm(a01, a23, 0x7632),
                                        __byte_perm(b01, b23, 0x5410), __byte_perm(b01, b23, 0x7632)};
#pragma unroll
                for (int j2 = 0; j2 < 2; ++j2) {
                    uint32_t c0 = ch[2 * j2], c1 = ch[2 * j2 + 1];
                    const int j = 2 * x + j2;
                    if (slow) {
                        const uint32_t n0 = nan_bytes(c0) >> 7, n1 = nan_bytes(c1) >> 7;   // 1 in each NaN byte
                        c0 &= ~(n0 * 0xFFu);
                        c1 &= ~(n1 * 0xFFu);
                        const auto ones = [](uint32_t n) { return ((n & 1u) | (n >> 8 & 1u) << 16) * 0x3C00u; };
                        const uint32_t na[4] = {ones(n0), ones(n1), ones(n0 >> 16), ones(n1 >> 16)};
#pragma unroll
                        for (int hf = 0; hf < kHalf; ++hf) {
                            uint32_t vis[2];
#pragma unroll
                            for (int n = 0; n < 2; ++n) {
                                const int tok = unit + 16 * hh + 8 * n + 2 * t;
                                vis[n] = (tok >= see[hf].lo && tok < see[hf].hi ? 0x3C00u : 0u) |
                                         (tok + 1 >= see[hf].lo && tok + 1 < see[hf].hi ? 0x3C000000u : 0u);
                            }
                            float cnt[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                            mma_f16(cnt, na, vis[0], vis[1]);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (cnt[e] > 0.0f)
                                    o[hf][j][e] = __uint_as_float(0x7FC00000u);
                        }
                    }
                    const uint2 v0 = e4m3x4_to_f16x4(c0), v1 = e4m3x4_to_f16x4(c1);
                    const uint32_t av[4] = {v0.x, v1.x, v0.y, v1.y};
#pragma unroll
                    for (int hf = 0; hf < kHalf; ++hf)
                        mma_f16(o[hf][j], av, pb[hf][2 * hh], pb[hf][2 * hh + 1]);
                }
            }
        }
        __syncwarp();   // every lane has read the stage that the next copies overwrite
        if (lane == 0 && unit + kStages * kTokens < end)
            fetch(unit + kStages * kTokens, stage);
        stage = stage + 1 == kStages ? 0 : stage + 1;
        parity ^= stage == 0;
    }
    }   // of the segment

    // Join the warps: each one's mean and the logarithm of its sum, the means through shared memory (the rings are drained).
#pragma unroll
    for (int hf = 0; hf < kHalf; ++hf) {
        l[hf] += __shfl_xor_sync(0xFFFFFFFFu, l[hf], 1);
        l[hf] += __shfl_xor_sync(0xFFFFFFFFu, l[hf], 2);
        const float ref = far_scales ? sum_ref[warp][g + 8 * hf] : m[hf];
        const float inv = reciprocal_sum(l[hf]) * (far_scales && l[hf] > 0.0f ? ex2(m[hf] - ref) : 1.0f);
        if (t == 0)
            part_log[warp][g + 8 * hf] = log_of_sum(ref, l[hf]);
        const float f0 = __shfl_sync(0xFFFFFFFFu, inv, 8 * t), f1 = __shfl_sync(0xFFFFFFFFu, inv, 8 * t + 4);   // as above
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
            o[hf][j][0] *= f0;
            o[hf][j][1] *= f1;
            o[hf][j][2] *= f0;
            o[hf][j][3] *= f1;
        }
    }
    if (__syncthreads_or(!ok)) {   // the same in the whole CTA; what it would have written stays as it was
        if (threadIdx.x == 0)
            atomicOr(&g_error, ERR_ATTN_WAIT);
        if (plan.cluster) {
            cluster_sync();
            cluster_sync();
        }
        return;
    }
    float *part = reinterpret_cast<float *>(dyn);   // [warp][row][kDim]
#pragma unroll
    for (int hf = 0; hf < kHalf; ++hf)
#pragma unroll
        for (int j = 0; j < kSteps; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e)   // channels (kDim/8) g + 2j and + 1
                *reinterpret_cast<float2 *>(part + (warp * kRows + 8 * hf + 2 * t + e) * kDim + (kDim / 8) * g + 2 * j) =
                    make_float2(o[hf][j][e], o[hf][j][e + 2]);
    __syncthreads();
    float *joined = part + kWarps * kRows * kDim;                                 // [row][kDim], with a cluster
    float *joined_log = joined + kRows * kDim;                                    // [row]
    const auto finish = [&](int r, int c, float log, float4 mean) {
        const int64_t row = s.row + (row0 + r) / group;
        const int head = kh * group + (row0 + r) % group;
        const __nv_bfloat162 x = __floats2bfloat162_rn(mean.x, mean.y), y = __floats2bfloat162_rn(mean.z, mean.w);
        *reinterpret_cast<uint2 *>(a.out + row * a.ot + head * a.oh + c) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y));
        if (a.lse != nullptr && c == 0)
            a.lse[row * a.heads + head] = log * kLn2;
    };
    for (int i = threadIdx.x; i < kRows * (kDim / 4); i += kThreads) {
        const int r = i / (kDim / 4), c = (i % (kDim / 4)) * 4;
        if (row0 + r >= rows)
            continue;
        float top = part_log[0][r], total = 0.0f;
#pragma unroll
        for (int w = 1; w < kWarps; ++w)
            top = fmaxf(top, part_log[w][r]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            total += of_top(part_log[w][r], top);
        const float inv = reciprocal_sum(total), log = log_of_sum(top, total);
        float4 mean = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            join(mean, *reinterpret_cast<const float4 *>(part + (w * kRows + r) * kDim + c), half_of_top(part_log[w][r], top), inv);
        if (plan.cluster) {
            *reinterpret_cast<float4 *>(joined + r * kDim + c) = mean;
            if (c == 0)
                joined_log[r] = log;
        } else if (whole) {
            finish(r, c, log, mean);
        } else {   // a CTA's first segment goes to its first place, another (its last) to the second
            const int64_t at = (blockIdx.x * 2 + (x != x_first)) * kRows + r;
            *reinterpret_cast<float4 *>(ws_out + at * kDim + c) = mean;
            if (c == 0)
                ws_log[at] = log;
        }
    }
    if (plan.cluster) {   // each CTA joins a share of the rows' pieces over all parts
        cluster_sync();
        const uint32_t j0 = smem_u32(joined), s0 = smem_u32(joined_log);
        for (int i = (blockIdx.x % plan.splits) * kThreads + threadIdx.x; i < kRows * (kDim / 4); i += kThreads * plan.splits) {
            const int r = i / (kDim / 4), c = (i % (kDim / 4)) * 4;
            if (row0 + r >= rows)
                continue;
            float top = -INFINITY, total = 0.0f;
            for (int p = 0; p < plan.splits; ++p)
                top = fmaxf(top, ld_cluster_f32(mapa_shared(s0 + 4 * r, p)));
            for (int p = 0; p < plan.splits; ++p)
                total += of_top(ld_cluster_f32(mapa_shared(s0 + 4 * r, p)), top);
            const float inv = reciprocal_sum(total);
            float4 mean = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int p = 0; p < plan.splits; ++p)
                join(mean, ld_cluster_v4(mapa_shared(j0 + (r * kDim + c) * 4, p)),
                     half_of_top(ld_cluster_f32(mapa_shared(s0 + 4 * r, p)), top), inv);
            finish(r, c, log_of_sum(top, total), mean);
        }
        cluster_sync();   // nobody leaves while its part may be read
    }
    x = next;
    fence_proxy_async_smem();   // the join's plain accesses come before the next segment's copies to the same place
    __syncthreads();
    }
}

constexpr int kJoinThreads = 1024;

// Joins the parts of the rows whose units lie with several CTAs: a CTA for each
// sequence, row tile and cache head, a thread for 4 channels of a row and every
// kGroups-th part (one long request has as many parts as there are CTAs for a
// cache head, 57 at 8 of them: one warp a row took 15 us over those).
template <int kDim, int kRows>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(AttnArgs a, int ctas, const float *ws_log, const float *ws_out)
{
    constexpr int kPieces = kRows * kDim / 4;
    constexpr int kGroups = kJoinThreads / kPieces;
    __shared__ float4 means[kGroups][kPieces];
    const int lane = threadIdx.x & 31, b = blockIdx.y, group = a.heads / a.cache.heads;
    const int kh = blockIdx.x % a.cache.heads, tile = blockIdx.x / a.cache.heads;
    const KvSequence s = kv_sequence(a.batch, b, a.tokens);   // (not written by the kernel before)
    const Units u = units_of<kRows>(a, s);
    int64_t ahead = 0, total = 0;   // units of the sequences before this one, and of all
    for (int i = lane; i < a.batch.batch; i += 32) {
        const Units v = units_of<kRows>(a, kv_sequence(a.batch, i, a.tokens));
        const int64_t n = static_cast<int64_t>(v.count) * v.tiles * a.cache.heads;
        total += n;
        ahead += i < b ? n : 0;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
        ahead += __shfl_xor_sync(0xFFFFFFFFu, ahead, o);
    }
    int64_t c0 = 0, c1 = 0, slot0 = 0;
    const bool mine = u.count > 0 && tile < u.tiles;
    if (mine) {
        const int64_t x0 = ahead + (static_cast<int64_t>(tile) * a.cache.heads + kh) * u.count;
        const int64_t takers = min(static_cast<int64_t>(ctas), total);
        c0 = cta_of(x0, takers, total);
        c1 = cta_of(x0 + u.count - 1, takers, total);
        slot0 = c0 * 2 + (divide(c0 * total, takers) != x0);   // the first part may be its CTA's second segment
    }
    // Every thread waits here until the parts are written: this grid must not end before the one that it followed.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (c0 == c1)
        return;   // nothing, or one CTA had them all and has written the output
    const int part0 = threadIdx.x / kPieces, piece = threadIdx.x % kPieces, r = piece / (kDim / 4), c = piece % (kDim / 4) * 4;
    const int row_in = tile * kRows + r;
    const bool live = row_in < s.n * group;
    const auto place = [&](int64_t p) { return (p == c0 ? slot0 : p * 2) * kRows + r; };
    float top = -INFINITY, sum = 0.0f;   // of the row's logarithms: their maximum, and the sum against it
    if (live) {
        for (int64_t p = c0 + lane % (kDim / 4); p <= c1; p += kDim / 4)   // a row's lanes: kDim / 4 neighbours
            add_log(top, sum, ws_log[place(p)], 1.0f);
    }
#pragma unroll
    for (int o = kDim / 8; o > 0; o >>= 1) {
        const float other = __shfl_xor_sync(0xFFFFFFFFu, top, o), its = __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        add_log(top, sum, other, its);
    }
    const float inv = reciprocal_sum(sum);
    float4 mean = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (live) {
#pragma unroll 8
        for (int64_t p = c0 + part0; p <= c1; p += kGroups)
            join(mean, *reinterpret_cast<const float4 *>(ws_out + place(p) * kDim + c), half_of_top(ws_log[place(p)], top), inv);
    }
    if (kGroups > 1) {
        means[part0][piece] = mean;
        __syncthreads();
        if (part0 > 0)
            return;
#pragma unroll
        for (int i = 1; i < kGroups; ++i) {
            const float4 v = means[i][piece];
            mean = make_float4(mean.x + v.x, mean.y + v.y, mean.z + v.z, mean.w + v.w);
        }
    }
    if (!live)
        return;
    const int64_t row = s.row + row_in / group;
    const int head = kh * group + row_in % group;
    const __nv_bfloat162 x = __floats2bfloat162_rn(mean.x, mean.y), y = __floats2bfloat162_rn(mean.z, mean.w);
    *reinterpret_cast<uint2 *>(a.out + row * a.ot + head * a.oh + c) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y));
    if (a.lse != nullptr && c == 0)
        a.lse[row * a.heads + head] = log_of_sum(top, sum) * kLn2;
}

}  // namespace

// Two ways to spread the keys.
// Small calls, where each unit of 128 tokens can have a CTA of its own and a
// row has 8 units at most: a cluster a row, joined over its shared memory.  No
// workspace and no second launch (one request of 777 keys, 56 heads: 12.4 us
// against 14.5).
// Others: as many CTAs as the SMs hold, each with an equal share of all units,
// whatever the lengths of the batch (equal parts per sequence, sized for the
// longest, left SMs idle: 32 ragged requests took 87 us, then 73); rows that
// lie with several CTAs are joined by a second kernel.
SplitPlan plan_rows(const AttnShape &s)
{
    const int64_t rows = static_cast<int64_t>(s.max_tokens) * (s.heads / s.kv_heads);
    const int64_t tile = rows <= 8 ? 8 : 16;
    const int64_t fit = sm_count() * (s.head_dim == 128 ? (tile == 8 ? resident<128, 8>() : resident<128, 16>())
                                                        : (tile == 8 ? resident<64, 8>() : resident<64, 16>()));
    const int64_t per_row = s.max_kv < 1 ? 1 : (s.max_kv + kWarps * kUnit - 1) / (kWarps * kUnit);
    if (per_row <= 8 && rows <= 16 && per_row * s.batch * s.kv_heads <= fit)
        return SplitPlan{static_cast<int32_t>(per_row), 0, 0, true};
    return SplitPlan{static_cast<int32_t>(fit), 0, fit * 2 * tile, false};
}

namespace {

// Tensor map over a cache's codes [blocks, page_size, head_dim] (a block: a page
// of one head), boxes of box_tokens tokens, 16-byte pieces swizzled by the
// 128-byte line (all eight of a line at 128 channels, four of a row at 64).
bool encode_cache_map(CUtensorMap *tm, const void *codes, int head_dim, int page_size, int64_t blocks, int box_tokens)
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    if (fn == nullptr)
        return false;
    const cuuint64_t row = static_cast<cuuint64_t>(head_dim), page = static_cast<cuuint64_t>(page_size);
    const cuuint64_t dims[3] = {row, page, static_cast<cuuint64_t>(blocks)}, strides[2] = {row, row * page};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(head_dim), static_cast<cuuint32_t>(box_tokens), 1}, step[3] = {1, 1, 1};
    return fn(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(codes), dims, strides, box, step,
              CU_TENSOR_MAP_INTERLEAVE_NONE, head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kDim, int kRows, bool kWithhold = false>
cudaError_t run_rows(const AttnArgs &a, const SplitPlan &plan, float *logs, float *part, cudaStream_t st, uint64_t wait_ns = kWaitNs)
{
    constexpr int kRing = kWarps * kStages * 2 * kUnit * kDim, kJoin = (kWarps + 1) * kRows * kDim * 4 + kRows * 4;
    constexpr int kSmem = kRing > kJoin ? kRing : kJoin;
    cudaError_t e = allow_shared<rows_kernel<kDim, kRows, kWithhold>>(kSmem);
    if (e != cudaSuccess)
        return e;
    CUtensorMap k_map, v_map;
    const int64_t blocks = static_cast<int64_t>(a.cache.num_pages) * a.cache.heads;
    const int box = a.cache.page_size < kUnit ? a.cache.page_size : kUnit;
    if (blocks == 0) {   // no pages: nothing is copied through the maps
        memset(&k_map, 0, sizeof(k_map));
        v_map = k_map;
    } else if (!encode_cache_map(&k_map, a.cache.k_codes, kDim, a.cache.page_size, blocks, box) ||
               !encode_cache_map(&v_map, a.cache.v_codes, kDim, a.cache.page_size, blocks, box)) {
        return cudaErrorInvalidValue;
    }
    const int64_t rows = static_cast<int64_t>(a.batch.max_tokens) * (a.heads / a.cache.heads);
    const int64_t joins = (rows + kRows - 1) / kRows * a.cache.heads, x = static_cast<int64_t>(plan.splits) * a.cache.heads;
    if (x > INT32_MAX || joins > INT32_MAX)
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr;
    cfg.gridDim = plan.cluster ? dim3(static_cast<unsigned>(x), static_cast<unsigned>(a.batch.batch))
                               : dim3(static_cast<unsigned>(plan.splits));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = st;
    cfg.attrs = &attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(plan.splits);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.numAttrs = plan.cluster ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, rows_kernel<kDim, kRows, kWithhold>, a, plan, logs, part, k_map, v_map, wait_ns);
    if (e != cudaSuccess || plan.cluster || kWithhold)
        return e;
    // The join may be scheduled while the last CTAs run; it waits for them before it reads what they wrote.
    cfg.gridDim = dim3(static_cast<unsigned>(joins), static_cast<unsigned>(a.batch.batch));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.dynamicSmemBytes = 0;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, join_kernel<kDim, kRows>, a, static_cast<int>(plan.splits), static_cast<const float *>(logs),
                              static_cast<const float *>(part));
}

}  // namespace

cudaError_t launch_attention_rows(const AttnArgs &a, const SplitPlan &plan, float *logs, float *part, cudaStream_t st)
{
    const bool small = static_cast<int64_t>(a.batch.max_tokens) * (a.heads / a.cache.heads) <= 8;
    if (a.cache.head_dim == 64)
        return small ? run_rows<64, 8>(a, plan, logs, part, st) : run_rows<64, 16>(a, plan, logs, part, st);
    return small ? run_rows<128, 8>(a, plan, logs, part, st) : run_rows<128, 16>(a, plan, logs, part, st);
}

cudaError_t launch_attention_rows_timeout(const AttnArgs &a, const SplitPlan &plan, float *logs, float *part, uint64_t wait_ns,
                                          cudaStream_t st)
{
    return run_rows<128, 8, true>(a, plan, logs, part, st, wait_ns);
}

cudaError_t read_attention_rows_error(uint32_t *code)
{
    uint32_t v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_error, sizeof(v));
    if (e != cudaSuccess)
        return e;
    const uint32_t zero = 0;
    e = cudaMemcpyToSymbol(g_error, &zero, sizeof(zero));
    *code = v;
    return e;
}

}  // namespace h3fp4

// attention_tile.cu -- attention of many queries: two tiles of 128 rows per
// CTA against tiles of 128 keys, both products on the tcgen05 tensor cores.
//
// The work is 4 * dim FLOP a visible pair and row; the floor is the FP16 tensor
// rate (4 x 512 SM cycles a step of 256 rows and 128 keys at dim 128).  The
// parts:
//  - 8 softmax warps, a thread a row: S from TMEM (tcgen05.ld), one pass for
//    the maximum and one for the weights, which go back to TMEM as FP16 over
//    S's own columns, the A operand of the second product.  The two row tiles
//    alternate, one in the tensor cores while the other is in the softmax.
//    The output accumulator in TMEM is rescaled only when a row's maximum has
//    grown by more than 2^8 since it was last; FP16 and FP32 hold weights of up
//    to 2^15 as well as up to 1.
//  - 4 conversion warps: codes straight from global memory to registers (they
//    are in L2: every row tile of a head reads them), E4M3 -> FP16, which is
//    exact, and into shared memory in the 128-byte-swizzled operand layout.
//    Keys are the first product's K-major B operand; values have the same
//    layout, read as the second product's MN-major B operand.
//  - 2 warps issue the MMAs, one for each row tile.
// Shared memory at dim 128: queries 64 KB, two stages of keys and of values 32
// KB each.
//
// Measured: 5,042 tokens of 56 heads of 128 channels against 37,810 keys 5.01
// ms, 1.09 PFLOP/s, about 4,100 cycles a step; with a window of 16,384 and 3,600
// sinks 3.06 ms, 1.06 PFLOP/s.  No pipe is full (tensor 43 to 50 %,
// exponentials 21 %, issue 45 %, shared memory 32 %), and leaving out any
// one part of the arithmetic but the exponentials changes nothing.  What is
// left is the length of a tile's chain -- scores, softmax, weights, product,
// the next scores, of which some 500 cycles lie between a product's end and the
// issue of the next scores -- with two tiles in turn, and the last wave: 1,120
// CTAs of equal length on 152 SMs are 7.4 waves run as 8.  Short CTAs (13
// steps: 1,560 tokens over as many) lose more: of 80,000 cycles 15,000 go by
// until the first step is done (set-up 2,600, the queries' way through DRAM and
// into shared memory 8,000), and 5,000 after the last.
// Tried and slower: half steps of 64 keys with two score buffers (5.65 ms), the
// next scores' first half issued while the softmax works (4 %), two threads a
// row (8.2 ms), a quarter of the exponentials as polynomials (16 %).
#include <algorithm>
#include <type_traits>

#include "attention.cuh"
#include "ptx_attention.cuh"

namespace h3fp4 {
namespace {

__device__ uint32_t g_error;
constexpr uint64_t kWaitNs = 2000000000ull;

constexpr int kKeys = 128;                     // keys per step
constexpr int kTiles = 2;                      // row tiles of 128 per CTA
constexpr int kSoftmaxWarps = 4 * kTiles;
constexpr int kConvertWarps = 4;
constexpr int kMmaWarp = kSoftmaxWarps + kConvertWarps;
constexpr int kThreads = 32 * (kMmaWarp + 4);  // whole warpgroups, for the register split; two warps idle
// Registers per thread of the three kinds of warpgroup, out of the 128 that 512 threads launch with (run_tile checks):
// a softmax thread holds its row's 128 scores.  (184, 112 and 32 left the conversion with sinks short: 5.21 ms where all is
// seen, 5.09 now; without sinks 5.12 and 5.10.  176, 128 and 32: 5.00 with sinks, 5.59 without.)
constexpr int kSoftmaxRegs = 184, kConvertRegs = 120, kMmaRegs = 24;
constexpr int kSplitRegs = 2 * kSoftmaxRegs + kConvertRegs + kMmaRegs;
static_assert(kSplitRegs <= 4 * 128 && kConvertRegs <= 128 && kMmaRegs <= 128, "the launch's registers cover the split");
constexpr int kStages = 2;
constexpr int kEntrySlots = 4;
// Weights are FP16 and stand against a reference: the row's maximum less kLift when it was set, held until a maximum passes
// it by kPast (log2).  So the largest weight lies between 2^kLift and 2^kPast, below FP16's limit of nearly 2^16, and one
// 2^-21 as large is still a normal number, one 2^-32 as large not yet nothing.
constexpr float kLift = 7.0f, kPast = 15.0f;

template <int kDim>
struct __align__(1024) Smem {
    uint8_t q[kTiles][128 * kDim * 2];
    uint8_t k[kStages][kKeys * kDim * 2];
    uint8_t v[kStages][kKeys * kDim * 2];
    PageEntry entry[kEntrySlots][kKeys / 16];
    uint16_t nan_mask[kStages][kKeys][kDim / 16];   // NaN codes of the value rows of a conversion warp that found any
    uint16_t row_nan[kTiles * 128][kDim / 16];      // channels in which a row has met NaN in an edge step
    int32_t nan_step[kStages][kConvertWarps];       // 1 + the last edge step in which that warp found a NaN
    uint64_t q_full[kTiles], s_full[kTiles], p_half[kTiles], p_full[kTiles], o_full[kTiles];
    uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages], entry_full[kEntrySlots];
    uint64_t drained;
    uint32_t tmem;
    int32_t far_from;   // first step with a far scale
};

// Byte offset of 16-byte piece c (8 halves) of row r in the operand layout: blocks of 64 channels, rows of 128 bytes
// swizzled in 16-byte pieces by the row's low three bits.
__device__ __forceinline__ uint32_t operand_at(int r, int c)
{
    return static_cast<uint32_t>((c >> 3) * (128 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

constexpr uint32_t idesc_f16(int n, bool b_mn_major)   // M = 128, FP32 accumulator
{
    return (1u << 4) | (b_mn_major ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) | (128u >> 4 << 24);
}

// Waits for the phase with this parity, two seconds at most.  The timer is read once in 64 tries only: a read takes about
// 1,000 cycles, and a try may come back empty-handed long before the phase completes.  The outcome is a vote, so that
// control flow that hangs on it is warp-uniform (and operands computed there can live in uniform registers).
__device__ __forceinline__ bool wait_for(const uint64_t &bar, uint32_t parity)
{
    const uint32_t at = smem_u32(&bar);
    uint64_t since = 0;
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 64; ++i)
            if (__all_sync(0xFFFFFFFFu, mbar_try_wait(at, parity)))
                return true;
        const uint64_t now = globaltimer_ns();
        if (since == 0)
            since = now;
        if (__any_sync(0xFFFFFFFFu, now - since > kWaitNs)) {
            atomicOr(&g_error, ERR_ATTN_WAIT);
            return false;
        }
    }
}

// What turns a score's product into the exponent: the row's factor times the keys' scale.  Never 0, so that a hidden
// key's -infinity stays one; at the least normal number all of a step's products (below 2^32) still come to nothing.
__device__ __forceinline__ float step_factor(float c_row, float ks) { return fmaxf(c_row * ks, 0x1p-126f); }

// One arrival for a warp whose lanes have each done (and fenced) their part.
__device__ __forceinline__ void warp_arrive(const uint64_t &bar)
{
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
        mbar_arrive(smem_u32(&bar));
}

// Every by-th row of a sequence and cache head: its token and the query head among the cache head's, with one division.
struct RowWalk {
    int row, token, head, by, by_tokens, by_heads, group;

    __device__ __forceinline__ RowWalk(int first, int by, int group)
        : row(first), token(first / group), head(first % group), by(by), by_tokens(by / group), by_heads(by % group), group(group)
    {
    }
    __device__ __forceinline__ void step()
    {
        row += by;
        token += by_tokens;
        head += by_heads;
        if (head >= group) {
            head -= group;
            ++token;
        }
    }
};

template <int kRegs>
__device__ __forceinline__ void grow_registers()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}

template <int kRegs>
__device__ __forceinline__ void shrink_registers()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

template <int kDim, int kGroup, int kForm>
__global__ void __launch_bounds__(kThreads, 1)
    tile_kernel(AttnArgs a, SplitPlan plan, int row_tiles, bool longest_first, float2 *ws_stat, float *ws_out)
{
    extern __shared__ uint8_t dyn[];
    Smem<kDim> &sm = *reinterpret_cast<Smem<kDim> *>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int page = a.cache.page_size, group = a.heads / a.cache.heads;
    if (kForm != kWhole)   // what follows waits for this grid's end itself: the join, or the half over the sequences' own keys
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    int tile, rest;   // the order of the grid, see by_length()
    if (longest_first) {
        const int others = a.cache.heads * plan.splits * a.batch.batch;
        tile = row_tiles - 1 - static_cast<int>(blockIdx.x / others);
        rest = blockIdx.x % others;
    } else {
        tile = blockIdx.x % row_tiles;
        rest = blockIdx.x / row_tiles;
    }
    const int kh = rest % a.cache.heads, split = rest / a.cache.heads % plan.splits, b = rest / a.cache.heads / plan.splits;
    const KvSequence s = kv_sequence(a.batch, b, a.tokens);
    if (s.n == 0) {
        after_prefix<kForm>();
        return;   // without queries its length and pages are not looked at
    }
    if (!in_range(a, s)) {
        if (threadIdx.x == 0)
            atomicOr(&g_error, ERR_KV_RANGE);
        if (tile == 0 && kh == 0 && split == 0)
            refuse_rows<kForm>(a, s);
        after_prefix<kForm>();
        return;
    }
    const int rows = s.n * group;   // below 2^31 (run_tile checks max_tokens)
    const int row0 = tile * (kTiles * 128);
    if (row0 >= rows || (split > 0 && split * plan.chunk >= s.len)) {
        after_prefix<kForm>();
        return;
    }
    const int row_end = min(rows, row0 + kTiles * 128);
    const Span first = seen_by(a, s, row0 / group), last = seen_by(a, s, (row_end - 1) / group);
    // With sinks everything below is in places (see Fold): what a row sees, less the gap, and the sinks, which end before it.
    const Fold places = fold<kForm>(a, min(first.lo, last.lo), max(first.hi, last.hi), kKeys);
    const int in_lo = max(first.lo, last.lo) - places.gap, in_hi = min(first.hi, last.hi) - places.gap;   // seen by every row
    const int out_lo = min(first.lo, last.lo) - places.gap, out_hi = max(first.hi, last.hi) - places.gap; // seen by any
    const int begin = kForm == kSinks ? split * plan.chunk : max(split * plan.chunk, out_lo & ~(kKeys - 1));
    const int end = min(min((split + 1) * plan.chunk, s.len), out_hi);
    const int steps = end > begin ? (end - begin + kKeys - 1) / kKeys : 0;
    const int tiles = row_end - row0 > 128 ? 2 : 1;

    constexpr int kRowLanes = kDim / 8, kRowsAtOnce = 32 / kRowLanes;
    const int shift = 31 - __clz(page);
    const auto page_ids = [&](int j) -> int32_t {
        const int64_t tok = begin + static_cast<int64_t>(j) * kKeys + lane * page;
        const int gap = kForm == kSinks && tok >= places.keep ? places.gap >> shift : 0;
        return lane < kKeys / page && tok < end && (tok + page > out_lo || (kForm == kSinks && tok < a.sinks))
                   ? a.batch.page_table[b * a.batch.ld_table + (tok >> shift) + gap] : -2;
    };

    if (threadIdx.x == 0) {
        for (int i = 0; i < kTiles; ++i) {
            mbar_init(smem_u32(&sm.q_full[i]), 4);
            mbar_init(smem_u32(&sm.s_full[i]), 1);
            mbar_init(smem_u32(&sm.p_half[i]), 4);
            mbar_init(smem_u32(&sm.p_full[i]), 4);
            mbar_init(smem_u32(&sm.o_full[i]), 1);
        }
        for (int i = 0; i < kStages; ++i) {
            mbar_init(smem_u32(&sm.k_full[i]), kConvertWarps);
            mbar_init(smem_u32(&sm.v_full[i]), kConvertWarps);
            mbar_init(smem_u32(&sm.k_empty[i]), tiles);
            mbar_init(smem_u32(&sm.v_empty[i]), tiles);
            for (int w = 0; w < kConvertWarps; ++w)
                sm.nan_step[i][w] = 0;
        }
        sm.far_from = INT32_MAX;
        for (int i = 0; i < kEntrySlots; ++i)
            mbar_init(smem_u32(&sm.entry_full[i]), 1);
        mbar_init(smem_u32(&sm.drained), tiles);
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        // One CTA per SM (the shared memory sees to that), so the whole TMEM is free.
        tmem_alloc(smem_u32(&sm.tmem), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // All 512 columns are this CTA's, so they start at 0: S of tile t at column 128 t, its output at 256 + kDim t.
    if (sm.tmem != 0) {
        if (threadIdx.x == 0)
            atomicOr(&g_error, ERR_ATTN_WAIT);
        __syncthreads();
        if (warp == kMmaWarp)
            tmem_dealloc(sm.tmem, 512);
        after_prefix<kForm>();
        return;
    }

    if (warp < kSoftmaxWarps) {
        grow_registers<kSoftmaxRegs>();
        const int t = warp >> 2, in_tile = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const int r = row0 + 128 * t + in_tile;
        const bool live = r < rows;
        if (t < tiles) {
            const int tok = live ? r / group : 0, head = kh * group + (live ? r % group : 0);
            Span see = live ? seen_by(a, s, tok) : Span{0, 0};
            if (kForm == kSinks)
                see = Span{see.lo - places.gap, see.hi - places.gap};
            // what the tile's rows all see
            const Span tf = seen_by(a, s, (row0 + 128 * t) / group), tl = seen_by(a, s, (min(rows, row0 + 128 * t + 128) - 1) / group);
            const int t_lo = max(tf.lo, tl.lo) - places.gap, t_hi = min(tf.hi, tl.hi) - places.gap;
            // The warp's 32 rows, kDim / 8 lanes a row: whole rows are read at a time.
            uint4 query[kRowLanes];
            RowWalk at(row0 + 32 * warp + lane / kRowLanes, kRowsAtOnce, group);
            const uint16_t *first_head = a.q + s.row * a.qt + kh * group * a.qh + 8 * (lane % kRowLanes);
#pragma unroll
            for (int y = 0; y < kRowLanes; ++y) {
                query[y] = at.row < rows ? *reinterpret_cast<const uint4 *>(first_head + at.token * a.qt + at.head * a.qh) : make_uint4(0, 0, 0, 0);
                at.step();
            }
            // Each row's largest channel: the lanes of a row give away half of their rows' maxima at each exchange, until lane
            // y of them holds that of row y.
            float c_row;
            {
                uint32_t top[kRowLanes];
#pragma unroll
                for (int y = 0; y < kRowLanes; ++y) {
                    const uint32_t m2 =
                        bf16x2_absmax(bf16x2_absmax(bf16x2_absmax(bf16x2_absmax(0, query[y].x), query[y].y), query[y].z), query[y].w);
                    top[y] = max(m2 & 0xFFFFu, m2 >> 16);
                }
#pragma unroll
                for (int x = kRowLanes / 2; x > 0; x >>= 1) {
                    const bool upper = (lane & x) != 0;
#pragma unroll
                    for (int y = 0; y < x; ++y)
                        top[y] = max(upper ? top[y + x] : top[y], __shfl_xor_sync(0xFFFFFFFFu, upper ? top[y] : top[y + x], x));
                }
                const float2 p = row_power(top[0]);
                c_row = fabsf(a.scale) * kLog2e * __shfl_sync(0xFFFFFFFFu, p.y, lane % kRowsAtOnce * kRowLanes + lane / kRowsAtOnce);
                const float mine = a.scale < 0.0f ? -p.x : p.x;
#pragma unroll
                for (int y = 0; y < kRowLanes; ++y) {
                    const float f = __shfl_sync(0xFFFFFFFFu, mine, (lane & -kRowLanes) + y);
                    st_shared_v4(smem_u32(sm.q[t]) + operand_at((warp & 3) * 32 + y * kRowsAtOnce + lane / kRowLanes, lane % kRowLanes),
                                 bf16x2_to_half2(query[y].x, f), bf16x2_to_half2(query[y].y, f), bf16x2_to_half2(query[y].z, f),
                                 bf16x2_to_half2(query[y].w, f));
                }
                fence_proxy_async_smem();
                warp_arrive(sm.q_full[t]);
            }
            float ref = -INFINITY, l = 0.0f;
            bool met_nan = false;
            const uint32_t sc = 128u * t + lanes, oc = 256u + static_cast<uint32_t>(kDim) * t + lanes;
            float apart_ref = -INFINITY, apart_l = 0.0f;   // with far scales: a sum against a reference of its own
            // One step; false: a wait gave up, or (kFar false) the first step with a far scale has come.  Those that follow are a
            // loop of their own, so that they cost the others a comparison (a chunk 5,118 us, prompts 99-100; with a choice
            // inside of one loop 5,420 and 104).
            const auto step = [&](auto far_scales, int j) -> bool {
                constexpr bool kFar = decltype(far_scales)::value;
                const int k0 = begin + j * kKeys;
                const bool edge = !all_seen<kForm>(a, t_lo, t_hi, k0, kKeys);
                if (!wait_for(sm.entry_full[j % kEntrySlots], (j / kEntrySlots) & 1) || (!kFar && j >= sm.far_from) ||
                    !wait_for(sm.s_full[t], j & 1))
                    return false;
                tc_fence_after();
                const PageEntry *pe = sm.entry[j % kEntrySlots];
                const int lo = see.lo - k0, hi = see.hi - k0;
                const auto visible = [&](int col) { return seen<kForm>(a, see, k0 + col); };
                // A step in which some rows do not see some keys: minus infinity goes over those scores in TMEM, so that
                // the straight code below is the same for all steps (masking its registers there, under a branch, made
                // every step 13 % slower).
                if (edge) {
#pragma unroll 1
                    for (int n = 0; n < kKeys / 16; ++n) {
                        if (__all_sync(0xFFFFFFFFu, all_seen<kForm>(a, see.lo, see.hi, k0 + 16 * n, 16)))
                            continue;
                        uint32_t x[16];
                        tmem_ld_32x32b_x16_wait(sc + 16 * n, x);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            x[i] = visible(16 * n + i) ? x[i] : 0xFF800000u;
                        tmem_st_32x32b_x16(sc + 16 * n, x);
                    }
                    tmem_st_wait();
                }
                float v[128], top = -INFINITY;
                tmem_ld_32x32b_x64(sc, v);
                tmem_ld_32x32b_x64(sc + 64, v + 64);
                tmem_ld_wait_x64(v);
                tmem_ld_wait_x64(v + 64);
#pragma unroll
                for (int n = 0; n < kKeys / kGroup; ++n) {
                    const PageEntry e = pe[(kGroup * n) >> shift];
                    const float *x = v + kGroup * n;
                    float g0 = max3(x[0], x[1], x[2]), g1 = max3(x[3], x[4], x[5]);
#pragma unroll
                    for (int i = 6; i + 3 < kGroup; i += 4) {
                        g0 = max3(g0, x[i], x[i + 1]);
                        g1 = max3(g1, x[i + 2], x[i + 3]);
                    }
                    top = fmaxf(top, fmaf(max3(g0, g1, fmaxf(x[kGroup - 2], x[kGroup - 1])), step_factor(c_row, e.ks), e.lv));
                }
                const bool move = top - ref > kPast;   // (a difference, which is exact on any grid; two infinities: no)
                if (__any_sync(0xFFFFFFFFu, move)) {
                    const float next = move ? top - kLift : ref;
                    const float f = ref == -INFINITY ? 0.0f : ex2(ref - next);
                    l *= f;
                    ref = next;
                    if (j > 0) {   // the accumulator's last product has completed: S of this step was issued after it
#pragma unroll 1
                        for (int c = 0; c < kDim / 16; ++c) {
                            uint32_t o[16];
                            tmem_ld_32x32b_x16_wait(oc + 16 * c, o);
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            tmem_st_32x32b_x16(oc + 16 * c, o);
                        }
                    }
                }
                const float at = ref == -INFINITY ? 0.0f : ref;
                // The exponent is one fused multiply-add.  For a row past 2^20 the reference's own rounding would show in
                // it (and could reach FP16's limit): there the score is rounded first, so that the largest one meets its
                // own copy in the reference.  A step with such a row takes a short loop instead of the long straight
                // code, with the same operations in the same order for every other row, so that a row's bits do not
                // depend on its neighbours.
                const bool far = fabsf(at) > 0x1p20f, plain = !kFar && !__any_sync(0xFFFFFFFFu, far);
                if (!plain) {
                    if constexpr (kFar) {
                        float u = -INFINITY, sum = 0.0f;
#pragma unroll 1
                        for (int n = 0; n < kKeys / 16; ++n) {
                            const float ck = step_factor(c_row, pe[(16 * n) >> shift].ks);
                            uint32_t x[16];
                            tmem_ld_32x32b_x16_wait(sc + 16 * n, x);
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                u = fmaxf(u, __fmul_rn(__uint_as_float(x[i]), ck));
                        }
                        const float was = apart_ref, next = fmaxf(was, u), base = next == -INFINITY ? 0.0f : next;
#pragma unroll 1
                        for (int n = 0; n < kKeys / 16; ++n) {
                            const float ck = step_factor(c_row, pe[(16 * n) >> shift].ks);
                            uint32_t x[16];
                            tmem_ld_32x32b_x16_wait(sc + 16 * n, x);
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                sum += ex2(__fmul_rn(__uint_as_float(x[i]), ck) - base);
                        }
                        apart_l = fmaf(apart_l, ex2(was - base), sum);
                        apart_ref = next;
                    }
                    float2 s0 = make_float2(0.0f, 0.0f), s1 = s0;
#pragma unroll 1
                    for (int n = 0; n < kKeys / 16; ++n) {
                        const PageEntry e = pe[(16 * n) >> shift];
                        const float ck = step_factor(c_row, e.ks), off = e.lv - at;
                        uint32_t x[16], p[8];
                        tmem_ld_32x32b_x16_wait(sc + 16 * n, x);
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            float w[2];
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const int col = 16 * n + i + y;
                                const float z = __uint_as_float(x[i + y]);
                                w[y] = visible(col) ? ex2(far ? fmaf(z, ck, e.lv) - at : fmaf(z, ck, off)) : 0.0f;
                            }
                            p[i / 2] = pack_half2(w[0], w[1]);
                            float2 &sum = (i & 2) == 0 ? s0 : s1;
                            sum = __fadd2_rn(sum, make_float2(w[0], w[1]));
                        }
                        if ((16 * n + 16) % kGroup == 0) {
                            s0 = __fadd2_rn(s0, s1);
                            l = fmaf(s0.x + s0.y, e.inv_vs, l);
                            s0 = s1 = make_float2(0.0f, 0.0f);
                        }
                        tmem_st_32x32b_x8(sc + 8 * n, p);   // over columns of S that are read already
                    }
                    tmem_st_wait();
                    tc_fence_before();
                    warp_arrive(sm.p_half[t]);
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        float *x = v + 32 * c;
#pragma unroll
                        for (int n = 0; n < 32; n += kGroup) {
                            const PageEntry e = pe[(32 * c + n) >> shift];
                            const float ck = step_factor(c_row, e.ks);
                            const float2 ck2 = make_float2(ck, ck), off2 = make_float2(e.lv - at, e.lv - at);
#pragma unroll
                            for (int i = n; i < n + kGroup; i += 2) {
                                const float2 w = __ffma2_rn(make_float2(x[i], x[i + 1]), ck2, off2);
                                x[i] = ex2(w.x);
                                x[i + 1] = ex2(w.y);
                            }
                        }
                        uint32_t p[16];
#pragma unroll
                        for (int i = 0; i < 32; i += 2)
                            p[i / 2] = pack_half2(x[i], x[i + 1]);
                        tmem_st_32x32b_x16(sc + 16 * c, p);
                        if (c == 1) {   // the first half's product can start
                            tmem_st_wait();
                            tc_fence_before();
                            warp_arrive(sm.p_half[t]);
                        }
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                if (!all_seen<kForm>(a, in_lo, in_hi, k0, kKeys)) {   // the conversion warps keep NaN out of such a step's values
                    if (!wait_for(sm.v_full[j % kStages], (j / kStages) & 1))
                        return false;
                    constexpr int kRowsPerWarp = 32 / (kDim / 16);   // of a conversion warp, among kConvertWarps * that
                    for (int w = 0; w < kConvertWarps; ++w) {
                        if (sm.nan_step[j % kStages][w] != j + 1)
                            continue;
                        uint16_t *mine = sm.row_nan[128 * t + in_tile];
                        for (int c = 0; c < kDim / 16; ++c) {
                            uint32_t m = met_nan ? mine[c] : 0u;
                            for (int x = kForm == kSinks ? 0 : max(lo, 0); x < min(hi, kKeys); ++x)
                                if ((kForm != kSinks || visible(x)) && x / kRowsPerWarp % kConvertWarps == w)
                                    m |= sm.nan_mask[j % kStages][x][c];
                            mine[c] = static_cast<uint16_t>(m);
                        }
                        met_nan = true;
                    }
                }
                warp_arrive(sm.p_full[t]);
                if (plain) {   // the sum, off the way to the product
#pragma unroll
                    for (int n = 0; n < kKeys / kGroup; ++n) {
                        const float *x = v + kGroup * n;
                        float2 s0 = make_float2(x[0], x[1]), s1 = make_float2(x[2], x[3]);
#pragma unroll
                        for (int i = 4; i < kGroup; i += 4) {
                            s0 = __fadd2_rn(s0, make_float2(x[i], x[i + 1]));
                            s1 = __fadd2_rn(s1, make_float2(x[i + 2], x[i + 3]));
                        }
                        s0 = __fadd2_rn(s0, s1);
                        l = fmaf(s0.x + s0.y, pe[(kGroup * n) >> shift].inv_vs, l);
                    }
                }
                return true;
            };
            int j = 0;
            while (j < steps && step(std::false_type{}, j))
                ++j;
            bool ok = j == steps || j >= sm.far_from;
            float o_factor = 1.0f;
            if (ok && j < steps) {
                apart_ref = log_of_sum(ref, l);
                apart_l = own_sum(l);
                for (; ok && j < steps; ++j)
                    ok = step(std::true_type{}, j);
                o_factor = apart_l > 0.0f ? ex2(ref - apart_ref) : 1.0f;
                ref = apart_ref;
                l = apart_l;
            }
            if (ok && steps > 0)
                ok = wait_for(sm.o_full[t], (steps - 1) & 1);
            if (ok) {
                tc_fence_after();
                const int64_t row = s.row + tok, at = row * a.heads + head;
                const bool final = plan.splits == 1;
                const float inv = reciprocal_sum(l) * o_factor;
                Shares share{};
                bool other_half = false, written = live;
                if (kForm == kOwn && final) {
                    after_prefix<kForm>();
                    const float other = live ? prefix_log(a, row, head) : -INFINITY;
                    other_half = other != -INFINITY;   // (else its mean may be anything)
                    share = shares_of(log_of_sum(ref, l), other);
                    written = live && !refused(other);
                }
                const uint32_t rows_written = kForm == kOwn ? __ballot_sync(0xFFFFFFFFu, written) : 0;
                // Rows are written through shared memory in whole sectors, or, where that gains nothing, straight from the
                // threads that hold them (128 channels: 1,560 tokens over as many keys 5,700 cycles a CTA, 7,000 straight; 64
                // channels, ragged prompts: 99.2 us, 97.5 straight; with sinks, a chunk: 3,105 us, 3,055).
                constexpr bool kStaged = kDim == 128 && kForm != kSinks;
                const bool narrow = final && kForm != kPrefix;   // bf16 to the output, else FP32 for a join
                const int pieces = narrow ? 4 : 8;
                const auto place_of = [&](int64_t to_row, int64_t to_head) -> uint8_t * {
                    const int64_t to = to_row * a.heads + to_head;
                    return narrow ? reinterpret_cast<uint8_t *>(a.out + to_row * a.ot + to_head * a.oh)
                                  : reinterpret_cast<uint8_t *>(kForm == kPrefix && final ? a.half_mean + to * kDim
                                                                                          : ws_out + (to * plan.splits + split) * kDim);
                };
                uint8_t *to[8];
                if constexpr (kStaged) {   // of this lane's pieces
                    RowWalk at_row(row0 + 32 * warp + lane / pieces, 32 / pieces, group);
                    const int first_row = row0 + 32 * warp, last_row = min(rows, first_row + 32);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        bool mine = at_row.row < last_row;
                        if (kForm == kOwn)
                            mine = mine && (rows_written >> (at_row.row - first_row) & 1) != 0;
                        to[i] = mine ? place_of(s.row + at_row.token, kh * group + at_row.head) + 16 * (lane & (pieces - 1)) : nullptr;
                        at_row.step();
                    }
                } else {
                    to[0] = written ? place_of(row, head) : nullptr;
                }
#pragma unroll 1
                for (int c = 0; c < kDim / 32; ++c) {
                    uint32_t v[32];
                    if (steps > 0) {
                        tmem_ld_32x32b_x32(oc + 32 * c, v);
                        tmem_ld_wait_regs(v);
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            v[i] = 0u;
                    }
                    float o[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        o[i] = __uint_as_float(v[i]) * inv;
                    if (met_nan) {
                        const uint32_t m = sm.row_nan[128 * t + in_tile][2 * c] | sm.row_nan[128 * t + in_tile][2 * c + 1] << 16;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            o[i] = m >> i & 1 ? __uint_as_float(0x7FC00000u) : o[i];
                    }
                    if (kForm == kOwn && final) {
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            const float4 p = other_half ? *reinterpret_cast<const float4 *>(a.half_mean + at * kDim + 32 * c + i)
                                                        : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                            o[i] = join_share(o[i], p.x, share);
                            o[i + 1] = join_share(o[i + 1], p.y, share);
                            o[i + 2] = join_share(o[i + 2], p.z, share);
                            o[i + 3] = join_share(o[i + 3], p.w, share);
                        }
                    }
                    const auto bf16_piece = [&](int i) {   // 8 channels
                        uint32_t x[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const __nv_bfloat162 z = __floats2bfloat162_rn(o[8 * i + 2 * y], o[8 * i + 2 * y + 1]);
                            x[y] = *reinterpret_cast<const uint32_t *>(&z);
                        }
                        return make_uint4(x[0], x[1], x[2], x[3]);
                    };
                    const auto float_piece = [&](int i) {   // 4 channels
                        return make_uint4(__float_as_uint(o[4 * i]), __float_as_uint(o[4 * i + 1]), __float_as_uint(o[4 * i + 2]),
                                          __float_as_uint(o[4 * i + 3]));
                    };
                    if constexpr (kStaged) {
                        // The queries' place is free (all that read them is done): 4 KB a warp, pieces moved by the row's number.
                        const uint32_t stage = smem_u32(sm.q[t]) + (warp & 3) * 4096;
                        const auto at_piece = [&](int in, int x) { return stage + in * 128 + ((x ^ (in & 7)) << 4); };
                        const auto put = [&](int x, const uint4 &p) { st_shared_v4(at_piece(lane, x), p.x, p.y, p.z, p.w); };
                        __syncwarp();
                        if (narrow) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                put(i, bf16_piece(i));
                        } else {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                put(i, float_piece(i));
                        }
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (to[i] != nullptr)
                                *reinterpret_cast<uint4 *>(to[i] + c * (16 * pieces)) =
                                    ld_shared_v4(at_piece(lane / pieces + i * (32 / pieces), lane & (pieces - 1)));
                    } else if (written && narrow) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            *reinterpret_cast<uint4 *>(to[0] + 64 * c + 16 * i) = bf16_piece(i);
                    } else if (written) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            *reinterpret_cast<uint4 *>(to[0] + 128 * c + 16 * i) = float_piece(i);
                    }
                }
                if (live && !final)
                    ws_stat[at * plan.splits + split] = make_float2(ref, l);
                else if (live && kForm == kPrefix)
                    a.half_log[at] = log_of_sum(ref, l);
                else if (written && a.lse != nullptr)
                    a.lse[at] = (kForm == kOwn ? share.log : log_of_sum(ref, l)) * kLn2;
                tc_fence_before();
            }
        }
    } else if (warp < kMmaWarp) {
        // ------------------------------------------------------------------ conversion
        shrink_registers<kConvertRegs>();
        constexpr int kPieces = kDim / 16;                        // 16-byte pieces of codes per token
        constexpr int kRowStep = 32 * kConvertWarps / kPieces;    // tokens between a thread's pieces
        constexpr int kPer = kKeys / kRowStep;
        // Each group of 8 lanes (a store's phase) takes 4 pieces of two adjacent rows: their swizzles differ in the lowest
        // bit, so that the first halves of the pieces, at even places, and then the second fill all banks.
        const int w0 = warp - kSoftmaxWarps;
        const int r0 = kDim == 128 ? 4 * w0 + ((lane >> 2) & 1) + ((lane >> 4) << 1) : 8 * w0 + (lane >> 2);
        const int c = kDim == 128 ? (lane & 3) | ((lane >> 3) & 1) << 2 : lane & 3;
        const auto checked = [&](int32_t id) -> int32_t {        // -2: no page; out of range: reported, page 0 instead
            if (id == -2 || (id >= 0 && id < a.cache.num_pages))
                return id;
            atomicOr(&g_error, ERR_KV_RANGE);
            return 0;
        };
        int32_t id[kPer];   // pages of the step whose codes are loaded next, by piece
        const auto ids = [&](int32_t of_lane) {
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                id[i] = __shfl_sync(0xFFFFFFFFu, kForm == kSinks ? max(of_lane, 0) : of_lane, (r0 + i * kRowStep) >> shift);
        };
        // A piece's group of kRowStep tokens lies in one page (dim 128: 16 tokens) or in two (dim 64: 32).
        const int64_t page_bytes = static_cast<int64_t>(a.cache.heads) * page * kDim;
        const int64_t mine = static_cast<int64_t>(kh) * page * kDim + 16 * c;
        const auto load = [&](const uint8_t *codes, int k0, uint4 (&w)[kPer]) {
            const uint8_t *base = codes + mine;
            if constexpr (kForm == kSinks) {
                // Whole steps, whoever sees them, and page 0 in place of pages that nobody sees (or past the end): such a step
                // is at an edge for every row, where scores are masked and NaN is kept out of the values.  (A test here of
                // which of the step's keys are seen cost every step: 5.42 ms for a call that takes 5.09 with it gone and 5.10
                // without sinks.)
#pragma unroll
                for (int i = 0; i < kPer; ++i)
                    w[i] = *reinterpret_cast<const uint4 *>(base + id[i] * page_bytes + ((r0 + i * kRowStep) & (page - 1)) * kDim);
            } else if (k0 >= out_lo && k0 + kKeys <= end) {
#pragma unroll
                for (int i = 0; i < kPer; ++i)
                    w[i] = *reinterpret_cast<const uint4 *>(base + id[i] * page_bytes + ((r0 + i * kRowStep) & (page - 1)) * kDim);
            } else {   // positions that no row sees stay zero
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const int tok = k0 + r0 + i * kRowStep;
                    w[i] = make_uint4(0, 0, 0, 0);
                    if (tok >= out_lo && tok < end)
                        w[i] = *reinterpret_cast<const uint4 *>(base + id[i] * page_bytes + (tok & (page - 1)) * kDim);
                }
            }
        };
        const uint32_t piece0 = operand_at(r0, 2 * c), piece1 = operand_at(r0, 2 * c + 1);
        const auto store = [&](uint32_t dst, const uint4 &w, int i) {
            const uint2 x = e4m3x4_to_f16x4(w.x), y = e4m3x4_to_f16x4(w.y), z = e4m3x4_to_f16x4(w.z), u = e4m3x4_to_f16x4(w.w);
            // rows kRowStep apart have the same swizzle
            st_shared_v4(dst + piece0 + i * (kRowStep * 128), x.x, x.y, y.x, y.y);
            st_shared_v4(dst + piece1 + i * (kRowStep * 128), z.x, z.y, u.x, u.y);
        };
        // A step's codes are loaded while the step before it is converted, its pages' numbers one step earlier still.
        uint4 kw[kPer], vw[kPer];
        int32_t lane_id = checked(page_ids(0)), next_id = page_ids(1);
        float ks = 1.0f, vs = 1.0f;   // the scales of lane_id's page, loaded as early as its codes
        const auto scales = [&] {
            ks = vs = 1.0f;
            if (warp == kSoftmaxWarps && lane_id >= 0) {
                const int64_t bh = static_cast<int64_t>(lane_id) * a.cache.heads + kh;
                ks = a.cache.k_scale[bh];
                vs = a.cache.v_scale[bh];
            }
        };
        scales();
        ids(lane_id);
        if (kForm != kSinks || steps > 0) {   // (without keys there may be no pages)
            load(a.cache.k_codes, begin, kw);
            load(a.cache.v_codes, begin, vw);
        }
        for (int j = 0; j < steps; ++j) {
            const int k0 = begin + j * kKeys, st = j % kStages;
            const bool edge = !all_seen<kForm>(a, in_lo, in_hi, k0, kKeys);
            if (!wait_for(sm.k_empty[st], ((j / kStages) & 1) ^ 1))
                break;
            if (warp == kSoftmaxWarps) {   // the step's page entries, 8 at most
                if (__any_sync(0xFFFFFFFFu, lane_id >= 0 && far_scale(vs)) && lane == 0)
                    sm.far_from = min(sm.far_from, j);
                const float lv = lg2(vs);
                if (lane < kKeys / page)
                    sm.entry[j % kEntrySlots][lane] = PageEntry{lane_id, ks, lv, ex2(-lv)};
                warp_arrive(sm.entry_full[j % kEntrySlots]);
            }
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                store(smem_u32(sm.k[st]), kw[i], i);
            fence_proxy_async_smem();
            warp_arrive(sm.k_full[st]);
            lane_id = checked(next_id);
            next_id = page_ids(j + 2);
            scales();
            ids(lane_id);
            load(a.cache.k_codes, k0 + kKeys, kw);   // zeros past the end

            if (!wait_for(sm.v_empty[st], ((j / kStages) & 1) ^ 1))
                break;
            if (edge) {   // NaN that only some rows see stays out of the product (a weight of zero would not stop it)
                uint32_t odd = 0;
#pragma unroll
                for (int i = 0; i < kPer; ++i)
                    odd |= nan_bytes(vw[i].x) | nan_bytes(vw[i].y) | nan_bytes(vw[i].z) | nan_bytes(vw[i].w);
                if (__any_sync(0xFFFFFFFFu, odd != 0)) {
#pragma unroll
                    for (int i = 0; i < kPer; ++i) {
                        uint32_t x[4] = {vw[i].x, vw[i].y, vw[i].z, vw[i].w}, m = 0;
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const uint32_t n = nan_bytes(x[y]) >> 7;   // 1 in each NaN byte
                            x[y] &= ~(n * 0xFFu);
                            m |= ((n & 1u) | (n >> 7 & 2u) | (n >> 14 & 4u) | (n >> 21 & 8u)) << (4 * y);
                        }
                        vw[i] = make_uint4(x[0], x[1], x[2], x[3]);
                        sm.nan_mask[st][r0 + i * kRowStep][c] = static_cast<uint16_t>(m);
                    }
                    if (lane == 0)
                        sm.nan_step[st][w0] = j + 1;
                }
            }
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                store(smem_u32(sm.v[st]), vw[i], i);
            fence_proxy_async_smem();
            warp_arrive(sm.v_full[st]);
            load(a.cache.v_codes, k0 + kKeys, vw);
        }
    } else {
        // ------------------------------------------------------------------ MMA issue
        shrink_registers<kMmaRegs>();
    }
    if (warp >= kMmaWarp && warp - kMmaWarp < tiles) {
        constexpr uint32_t kQk = idesc_f16(kKeys, false), kPv = idesc_f16(kDim, true);
        const uint32_t q_lo = (smem_u32(sm.q) & 0x3FFFFu) >> 4 | 1u << 16, k_lo = (smem_u32(sm.k) & 0x3FFFFu) >> 4 | 1u << 16;
        const uint32_t v_lo = (smem_u32(sm.v) & 0x3FFFFu) >> 4 | (128u * 128u >> 4) << 16;   // 64-channel blocks 16 KB apart
        constexpr uint32_t kHi = (1024u >> 4) | 1u << 14 | 2u << 29;   // 8 rows 1 KB apart, version 1, 128-byte swizzle
        constexpr uint32_t kTileUnits = 128 * kDim * 2 / 16;           // an operand tile in 16-byte units
        const auto qk = [&](uint32_t t, uint32_t st) {
#pragma unroll
            for (int x = 0; x < kDim / 16; ++x) {
                const uint32_t off = (x >> 2) * (128 * 128 / 16) + (x & 3) * 2;
                tc_mma_f16_elect(128 * t, q_lo + t * kTileUnits + off, kHi, k_lo + st * kTileUnits + off, kHi, kQk, x > 0);
            }
            tc_commit_elect(smem_u32(&sm.s_full[t]));
        };
        const auto pv = [&](uint32_t t, uint32_t st, int half, bool accumulate) {
#pragma unroll
            for (int y = 0; y < kKeys / 32; ++y) {   // 8-token groups 1 KB apart
                const int x = half * (kKeys / 32) + y;
                tc_mma_f16_ts_elect(256 + kDim * t, 128 * t + 8 * x, v_lo + st * kTileUnits + x * (2048 / 16), kHi, kPv,
                                    accumulate || x > 0);
            }
        };
        // A warp for each tile, with no more between a wait and an issue than the issue needs: scores, then for each
        // step the first half's product, the second half's, and -- that done, for the next scores go over the weights
        // it reads -- the next scores.
        const uint32_t t = warp - kMmaWarp;
        bool ok = steps > 0 && wait_for(sm.q_full[t], 0) && wait_for(sm.k_full[0], 0);
        if (ok) {
            tc_fence_after();
            qk(t, 0);
            tc_commit_elect(smem_u32(&sm.k_empty[0]));
        }
        for (int j = 0; ok && j < steps; ++j) {
            const uint32_t st = j & (kStages - 1), nx = st ^ 1u;
            if (!(ok = wait_for(sm.v_full[st], (j / kStages) & 1) && wait_for(sm.p_half[t], j & 1)))
                break;
            tc_fence_after();
            pv(t, st, 0, j > 0);
            if (!(ok = wait_for(sm.p_full[t], j & 1)))
                break;
            tc_fence_after();
            pv(t, st, 1, true);
            tc_commit_elect(smem_u32(&sm.o_full[t]));
            tc_commit_elect(smem_u32(&sm.v_empty[st]));
            if (j + 1 < steps) {
                if (!(ok = wait_for(sm.k_full[nx], ((j + 1) / kStages) & 1) && wait_for(sm.o_full[t], j & 1)))
                    break;
                tc_fence_after();
                qk(t, nx);
                tc_commit_elect(smem_u32(&sm.k_empty[nx]));
            }
        }
        tc_commit_elect(smem_u32(&sm.drained));   // nothing of this CTA is in the tensor cores when TMEM is freed
        wait_for(sm.drained, 0);
        tc_fence_before();
    }
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(0, 512);
    }
    after_prefix<kForm>();
}

constexpr int kJoinThreads = 128;

// Joins the parts of each row: one warp per query token and head.
template <int kDim, int kForm>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(AttnArgs a, SplitPlan plan, const float2 *ws_stat, const float *ws_out)
{
    let_next_start<kForm>();
    if (kForm != kWhole)   // launched to overlap with the kernel before
        asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, b = blockIdx.y;
    const int64_t w = static_cast<int64_t>(blockIdx.x) * (kJoinThreads / 32) + (threadIdx.x >> 5);
    const KvSequence s = kv_sequence(a.batch, b, a.tokens);
    if (!in_range(a, s) || w >= static_cast<int64_t>(s.n) * a.heads)
        return;
    const int64_t row = s.row + w / a.heads;
    const int head = static_cast<int>(w % a.heads);
    const int64_t at = row * a.heads + head;
    const int parts = min(plan.splits, max(1, (s.len + plan.chunk - 1) / plan.chunk));   // (folded: fewer than the length has)
    const float2 *stat = ws_stat + at * plan.splits;
    const auto log_of = [&](int i) { return log_of_sum(stat[i].x, stat[i].y); };
    float top = -INFINITY, sum = 0.0f;
    for (int i = lane; i < parts; i += 32)
        add_log(top, sum, log_of(i), 1.0f);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) {
        const float other = __shfl_xor_sync(0xFFFFFFFFu, top, x), its = __shfl_xor_sync(0xFFFFFFFFu, sum, x);
        add_log(top, sum, other, its);
    }
    const float inv = reciprocal_sum(sum);
    constexpr int kPer = kDim / 32;
    float mean[kPer];
#pragma unroll
    for (int c = 0; c < kPer; ++c)
        mean[c] = 0.0f;
#pragma unroll 4
    for (int i = 0; i < parts; ++i) {
        const float half = half_of_top(log_of(i), top), rest = half * inv;   // the part's share in two halves: see half_of_top
        const float *src = ws_out + (at * plan.splits + i) * kDim + lane * kPer;
#pragma unroll
        for (int c = 0; c < kPer; c += 2) {
            const float2 v = *reinterpret_cast<const float2 *>(src + c);
            mean[c] = fmaf(v.x * half, rest, mean[c]);
            mean[c + 1] = fmaf(v.y * half, rest, mean[c + 1]);
        }
    }
    float log = log_of_sum(top, sum);
    if (kForm == kOwn) {
        const float other = prefix_log(a, row, head);
        if (refused(other))
            return;
        const Shares share = shares_of(log, other);
        const float *half = a.half_mean + at * kDim + lane * kPer;
#pragma unroll
        for (int c = 0; c < kPer; ++c)
            mean[c] = join_share(mean[c], other != -INFINITY ? half[c] : 0.0f, share);
        log = share.log;
    }
    if (kForm == kPrefix) {
#pragma unroll
        for (int c = 0; c < kPer; c += 2)
            *reinterpret_cast<float2 *>(a.half_mean + at * kDim + lane * kPer + c) = make_float2(mean[c], mean[c + 1]);
        if (lane == 0)
            a.half_log[at] = log;
        return;
    }
    uint16_t *dst = a.out + row * a.ot + head * a.oh + lane * kPer;
#pragma unroll
    for (int c = 0; c < kPer; c += 2) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(mean[c], mean[c + 1]);
        *reinterpret_cast<uint32_t *>(dst + c) = *reinterpret_cast<const uint32_t *>(&v);
    }
    if (a.lse != nullptr && lane == 0)
        a.lse[at] = log * kLn2;
}

// kGroup: scores in a row that are sure to lie in one page.
// Order of the grid.  The CTAs of causal attention differ in length, by their place in the sequence and by the sequence, and
// the last ones should be short: the tiles that lie furthest back go first, over all heads and sequences (6 ragged prompts
// of up to 2,050 tokens with a window: 96 us, 106 with a head's tiles side by side; 8,192 tokens, 56 heads of 128 channels:
// 1,034 us, 1,121).  But the CTAs that run together then read all heads' keys, and where those are more than L2 holds a
// head's tiles side by side are faster (5,042 tokens against 37,810, 542 MB of codes: 4,753 us, 4,887), as they are where
// all tiles have one length (the same without the causal mask: 5,045 us, 5,229).
bool by_length(const AttnArgs &a)
{
    return a.causal && 2.0 * a.batch.batch * a.cache.heads * a.max_kv * a.cache.head_dim <= 128.0 * 1048576;
}

template <int kDim, int kGroup, int kForm>
cudaError_t run_tile(const AttnArgs &a, const SplitPlan &plan, float2 *stat, float *part, cudaStream_t st)
{
    // More than half of an SM's shared memory even at dim 64: a second CTA on the SM would wait for the first one's TMEM.
    constexpr int kNeed = sizeof(Smem<kDim>) + 1024, kSmem = kNeed > 120 * 1024 ? kNeed : 120 * 1024;
    static_assert(kSmem <= 227 * 1024, "fits an SM");
    cudaError_t e = allow_shared<tile_kernel<kDim, kGroup, kForm>>(kSmem);
    if (e != cudaSuccess)
        return e;
    static const bool registers_fit = [] {   // a property of the build
        cudaFuncAttributes f;
        return cudaFuncGetAttributes(&f, tile_kernel<kDim, kGroup, kForm>) == cudaSuccess && 4 * f.numRegs >= kSplitRegs && f.numRegs >= kConvertRegs;
    }();
    if (!registers_fit)
        return cudaErrorLaunchOutOfResources;
    const int64_t most = std::min<int64_t>(most_rows(a.batch), a.tokens);   // of a sequence
    const int64_t tiles = (most * (a.heads / a.cache.heads) + kTiles * 128 - 1) / (kTiles * 128), x = tiles * a.cache.heads * plan.splits * a.batch.batch;
    if (x > INT32_MAX || tiles * (kTiles * 128) > INT32_MAX)
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr = overlap_with_last();
    cfg.gridDim = dim3(static_cast<unsigned>(x));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = kForm == kOwn ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, tile_kernel<kDim, kGroup, kForm>, a, plan, static_cast<int>(tiles), by_length(a), stat, part);
}

}  // namespace

// Parts of the keys: as many as give every SM a CTA, of 256 keys at least (256
// rows of 8 heads of 128 channels against 2,000 keys: 23.5 us, 27.2 with 512 at
// least, 22.5 with 128, 48.5 in one part; against 300: 20.4, 19.3, 22.1).
SplitPlan plan_tile(const AttnShape &s)
{
    const int64_t rows = static_cast<int64_t>(s.max_tokens) * (s.heads / s.kv_heads);
    const int64_t ctas = static_cast<int64_t>(s.batch) * s.kv_heads * ((rows + kTiles * 128 - 1) / (kTiles * 128));
    const int64_t group = s.heads / s.kv_heads, kv = s.max_kv < 1 ? 1 : s.max_kv;
    int64_t splits = ctas > 0 ? sm_count() / ctas : 1;
    const int64_t most = (kv + 255) / 256;
    splits = splits > most ? most : splits < 1 ? 1 : splits;
    int64_t chunk = ((kv + splits - 1) / splits + kKeys - 1) / kKeys * kKeys;
    splits = (kv + chunk - 1) / chunk;
    // Under a window that lies within a part most parts have nothing to do but to write that down (4,674 tokens of 2 heads,
    // window 5: 24.2 us in one part, 32.4 in four).
    const int64_t tokens = kTiles * 128 / group + 1;   // of a CTA's rows
    if (s.sinks > 0) {   // parts of what is left of the keys, no more than above
        const int64_t left = folded_keys(s, s.causal ? tokens : s.max_tokens), parts = std::min(splits, (left + 255) / 256);
        chunk = ((left + parts - 1) / parts + kKeys - 1) / kKeys * kKeys;
        splits = (left + chunk - 1) / chunk;
    } else if (s.reach > 0 && s.reach + tokens <= chunk) {
        splits = 1;
        chunk = (kv + kKeys - 1) / kKeys * kKeys;
    }
    return SplitPlan{static_cast<int32_t>(splits), static_cast<int32_t>(chunk), splits > 1 ? s.tokens * s.heads * splits : 0, false};
}

template <int kForm>
static cudaError_t run_tile_form(const AttnArgs &a, const SplitPlan &plan, float2 *stat, float *part, cudaStream_t st)
{
    cudaError_t e;
    if (a.cache.page_size == 16)
        e = a.cache.head_dim == 64 ? run_tile<64, 16, kForm>(a, plan, stat, part, st) : run_tile<128, 16, kForm>(a, plan, stat, part, st);
    else
        e = a.cache.head_dim == 64 ? run_tile<64, 32, kForm>(a, plan, stat, part, st) : run_tile<128, 32, kForm>(a, plan, stat, part, st);
    if (e != cudaSuccess || plan.splits == 1)
        return e;
    constexpr int kJoinWarps = kJoinThreads / 32;
    const int64_t x = (std::min<int64_t>(most_rows(a.batch), a.tokens) * a.heads + kJoinWarps - 1) / kJoinWarps;
    if (x > INT32_MAX)
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr = overlap_with_last();
    cfg.gridDim = dim3(static_cast<unsigned>(x), static_cast<unsigned>(a.batch.batch));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = kForm != kWhole ? 1 : 0;
    const float2 *const stats = stat;
    const float *const parts = part;
    return a.cache.head_dim == 64 ? cudaLaunchKernelEx(&cfg, join_kernel<64, kForm>, a, plan, stats, parts)
                                  : cudaLaunchKernelEx(&cfg, join_kernel<128, kForm>, a, plan, stats, parts);
}

cudaError_t launch_attention_tile(const AttnArgs &a, Form form, const SplitPlan &plan, float2 *stat, float *part, cudaStream_t st)
{
    switch (form) {
    case kSinks: return run_tile_form<kSinks>(a, plan, stat, part, st);
    case kPrefix: return run_tile_form<kPrefix>(a, plan, stat, part, st);
    case kOwn: return run_tile_form<kOwn>(a, plan, stat, part, st);
    default: return run_tile_form<kWhole>(a, plan, stat, part, st);
    }
}

cudaError_t read_attention_tile_error(uint32_t *code)
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

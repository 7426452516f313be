// norm_rope.cu -- per-head RMS norm of queries and keys with their rotation in
// the same pass (h3fp4_norm_rope), and its gradients (h3fp4_norm_rope_backward).
//
//   r = 1 / sqrt(mean(x^2) + eps),  y = R (x r w)
//   g = R^T dy,  dw = sum over tokens and heads of g x r,
//   dx = r (w g - x r^2 mean(w g x))
//
// R turns pairs of channels, so that y = r (x A + partner(x) B) with A = w cos
// and B = -+ w(partner) sin, which serve all heads of a token; one sum over a
// head's lanes (two for the gradient) lies between its loads and its stores.
// Everything is FP32 until the one rounding to bf16.
//
// A lane holds 16 channels of a head, two chunks of eight.  Pairs that are
// interleaved lie within a chunk; of halves whose sections are whole chunks
// the lane's second chunk is the partner of its first; other halves are
// exchanged through shared memory.  FP32 pairs go through the packed
// instructions.  (With 8 channels a lane and single FP32 instructions the
// forward kernel issued 147 for each 512 bytes read, and that bound it: 452 us
// where it takes 320 now.)
//
// Reads and writes each value once, so HBM bounds both: 37,810 tokens of 56 +
// 56 heads of 128 channels forward 320 us, 6.8 TB/s (the copy rate); 5,042
// tokens' gradients 72 us, 6.0 TB/s, 20,000 tokens' 259 us, 6.6 TB/s.  What is
// left of the gradient's is a launch, the first loads and the join of dw (3
// us); of small calls a launch and a chain of dependent loads (32 tokens of 72
// heads 4.1 us).  Exchanged halves cost the shared-memory pipe: 20,000
// tokens 213 us (gradients 277), interleaved pairs 175 (259).  Halves that face
// each other take 174 (260) as one section; in several a lane's chunks lie in
// shorter runs: (32, 32, 64) 189 (311), (32, 48, 48) 221 (359).  Heads of 256
// channels, half as many: exchanged 217 (290), else 181 (279).  All in a graph of
// 10 passes.
#include <cuda_bf16.h>

#include "norm_exchange.h"
#include "norm_rope.cuh"
#include "rope.cuh"

namespace h3fp4 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// Units of a warp that are loaded or on their way: 1 KB each forward, 2 KB for the gradients, half of the ring in a burst (a
// unit at a time 371 us, 357 in bursts, both in one wave: longer runs of addresses).  Forward with half as many 338 us (326);
// 5,042 tokens' gradients with half as many 77 us (72).
constexpr int kForwardStages = 8, kBackwardStages = 8;
// CTAs of an SM: three forward 424 us against 360 (more streams of addresses at a time), two for the gradients 79 against 78.
constexpr int kForwardCtas = 2, kBackwardCtas = 1;
// Forward calls come in waves of short CTAs, which even out what SMs get of the memory and read it in order (one wave 357 us, 8
// waves 342, 16 and 32 326), as long as a warp has kWaveUnits units in each (20,000 tokens 177 us; with 14 units 184).  Gradients take one wave
// (two: 89 us against 80): each CTA leaves its part of dw.
constexpr int kForwardWaves = 16, kWaveUnits = 28;
static_assert((kForwardStages & (kForwardStages - 1)) == 0 && (kBackwardStages & (kBackwardStages - 1)) == 0, "stages wrap by a mask");

// Where a channel's partner is: beside it, anywhere (exchanged), or at its place in the lane's other chunk (axes of 16 n
// channels).
enum Mode { kInterleaved, kExchanged, kFacing };

// 16 channels as pairs for the packed instructions: [4 j + 2 h + o] holds channels 8 j + 4 h + o and + 2 (of the lane's chunk
// j), so that interleaved partners lie in pairs next to one another.
struct Lane16 {
    float2 p[8];
};

__device__ __forceinline__ int channel_of(int k, bool second) { return (k >> 2) * 8 + (k >> 1 & 1) * 4 + (k & 1) + (second ? 2 : 0); }

__device__ __forceinline__ Lane16 unpack(const uint4 (&raw)[2])
{
    Lane16 v;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            v.p[4 * j + 2 * h] = make_float2(__uint_as_float(w[2 * h] << 16), __uint_as_float(w[2 * h + 1] << 16));
            v.p[4 * j + 2 * h + 1] = make_float2(__uint_as_float(w[2 * h] & 0xFFFF0000u), __uint_as_float(w[2 * h + 1] & 0xFFFF0000u));
        }
    }
    return v;
}

__device__ __forceinline__ uint32_t bf_pack(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ uint4 pack(const Lane16 &v, int j)
{
    const float2 *p = v.p + 4 * j;
    return make_uint4(bf_pack(p[0].x, p[1].x), bf_pack(p[0].y, p[1].y), bf_pack(p[2].x, p[3].x), bf_pack(p[2].y, p[3].y));
}

__device__ __forceinline__ float2 twice(float v) { return make_float2(v, v); }

__device__ __forceinline__ float rsqrt_normal(float x)   // of a normal number
{
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Sum over the kLanes neighbours that hold a head; the same bits in all of them (each step adds the same two numbers).
template <int kLanes>
__device__ __forceinline__ float head_sum(float v)
{
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

__device__ __forceinline__ float sum_of(const Lane16 &a, const Lane16 &b)   // of products
{
    float2 s0 = __fmul2_rn(a.p[0], b.p[0]), s1 = __fmul2_rn(a.p[1], b.p[1]);
#pragma unroll
    for (int k = 2; k < 8; k += 2) {
        s0 = __ffma2_rn(a.p[k], b.p[k], s0);
        s1 = __ffma2_rn(a.p[k + 1], b.p[k + 1], s1);
    }
    s0 = __fadd2_rn(s0, s1);
    return s0.x + s0.y;
}

// Squares of a row past 2^50 could leave FP32's range: such a row is taken times this (exact; what becomes subnormal is
// nothing next to the rest), without eps, which is nothing next to it either.
constexpr float kFarRow = 0x1p100f, kFarScale = 0x1p-80f;

// 1 / sqrt(mean + eps) of the rows of a warp, and what a far one was taken times (v then is too).
template <int kLanes>
__device__ __forceinline__ float2 norm_of(Lane16 &v, float per_channel, float eps)
{
    float sum = head_sum<kLanes>(sum_of(v, v)), f = 1.0f;
    if (__any_sync(0xFFFFFFFFu, !(sum < kFarRow))) {
        const bool far = !(sum < kFarRow);
        f = far ? kFarScale : 1.0f;
        eps = far ? 0.0f : eps;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v.p[k] = __fmul2_rn(v.p[k], twice(f));
        sum = head_sum<kLanes>(sum_of(v, v));
    }
    return make_float2(rsqrt_normal(fmaf(sum, per_channel, eps)), f);
}

__device__ __forceinline__ float weight_at(const void *weight, bool wide, int c)
{
    if (weight == nullptr)
        return 1.0f;
    return wide ? static_cast<const float *>(weight)[c]
                : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(weight)[c]) << 16);
}

// What a CTA keeps, and a warp: cosines and sines of the token it is at, by pair, or with kExchanged by channel (the sine then
// with its sign).
template <int kMode, int kLanes>
struct __align__(16) Tables {
    static constexpr bool kEach = kMode == kExchanged;
    float2 cs[kWarps][(kEach ? 16 : 8) * kLanes];
    float weight[kEach ? 4 : 2][16 * kLanes];   // of queries and keys, then those of each channel's partner
    float2 turns[8 * kLanes];                   // FP64 is slow here: once a pair, not once a pair and token
    uint32_t swap[kEach ? kWarps : 1][kEach ? kExchangeWords : 4];
    ushort2 members[kEach ? 8 * kLanes : 1];    // a pair's channels
    uint16_t partner[kEach ? 16 * kLanes : 2];  // a channel's (itself where it does not turn)
};

template <int kMode, int kLanes, class Side>
__device__ __forceinline__ void fill_tables(Tables<kMode, kLanes> &s, const Side &q, const Side &k, int dim, const RopeArgs &r)
{
    for (int p = threadIdx.x; p < r.pairs; p += kThreads)
        s.turns[p] = rope_turns(r, p);
    for (int i = threadIdx.x; i < 2 * dim; i += kThreads) {
        const bool first = i < dim;
        const int c = first ? i : i - dim;
        const void *weight = first ? q.weight : k.weight;
        const bool wide = (first ? q.wide : k.wide) != 0;
        s.weight[first ? 0 : 1][c] = weight_at(weight, wide, c);
        if constexpr (kMode == kExchanged) {
            const RopeChannel ch = rope_channel(r, c);
            s.weight[first ? 2 : 3][c] = weight_at(weight, wide, ch.partner);
            s.partner[c] = static_cast<uint16_t>(ch.partner);
            if (ch.pair >= 0 && ch.first)
                s.members[ch.pair] = make_ushort2(static_cast<unsigned short>(c), static_cast<unsigned short>(ch.partner));
        }
    }
    for (int p = threadIdx.x & 31; p < static_cast<int>(sizeof(s.cs[0]) / sizeof(float2)); p += 32)
        s.cs[threadIdx.x >> 5][p] = make_float2(1.0f, 0.0f);   // channels that do not turn
    __syncthreads();
}

// A warp's way through the work: units of 32 / kLanes heads of a token, its queries' and then its keys', token by token.  Warps
// take equal shares, whatever the numbers of tokens and heads are, and are on their own from one unit to the next.
struct Walk {
    int left, t, unit;   // units to do (an output of 2^31 of them would not fit any memory); the token; the unit of its heads

    __device__ __forceinline__ Walk(int tokens, int units)
    {
        const int64_t all = static_cast<int64_t>(tokens) * units, warps = static_cast<int64_t>(gridDim.x) * kWarps;
        const int64_t w = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5), at = w * all / warps;
        left = static_cast<int>((w + 1) * all / warps - at);
        t = static_cast<int>(at / units);
        unit = static_cast<int>(at - static_cast<int64_t>(t) * units);
    }
};

// A lane's 16 bytes of a later unit on their way into a place of its own (zeros where they are none of its).
__device__ __forceinline__ void copy_ahead(uint4 *to, const uint16_t *from, bool live)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(to))), "l"(from),
                 "r"(live ? 16 : 0)
                 : "memory");
}

__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int kLater>
__device__ __forceinline__ void wait_for_all_but()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(kLater) : "memory");
}

// The positions of token t, axis a's in lane a.
__device__ __forceinline__ float positions_of(const RopeArgs &r, int t, int tokens, int lane)
{
    return r.pairs > 0 && lane <= rope_axis(r, r.pairs - 1) && t < tokens ? r.positions[static_cast<int64_t>(t) * r.ld_positions + lane]
                                                                           : 0.0f;
}

template <int kMode, int kLanes>
__device__ __forceinline__ void fill_angles(Tables<kMode, kLanes> &s, const RopeArgs &r, float positions, int warp, int lane)
{
    __syncwarp();   // the last token's readers are done
    for (int p0 = 0; p0 < r.pairs; p0 += 32) {
        const int p = min(p0 + lane, r.pairs - 1);
        const float pos = __shfl_sync(0xFFFFFFFFu, positions, rope_axis(r, p));
        if (p0 + lane >= r.pairs)
            continue;
        const float2 v = rope_cos_sin(pos, s.turns[p]);
        if constexpr (kMode == kExchanged) {
            const ushort2 m = s.members[p];
            s.cs[warp][m.x] = make_float2(v.x, -v.y);
            s.cs[warp][m.y] = v;
        } else {
            s.cs[warp][p] = v;
        }
    }
    __syncwarp();
}

// Lane and chunk of a channel in kFacing: lane l holds pairs 8 l .. 8 l + 7, first members and second, and past those the
// channels that do not turn.
__device__ __forceinline__ int2 facing_place(const RopeArgs &r, int c)
{
    if (c >= 2 * r.pairs)
        return make_int2((r.pairs >> 3) + ((c - 2 * r.pairs) >> 4), (c - 2 * r.pairs) >> 3 & 1);
    const RopeChannel ch = rope_channel(r, c);
    return make_int2(ch.pair >> 3, ch.first ? 0 : 1);
}

// A lane's place: its two chunks (either may be none), and with kExchanged where each channel's partner stands in the warp's
// buffer.
template <int kMode, int kLanes>
struct Place {
    int c[2];          // first channel of each chunk
    bool live[2];
    bool still;        // kFacing: channels that do not turn
    int16_t from[kMode == kExchanged ? 16 : 1];

    __device__ __forceinline__ Place(const RopeArgs &r, int dim, int lane)
    {
        const int l = lane % kLanes, chunks = dim >> 3, half = (chunks + 1) >> 1;
        if constexpr (kMode == kFacing) {
            still = 8 * l >= r.pairs;
            int first_channel = 2 * r.pairs + 16 * (l - (r.pairs >> 3)), apart = 8;
            if (!still) {   // the section of pair 8 l
                int start = 0, end = r.end[0];
#pragma unroll
                for (int i = 0; i < H3FP4_ROPE_MAX_AXES - 1; ++i)
                    if (16 * l >= r.end[i]) {
                        start = r.end[i];
                        end = r.end[i + 1];
                    }
                first_channel = start / 2 + 8 * l;
                apart = (end - start) >> 1;
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int at = first_channel + j * apart;
                live[j] = at < dim;
                c[j] = live[j] ? at : 0;
            }
        } else {
            live[0] = l < half;
            live[1] = l < half && l + half < chunks;
            c[0] = live[0] ? 8 * l : 0;
            c[1] = live[1] ? 8 * (l + half) : 0;
        }
    }

    __device__ __forceinline__ void find_partners(const uint16_t *partner, int lane)
    {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int at = partner[c[i >> 3] + (i & 7)];
            from[i] = static_cast<int16_t>(2 * exchange_at<kLanes>(lane / kLanes, at) + (at & 1));
        }
    }
};

// Cosines and signed sines (+ where the partner is added) of a lane's channels.
template <int kMode, int kLanes>
__device__ __forceinline__ void angles_of(const Place<kMode, kLanes> &at, const float2 *cs, Lane16 &cosv, Lane16 &sinv)
{
    const int l = threadIdx.x % kLanes;
    if constexpr (kMode == kInterleaved) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float4 v = *reinterpret_cast<const float4 *>(cs + at.c[j] / 2 + 2 * h);   // two pairs
                cosv.p[4 * j + 2 * h] = cosv.p[4 * j + 2 * h + 1] = make_float2(v.x, v.z);
                sinv.p[4 * j + 2 * h] = make_float2(-v.y, -v.w);
                sinv.p[4 * j + 2 * h + 1] = make_float2(v.y, v.w);
            }
    } else if constexpr (kMode == kFacing) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4 v = *reinterpret_cast<const float4 *>(cs + 8 * l + 4 * h), w = *reinterpret_cast<const float4 *>(cs + 8 * l + 4 * h + 2);
            cosv.p[2 * h] = cosv.p[4 + 2 * h] = make_float2(v.x, w.x);
            cosv.p[2 * h + 1] = cosv.p[4 + 2 * h + 1] = make_float2(v.z, w.z);
            sinv.p[2 * h] = make_float2(-v.y, -w.y);
            sinv.p[2 * h + 1] = make_float2(-v.w, -w.w);
            sinv.p[4 + 2 * h] = make_float2(v.y, w.y);
            sinv.p[4 + 2 * h + 1] = make_float2(v.w, w.w);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {   // channels 4 h .. 4 h + 3
                const float4 v = *reinterpret_cast<const float4 *>(cs + at.c[j] + 4 * h), w = *reinterpret_cast<const float4 *>(cs + at.c[j] + 4 * h + 2);
                cosv.p[4 * j + 2 * h] = make_float2(v.x, w.x);
                cosv.p[4 * j + 2 * h + 1] = make_float2(v.z, w.z);
                sinv.p[4 * j + 2 * h] = make_float2(v.y, w.y);
                sinv.p[4 * j + 2 * h + 1] = make_float2(v.w, w.w);
            }
    }
}

template <int kMode, int kLanes>
__device__ __forceinline__ Lane16 weights_of(const Place<kMode, kLanes> &at, const float *weight)
{
    Lane16 w;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4 v = *reinterpret_cast<const float4 *>(weight + at.c[j] + 4 * h);
            w.p[4 * j + 2 * h] = make_float2(v.x, v.z);
            w.p[4 * j + 2 * h + 1] = make_float2(v.y, v.w);
        }
    return w;
}

// Each channel's partner.  kExchanged: from the raw words, and for channels that do not turn the channel itself; otherwise
// those get zeros (their sine is zero, but an infinity for a partner would make NaN of it).
template <int kMode, int kLanes>
__device__ __forceinline__ Lane16 partners_of(const Place<kMode, kLanes> &at, const RopeArgs &r, int dim, const Lane16 &v, const uint4 (&raw)[2],
                                              uint32_t *swap, int lane)
{
    Lane16 x;
    if constexpr (kMode == kExchanged) {
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (at.live[j]) {
                uint32_t *to = swap + exchange_at<kLanes>(lane / kLanes, at.c[j]);
                to[0] = raw[j].x;
                to[1] = raw[j].y;
                to[2] = raw[j].z;
                to[3] = raw[j].w;
            }
        __syncwarp();
        const uint16_t *half = reinterpret_cast<const uint16_t *>(swap);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            x.p[k] = make_float2(__uint_as_float(static_cast<uint32_t>(half[at.from[channel_of(k, false)]]) << 16),
                                 __uint_as_float(static_cast<uint32_t>(half[at.from[channel_of(k, true)]]) << 16));
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            x.p[k] = v.p[kMode == kInterleaved ? k ^ 1 : k ^ 4];
        if (kMode == kInterleaved && 2 * r.pairs < dim) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int c = at.c[k >> 2] + (channel_of(k, false) & 7);
                x.p[k].x = c < 2 * r.pairs ? x.p[k].x : 0.0f;
                x.p[k].y = c + 2 < 2 * r.pairs ? x.p[k].y : 0.0f;
            }
        }
        if (kMode == kFacing && at.still) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                x.p[k] = twice(0.0f);
        }
    }
    return x;
}

template <int kMode, int kLanes>
struct Shared : Tables<kMode, kLanes> {
    uint4 ring[kForwardStages][2][kThreads];
};

// kLanes: lanes of a head, a power of two; those past its chunks idle.
template <int kMode, int kLanes>
__global__ void __launch_bounds__(kThreads, kForwardCtas)
    norm_rope_kernel(NormSide qs, NormSide ks, int tokens, int q_units, int units, int dim, float eps, RopeArgs rope)
{
    constexpr int kPerWarp = 32 / kLanes, kStages = kForwardStages;
    extern __shared__ __align__(16) uint8_t dyn[];
    Shared<kMode, kLanes> &s = *reinterpret_cast<Shared<kMode, kLanes> *>(dyn);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / kLanes;
    Place<kMode, kLanes> place(rope, dim, lane);
    const Walk at(tokens, units);
    // Some units ahead: those of one side of a token lie a step apart.
    int to_copy = at.left, copy_t = at.t, copy_unit = at.unit, run = 0, head = 0, heads = 0;
    const uint16_t *xp = nullptr, *const some = qs.heads > 0 ? qs.x : ks.x;   // (an address for copies of nothing)
    int64_t x_step = 0;
    const auto fetch = [&](int first) {   // half of the ring; past the last unit, nothing
#pragma unroll
        for (int y = 0; y < kStages / 2 && to_copy > 0; ++y) {
            const int stage = first + y;
            if (run == 0) {
                const bool q = copy_unit < q_units;
                run = (q ? q_units : units) - copy_unit;
                head = (q ? copy_unit : copy_unit - q_units) * kPerWarp + sub;
                heads = q ? qs.heads : ks.heads;
                const int64_t xh = q ? qs.xh : ks.xh;
                xp = (q ? qs.x + copy_t * qs.xt : ks.x + copy_t * ks.xt) + head * xh;
                x_step = xh * kPerWarp;
                copy_unit = q && q_units < units ? q_units : 0;
                copy_t += copy_unit == 0 ? 1 : 0;
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
                copy_ahead(&s.ring[stage][j][threadIdx.x], (head < heads ? xp : some) + place.c[j], head < heads && place.live[j]);
            xp += x_step;
            head += kPerWarp;
            --run;
            --to_copy;
        }
        copies_end();
    };
    fetch(0);
    float positions = at.left > 0 ? positions_of(rope, at.t, tokens, lane) : 0.0f;
    fill_tables(s, qs, ks, dim, rope);
    if constexpr (kMode == kExchanged)
        place.find_partners(s.partner, lane);
    const float per_channel = 1.0f / static_cast<float>(dim);
    Lane16 a, b;
    int left = at.left, t = at.t, unit = at.unit, stage = 0;
    bool new_token = true;
    while (left > 0) {   // a side of a token, the same in the whole warp
        if (new_token) {
            fill_angles(s, rope, positions, warp, lane);
            positions = positions_of(rope, t + 1, tokens, lane);   // the next token's
        }
        const bool q = unit < q_units;
        {
            Lane16 sinv;
            angles_of(place, s.cs[warp], a, sinv);
            const float *weight = s.weight[q ? 0 : 1];
            const Lane16 w = weights_of(place, weight);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                a.p[k] = __fmul2_rn(a.p[k], w.p[k]);
            if constexpr (kMode == kExchanged) {
                const Lane16 other = weights_of(place, s.weight[q ? 2 : 3]);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    b.p[k] = __fmul2_rn(sinv.p[k], other.p[k]);
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    b.p[k] = __fmul2_rn(sinv.p[k], w.p[kMode == kInterleaved ? k ^ 1 : k ^ 4]);
            }
        }
        const int n = min(left, (q ? q_units : units) - unit), side_heads = q ? qs.heads : ks.heads;
        int h = (q ? unit : unit - q_units) * kPerWarp + sub;
        const int64_t oh = q ? qs.oh : ks.oh;
        uint16_t *op = (q ? qs.out + t * qs.ot : ks.out + t * ks.ot) + h * oh;
        for (int i = 0; i < n; ++i) {
            if ((stage & (kStages / 2 - 1)) == 0) {
                fetch(stage ^ kStages / 2);
                wait_for_all_but<1>();
            }
            const uint4 raw[2] = {s.ring[stage][0][threadIdx.x], s.ring[stage][1][threadIdx.x]};
            stage = (stage + 1) & (kStages - 1);
            Lane16 v = unpack(raw);
            const float2 norm = norm_of<kLanes>(v, per_channel, eps);
            Lane16 x = partners_of(place, rope, dim, v, raw, s.swap[kMode == kExchanged ? warp : 0], lane);
            if (kMode == kExchanged && norm.y != 1.0f) {   // (taken from the raw words)
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    x.p[k] = __fmul2_rn(x.p[k], twice(norm.y));
            }
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v.p[k] = __fmul2_rn(twice(norm.x), __ffma2_rn(v.p[k], a.p[k], __fmul2_rn(x.p[k], b.p[k])));
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (place.live[j] && h < side_heads)
                    *reinterpret_cast<uint4 *>(op + place.c[j]) = pack(v, j);
            op += kPerWarp * oh;
            h += kPerWarp;
        }
        left -= n;
        unit += n;
        new_token = unit == units;
        t += new_token ? 1 : 0;
        unit = new_token ? 0 : unit;
    }
}

template <int kMode, int kLanes>
struct GradShared : Tables<kMode, kLanes> {
    float4 sums[2][4][kThreads];   // dw of each thread's 16 channels, of both sides
    uint4 ring[kBackwardStages][4][kThreads];
};

// As above; a lane keeps its share of a side's dw in registers from one change of the side to the next, and the CTA leaves its
// own in parts [side][CTA][dim].
template <int kMode, int kLanes>
__global__ void __launch_bounds__(kThreads, kBackwardCtas)
    norm_rope_grad_kernel(NormGradSide qs, NormGradSide ks, int tokens, int q_units, int units, int dim, float eps, RopeArgs rope,
                          float *parts)
{
    constexpr int kPerWarp = 32 / kLanes, kStages = kBackwardStages;
    extern __shared__ __align__(16) uint8_t dyn[];
    GradShared<kMode, kLanes> &s = *reinterpret_cast<GradShared<kMode, kLanes> *>(dyn);
    auto &sums = s.sums;
    // What joins the parts may be scheduled as places fall free; it waits for this grid's end before it reads them.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / kLanes;
    Place<kMode, kLanes> place(rope, dim, lane);
    const Walk at(tokens, units);
    // Some units ahead, as above.
    int to_copy = at.left, copy_t = at.t, copy_unit = at.unit, run = 0, head = 0, heads = 0;
    const uint16_t *xp = nullptr, *gp = nullptr, *const some = qs.heads > 0 ? qs.x : ks.x;
    int64_t x_step = 0, g_step = 0;
    const auto fetch = [&](int first) {
#pragma unroll
        for (int y = 0; y < kStages / 2 && to_copy > 0; ++y) {
            const int stage = first + y;
            if (run == 0) {
                const bool q = copy_unit < q_units;
                run = (q ? q_units : units) - copy_unit;
                head = (q ? copy_unit : copy_unit - q_units) * kPerWarp + sub;
                heads = q ? qs.heads : ks.heads;
                const int64_t xh = q ? qs.xh : ks.xh, gh = q ? qs.gh : ks.gh;
                xp = (q ? qs.x + copy_t * qs.xt : ks.x + copy_t * ks.xt) + head * xh;
                gp = (q ? qs.dy + copy_t * qs.gt : ks.dy + copy_t * ks.gt) + head * gh;
                x_step = xh * kPerWarp;
                g_step = gh * kPerWarp;
                copy_unit = q && q_units < units ? q_units : 0;
                copy_t += copy_unit == 0 ? 1 : 0;
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                copy_ahead(&s.ring[stage][j][threadIdx.x], (head < heads ? xp : some) + place.c[j], head < heads && place.live[j]);
                copy_ahead(&s.ring[stage][2 + j][threadIdx.x], (head < heads ? gp : some) + place.c[j], head < heads && place.live[j]);
            }
            xp += x_step;
            gp += g_step;
            head += kPerWarp;
            --run;
            --to_copy;
        }
        copies_end();
    };
    fetch(0);
    float positions = at.left > 0 ? positions_of(rope, at.t, tokens, lane) : 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        sums[0][i][threadIdx.x] = sums[1][i][threadIdx.x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    fill_tables(s, qs, ks, dim, rope);
    if constexpr (kMode == kExchanged)
        place.find_partners(s.partner, lane);
    const float per_channel = 1.0f / static_cast<float>(dim);
    Lane16 dw, cosv, sinv;
#pragma unroll
    for (int k = 0; k < 8; ++k)
        dw.p[k] = twice(0.0f);
    const auto flush = [&](int side) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float4 &v = sums[side][i][threadIdx.x];
            const float4 w = v;
            v = make_float4(w.x + dw.p[2 * i].x, w.y + dw.p[2 * i].y, w.z + dw.p[2 * i + 1].x, w.w + dw.p[2 * i + 1].y);
            dw.p[2 * i] = dw.p[2 * i + 1] = twice(0.0f);
        }
    };
    int left = at.left, t = at.t, unit = at.unit, stage = 0;
    bool new_token = true;
    while (left > 0) {   // a side of a token, the same in the whole warp
        if (new_token) {
            fill_angles(s, rope, positions, warp, lane);
            positions = positions_of(rope, t + 1, tokens, lane);   // the next token's
            angles_of(place, s.cs[warp], cosv, sinv);
        }
        const bool q = unit < q_units;
        const int n = min(left, (q ? q_units : units) - unit), side_heads = q ? qs.heads : ks.heads;
        int h = (q ? unit : unit - q_units) * kPerWarp + sub;
        const int64_t oh = q ? qs.oh : ks.oh;
        uint16_t *op = (q ? qs.dx + t * qs.ot : ks.dx + t * ks.ot) + h * oh;
        for (int i = 0; i < n; ++i) {
            if ((stage & (kStages / 2 - 1)) == 0) {
                fetch(stage ^ kStages / 2);
                wait_for_all_but<1>();
            }
            const uint4 rx[2] = {s.ring[stage][0][threadIdx.x], s.ring[stage][1][threadIdx.x]};
            const uint4 rg[2] = {s.ring[stage][2][threadIdx.x], s.ring[stage][3][threadIdx.x]};
            stage = (stage + 1) & (kStages - 1);
            Lane16 g = unpack(rg);
            const Lane16 other = partners_of(place, rope, dim, g, rg, s.swap[kMode == kExchanged ? warp : 0], lane);
#pragma unroll
            for (int k = 0; k < 8; ++k)   // turned back: the sine's sign the other way round
                g.p[k] = __ffma2_rn(g.p[k], cosv.p[k], __fmul2_rn(other.p[k], make_float2(-sinv.p[k].x, -sinv.p[k].y)));
            Lane16 v = unpack(rx);
            const float2 norm = norm_of<kLanes>(v, per_channel, eps);
            const Lane16 w = weights_of(place, s.weight[q ? 0 : 1]);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                v.p[k] = __fmul2_rn(v.p[k], twice(norm.x));   // the normed value
                dw.p[k] = __ffma2_rn(g.p[k], v.p[k], dw.p[k]);
                g.p[k] = __fmul2_rn(g.p[k], w.p[k]);
            }
            const float along = -head_sum<kLanes>(sum_of(g, v)) * per_channel, r = norm.x * norm.y;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v.p[k] = __fmul2_rn(twice(r), __ffma2_rn(v.p[k], twice(along), g.p[k]));
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (place.live[j] && h < side_heads)
                    *reinterpret_cast<uint4 *>(op + place.c[j]) = pack(v, j);
            op += kPerWarp * oh;
            h += kPerWarp;
        }
        flush(q ? 0 : 1);
        left -= n;
        unit += n;
        new_token = unit == units;
        t += new_token ? 1 : 0;
        unit = new_token ? 0 : unit;
    }
    __syncthreads();
    // Channel c of each head that the CTA has held at a time, in the order of the threads.
    for (int i = threadIdx.x; i < 2 * dim; i += kThreads) {
        const int of_side = i < dim ? 0 : 1, c = i < dim ? i : i - dim;
        if ((of_side == 0 ? qs.dweight : ks.dweight) == nullptr)
            continue;
        const int chunk = c >> 3, half = ((dim >> 3) + 1) >> 1, e = c & 7;
        const int2 lane_of = kMode == kFacing ? facing_place(rope, c) : make_int2(chunk >= half ? chunk - half : chunk, chunk >= half ? 1 : 0);
        const int l = lane_of.x, k = 4 * lane_of.y + (e >> 2) * 2 + (e & 1);   // the lane, its pair, and the place there
        const float *from = reinterpret_cast<const float *>(&sums[of_side][k >> 1][l]) + (k & 1) * 2 + (e >> 1 & 1);
        float sum = 0.0f;
#pragma unroll 8
        for (int x = 0; x < kWarps * kPerWarp; ++x)
            sum += from[x * kLanes * 4];
        parts[(static_cast<int64_t>(of_side) * gridDim.x + blockIdx.x) * dim + c] = sum;
    }
}

constexpr int kJoinThreads = 1024;

// dw of 32 channels of a side: 32 warps sum every 32nd part each, then one the 32 sums.
__global__ void __launch_bounds__(kJoinThreads) weight_grad_kernel(float *q_dweight, float *k_dweight, const float *parts, int ctas, int dim)
{
    __shared__ float sums[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float *out = blockIdx.y == 0 ? q_dweight : k_dweight;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (out == nullptr)
        return;
    float sum = 0.0f;
    if (c < dim) {
#pragma unroll 8
        for (int p = warp; p < ctas; p += 32)
            sum += parts[(static_cast<int64_t>(blockIdx.y) * ctas + p) * dim + c];
    }
    sums[warp][lane] = sum;
    __syncthreads();
    if (warp != 0 || c >= dim)
        return;
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i)
        sum += sums[i][lane];
    out[c] = sum;
}

// Units of a token's heads, and CTAs of a call: as many waves of what the SMs hold as leave a warp kWaveUnits, or a unit a warp.
struct Split {
    int q_units, units, ctas;
};

Split split_of(int64_t tokens, int q_heads, int k_heads, int per_unit, int resident, int most_waves)
{
    const int q = (q_heads + per_unit - 1) / per_unit, units = q + (k_heads + per_unit - 1) / per_unit;
    const int64_t ctas = (tokens * units + kWarps - 1) / kWarps, waves = ctas / (int64_t(resident) * kWaveUnits);
    const int64_t most = resident * (waves < 1 ? 1 : waves < most_waves ? waves : most_waves);
    return Split{q, units, static_cast<int>(ctas < most ? ctas : most)};
}

Mode mode_of(const RopeArgs &r, int dim)
{
    if (r.layout == 0 || r.pairs == 0)
        return kInterleaved;
    for (int i = 0; i < H3FP4_ROPE_MAX_AXES; ++i)
        if (r.end[i] % 16 != 0)
            return kExchanged;
    return kFacing;
}

template <int kMode, int kLanes>
cudaError_t run(const NormSide &q, const NormSide &k, int64_t tokens, int dim, float eps, const RopeArgs &r, cudaStream_t st)
{
    const Split p = split_of(tokens, q.heads, k.heads, 32 / kLanes, kForwardCtas * sm_count(), kForwardWaves);
    constexpr int kSmem = sizeof(Shared<kMode, kLanes>);
    const cudaError_t e = allow_shared<norm_rope_kernel<kMode, kLanes>>(kSmem);
    if (e != cudaSuccess)
        return e;
    norm_rope_kernel<kMode, kLanes><<<p.ctas, kThreads, kSmem, st>>>(q, k, static_cast<int>(tokens), p.q_units, p.units, dim, eps, r);
    return cudaGetLastError();
}

int grad_ctas() { return kBackwardCtas * sm_count(); }

template <int kMode, int kLanes>
cudaError_t run_grad(const NormGradSide &q, const NormGradSide &k, int64_t tokens, int dim, float eps, const RopeArgs &r, float *parts,
                     cudaStream_t st)
{
    const Split p = split_of(tokens, q.heads, k.heads, 32 / kLanes, grad_ctas(), 1);
    if (p.ctas > 0) {
        constexpr int kSmem = sizeof(GradShared<kMode, kLanes>);
        cudaError_t e = allow_shared<norm_rope_grad_kernel<kMode, kLanes>>(kSmem);
        if (e != cudaSuccess)
            return e;
        norm_rope_grad_kernel<kMode, kLanes><<<p.ctas, kThreads, kSmem, st>>>(q, k, static_cast<int>(tokens), p.q_units, p.units, dim, eps, r,
                                                                              parts);
        if ((e = cudaGetLastError()) != cudaSuccess)
            return e;
    }
    if (q.dweight == nullptr && k.dweight == nullptr)
        return cudaSuccess;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(static_cast<unsigned>((dim + 31) / 32), 2);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = p.ctas > 0 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, weight_grad_kernel, q.dweight, k.dweight, static_cast<const float *>(parts), p.ctas, dim);
}

template <int kMode>
cudaError_t run_mode(const NormSide &q, const NormSide &k, int64_t tokens, int dim, float eps, const RopeArgs &r, cudaStream_t st)
{
    return dim <= 64 ? run<kMode, 4>(q, k, tokens, dim, eps, r, st) : dim <= 128 ? run<kMode, 8>(q, k, tokens, dim, eps, r, st)
                                                                                 : run<kMode, 16>(q, k, tokens, dim, eps, r, st);
}

template <int kMode>
cudaError_t run_grad_mode(const NormGradSide &q, const NormGradSide &k, int64_t tokens, int dim, float eps, const RopeArgs &r, float *parts,
                          cudaStream_t st)
{
    return dim <= 64    ? run_grad<kMode, 4>(q, k, tokens, dim, eps, r, parts, st)
           : dim <= 128 ? run_grad<kMode, 8>(q, k, tokens, dim, eps, r, parts, st)
                        : run_grad<kMode, 16>(q, k, tokens, dim, eps, r, parts, st);
}

}  // namespace

int64_t norm_grad_workspace(int dim) { return 2 * static_cast<int64_t>(grad_ctas()) * dim * 4; }

cudaError_t launch_norm_rope(const NormSide &q, const NormSide &k, int64_t tokens, int dim, float eps, const RopeArgs &r, cudaStream_t st)
{
    switch (mode_of(r, dim)) {
    case kInterleaved: return run_mode<kInterleaved>(q, k, tokens, dim, eps, r, st);
    case kFacing: return run_mode<kFacing>(q, k, tokens, dim, eps, r, st);
    default: return run_mode<kExchanged>(q, k, tokens, dim, eps, r, st);
    }
}

cudaError_t launch_norm_rope_grad(const NormGradSide &q, const NormGradSide &k, int64_t tokens, int dim, float eps, const RopeArgs &r,
                                  void *workspace, cudaStream_t st)
{
    float *parts = static_cast<float *>(workspace);
    switch (mode_of(r, dim)) {
    case kInterleaved: return run_grad_mode<kInterleaved>(q, k, tokens, dim, eps, r, parts, st);
    case kFacing: return run_grad_mode<kFacing>(q, k, tokens, dim, eps, r, parts, st);
    default: return run_grad_mode<kExchanged>(q, k, tokens, dim, eps, r, parts, st);
    }
}

}  // namespace h3fp4

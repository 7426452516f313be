// rope.cuh -- rotary positions with several axes: the channel layout, the
// angles and the rotation shared by rope.cu and the cache writer.
//
// A pair (a, b) at position p with frequency w turns by phi = p w.  The
// frequency comes in FP64 and is split once into turns per unit of position,
// w / 2 pi = hi + lo (two floats); p hi is formed with its rounding error (one
// fused multiply-add), the nearest whole number of turns is taken off exactly
// and the rest, at most half a turn, goes to sincospi.  So the angle's error
// is that of a number below one half, whatever the position.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "launch.h"

namespace h3fp4 {

constexpr int kRopeMaxPairs = 128;   // head_dim 256

// Turns per unit of position of pair `p`, as hi + lo.
__device__ __forceinline__ float2 rope_turns(const RopeArgs &r, int p)
{
    const double t = r.freqs[p] * 0.15915494309189533577;   // 1 / (2 pi)
    const float hi = static_cast<float>(t);
    return make_float2(hi, static_cast<float>(t - hi));
}

// Axis of pair p (p < r.pairs).
__device__ __forceinline__ int rope_axis(const RopeArgs &r, int p)
{
    int a = 0;
#pragma unroll
    for (int i = 0; i < H3FP4_ROPE_MAX_AXES - 1; ++i)
        a += 2 * p >= r.end[i] ? 1 : 0;   // axes past the last one end at the total, which 2 p never reaches
    return a;
}

__device__ __forceinline__ float2 rope_cos_sin(float pos, float2 turns)
{
    const float p = __fmul_rn(pos, turns.x);
    const float e = __fmaf_rn(pos, turns.y, __fmaf_rn(pos, turns.x, -p));
    const float t = (p - rintf(p)) + e;
    float s, c;
    sincospif(2.0f * t, &s, &c);
    return make_float2(c, s);
}

// Where channel c stands: its pair, its partner's channel, and whether it is
// the pair's first (a) or second (b) member.  pair < 0: not turned.
struct RopeChannel {
    int pair, partner;
    bool first;
};

__device__ __forceinline__ RopeChannel rope_channel(const RopeArgs &r, int c)
{
    if (c >= 2 * r.pairs)
        return RopeChannel{-1, c, true};
    if (r.layout == 0)
        return RopeChannel{c >> 1, c ^ 1, (c & 1) == 0};
    int start = 0, end = r.end[0];
#pragma unroll
    for (int i = 0; i < H3FP4_ROPE_MAX_AXES - 1; ++i)
        if (c >= r.end[i]) {
            start = r.end[i];
            end = r.end[i + 1];
        }
    const int h = (end - start) >> 1, l = c - start;
    const bool first = l < h;
    return RopeChannel{(start >> 1) + (first ? l : l - h), first ? c + h : c - h, first};
}

// One member of a pair in FP32: x cos -+ partner sin, `ss` carrying the sign.
__device__ __forceinline__ float rope_mix(float x, float partner, float cosv, float ss)
{
    return __fmaf_rn(x, cosv, __fmul_rn(partner, ss));
}

// A lane's eight channels c0 .. c0 + 7 of a head whose lanes are neighbours:
// which of them turn, which are a pair's first member, the pair of each, and
// (halves) where the partner stands in the warp's exchange buffer.
template <int kLayout>
struct RopeLane {
    uint32_t turned, first;
    int16_t pair[8], from[8];

    __device__ __forceinline__ RopeLane(const RopeArgs &r, int c0, int first_lane)
    {
        turned = first = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const RopeChannel ch = rope_channel(r, c0 + e);
            turned |= ch.pair >= 0 ? 1u << e : 0u;
            first |= ch.first ? 1u << e : 0u;
            pair[e] = static_cast<int16_t>(max(ch.pair, 0));
            from[e] = static_cast<int16_t>((ch.partner & 6) * 32 + 2 * (first_lane + (ch.partner >> 3)) + (ch.partner & 1));
        }
    }
};

// The partners of a lane's eight bf16 values (words w).  Interleaved pairs lie
// within the lane; halves meet in `swap`, 128 words of the warp's own: word i
// of each lane's four side by side, so that four stores and eight 16-bit reads
// meet no bank conflicts (20,000 tokens of 56 heads, 128 channels: 2 % faster
// than stored member by member).  Whole warp.
template <int kLayout>
__device__ __forceinline__ void rope_partners(const RopeLane<kLayout> &l, const uint32_t (&w)[4], uint32_t *swap, float (&partner)[8])
{
    if constexpr (kLayout == 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            partner[e ^ 1] = __uint_as_float((e & 1) != 0 ? w[e >> 1] & 0xFFFF0000u : w[e >> 1] << 16);
    } else {
        const int lane = threadIdx.x & 31;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i)
            swap[i * 32 + lane] = w[i];
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 8; ++e)
            partner[e] = __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(swap)[l.from[e]]) << 16);
    }
}

}  // namespace h3fp4

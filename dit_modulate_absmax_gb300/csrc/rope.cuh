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

}  // namespace h3fp4

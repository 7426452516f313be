// rope.cu -- rotary positions with several axes (h3fp4_rope_axes).
//
// Reads and writes each value once: 4 bytes a channel, bound by HBM (37,810
// tokens of 112 heads of 128 channels: 328 us, 6.6 TB/s).  Times here are those
// of a launch among others in a graph; launched by itself each takes 2 to 3 us
// longer (a token of 112 heads 6.2, and 14 called from Python; 5,042 tokens of
// 56 heads in halves 34 to 35).  A CTA takes 4 tokens
// (or 8) and a range of heads.  It first computes the cosines and sines of its
// tokens' pairs into shared memory (they serve every head), then two warps (or
// one) walk each token's heads, a lane holding 8 channels (16 bytes) and their
// coefficients in registers.
#include <cuda_bf16.h>

#include "rope.cuh"

namespace h3fp4 {
namespace {

constexpr int kThreads = 256;
constexpr int kInFlight = 4;                     // head groups in flight per warp

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t bf_pack(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

template <int kLayout, int kTokens>   // kTokens per CTA
__global__ void __launch_bounds__(kThreads)
    rope_kernel(const uint16_t *x, int64_t xt, int64_t xh, uint16_t *out, int64_t ot, int64_t oh, int64_t tokens,
                int heads, int dim, int heads_per_cta, RopeArgs r)
{
    constexpr int kWarpsPerToken = kThreads / 32 / kTokens;
    __shared__ float2 cs[kTokens][kRopeMaxPairs];
    __shared__ uint32_t swap[kLayout == 0 ? 1 : kThreads / 32][kLayout == 0 ? 1 : 128];
    __shared__ float2 turns[kRopeMaxPairs];   // FP64 is slow here: once a pair, not once a pair and token
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTokens;
    for (int p = threadIdx.x; p < r.pairs; p += kThreads)
        turns[p] = rope_turns(r, p);
    __syncthreads();
    for (int i = threadIdx.x; i < kTokens * r.pairs; i += kThreads) {
        const int tt = i / r.pairs, p = i - tt * r.pairs;
        if (t0 + tt < tokens) {
            const float pos = r.positions[(t0 + tt) * r.ld_positions + rope_axis(r, p)];
            cs[tt][p] = rope_cos_sin(r.inverse ? -pos : pos, turns[p]);
        }
    }
    __syncthreads();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tt = warp % kTokens;
    const int64_t t = t0 + tt;
    if (t >= tokens)
        return;
    const int per_head = dim >> 3, per_warp = 32 / per_head;
    const int sub = lane / per_head, c0 = (lane - sub * per_head) * 8;
    const bool live = sub < per_warp;

    const RopeLane<kLayout> of(r, c0, live ? sub * per_head : 0);   // (lanes without a head stay within the buffer)
    float cosv[8], ss[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float2 v = live ? cs[tt][of.pair[e]] : make_float2(1.0f, 0.0f);
        cosv[e] = v.x;
        ss[e] = (of.first >> e) & 1u ? -v.y : v.y;
    }
    const int begin = blockIdx.y * heads_per_cta, end = min(heads, begin + heads_per_cta);
    const int step = kWarpsPerToken * per_warp;
    const uint16_t *xp = x + t * xt + c0;
    uint16_t *op = out + t * ot + c0;
    for (int h0 = begin + (warp / kTokens) * per_warp; h0 < end; h0 += kInFlight * step) {   // the same in the whole warp
        uint4 raw[kInFlight];
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
            const int h = h0 + u * step + sub;
            raw[u] = live && h < end ? *reinterpret_cast<const uint4 *>(xp + h * xh) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
            const int h = h0 + u * step + sub;
            const uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
            float v[8], partner[8], y[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = bf_lo(w[i]);
                v[2 * i + 1] = bf_hi(w[i]);
            }
            rope_partners(of, w, swap[kLayout == 0 ? 0 : warp], partner);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                y[e] = (of.turned >> e) & 1u ? rope_mix(v[e], partner[e], cosv[e], ss[e]) : v[e];
            if (live && h < end)
                *reinterpret_cast<uint4 *>(op + h * oh) =
                    make_uint4(bf_pack(y[0], y[1]), bf_pack(y[2], y[3]), bf_pack(y[4], y[5]), bf_pack(y[6], y[7]));
        }
    }
}

}  // namespace

cudaError_t launch_rope(const uint16_t *x, int64_t xt, int64_t xh, uint16_t *out, int64_t ot, int64_t oh,
                        int64_t tokens, int heads, int dim, const RopeArgs &r, cudaStream_t st)
{
    // Halves take a warp some time to find its partners, which more tokens' worth of heads pay for: 8 tokens a CTA, a warp
    // each, once that gives every SM two CTAs (5,042 tokens of 56 heads 31.6 us, 33.4 with 4; 20,000: 100, 115; 500: 7.1,
    // 6.2; interleaved 29.0, 28.4).
    const int each = r.layout == 1 && tokens >= 16 * sm_count() ? 8 : 4;
    const int64_t groups = (tokens + each - 1) / each;
    // Few tokens: their heads are spread over several CTAs until every SM has one (a token of 112 heads: 3.1 us, 6.2 in one
    // CTA; 100 tokens 4.1, 6.5).
    const int per_pass = kThreads / 32 / each * (32 / (dim / 8));
    int64_t split = (sm_count() + groups - 1) / groups;
    const int64_t most = (heads + per_pass - 1) / per_pass;
    split = split < 1 ? 1 : split > most ? most : split;
    const int heads_per_cta = static_cast<int>(((heads + split - 1) / split + per_pass - 1) / per_pass) * per_pass;
    const dim3 grid(static_cast<unsigned>(groups), static_cast<unsigned>((heads + heads_per_cta - 1) / heads_per_cta));
    const auto kernel = r.layout == 0 ? rope_kernel<0, 4> : each == 4 ? rope_kernel<1, 4> : rope_kernel<1, 8>;
    kernel<<<grid, kThreads, 0, st>>>(x, xt, xh, out, ot, oh, tokens, heads, dim, heads_per_cta, r);
    return cudaGetLastError();
}

}  // namespace h3fp4

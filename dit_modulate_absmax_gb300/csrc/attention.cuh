// attention.cuh -- what the attention kernels share: the rows of a tile, what
// they see, and the queries' conversion to FP16.
//
// All of a cache head's query heads are taken together: row r of sequence b
// and cache head kh is query token r / group, head kh * group + r % group, so
// that keys and values are read once for the group.
//
// Softmax in base 2 with the values' scales inside: a key j in page P has
//     s'_j = S_j * (c * k_scale_P) + log2(v_scale_P),   S = q~ . k codes,
// where q~ is the query row times a power of two that brings its largest
// channel to [2^14, 2^15) (exact in FP16 but for channels below 2^-28 of it)
// and c = |softmax_scale| * log2(e) / that power (the sign goes into q~).
// The weight that meets the value codes is 2^(s'_j - m'), with m' the running
// maximum of s' less a constant: the largest CONTRIBUTION to the output, not
// the largest probability, stands near the top of FP16's range, and that range
// serves it whatever the pages' scales.
// Dividing a page's weights by its scale gives the softmax's own sum -- as long
// as the values' scales do not lie too far apart.  Where they may (far_scale),
// a key that counts in the sum may have a weight below FP32's smallest; from
// the first step with such a page on the sum has a reference of its own, the
// running maximum of S_j * (c * k_scale_P), and exponentials of its own.
//
// A part of the keys leaves its mean (output over sum) and log2 of its sum, or
// the sum and its reference; parts are joined as the means weighted by their
// sums, whatever those were kept against.
#pragma once

#include "kvcache.cuh"

namespace h3fp4 {

constexpr uint32_t ERR_ATTN_WAIT = 1u << 10;   // a pipeline wait gave up

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float lg2(float x)
{
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Positions [lo, hi) that query i of a sequence sees.
struct Span {
    int lo, hi;
};

__device__ __forceinline__ Span seen_by(const AttnArgs &a, const KvSequence &s, int i)
{
    const int pos = s.len - s.n + i;   // may be negative: nothing seen if causal
    Span r{0, s.len};
    if (a.causal)
        r.hi = min(s.len, pos + 1);
    if (a.window > 0)
        r.lo = max(0, pos - a.window + 1);   // pos >= -2^20 and window <= 2^31 - 1: no wrap
    if (r.hi <= r.lo)
        r.hi = r.lo = max(0, min(r.lo, s.len));   // empty
    return r;
}

// Power of two that brings a row whose largest magnitude is amax (a bf16
// pattern) to [2^14, 2^15), and its inverse; 1 for zero and non-finite rows.
__device__ __forceinline__ float2 row_power(uint32_t amax_bf16)
{
    const int e = static_cast<int>(amax_bf16 >> 7);   // biased exponent
    if (amax_bf16 == 0 || e == 255)
        return make_float2(1.0f, 1.0f);
    const int s = min(14 - (e - 127), 126);           // tiny rows: as far as a float's power goes
    return make_float2(__uint_as_float(static_cast<uint32_t>(s + 127) << 23),
                       __uint_as_float(static_cast<uint32_t>(127 - s) << 23));
}

// Largest magnitude among the two bf16 of each word, as a pattern.
__device__ __forceinline__ uint32_t bf16x2_absmax(uint32_t m2, uint32_t w) { return __vmaxu2(m2, w & 0x7FFF7FFFu); }

// Two bf16 times a power of two, as FP16.
__device__ __forceinline__ uint32_t bf16x2_to_half2(uint32_t w, float f)
{
    return pack_half2(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xFFFF0000u) * f);
}

// Whether a values' scale lies outside [2^-40, 2^41): a part with such a page keeps its sum against a reference of its own.
// All others lie within 2^81 of each other, where 2^-126 as the least weight leaves out keys below 2^-45 of the largest
// probability.  (Of the scales that a write sets, those of values from 2^49 on are outside.)
__device__ __forceinline__ bool far_scale(float scale) { return abs(static_cast<int>(__float_as_uint(scale) >> 23 & 0xFFu) - 127) > 40; }

// 1 / sum; a row that has seen nothing stays zero, NaN stays NaN.
__device__ __forceinline__ float reciprocal_sum(float sum) { return sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f; }

// ref + log2(sum), the sum's exponent taken apart: lg2's error is 2^-22 of its result, which near 0 is small and at a
// lifted reference or a scale of 2^-40 is not.  (Exact at powers of two.)
__device__ __forceinline__ float log_of_sum(float ref, float sum)
{
    if (!(sum >= 0x1p-126f && sum < INFINITY))
        return ref + lg2(sum);   // nothing, or not a number
    const uint32_t bits = __float_as_uint(sum);
    return (ref + static_cast<float>(static_cast<int>(bits >> 23) - 127)) + lg2(__uint_as_float((bits & 0x7FFFFFu) | 0x3F800000u));
}

// A sum against its own logarithm: 1, or still nothing, or NaN.
__device__ __forceinline__ float own_sum(float sum) { return sum > 0.0f ? 1.0f : sum; }

// 2^(log - top), nothing for two that have seen nothing.
__device__ __forceinline__ float of_top(float log, float top) { return ex2(log - (top == -INFINITY ? 0.0f : top)); }

// Its square root: a part's mean times this twice keeps what is left of very large values down to shares of 2^-252.
__device__ __forceinline__ float half_of_top(float log, float top) { return ex2(0.5f * (log - (top == -INFINITY ? 0.0f : top))); }

// Adds its * 2^log to a sum kept against top.  Products and sum are rounded apart, so that two lanes that exchange theirs
// come to the same bits.
__device__ __forceinline__ void add_log(float &top, float &sum, float log, float its)
{
    const float next = fmaxf(top, log);
    sum = __fadd_rn(__fmul_rn(sum, of_top(top, next)), __fmul_rn(its, of_top(log, next)));
    top = next;
}

// A page's table entry as the kernels keep it: id (< 0: none), the keys'
// scale, log2 of the values' scale and its inverse: that of the logarithm as
// it was rounded, so that the two cancel in the sum.
struct PageEntry {
    int32_t id;
    float ks, lv, inv_vs;
};

// Bit 7 of each byte that is an E4M3 NaN.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w)
{
    return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

// How a launch spreads the keys.  Tiles: `splits` parts of `chunk` keys each.
// Rows: clusters of `splits` CTAs, or `splits` CTAs with equal shares.
// part_rows: rows of partial results (a mean and its sum) that the workspace
// has room for.
struct SplitPlan {
    int32_t splits, chunk;
    int64_t part_rows;
    bool cluster;
};

SplitPlan plan_rows(const AttnShape &s);
cudaError_t launch_attention_rows(const AttnArgs &a, const SplitPlan &plan, float *logs, float *part, cudaStream_t st);
cudaError_t launch_attention_rows_timeout(const AttnArgs &a, const SplitPlan &plan, float *logs, float *part, uint64_t wait_ns,
                                          cudaStream_t st);   // 128 channels, 8 rows at most
SplitPlan plan_tile(const AttnShape &s);
cudaError_t launch_attention_tile(const AttnArgs &a, const SplitPlan &plan, float2 *stat, float *part, cudaStream_t st);
cudaError_t read_attention_tile_error(uint32_t *code);
cudaError_t read_attention_rows_error(uint32_t *code);

}  // namespace h3fp4

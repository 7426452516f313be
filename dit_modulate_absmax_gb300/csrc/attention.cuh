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

// Forms of the kernels: all that a query sees in one call; the same with first positions that stay visible under a window;
// the half over shared prefixes, and the half over a sequence's own keys that is joined to it.
enum Form { kWhole, kSinks, kPrefix, kOwn };

// Positions [lo, hi) that query i of a sequence sees.  With kSinks also those below a.sinks, as far as they lie below hi.
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

// Whether a sequence's rows, length and pages are within the arrays.  (A cache without pages has no arrays either: nothing of
// it may be read.)
__device__ __forceinline__ bool in_range(const AttnArgs &a, const KvSequence &s)
{
    return s.ok && s.len <= a.max_kv && (s.len <= 0 || ((s.len - 1) / a.cache.page_size < a.batch.ld_table && a.cache.num_pages != 0));
}

template <int kForm>
__device__ __forceinline__ bool seen(const AttnArgs &a, const Span &s, int tok)
{
    return tok < s.hi && (tok >= s.lo || (kForm == kSinks && tok < a.sinks));
}

// Whether [tok, tok + n) is seen as a whole by those that all see [lo, hi).
template <int kForm>
__device__ __forceinline__ bool all_seen(const AttnArgs &a, int lo, int hi, int tok, int n)
{
    return tok + n <= hi && (tok >= lo || (kForm == kSinks && tok + n <= a.sinks));
}

// The keys that some rows see, [lo, hi) and the sinks, as one run of places: place v below `keep` is position v, one from
// there on position v + gap.  Both are multiples of `align` (a page and a kernel's step at least), so that neither a page nor
// a step lies on both sides.  Sinks that reach to lo's step leave no gap.  Where there is one, lo lies past keep for all rows,
// so that a row sees place v if that is a sink or in [lo - gap, hi - gap): seen() holds of places too, with that span.
struct Fold {
    int keep, gap;
};

template <int kForm>
__device__ __forceinline__ Fold fold(const AttnArgs &a, int lo, int hi, int align)
{
    Fold f{0, 0};
    if (kForm == kSinks) {
        const int keep = (min(a.sinks, hi) + align - 1) & -align, from = lo & -align;
        if (from > keep)
            f = Fold{keep, from - keep};
    }
    return f;
}

template <int kForm>
__device__ __forceinline__ int position(const Fold &f, int v)
{
    return kForm == kSinks && v >= f.keep ? v + f.gap : v;
}

// Waits, where this kernel was launched to overlap with it, for the one before, whose half of a row is read from here on.
// Every thread of the kernel comes by here before it ends: what follows takes this grid's end for that of both.
template <int kForm>
__device__ __forceinline__ void after_prefix()
{
    if (kForm == kOwn)
        asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <int kForm>
__device__ __forceinline__ void let_next_start()
{
    if (kForm == kPrefix)
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
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

// The shares of a row's two halves whose sums have these logarithms: each mean counts half^2 inv.
struct Shares {
    float own, prefix, inv, log;   // square roots of the shares before inv; log2 of the whole sum
};

__device__ __forceinline__ Shares shares_of(float own_log, float prefix_log)
{
    const float top = fmaxf(own_log, prefix_log), total = of_top(own_log, top) + of_top(prefix_log, top);
    return Shares{half_of_top(own_log, top), half_of_top(prefix_log, top), reciprocal_sum(total), log_of_sum(top, total)};
}

// In place of the logarithm of a row whose group is out of range: a NaN that arithmetic does not make.  Such rows are left as
// they were, as those of a sequence that is.
constexpr uint32_t kRefusedLog = 0x7FBADBADu;

__device__ __forceinline__ bool refused(float log) { return __float_as_uint(log) == kRefusedLog; }

// Says so of a group's rows, as far as they lie in the arrays.  All threads of a CTA.
template <int kForm>
__device__ __forceinline__ void refuse_rows(const AttnArgs &a, const KvSequence &s)
{
    if (kForm != kPrefix)
        return;
    const int64_t first = s.row > 0 ? s.row : 0, end = min(s.row + s.n, a.tokens) * a.heads;
    for (int64_t i = first * a.heads + threadIdx.x; i < end; i += blockDim.x)
        a.half_log[i] = __uint_as_float(kRefusedLog);
}

// log2 of the sum of a row's prefix half; minus infinity for a row of no group.
__device__ __forceinline__ float prefix_log(const AttnArgs &a, int64_t row, int head)
{
    const bool covered = row >= a.prefix_cu[0] && row < a.prefix_cu[a.prefix_groups];
    return covered ? a.half_log[row * a.heads + head] : -INFINITY;
}

__device__ __forceinline__ float join_share(float own, float prefix, const Shares &s)
{
    return fmaf(prefix * s.prefix, s.prefix * s.inv, own * s.own * (s.own * s.inv));
}

// Writes four channels of a row: its output, its prefix half, or its output from both halves.
template <int kForm>
__device__ __forceinline__ void finish_row(const AttnArgs &a, int64_t row, int head, int c, float log, float4 mean)
{
    const int64_t at = row * a.heads + head;
    if (kForm == kPrefix) {
        *reinterpret_cast<float4 *>(a.half_mean + at * a.cache.head_dim + c) = mean;
        if (c == 0)
            a.half_log[at] = log;
        return;
    }
    if (kForm == kOwn) {
        const float other = prefix_log(a, row, head);
        if (refused(other))
            return;
        const Shares s = shares_of(log, other);
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (other != -INFINITY)
            v = *reinterpret_cast<const float4 *>(a.half_mean + at * a.cache.head_dim + c);
        mean = make_float4(join_share(mean.x, v.x, s), join_share(mean.y, v.y, s), join_share(mean.z, v.z, s), join_share(mean.w, v.w, s));
        log = s.log;
    }
    const __nv_bfloat162 x = __floats2bfloat162_rn(mean.x, mean.y), y = __floats2bfloat162_rn(mean.z, mean.w);
    *reinterpret_cast<uint2 *>(a.out + row * a.ot + head * a.oh + c) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y));
    if (a.lse != nullptr && c == 0)
        a.lse[at] = log * kLn2;
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
    int32_t warps = 0;   // rows: of a CTA
};

// For a launch that may begin while the one before it ends (it waits for that end itself).
inline cudaLaunchAttribute overlap_with_last()
{
    cudaLaunchAttribute a;
    a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a.val.programmaticStreamSerializationAllowed = 1;
    return a;
}

// Most tokens of a sequence for which a call is launched: groups that are all to be empty are looked at all the same, for one
// that is not is out of range.
inline int32_t most_rows(const KvBatch &b) { return b.max_tokens > 1 ? b.max_tokens : 1; }

// Most keys that a window of s.reach and s.sinks leave to rows of `tokens` neighbouring queries, folded in steps of up to 128.
inline int64_t folded_keys(const AttnShape &s, int64_t tokens)
{
    const int64_t kv = s.max_kv < 1 ? 1 : s.max_kv, most = int64_t(s.sinks) + s.reach + tokens + 256;
    return s.sinks > 0 && s.reach > 0 && most < kv ? most : kv;
}

SplitPlan plan_rows(const AttnShape &s);
cudaError_t launch_attention_rows(const AttnArgs &a, Form form, const SplitPlan &plan, float *logs, float *part, cudaStream_t st);
cudaError_t launch_attention_rows_timeout(const AttnArgs &a, const SplitPlan &plan, float *logs, float *part, uint64_t wait_ns,
                                          cudaStream_t st);   // 128 channels, 8 rows at most
SplitPlan plan_tile(const AttnShape &s);
cudaError_t launch_attention_tile(const AttnArgs &a, Form form, const SplitPlan &plan, float2 *stat, float *part, cudaStream_t st);
cudaError_t read_attention_tile_error(uint32_t *code);
cudaError_t read_attention_rows_error(uint32_t *code);

}  // namespace h3fp4

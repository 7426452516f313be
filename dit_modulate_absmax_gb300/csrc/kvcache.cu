// kvcache.cu -- writing keys and values into the 8-bit paged cache, and
// reading them back as bf16.
//
// A page and head is one block: page_size x head_dim values under one scale
// 2^e, the smallest power of two that keeps the block's largest magnitude
// within E4M3's 448.  Powers of two make code * scale exact in bf16 and the
// re-encoding of a block whose scale grows (tokens are appended one call
// after another) a shift of the exponents, so that repeated appends do not
// round the same value again and again.
//
// Writing moves 3 bytes a value and reading 3, both bound by HBM.  A CTA of
// the writer holds a head's new keys and values of its page in registers
// between the maximum and the encoding, so that each is read once, and goes on
// to the next with one barrier between, its loads under way meanwhile; the
// cosines and sines of its tokens serve all its heads.  37,810 tokens of 56
// heads of 128 channels are read back in 240 us, at the rate of a plain copy;
// 5,042 such tokens are written in 45 us (4.8 TB/s), with a rotation in 68 (in
// halves 98): neither HBM (35 %) nor issue (62 %) is full there, so that form
// has no bound yet.
#include <type_traits>

#include "kvcache.cuh"
#include "rope.cuh"

namespace h3fp4 {
namespace {

__device__ uint32_t g_error;

constexpr int kMaxThreads = 1024;
constexpr int kReadThreads = 256;
constexpr int kReadTurns = 4;             // chunks of keys and of values in flight per thread
constexpr int kScaleExpMin = -40, kScaleExpMax = 119;

__device__ __forceinline__ uint32_t bf_pack(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Largest finite magnitude of eight bf16 values as a bf16 pattern, with bit 16
// set if any of them is not finite.
__device__ __forceinline__ uint32_t finite_absmax8(const uint4 &v)
{
    const uint32_t w[4] = {v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu, v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu};
    const uint32_t m2 = __vmaxu2(__vmaxu2(w[0], w[1]), __vmaxu2(w[2], w[3]));
    uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
    if (m >= 0x7F80u) {   // rare: look at each value
        m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = w[i] & 0xFFFFu, hi = w[i] >> 16;
            m = max(m, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
        }
        m |= 0x10000u;
    }
    return m;
}

// 2^e with the smallest e in [-40, 119] such that amax <= 448 * 2^e; 448 is
// 1.75 * 2^8, so e is amax's exponent less 8, plus one if its significand is
// above 1.75.
__device__ __forceinline__ float block_scale_of(uint32_t amax_bf16)
{
    const int biased = static_cast<int>(((amax_bf16 << 16) + 0x1FFFFFu) >> 23);
    const int e = min(max(biased - 127 - 8, kScaleExpMin), kScaleExpMax);
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// x / scale: an exact multiplication where the scale is a power of two (those
// this writer chose), a division by a scale that a caller put there.
struct Divisor {
    float scale, inv;
    bool pow2;
};

__device__ __forceinline__ Divisor divisor(float scale)
{
    return Divisor{scale, __frcp_rn(scale), (__float_as_uint(scale) & 0x7FFFFFu) == 0};
}

__device__ __forceinline__ float over(float x, const Divisor &d)
{
    return d.pow2 ? __fmul_rn(x, d.inv) : __fdiv_rn(x, d.scale);
}

// Codes of eight values under a power-of-two scale, its inverse given.
__device__ __forceinline__ uint2 encode8_pow2(const uint4 &v, float inv)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 q = __fmul2_rn(make_float2(bf_lo(w[i]), bf_hi(w[i])), make_float2(inv, inv));
        c[i] = floats_to_e4m3x2(q.x, q.y);
    }
    return make_uint2(__byte_perm(c[0], c[1], 0x5410), __byte_perm(c[2], c[3], 0x5410));
}

// ... under any scale, with values that may not be finite: infinities would
// saturate, they become NaN like NaNs.
__device__ __noinline__ uint2 encode8_any(uint4 v, Divisor d)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[2] = {0, 0};
    for (int i = 0; i < 8; ++i) {
        const uint32_t x = w[i >> 1] >> (16 * (i & 1)) & 0xFFFFu;
        const uint32_t c = (x & 0x7F80u) == 0x7F80u ? 0x7Fu : floats_to_e4m3x2(over(__uint_as_float(x << 16), d), 0.0f) & 0xFFu;
        o[i >> 2] |= c << (8 * (i & 3));
    }
    return make_uint2(o[0], o[1]);
}

__device__ __forceinline__ uint32_t reencode4(uint32_t c, float was, const Divisor &d)
{
    const float2 a = e4m3x2_to_float2(c & 0xFFFFu), b = e4m3x2_to_float2(c >> 16);
    return floats_to_e4m3x2(over(__fmul_rn(a.x, was), d), over(__fmul_rn(a.y, was), d)) |
           floats_to_e4m3x2(over(__fmul_rn(b.x, was), d), over(__fmul_rn(b.y, was), d)) << 16;
}

struct WriteArgs {
    KvCache cache;
    KvBatch batch;
    const uint16_t *x[2];            // keys, values
    int64_t token_stride[2], head_stride[2];
    int64_t tokens;
    RopeArgs rope;                   // pairs = 0: none
};

// One CTA: a page's blocks of every head in [blockIdx.x * heads_per_cta, ...).
// kPer chunks of 8 values per thread cover the page (kPer * blockDim.x * 8 =
// page * dim), all at the same channels.  kRope: 0 none, 1 interleaved, 2 halves.
// Its largest launch, 1,024 threads (pages of 128 with 128 channels, rotated),
// leaves every form 64 registers: <2, 2> spills 64 bytes, <4, 0> 20.
template <int kPer, int kRope>
__global__ void __launch_bounds__(kMaxThreads) write_kernel(WriteArgs a, int heads_per_cta)
{
    extern __shared__ __align__(16) float2 cs[];                              // [page][dim / 2], with a rotation
    __shared__ uint32_t warp_max[2][kMaxThreads / 32];
    __shared__ uint32_t swap[kRope == 2 ? kMaxThreads / 32 : 1][kRope == 2 ? 128 : 1];
    const int b = blockIdx.z, page = a.cache.page_size, dim = a.cache.head_dim, heads = a.cache.heads;
    const KvSequence s = kv_sequence(a.batch, b, a.tokens);
    // positions in 64 bits: lengths near 2^31 must not wrap
    const int64_t last = static_cast<int64_t>(s.len) + s.n;
    if (!s.ok || (s.n > 0 && (last - 1) / page >= a.batch.ld_table)) {
        if (threadIdx.x == 0)
            atomicOr(&g_error, ERR_KV_RANGE);
        return;
    }
    const int64_t block = static_cast<int64_t>(s.len) / page + blockIdx.y, p0 = block * page;
    if (s.n == 0 || p0 >= last)
        return;
    const int32_t id = a.batch.page_table[b * a.batch.ld_table + block];
    if (id < 0 || id >= a.cache.num_pages) {
        if (threadIdx.x == 0)
            atomicOr(&g_error, ERR_KV_RANGE);
        return;
    }
    const int lo = static_cast<int>(s.len > p0 ? s.len - p0 : 0);            // the page's tokens [lo, hi) are new
    const int hi = static_cast<int>(last - p0 < page ? last - p0 : page);
    const int64_t row0 = s.row + p0 - s.len;                                  // row of the page's token 0

    const int per_row = dim >> 3, t0 = threadIdx.x / per_row, c0 = (threadIdx.x - t0 * per_row) * 8;
    const int t_step = blockDim.x / per_row;
    const int h0 = blockIdx.x * heads_per_cta, h_end = min(heads, h0 + heads_per_cta);
    const auto load = [&](int kv, int h, uint4 (&v)[kPer]) {
        const uint16_t *x = a.x[kv] + (row0 + t0) * a.token_stride[kv] + h * a.head_stride[kv] + c0;
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const int t = t0 + u * t_step;
            v[u] = t >= lo && t < hi ? *reinterpret_cast<const uint4 *>(x + static_cast<int64_t>(u * t_step) * a.token_stride[kv])
                                     : make_uint4(0, 0, 0, 0);
        }
    };
    uint4 x[2][kPer];
    load(0, h0, x[0]);
    // Where a token's row of `cs` holds pair p.  Halves: a lane's eight pairs apart, so that lanes side by side read pairs
    // side by side (5,042 tokens of 56 heads: 98 us; in order, with 8-way bank conflicts, 114 us).
    const auto place = [&](int p) { return kRope == 2 ? (p & 7) * (dim >> 4) + (p >> 3) : p; };
    if constexpr (kRope != 0) {
        __shared__ float2 turns[64];   // FP64 is slow here: once a pair, not once a pair and token
        for (int p = threadIdx.x; p < a.rope.pairs; p += blockDim.x)
            turns[p] = rope_turns(a.rope, p);
        __syncthreads();
        for (int i = threadIdx.x; i < page * (dim / 2); i += blockDim.x) {
            const int t = i / (dim / 2), p = i - t * (dim / 2);
            if (t >= lo && t < hi && p < a.rope.pairs) {
                const float pos = a.rope.positions[(row0 + t) * a.rope.ld_positions + rope_axis(a.rope, p)];
                cs[t * (dim / 2) + place(p)] = rope_cos_sin(a.rope.inverse ? -pos : pos, turns[p]);
            }
        }
        __syncthreads();
    }
    const RopeLane<kRope == 2 ? 1 : 0> lane_of(a.rope, c0, (threadIdx.x & 31) / per_row * per_row);

    // One of a head's two blocks, whose values are in registers.
    const auto block_of = [&](auto kv_constant, int h) {
        constexpr int kKv = decltype(kv_constant)::value;
        const int64_t bh = static_cast<int64_t>(id) * heads + h;
        float *const scale_at = (kKv == 0 ? a.cache.k_scale : a.cache.v_scale) + bh;
        const float was = lo > 0 ? *scale_at : 0.0f;
        if constexpr (kRope != 0 && kKv == 0) {
#pragma unroll
            for (int u = 0; u < kPer; ++u) {
                const int t = t0 + u * t_step;
                uint32_t w[4] = {x[0][u].x, x[0][u].y, x[0][u].z, x[0][u].w};
                float partner[8];
                rope_partners(lane_of, w, swap[kRope == 2 ? threadIdx.x >> 5 : 0], partner);
                if (t < lo || t >= hi)
                    continue;
                const float2 *f = cs + t * (dim / 2);
                float2 turn[8];   // of each channel
                if constexpr (kRope == 1) {
                    const float4 *g = reinterpret_cast<const float4 *>(f + (c0 >> 1));
                    const float4 q0 = g[0], q1 = g[1];
                    turn[0] = turn[1] = make_float2(q0.x, q0.y);
                    turn[2] = turn[3] = make_float2(q0.z, q0.w);
                    turn[4] = turn[5] = make_float2(q1.x, q1.y);
                    turn[6] = turn[7] = make_float2(q1.z, q1.w);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        turn[e] = f[place(lane_of.pair[e])];
                }
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float2 v = turn[e];
                    const bool first = kRope == 1 ? (e & 1) == 0 : (lane_of.first >> e & 1u) != 0;
                    y[e] = rope_mix((e & 1) != 0 ? bf_hi(w[e >> 1]) : bf_lo(w[e >> 1]), partner[e], v.x, first ? -v.y : v.y);
                }
                if (lane_of.turned != 0xFFu)   // channels past the axes
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if ((lane_of.turned >> e & 1u) == 0)
                            y[e] = (e & 1) != 0 ? bf_hi(w[e >> 1]) : bf_lo(w[e >> 1]);
                x[0][u] = make_uint4(bf_pack(y[0], y[1]), bf_pack(y[2], y[3]), bf_pack(y[4], y[5]), bf_pack(y[6], y[7]));
            }
        }
        uint32_t m = 0, odd = 0;   // maximum; chunks with a value that is not finite
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const uint32_t f = finite_absmax8(x[kKv][u]);
            odd |= (f >> 16) << u;
            m = max(m, f & 0xFFFFu);
        }
        m = __reduce_max_sync(0xFFFFFFFFu, m);
        if ((threadIdx.x & 31) == 0)
            warp_max[kKv][threadIdx.x >> 5] = m;
        __syncthreads();   // and the old scale is read; the next block uses the other half of warp_max
        m = 0;
        for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w)
            m = max(m, warp_max[kKv][w]);
        float scale = block_scale_of(m);
        if (lo > 0)
            scale = fmaxf(scale, was);
        const Divisor d = divisor(scale);
        if (threadIdx.x == 0)
            *scale_at = scale;
        const bool grown = lo > 0 && scale != was;
        uint2 *codes = reinterpret_cast<uint2 *>((kKv == 0 ? a.cache.k_codes : a.cache.v_codes) + bh * page * dim) + threadIdx.x;
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const int t = t0 + u * t_step;
            uint2 *dst = codes + u * blockDim.x;
            if (t >= lo && t < hi) {
                *dst = d.pow2 && ((odd >> u) & 1u) == 0 ? encode8_pow2(x[kKv][u], d.inv) : encode8_any(x[kKv][u], d);
            } else if (t < lo && grown) {
                const uint2 c = *dst;
                *dst = make_uint2(reencode4(c.x, was, d), reencode4(c.y, was, d));
            }
        }
    };
    for (int h = h0; h < h_end; ++h) {   // one block's loads are on their way while the other is encoded
        load(1, h, x[1]);
        block_of(std::integral_constant<int, 0>{}, h);
        if (h + 1 < h_end)
            load(0, h + 1, x[0]);
        block_of(std::integral_constant<int, 1>{}, h);
    }
}

struct ReadArgs {
    KvCache cache;
    KvBatch batch;
    uint16_t *x[2];
    int64_t token_stride[2], head_stride[2];
    int64_t tokens;
};

__device__ __forceinline__ uint32_t decode2(uint32_t c, float scale)
{
    const float2 f = e4m3x2_to_float2(c);
    const __nv_bfloat162 v = __floats2bfloat162_rn(__fmul_rn(f.x, scale), __fmul_rn(f.y, scale));
    return *reinterpret_cast<const uint32_t *>(&v);
}

// One CTA: a page of a head, or of several where that has fewer codes than a turn
// of all threads (pages of 16, 64 channels, 51 heads of 31 ragged sequences: 33
// us, 92 a head each); 8 codes a thread and turn (16-byte stores side by side:
// 16 codes a thread, whose two stores leave gaps for each other, took 10 %
// longer), several in flight.  Registers for 5 CTAs an SM: 37,810 tokens of 56
// heads 240 us (for 4: 249, for 6: 283).
__global__ void __launch_bounds__(kReadThreads, 5) read_kernel(ReadArgs a, int heads_per_cta)
{
    const int b = blockIdx.z, page = a.cache.page_size, dim = a.cache.head_dim, heads = a.cache.heads;
    const KvSequence s = kv_sequence(a.batch, b, a.tokens);
    const int64_t last = static_cast<int64_t>(s.len) + s.n;
    if (!s.ok || (s.n > 0 && (last - 1) / page >= a.batch.ld_table)) {
        if (threadIdx.x == 0)
            atomicOr(&g_error, ERR_KV_RANGE);
        return;
    }
    const int64_t block = static_cast<int64_t>(s.len) / page + blockIdx.y, p0 = block * page;
    if (s.n == 0 || p0 >= last)
        return;
    const int32_t id = a.batch.page_table[b * a.batch.ld_table + block];
    if (id < 0 || id >= a.cache.num_pages) {
        if (threadIdx.x == 0)
            atomicOr(&g_error, ERR_KV_RANGE);
        return;
    }
    const int lo = static_cast<int>(s.len > p0 ? s.len - p0 : 0);
    const int hi = static_cast<int>(last - p0 < page ? last - p0 : page);
    const int row_log = dim == 128 ? 4 : 3, head_log = row_log + 31 - __clz(page);   // chunks of a row, of a page and head
    const int h0 = blockIdx.x * heads_per_cta, n = min(heads_per_cta, heads - h0) << head_log;
    const int64_t row0 = s.row + p0 - s.len, bh = static_cast<int64_t>(id) * heads + h0, at = bh * page * dim;
    for (int i0 = threadIdx.x; i0 < n; i0 += kReadTurns * blockDim.x) {
        uint2 q[kReadTurns][2];
        float scale[kReadTurns][2];
#pragma unroll
        for (int u = 0; u < kReadTurns; ++u) {
            const int i = i0 + u * blockDim.x, t = (i >> row_log) & (page - 1);
#pragma unroll
            for (int kv = 0; kv < 2; ++kv)
                if (i < n && t >= lo && t < hi && a.x[kv] != nullptr) {
                    q[u][kv] = *reinterpret_cast<const uint2 *>((kv == 0 ? a.cache.k_codes : a.cache.v_codes) + at + 8 * i);
                    scale[u][kv] = (kv == 0 ? a.cache.k_scale : a.cache.v_scale)[bh + (i >> head_log)];
                }
        }
#pragma unroll
        for (int u = 0; u < kReadTurns; ++u) {
            const int i = i0 + u * blockDim.x, t = (i >> row_log) & (page - 1), c = (i & ((1 << row_log) - 1)) * 8;
            const int h = h0 + (i >> head_log);
#pragma unroll
            for (int kv = 0; kv < 2; ++kv)
                if (i < n && t >= lo && t < hi && a.x[kv] != nullptr) {
                    const uint2 v = q[u][kv];
                    const float f = scale[u][kv];
                    *reinterpret_cast<uint4 *>(a.x[kv] + (row0 + t) * a.token_stride[kv] + h * a.head_stride[kv] + c) =
                        make_uint4(decode2(v.x & 0xFFFFu, f), decode2(v.x >> 16, f), decode2(v.y & 0xFFFFu, f), decode2(v.y >> 16, f));
                }
        }
    }
}

template <auto kKernel>
struct kernel_constant {
    static constexpr auto value = kKernel;
};

// Heads that a CTA takes one after another: so many that no more than `per_sm`
// CTAs come to an SM, but `most` at most (where the grid is many waves anyway).
// 5,042 tokens of 56 heads, with a rotation: 68 us with 8 heads, 72 with 6 (a
// second wave), 76 with 12, 127 with one; plain 45 us with 4, 47 with one.
// per_sm is what fits with the 256 threads and more of those sizes; of smaller
// CTAs (64 threads, see launch_kv_write) more would fit, and the rule gives
// each of them more heads than filling the SMs takes.
int heads_each(const KvCache &cache, const KvBatch &batch, unsigned blocks, int per_sm, int most)
{
    const int64_t slots = static_cast<int64_t>(sm_count()) * per_sm;
    const int64_t n = (static_cast<int64_t>(blocks) * batch.batch * cache.heads + slots - 1) / slots;
    return n < 1 ? 1 : n > most ? most : static_cast<int>(n);
}

}  // namespace

cudaError_t launch_kv_write(const KvCache &cache, const KvBatch &batch, const uint16_t *k, int64_t kt, int64_t kh,
                            const uint16_t *v, int64_t vt, int64_t vh, int64_t tokens, const RopeArgs &rope,
                            cudaStream_t st)
{
    WriteArgs a{cache, batch, {k, v}, {kt, vt}, {kh, vh}, tokens, rope};
    const int chunks = cache.page_size * cache.head_dim / 8;
    // A rotation needs registers of its own: two chunks of keys and of values a thread at most, else four (5,042 tokens of
    // 56 heads of 128, pages of 64: 72 us turned with two chunks, 71 with four, in halves 98 and 123; plain 54 and 46).
    const int per = rope.pairs > 0 ? 2 : 4;
    // Fewer threads with more loads each, down to 64, are faster where pages are full of new tokens (5 prompts of 3,001
    // tokens, 16 heads of 64, from cold caches: 22.5 us, 29.7 with 256 at least), but not where few are (64 single tokens:
    // 10.2, 8.2).
    const int least = batch.max_tokens < cache.page_size ? 256 : 64;
    const int threads = chunks < least ? chunks : chunks / per < least ? least : chunks / per;
    const unsigned blocks = static_cast<unsigned>((batch.max_tokens + cache.page_size - 2) / cache.page_size + 1);
    const int heads_per_cta = heads_each(cache, batch, blocks, rope.pairs > 0 ? 4 : 8, rope.pairs > 0 ? 8 : 4);
    const dim3 grid(static_cast<unsigned>((cache.heads + heads_per_cta - 1) / heads_per_cta), blocks,
                    static_cast<unsigned>(batch.batch));
    const int smem = rope.pairs > 0 ? cache.page_size * cache.head_dim / 2 * static_cast<int>(sizeof(float2)) : 0;
    const auto turned = [&](auto kernel_of) {
        constexpr auto kernel = decltype(kernel_of)::value;
        const cudaError_t e = allow_shared<kernel>(64 * 1024);
        if (e == cudaSuccess)
            kernel<<<grid, threads, smem, st>>>(a, heads_per_cta);
        return e != cudaSuccess ? e : cudaGetLastError();
    };
    const int each = chunks / threads;
    if (rope.pairs == 0) {
        if (each == 1)
            write_kernel<1, 0><<<grid, threads, 0, st>>>(a, heads_per_cta);
        else if (each == 2)
            write_kernel<2, 0><<<grid, threads, 0, st>>>(a, heads_per_cta);
        else
            write_kernel<4, 0><<<grid, threads, 0, st>>>(a, heads_per_cta);
        return cudaGetLastError();
    }
    if (rope.layout == 0)
        return each == 1 ? turned(kernel_constant<write_kernel<1, 1>>{}) : turned(kernel_constant<write_kernel<2, 1>>{});
    return each == 1 ? turned(kernel_constant<write_kernel<1, 2>>{}) : turned(kernel_constant<write_kernel<2, 2>>{});
}

cudaError_t launch_kv_read(const KvCache &cache, const KvBatch &batch, uint16_t *k, int64_t kt, int64_t kh,
                           uint16_t *v, int64_t vt, int64_t vh, int64_t tokens, cudaStream_t st)
{
    ReadArgs a{cache, batch, {k, v}, {kt, vt}, {kh, vh}, tokens};
    const unsigned blocks = static_cast<unsigned>((batch.max_tokens + cache.page_size - 2) / cache.page_size + 1);
    const int block = cache.page_size * cache.head_dim, turn = 8 * kReadThreads * kReadTurns;
    const int heads_per_cta = block >= turn ? 1 : turn / block < cache.heads ? turn / block : cache.heads;
    const dim3 grid(static_cast<unsigned>((cache.heads + heads_per_cta - 1) / heads_per_cta), blocks,
                    static_cast<unsigned>(batch.batch));
    read_kernel<<<grid, kReadThreads, 0, st>>>(a, heads_per_cta);
    return cudaGetLastError();
}

cudaError_t read_kvcache_error(uint32_t *code)
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

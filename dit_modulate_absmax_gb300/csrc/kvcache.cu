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
// the writer holds its block's new values in registers between the maximum
// and the encoding, so that each is read once.
#include "kvcache.cuh"
#include "rope.cuh"

namespace h3fp4 {
namespace {

__device__ uint32_t g_error;

constexpr int kThreads = 256;
constexpr int kScaleExpMin = -40, kScaleExpMax = 119;

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

__device__ __forceinline__ uint32_t encode2(uint32_t w, const Divisor &d)
{
    return floats_to_e4m3x2(over(bf_lo(w), d), over(bf_hi(w), d));
}

__device__ __forceinline__ uint2 encode8(const uint4 &v, const Divisor &d, bool all_finite)
{
    uint32_t lo = encode2(v.x, d) | encode2(v.y, d) << 16, hi = encode2(v.z, d) | encode2(v.w, d) << 16;
    if (!all_finite) {   // infinities would saturate: they become NaN like NaNs
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (((w[i >> 1] >> (16 * (i & 1))) & 0x7F80u) == 0x7F80u) {
                uint32_t &o = i < 4 ? lo : hi;
                o = (o & ~(0xFFu << (8 * (i & 3)))) | 0x7Fu << (8 * (i & 3));
            }
        }
    }
    return make_uint2(lo, hi);
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

// Maximum over the CTA, in every thread.
__device__ __forceinline__ uint32_t cta_max(uint32_t v, uint32_t *warp_max)
{
    v = __reduce_max_sync(0xFFFFFFFFu, v);
    __syncthreads();   // the last call's readers are done
    if ((threadIdx.x & 31) == 0)
        warp_max[threadIdx.x >> 5] = v;
    __syncthreads();
    uint32_t m = 0;
    for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w)
        m = max(m, warp_max[w]);
    return m;
}

// One CTA: a page's block of every head in [blockIdx.x * heads_per_cta, ...).
// kPer chunks of 8 values per thread cover the page (kPer * blockDim.x * 8 = page * dim).
template <int kPer>
__global__ void __launch_bounds__(kThreads) write_kernel(WriteArgs a, int heads_per_cta)
{
    extern __shared__ __align__(16) uint8_t dyn[];
    __shared__ uint32_t warp_max[kThreads / 32];
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

    const bool turn = a.rope.pairs > 0;
    float2 *cs = reinterpret_cast<float2 *>(dyn);                             // [page][pairs]
    uint16_t *tile = reinterpret_cast<uint16_t *>(dyn + sizeof(float2) * page * a.rope.pairs);   // [page][dim]
    if (turn)
        for (int i = threadIdx.x; i < page * a.rope.pairs; i += blockDim.x) {
            const int t = i / a.rope.pairs, p = i - t * a.rope.pairs;
            if (t >= lo && t < hi) {
                const float pos = a.rope.positions[(row0 + t) * a.rope.ld_positions + rope_axis(a.rope, p)];
                cs[i] = rope_cos_sin(a.rope.inverse ? -pos : pos, rope_turns(a.rope, p));
            }
        }

    const int per_row = dim >> 3;
    for (int h = blockIdx.x * heads_per_cta; h < min(heads, (static_cast<int>(blockIdx.x) + 1) * heads_per_cta); ++h) {
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv) {
            const int64_t bh = static_cast<int64_t>(id) * heads + h;
            uint8_t *codes = (kv == 0 ? a.cache.k_codes : a.cache.v_codes) + bh * page * dim;
            float *scale = (kv == 0 ? a.cache.k_scale : a.cache.v_scale) + bh;
            const uint16_t *x = a.x[kv] + h * a.head_stride[kv];
            const float was = lo > 0 ? *scale : 0.0f;
            uint4 v[kPer];
#pragma unroll
            for (int u = 0; u < kPer; ++u) {
                const int i = threadIdx.x + u * blockDim.x, t = i / per_row, c = (i - t * per_row) * 8;
                v[u] = t >= lo && t < hi ? *reinterpret_cast<const uint4 *>(x + (row0 + t) * a.token_stride[kv] + c)
                                         : make_uint4(0, 0, 0, 0);
            }
            if (kv == 0 && turn) {
                __syncthreads();   // the last head's readers are done; cs is written
#pragma unroll
                for (int u = 0; u < kPer; ++u)
                    reinterpret_cast<uint4 *>(tile)[threadIdx.x + u * blockDim.x] = v[u];
                __syncthreads();
#pragma unroll
                for (int u = 0; u < kPer; ++u) {
                    const int i = threadIdx.x + u * blockDim.x, t = i / per_row, c = (i - t * per_row) * 8;
                    if (t < lo || t >= hi)
                        continue;
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const RopeChannel ch = rope_channel(a.rope, c + e);
                        const uint16_t own = tile[t * dim + c + e];
                        uint32_t y = own;
                        if (ch.pair >= 0) {
                            const float2 f = cs[t * a.rope.pairs + ch.pair];
                            const float r = rope_mix(__uint_as_float(static_cast<uint32_t>(own) << 16),
                                                     __uint_as_float(static_cast<uint32_t>(tile[t * dim + ch.partner]) << 16),
                                                     f.x, ch.first ? -f.y : f.y);
                            y = __bfloat16_as_ushort(__float2bfloat16_rn(r));
                        }
                        w[e >> 1] = (e & 1) ? w[e >> 1] | y << 16 : y;
                    }
                    v[u] = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            uint32_t m = 0;
            uint32_t odd = 0;   // chunks with a value that is not finite
#pragma unroll
            for (int u = 0; u < kPer; ++u) {
                const uint32_t f = finite_absmax8(v[u]);
                odd |= (f >> 16) << u;
                m = max(m, f & 0xFFFFu);
            }
            m = cta_max(m, warp_max);
            float s2 = block_scale_of(m);
            if (lo > 0)
                s2 = fmaxf(s2, was);
            const Divisor d = divisor(s2);
            if (threadIdx.x == 0)
                *scale = s2;   // every thread read the old one before cta_max's barriers
            const bool grown = lo > 0 && s2 != was;
#pragma unroll
            for (int u = 0; u < kPer; ++u) {
                const int i = threadIdx.x + u * blockDim.x, t = i / per_row;
                uint2 *dst = reinterpret_cast<uint2 *>(codes) + i;
                if (t >= lo && t < hi) {
                    *dst = encode8(v[u], d, ((odd >> u) & 1u) == 0);
                } else if (t < lo && grown) {
                    const uint2 c = *dst;
                    *dst = make_uint2(reencode4(c.x, was, d), reencode4(c.y, was, d));
                }
            }
        }
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

// One CTA: one page and head, keys and values.
__global__ void __launch_bounds__(kThreads) read_kernel(ReadArgs a)
{
    const int b = blockIdx.z, h = blockIdx.x, page = a.cache.page_size, dim = a.cache.head_dim;
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
    const int64_t bh = static_cast<int64_t>(id) * a.cache.heads + h;
    const int per_row = dim >> 3;
    for (int kv = 0; kv < 2; ++kv) {
        if (a.x[kv] == nullptr)
            continue;
        const uint2 *codes = reinterpret_cast<const uint2 *>((kv == 0 ? a.cache.k_codes : a.cache.v_codes) + bh * page * dim);
        const float scale = (kv == 0 ? a.cache.k_scale : a.cache.v_scale)[bh];
        uint16_t *x = a.x[kv] + h * a.head_stride[kv];
        for (int i = lo * per_row + threadIdx.x; i < hi * per_row; i += blockDim.x) {
            const int t = i / per_row, c = (i - t * per_row) * 8;
            const uint2 q = codes[i];
            *reinterpret_cast<uint4 *>(x + (s.row + p0 - s.len + t) * a.token_stride[kv] + c) =
                make_uint4(decode2(q.x & 0xFFFFu, scale), decode2(q.x >> 16, scale), decode2(q.y & 0xFFFFu, scale),
                           decode2(q.y >> 16, scale));
        }
    }
}

}  // namespace

cudaError_t launch_kv_write(const KvCache &cache, const KvBatch &batch, const uint16_t *k, int64_t kt, int64_t kh,
                            const uint16_t *v, int64_t vt, int64_t vh, int64_t tokens, const RopeArgs &rope,
                            cudaStream_t st)
{
    WriteArgs a{cache, batch, {k, v}, {kt, vt}, {kh, vh}, tokens, rope};
    const int chunks = cache.page_size * cache.head_dim / 8;
    const int threads = chunks < kThreads ? chunks : kThreads;
    const int heads_per_cta = rope.pairs > 0 ? 8 : 1;
    const unsigned blocks = static_cast<unsigned>((batch.max_tokens + cache.page_size - 2) / cache.page_size + 1);
    const dim3 grid(static_cast<unsigned>((cache.heads + heads_per_cta - 1) / heads_per_cta), blocks,
                    static_cast<unsigned>(batch.batch));
    const size_t smem = rope.pairs > 0 ? static_cast<size_t>(cache.page_size) * (8 * rope.pairs + 2 * cache.head_dim) : 0;
    const auto run = [&](auto kernel) {
        if (smem > 47 * 1024) {   // 48 KB, the static part included, need no leave
            const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                       static_cast<int>(smem));
            if (e != cudaSuccess)
                return e;
        }
        kernel<<<grid, threads, smem, st>>>(a, heads_per_cta);
        return cudaGetLastError();
    };
    switch (chunks / threads) {
    case 1: return run(write_kernel<1>);
    case 2: return run(write_kernel<2>);
    case 4: return run(write_kernel<4>);
    default: return run(write_kernel<8>);
    }
}

cudaError_t launch_kv_read(const KvCache &cache, const KvBatch &batch, uint16_t *k, int64_t kt, int64_t kh,
                           uint16_t *v, int64_t vt, int64_t vh, int64_t tokens, cudaStream_t st)
{
    ReadArgs a{cache, batch, {k, v}, {kt, vt}, {kh, vh}, tokens};
    const unsigned blocks = static_cast<unsigned>((batch.max_tokens + cache.page_size - 2) / cache.page_size + 1);
    const dim3 grid(static_cast<unsigned>(cache.heads), blocks, static_cast<unsigned>(batch.batch));
    read_kernel<<<grid, kThreads, 0, st>>>(a);
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

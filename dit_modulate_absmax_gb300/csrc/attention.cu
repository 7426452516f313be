// attention.cu -- attention over the 8-bit paged cache (h3fp4_kv_attention).
//
// One warp per query and head: a lane holds dim/32 channels, keys are taken
// one after another with a running maximum and sum.
#include "kvcache.cuh"

namespace h3fp4 {
namespace {

__device__ uint32_t g_error;

constexpr int kThreads = 128;

template <int kDim>
__global__ void __launch_bounds__(kThreads) attention_kernel(AttnArgs a)
{
    constexpr int kPer = kDim / 32;   // channels per lane
    const int lane = threadIdx.x & 31, b = blockIdx.z, h = blockIdx.y;
    const int i = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const KvSequence s = kv_sequence(a.batch, b, a.tokens);
    const int page = a.cache.page_size;
    if (!s.ok || s.len > a.max_kv || (s.len > 0 && (s.len - 1) / page >= a.batch.ld_table)) {
        if (threadIdx.x == 0)
            atomicOr(&g_error, ERR_KV_RANGE);
        return;
    }
    if (i >= s.n)
        return;
    const int64_t row = s.row + i;
    const int pos = s.len - s.n + i, kh = h / (a.heads / a.cache.heads);
    float q[kPer], o[kPer];
    for (int c = 0; c < kPer; ++c) {
        q[c] = __uint_as_float(static_cast<uint32_t>(a.q[row * a.qt + h * a.qh + lane * kPer + c]) << 16);
        o[c] = 0.0f;
    }
    float m = -INFINITY, l = 0.0f;
    const int end = a.causal ? min(s.len, pos + 1) : s.len;
    const int begin = a.window > 0 ? max(0, pos - a.window + 1) : 0;
    for (int j = begin; j < end; ++j) {
        const int32_t id = a.batch.page_table[b * a.batch.ld_table + j / page];
        if (id < 0 || id >= a.cache.num_pages) {
            if (lane == 0)
                atomicOr(&g_error, ERR_KV_RANGE);
            continue;
        }
        const int64_t bh = static_cast<int64_t>(id) * a.cache.heads + kh;
        const int64_t at = (bh * page + j % page) * kDim + lane * kPer;
        float k[kPer], v[kPer];
        for (int c = 0; c < kPer; c += 2) {
            const float2 f = e4m3x2_to_float2(*reinterpret_cast<const uint16_t *>(a.cache.k_codes + at + c));
            const float2 g = e4m3x2_to_float2(*reinterpret_cast<const uint16_t *>(a.cache.v_codes + at + c));
            k[c] = f.x; k[c + 1] = f.y;
            v[c] = g.x; v[c + 1] = g.y;
        }
        float d = 0.0f;
        for (int c = 0; c < kPer; ++c)
            d = fmaf(q[c], k[c], d);
        for (int o2 = 16; o2 > 0; o2 >>= 1)
            d += __shfl_xor_sync(0xFFFFFFFFu, d, o2);
        d *= a.cache.k_scale[bh] * a.scale;
        const float m2 = fmaxf(m, d), keep = expf(m - m2), p = expf(d - m2), pv = p * a.cache.v_scale[bh];
        m = m2;
        l = l * keep + p;
        for (int c = 0; c < kPer; ++c)
            o[c] = fmaf(pv, v[c], o[c] * keep);
    }
    for (int c = 0; c < kPer; ++c)
        a.out[row * a.ot + h * a.oh + lane * kPer + c] =
            __bfloat16_as_ushort(__float2bfloat16_rn(l > 0.0f || l != l ? o[c] / l : 0.0f));
    if (a.lse != nullptr && lane == 0)
        a.lse[row * a.heads + h] = m + logf(l);
}

}  // namespace

int64_t attention_workspace(const AttnShape &)
{
    return 0;
}

cudaError_t launch_attention(const AttnArgs &a, void *, cudaStream_t st)
{
    const dim3 grid((a.batch.max_tokens + kThreads / 32 - 1) / (kThreads / 32), a.heads, a.batch.batch);
    if (a.cache.head_dim == 64)
        attention_kernel<64><<<grid, kThreads, 0, st>>>(a);
    else
        attention_kernel<128><<<grid, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t read_attention_error(uint32_t *code)
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

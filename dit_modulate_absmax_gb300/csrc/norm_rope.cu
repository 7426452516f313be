// norm_rope.cu -- per-head RMS norm of queries and keys with their rotation in
// the same pass (h3fp4_norm_rope), and its gradients (h3fp4_norm_rope_backward).
//
//   r = 1 / sqrt(mean(x^2) + eps),  y = R (x r w)
//   g = R^T dy,  dw = sum over tokens and heads of g x r,
//   dx = r (w g - x r^2 mean(w g x))
//
// R turns pairs of channels, so that y = r (x A + partner(x) B) with A = w cos
// and B = -+ w(partner) sin: a lane keeps both for its 8 channels and serves
// every head of its token with them, and one sum over a head's lanes (two for
// the gradient) lies between its loads and its stores.  Everything is FP32
// until the one rounding to bf16.
#include <cuda_bf16.h>

#include "norm_rope.cuh"
#include "rope.cuh"

namespace h3fp4 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTokens = 4;                       // per CTA
constexpr int kWarpsPerToken = kWarps / kTokens;
constexpr int kMaxDim = 256;

__device__ __forceinline__ uint32_t bf_pack(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ void unpack(const uint4 &raw, uint32_t (&w)[4], float (&v)[8])
{
    w[0] = raw.x; w[1] = raw.y; w[2] = raw.z; w[3] = raw.w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 pack(const float (&y)[8])
{
    return make_uint4(bf_pack(y[0], y[1]), bf_pack(y[2], y[3]), bf_pack(y[4], y[5]), bf_pack(y[6], y[7]));
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

// Squares of a row past 2^50 could leave FP32's range: such a row is taken times this (exact; what becomes subnormal is
// nothing next to the rest), without eps, which is nothing next to it either.
constexpr float kFarRow = 0x1p100f, kFarScale = 0x1p-80f;

__device__ __forceinline__ float weight_at(const void *weight, bool wide, int c)
{
    if (weight == nullptr)
        return 1.0f;
    return wide ? static_cast<const float *>(weight)[c]
                : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(weight)[c]) << 16);
}

// What a CTA keeps for all its tokens and heads.
struct Tables {
    float2 cs[kTokens][kRopeMaxPairs];   // cosine and sine of each token's pairs
    float2 turns[kRopeMaxPairs];         // FP64 is slow here: once a pair, not once a pair and token
    float weight[2][kMaxDim];            // of queries and keys
};

__device__ __forceinline__ void fill_turns(Tables &s, const RopeArgs &r)
{
    for (int p = threadIdx.x; p < r.pairs; p += kThreads)
        s.turns[p] = rope_turns(r, p);
}

__device__ __forceinline__ void fill_angles(Tables &s, const RopeArgs &r, int64_t t0, int64_t tokens, bool inverse)
{
    for (int i = threadIdx.x; i < kTokens * r.pairs; i += kThreads) {
        const int tt = i / r.pairs, p = i - tt * r.pairs;
        if (t0 + tt < tokens) {
            const float pos = r.positions[(t0 + tt) * r.ld_positions + rope_axis(r, p)];
            s.cs[tt][p] = rope_cos_sin(inverse ? -pos : pos, s.turns[p]);
        }
    }
}

// kLanes: lanes of a head, a power of two; those past its channels idle.
template <int kLayout, int kLanes>
__global__ void __launch_bounds__(kThreads)
    norm_rope_kernel(NormSide qs, NormSide ks, int64_t tokens, int dim, int heads_per_cta, float eps, RopeArgs rope)
{
    constexpr int kInFlight = 4, kPerWarp = 32 / kLanes, kStep = kWarpsPerToken * kPerWarp;
    __shared__ Tables s;
    __shared__ uint32_t swap[kLayout == 0 ? 1 : kWarps][kLayout == 0 ? 1 : 128];
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTokens;
    fill_turns(s, rope);
    for (int i = threadIdx.x; i < 2 * dim; i += kThreads) {
        const NormSide &of = i < dim ? qs : ks;
        const int c = i < dim ? i : i - dim;
        s.weight[i >= dim][c] = weight_at(of.weight, of.wide != 0, c);
    }
    __syncthreads();
    fill_angles(s, rope, t0, tokens, false);
    __syncthreads();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tt = warp % kTokens;
    const int64_t t = t0 + tt;
    if (t >= tokens)
        return;
    const int sub = lane / kLanes, c0 = lane % kLanes * 8;
    const bool live = c0 < dim;
    const RopeLane<kLayout> of(rope, c0, sub * kLanes);
    const float per_channel = 1.0f / static_cast<float>(dim);
    const int all = qs.heads + ks.heads, begin = blockIdx.y * heads_per_cta, end = min(all, begin + heads_per_cta);
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
        const NormSide &x = side == 0 ? qs : ks;
        const int first = side == 0 ? 0 : qs.heads, lo = max(begin, first) - first, hi = min(end, first + x.heads) - first;
        if (lo >= hi)
            continue;
        float a[8], b[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const bool turned = live && (of.turned >> e & 1u) != 0;
            const int c = live ? c0 + e : 0;
            const float2 v = turned ? s.cs[tt][of.pair[e]] : make_float2(1.0f, 0.0f);
            a[e] = s.weight[side][c] * v.x;
            b[e] = turned ? s.weight[side][rope_channel(rope, c).partner] * ((of.first >> e & 1u) != 0 ? -v.y : v.y) : 0.0f;
        }
        const uint16_t *xp = x.x + t * x.xt + c0;
        uint16_t *op = x.out + t * x.ot + c0;
        for (int h0 = lo + (warp / kTokens) * kPerWarp; h0 < hi; h0 += kInFlight * kStep) {   // the same in the whole warp
            uint4 raw[kInFlight];
#pragma unroll
            for (int u = 0; u < kInFlight; ++u) {
                const int h = h0 + u * kStep + sub;
                raw[u] = live && h < hi ? *reinterpret_cast<const uint4 *>(xp + h * x.xh) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int u = 0; u < kInFlight; ++u) {
                const int h = h0 + u * kStep + sub;
                uint32_t w[4];
                float v[8], partner[8], y[8], sum = 0.0f, at = eps;
                unpack(raw[u], w, v);
                rope_partners(of, w, swap[kLayout == 0 ? 0 : warp], partner);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    sum = fmaf(v[e], v[e], sum);
                sum = head_sum<kLanes>(sum);
                if (__any_sync(0xFFFFFFFFu, !(sum < kFarRow))) {
                    const bool far = !(sum < kFarRow);
                    const float f = far ? kFarScale : 1.0f;
                    at = far ? 0.0f : eps;
                    sum = 0.0f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        v[e] *= f;
                        partner[e] *= f;
                        sum = fmaf(v[e], v[e], sum);
                    }
                    sum = head_sum<kLanes>(sum);
                }
                const float r = rsqrtf(fmaf(sum, per_channel, at));
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    y[e] = r * fmaf(v[e], a[e], (of.turned >> e & 1u) != 0 ? partner[e] * b[e] : 0.0f);
                if (live && h < hi)
                    *reinterpret_cast<uint4 *>(op + h * x.oh) = pack(y);
            }
        }
    }
}

// A CTA takes groups of kTokens tokens and a range of their heads in turn, keeps its share of dw in registers and leaves it
// in parts [side][CTA][dim].
template <int kLayout, int kLanes>
__global__ void __launch_bounds__(kThreads)
    norm_rope_grad_kernel(NormGradSide qs, NormGradSide ks, int64_t tokens, int dim, int heads_per_item, int64_t items, float eps,
                          RopeArgs rope, float *parts)
{
    constexpr int kInFlight = 2, kPerWarp = 32 / kLanes, kStep = kWarpsPerToken * kPerWarp;
    __shared__ Tables s;
    __shared__ uint32_t swap[kLayout == 0 ? 1 : kWarps][kLayout == 0 ? 1 : 128];
    __shared__ float rows[kWarps * kPerWarp][kLanes * 8 + 4];
    // What joins the parts may be scheduled as places fall free; it waits for this grid's end before it reads them.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    fill_turns(s, rope);
    for (int i = threadIdx.x; i < 2 * dim; i += kThreads) {
        const NormGradSide &of = i < dim ? qs : ks;
        const int c = i < dim ? i : i - dim;
        s.weight[i >= dim][c] = weight_at(of.weight, of.wide != 0, c);
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tt = warp % kTokens;
    const int sub = lane / kLanes, c0 = lane % kLanes * 8;
    const bool live = c0 < dim;
    const RopeLane<kLayout> of(rope, c0, sub * kLanes);
    const float per_channel = 1.0f / static_cast<float>(dim);
    const int all = qs.heads + ks.heads, ranges = (all + heads_per_item - 1) / heads_per_item;
    float dw[2][8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        dw[0][e] = dw[1][e] = 0.0f;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {   // the same in the whole CTA
        const int64_t t0 = item / ranges * kTokens, t = t0 + tt;
        const int begin = static_cast<int>(item % ranges) * heads_per_item, end = min(all, begin + heads_per_item);
        __syncthreads();   // the last item's readers are done (and the first one's turns are there)
        fill_angles(s, rope, t0, tokens, true);
        __syncthreads();
        if (t >= tokens)
            continue;
        float cosv[8], ss[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const bool turned = live && (of.turned >> e & 1u) != 0;
            const float2 v = turned ? s.cs[tt][of.pair[e]] : make_float2(1.0f, 0.0f);
            cosv[e] = v.x;
            ss[e] = (of.first >> e & 1u) != 0 ? -v.y : v.y;
        }
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            const NormGradSide &x = side == 0 ? qs : ks;
            const int first = side == 0 ? 0 : qs.heads, lo = max(begin, first) - first, hi = min(end, first + x.heads) - first;
            if (lo >= hi)
                continue;
            float w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                w[e] = live ? s.weight[side][c0 + e] : 0.0f;
            const uint16_t *xp = x.x + t * x.xt + c0, *gp = x.dy + t * x.gt + c0;
            uint16_t *op = x.dx + t * x.ot + c0;
            for (int h0 = lo + (warp / kTokens) * kPerWarp; h0 < hi; h0 += kInFlight * kStep) {   // the same in the whole warp
                uint4 rx[kInFlight], rg[kInFlight];
#pragma unroll
                for (int u = 0; u < kInFlight; ++u) {
                    const int h = h0 + u * kStep + sub;
                    const bool mine = live && h < hi;
                    rx[u] = mine ? *reinterpret_cast<const uint4 *>(xp + h * x.xh) : make_uint4(0, 0, 0, 0);
                    rg[u] = mine ? *reinterpret_cast<const uint4 *>(gp + h * x.gh) : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int u = 0; u < kInFlight; ++u) {
                    const int h = h0 + u * kStep + sub;
                    uint32_t words[4];
                    float v[8], g[8], partner[8], y[8], sum = 0.0f, along = 0.0f, at = eps, f = 1.0f;
                    unpack(rg[u], words, g);
                    rope_partners(of, words, swap[kLayout == 0 ? 0 : warp], partner);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        g[e] = (of.turned >> e & 1u) != 0 ? rope_mix(g[e], partner[e], cosv[e], ss[e]) : g[e];
                    unpack(rx[u], words, v);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        sum = fmaf(v[e], v[e], sum);
                    sum = head_sum<kLanes>(sum);
                    if (__any_sync(0xFFFFFFFFu, !(sum < kFarRow))) {
                        const bool far = !(sum < kFarRow);
                        f = far ? kFarScale : 1.0f;
                        at = far ? 0.0f : eps;
                        sum = 0.0f;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            v[e] *= f;
                            sum = fmaf(v[e], v[e], sum);
                        }
                        sum = head_sum<kLanes>(sum);
                    }
                    const float r = rsqrtf(fmaf(sum, per_channel, at));
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        v[e] *= r;   // the normed value
                        const float gw = w[e] * g[e];
                        along = fmaf(gw, v[e], along);
                        dw[side][e] = fmaf(g[e], v[e], dw[side][e]);
                        g[e] = gw;
                    }
                    along = head_sum<kLanes>(along) * per_channel;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        y[e] = r * f * fmaf(-v[e], along, g[e]);
                    if (live && h < hi)
                        *reinterpret_cast<uint4 *>(op + h * x.oh) = pack(y);
                }
            }
        }
    }
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
        if ((side == 0 ? qs : ks).dweight == nullptr)
            continue;
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e)
            rows[warp * kPerWarp + sub][c0 + e] = side == 0 ? dw[0][e] : dw[1][e];
        __syncthreads();
        for (int c = threadIdx.x; c < dim; c += kThreads) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kWarps * kPerWarp; ++i)
                sum += rows[i][c];
            parts[(static_cast<int64_t>(side) * gridDim.x + blockIdx.x) * dim + c] = sum;
        }
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

// Heads of a CTA: few tokens have theirs spread over several until every SM has one.
int heads_each(int64_t groups, int heads, int per_pass, int64_t ctas)
{
    int64_t split = (ctas + groups - 1) / groups;
    const int64_t most = (heads + per_pass - 1) / per_pass;
    split = split < 1 ? 1 : split > most ? most : split;
    return static_cast<int>(((heads + split - 1) / split + per_pass - 1) / per_pass) * per_pass;
}

template <int kLanes>
cudaError_t run(const NormSide &q, const NormSide &k, int64_t tokens, int dim, float eps, const RopeArgs &r, cudaStream_t st)
{
    const int64_t groups = (tokens + kTokens - 1) / kTokens;
    const int heads = q.heads + k.heads, each = heads_each(groups, heads, kWarpsPerToken * (32 / kLanes), sm_count());
    const dim3 grid(static_cast<unsigned>(groups), static_cast<unsigned>((heads + each - 1) / each));
    (r.layout == 0 ? norm_rope_kernel<0, kLanes> : norm_rope_kernel<1, kLanes>)<<<grid, kThreads, 0, st>>>(q, k, tokens, dim, each, eps, r);
    return cudaGetLastError();
}

// CTAs of the gradient: two an SM.
int grad_ctas() { return 2 * sm_count(); }

template <int kLanes>
cudaError_t run_grad(const NormGradSide &q, const NormGradSide &k, int64_t tokens, int dim, float eps, const RopeArgs &r, float *parts,
                     cudaStream_t st)
{
    const int64_t groups = (tokens + kTokens - 1) / kTokens;
    const int heads = q.heads + k.heads;
    int64_t ctas = 0;
    if (groups > 0 && heads > 0) {
        const int each = heads_each(groups, heads, kWarpsPerToken * (32 / kLanes), grad_ctas());
        const int64_t items = groups * ((heads + each - 1) / each);
        ctas = items < grad_ctas() ? items : grad_ctas();
        (r.layout == 0 ? norm_rope_grad_kernel<0, kLanes> : norm_rope_grad_kernel<1, kLanes>)<<<static_cast<unsigned>(ctas), kThreads, 0, st>>>(
            q, k, tokens, dim, each, items, eps, r, parts);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess)
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
    cfg.numAttrs = ctas > 0 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, weight_grad_kernel, q.dweight, k.dweight, static_cast<const float *>(parts), static_cast<int>(ctas), dim);
}

}  // namespace

int64_t norm_grad_workspace(int dim) { return 2 * static_cast<int64_t>(grad_ctas()) * dim * 4; }

cudaError_t launch_norm_rope(const NormSide &q, const NormSide &k, int64_t tokens, int dim, float eps, const RopeArgs &r, cudaStream_t st)
{
    return dim <= 64 ? run<8>(q, k, tokens, dim, eps, r, st) : dim <= 128 ? run<16>(q, k, tokens, dim, eps, r, st)
                                                                          : run<32>(q, k, tokens, dim, eps, r, st);
}

cudaError_t launch_norm_rope_grad(const NormGradSide &q, const NormGradSide &k, int64_t tokens, int dim, float eps, const RopeArgs &r,
                                  void *workspace, cudaStream_t st)
{
    float *parts = static_cast<float *>(workspace);
    return dim <= 64    ? run_grad<8>(q, k, tokens, dim, eps, r, parts, st)
           : dim <= 128 ? run_grad<16>(q, k, tokens, dim, eps, r, parts, st)
                        : run_grad<32>(q, k, tokens, dim, eps, r, parts, st);
}

}  // namespace h3fp4

// api.cu -- the extern "C" entry points declared in include/h3fp4.h.
//
// Each entry point checks its arguments on the host (null pointers, 16-byte
// alignment, leading dimensions, shape multiples, segment table) and only then
// enqueues its kernels; a failed check enqueues nothing.
#include <cuda_runtime.h>

#include <cstdint>
#include <optional>

#include "h3fp4.h"
#include "launch.h"

#ifndef H3FP4_VERSION
#define H3FP4_VERSION "0.1.0"
#endif
#define H3FP4_STR2(x) #x
#define H3FP4_STR(x) H3FP4_STR2(x)

namespace {

using h3fp4::SegTable;

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

cudaStream_t as_stream(void *s) { return static_cast<cudaStream_t>(s); }

h3fp4_status from_cuda(cudaError_t e) { return e == cudaSuccess ? H3FP4_OK : H3FP4_ERR_CUDA; }

// Fills `t` from the host offsets; checks 0 = off[0] <= ... <= off[nseg] = m.
h3fp4_status make_segments(const int32_t *off, int32_t nseg, int64_t m, SegTable *t)
{
    if (off == nullptr)
        return H3FP4_ERR_NULL;
    if (nseg < 1 || nseg > H3FP4_MAX_SEGMENTS)
        return H3FP4_ERR_SHAPE;
    if (off[0] != 0 || static_cast<int64_t>(off[nseg]) != m)
        return H3FP4_ERR_SHAPE;
    for (int32_t s = 0; s < nseg; ++s)
        if (off[s + 1] < off[s])
            return H3FP4_ERR_SHAPE;
    for (int32_t s = 0; s <= H3FP4_MAX_SEGMENTS; ++s)
        t->off[s] = s <= nseg ? off[s] : off[nseg];
    t->nseg = nseg;
    return H3FP4_OK;
}

// Shared checks of the modulation producer's inputs.
// x may be NULL when m == 0 (nothing is read from it).
h3fp4_status check_modulate(const void *x, int64_t ldx, int64_t m, int64_t d, const void *shift,
                            const void *scale, int64_t ld_mod)
{
    if ((x == nullptr && m != 0) || shift == nullptr || scale == nullptr)
        return H3FP4_ERR_NULL;
    if (m < 0 || m > INT32_MAX || d <= 0 || d % 256 != 0 || d > (int64_t(1) << 24))
        return H3FP4_ERR_SHAPE;
    if (ldx < d || ld_mod < d)
        return H3FP4_ERR_SHAPE;
    if (!aligned16(x) || !aligned16(shift) || !aligned16(scale) || ldx % 8 != 0 || ld_mod % 8 != 0)
        return H3FP4_ERR_ALIGN;
    return H3FP4_OK;
}

h3fp4_status check_pack_outputs(int64_t m, int64_t m_pad, const void *qdata, const void *sf)
{
    if (qdata == nullptr || sf == nullptr)
        return H3FP4_ERR_NULL;
    if (m_pad < m || m_pad % 16 != 0 || m_pad > INT32_MAX)   // the GEMM's descriptor M: a multiple of 16
        return H3FP4_ERR_SHAPE;
    if (!aligned16(qdata) || !aligned16(sf))
        return H3FP4_ERR_ALIGN;
    return H3FP4_OK;
}

}  // namespace

extern "C" {

h3fp4_status h3fp4_modulate_absmax(const void *x_bf16, int64_t ldx, int64_t m, int64_t d, const void *shift_bf16,
                                   const void *scale_bf16, int64_t ld_mod, const int32_t *seg_row_offsets,
                                   int32_t nseg, float *tensor_scale, uint32_t *scratch, void *stream)
{
    h3fp4_status s = check_modulate(x_bf16, ldx, m, d, shift_bf16, scale_bf16, ld_mod);
    if (s != H3FP4_OK)
        return s;
    if (tensor_scale == nullptr || scratch == nullptr)
        return H3FP4_ERR_NULL;
    SegTable seg;
    if ((s = make_segments(seg_row_offsets, nseg, m, &seg)) != H3FP4_OK)
        return s;
    return from_cuda(h3fp4::launch_modulate_absmax(
        static_cast<const uint16_t *>(x_bf16), ldx, m, d, static_cast<const uint16_t *>(shift_bf16),
        static_cast<const uint16_t *>(scale_bf16), ld_mod, seg, tensor_scale, scratch, as_stream(stream)));
}

h3fp4_status h3fp4_modulate_pack(const void *x_bf16, int64_t ldx, int64_t m, int64_t m_pad, int64_t d,
                                 const void *shift_bf16, const void *scale_bf16, int64_t ld_mod,
                                 const int32_t *seg_row_offsets, int32_t nseg, const float *tensor_scale,
                                 uint8_t *qdata, uint8_t *sfa, void *stream)
{
    h3fp4_status s = check_modulate(x_bf16, ldx, m, d, shift_bf16, scale_bf16, ld_mod);
    if (s != H3FP4_OK)
        return s;
    if (tensor_scale == nullptr)
        return H3FP4_ERR_NULL;
    if ((s = check_pack_outputs(m, m_pad, qdata, sfa)) != H3FP4_OK)
        return s;
    SegTable seg;
    if ((s = make_segments(seg_row_offsets, nseg, m, &seg)) != H3FP4_OK)
        return s;
    return from_cuda(h3fp4::launch_modulate_pack(
        static_cast<const uint16_t *>(x_bf16), ldx, m, m_pad, d, static_cast<const uint16_t *>(shift_bf16),
        static_cast<const uint16_t *>(scale_bf16), ld_mod, seg, tensor_scale, qdata, sfa, as_stream(stream)));
}

h3fp4_status h3fp4_modulate_produce(const void *x_bf16, int64_t ldx, int64_t m, int64_t m_pad, int64_t d,
                                    const void *shift_bf16, const void *scale_bf16, int64_t ld_mod,
                                    const int32_t *seg_row_offsets, int32_t nseg, float *tensor_scale,
                                    uint32_t *scratch, uint8_t *qdata, uint8_t *sfa, void *stream)
{
    h3fp4_status s = check_modulate(x_bf16, ldx, m, d, shift_bf16, scale_bf16, ld_mod);
    if (s != H3FP4_OK)
        return s;
    if (tensor_scale == nullptr || scratch == nullptr)
        return H3FP4_ERR_NULL;
    if ((s = check_pack_outputs(m, m_pad, qdata, sfa)) != H3FP4_OK)
        return s;
    SegTable seg;
    if ((s = make_segments(seg_row_offsets, nseg, m, &seg)) != H3FP4_OK)
        return s;
    return from_cuda(h3fp4::launch_modulate_produce(
        static_cast<const uint16_t *>(x_bf16), ldx, m, m_pad, d, static_cast<const uint16_t *>(shift_bf16),
        static_cast<const uint16_t *>(scale_bf16), ld_mod, seg, tensor_scale, scratch, qdata, sfa, as_stream(stream)));
}

h3fp4_status h3fp4_swiglu_pack(const void *gate_bf16, int64_t ldg, const void *up_bf16, int64_t ldu, int64_t m,
                               int64_t m_pad, int64_t f, float *tensor_scale, uint32_t *scratch, uint8_t *qdata,
                               uint8_t *sfa, void *h_workspace, void *stream)
{
    if (((gate_bf16 == nullptr || up_bf16 == nullptr) && m != 0) || tensor_scale == nullptr || scratch == nullptr)
        return H3FP4_ERR_NULL;
    if (m < 0 || m > INT32_MAX || f <= 0 || f % 256 != 0 || f > (int64_t(1) << 24) || ldg < f || ldu < f)
        return H3FP4_ERR_SHAPE;
    if (!aligned16(gate_bf16) || !aligned16(up_bf16) || ldg % 8 != 0 || ldu % 8 != 0 ||
        (h_workspace != nullptr && !aligned16(h_workspace)))
        return H3FP4_ERR_ALIGN;
    h3fp4_status s = check_pack_outputs(m, m_pad, qdata, sfa);
    if (s != H3FP4_OK)
        return s;
    return from_cuda(h3fp4::launch_swiglu_pack(
        static_cast<const uint16_t *>(gate_bf16), ldg, static_cast<const uint16_t *>(up_bf16), ldu, m, m_pad, f,
        tensor_scale, scratch, qdata, sfa, static_cast<uint16_t *>(h_workspace), as_stream(stream)));
}

h3fp4_status h3fp4_quantize_pack(const void *x_bf16, int64_t ldx, int64_t m, int64_t m_pad, int64_t d,
                                 float *tensor_scale, uint32_t *scratch, uint8_t *qdata, uint8_t *sfa, void *stream)
{
    if ((x_bf16 == nullptr && m != 0) || tensor_scale == nullptr || scratch == nullptr)
        return H3FP4_ERR_NULL;
    if (m < 0 || m > INT32_MAX || d <= 0 || d % 256 != 0 || d > (int64_t(1) << 24) || ldx < d)
        return H3FP4_ERR_SHAPE;
    if (!aligned16(x_bf16) || ldx % 8 != 0)
        return H3FP4_ERR_ALIGN;
    h3fp4_status s = check_pack_outputs(m, m_pad, qdata, sfa);
    if (s != H3FP4_OK)
        return s;
    return from_cuda(h3fp4::launch_quantize_pack(static_cast<const uint16_t *>(x_bf16), ldx, m, m_pad, d,
                                                 tensor_scale, scratch, qdata, sfa, as_stream(stream)));
}

namespace {

// Checks shared by both GEMM entry points; fills `c` with the configuration.
h3fp4_status check_gemm(const uint8_t *a_q, const uint8_t *a_sf, const float *a_tensor_scale, const uint8_t *b_q,
                        const uint8_t *b_sf, const float *b_tensor_scale, const void *c_bf16, int64_t ldc, int64_t m,
                        int64_t m_pad, int64_t n, int64_t k, const h3fp4_gemm_config *cfg, h3fp4_gemm_config *c)
{
    if (a_q == nullptr || a_sf == nullptr || a_tensor_scale == nullptr || b_q == nullptr || b_sf == nullptr ||
        b_tensor_scale == nullptr || (c_bf16 == nullptr && m != 0 && n != 0))
        return H3FP4_ERR_NULL;
    if (m < 0 || m > m_pad || m_pad % 16 != 0 || m_pad > INT32_MAX || n < 0 || n % 128 != 0 || n > INT32_MAX ||
        k <= 0 || k % 256 != 0 || k > (int64_t(1) << 24) || ldc < n)
        return H3FP4_ERR_SHAPE;
    if (!aligned16(a_q) || !aligned16(a_sf) || !aligned16(b_q) || !aligned16(b_sf) || !aligned16(c_bf16) ||
        ldc % 8 != 0)
        return H3FP4_ERR_ALIGN;
    *c = h3fp4_gemm_config{0, 0, 0, 0};
    if (cfg != nullptr) {
        *c = *cfg;
        if (c->n_group < 0 || c->stages != 0 || (c->cta_pair != 0 && c->cta_pair != 1 && c->cta_pair != 4) ||
            c->reserved != 0)
            return H3FP4_ERR_UNSUPPORTED;
    }
    return H3FP4_OK;
}

}  // namespace

h3fp4_status h3fp4_gemm(const uint8_t *a_q, const uint8_t *a_sf, const float *a_tensor_scale, const uint8_t *b_q,
                        const uint8_t *b_sf, const float *b_tensor_scale, void *c_bf16, int64_t ldc, int64_t m,
                        int64_t m_pad, int64_t n, int64_t k, const h3fp4_gemm_config *cfg, void *stream)
{
    h3fp4_gemm_config c;
    h3fp4_status s = check_gemm(a_q, a_sf, a_tensor_scale, b_q, b_sf, b_tensor_scale, c_bf16, ldc, m, m_pad, n, k, cfg, &c);
    if (s != H3FP4_OK)
        return s;
    return h3fp4::launch_gemm(a_q, a_sf, a_tensor_scale, b_q, b_sf, b_tensor_scale,
                              static_cast<uint16_t *>(c_bf16), ldc, m, m_pad, n, k, c, nullptr, as_stream(stream));
}

h3fp4_status h3fp4_gemm_gated_residual(const uint8_t *a_q, const uint8_t *a_sf, const float *a_tensor_scale,
                                       const uint8_t *b_q, const uint8_t *b_sf, const float *b_tensor_scale,
                                       const void *gate_bf16, int64_t ld_gate, const int32_t *seg_row_offsets,
                                       int32_t nseg, const void *residual_bf16, int64_t ldr, void *out_bf16,
                                       int64_t ldo, int64_t m, int64_t m_pad, int64_t n, int64_t k,
                                       const h3fp4_gemm_config *cfg, void *stream)
{
    h3fp4_gemm_config c;
    h3fp4_status s = check_gemm(a_q, a_sf, a_tensor_scale, b_q, b_sf, b_tensor_scale, out_bf16, ldo, m, m_pad, n, k,
                                cfg, &c);
    if (s != H3FP4_OK)
        return s;
    const bool rows = m != 0 && n != 0;
    if (rows && (gate_bf16 == nullptr || residual_bf16 == nullptr))
        return H3FP4_ERR_NULL;
    if (ld_gate < n || ldr < n)
        return H3FP4_ERR_SHAPE;
    if (!aligned16(gate_bf16) || !aligned16(residual_bf16) || ld_gate % 8 != 0 || ldr % 8 != 0)
        return H3FP4_ERR_ALIGN;
    SegTable seg;
    if ((s = make_segments(seg_row_offsets, nseg, m, &seg)) != H3FP4_OK)
        return s;
    if (rows) {   // the output either is the residual (same leading dimension) or does not overlap it
        const char *o = static_cast<const char *>(out_bf16), *r = static_cast<const char *>(residual_bf16);
        const int64_t ob = ((m - 1) * ldo + n) * 2, rb = ((m - 1) * ldr + n) * 2;
        const bool same = o == r && ldo == ldr;
        if (!same && o < r + rb && r < o + ob)
            return H3FP4_ERR_UNSUPPORTED;
    }
    h3fp4::GatedArgs g{static_cast<const uint16_t *>(gate_bf16), ld_gate, seg, residual_bf16, ldr};
    return h3fp4::launch_gemm(a_q, a_sf, a_tensor_scale, b_q, b_sf, b_tensor_scale, static_cast<uint16_t *>(out_bf16),
                              ldo, m, m_pad, n, k, c, &g, as_stream(stream));
}

namespace {

// Token arrays [tokens, heads, dim] with element strides of tokens and heads.
struct Strided {
    const void *p;
    int64_t token, head;
};

// Largest stride accepted: byte offsets (up to 2^31 tokens) stay within 63 bits.
constexpr int64_t kMaxStride = int64_t(1) << 30;

h3fp4_status check_strided(const Strided &a)
{
    if (a.p == nullptr)
        return H3FP4_ERR_NULL;
    if (a.token < 0 || a.head < 0 || a.token > kMaxStride || a.head > kMaxStride)
        return H3FP4_ERR_SHAPE;
    if (!aligned16(a.p) || a.token % 8 != 0 || a.head % 8 != 0)
        return H3FP4_ERR_ALIGN;
    return H3FP4_OK;
}

// An output's rows must be distinct: neither stride may fold two of them together.
h3fp4_status check_strided_out(const Strided &a, int64_t tokens, int64_t heads, int64_t dim)
{
    const h3fp4_status s = check_strided(a);
    if (s != H3FP4_OK)
        return s;
    const bool token_outer = a.token >= a.head;
    const int64_t inner = token_outer ? a.head : a.token, outer = token_outer ? a.token : a.head;
    const int64_t n_inner = token_outer ? heads : tokens, n_outer = token_outer ? tokens : heads;
    if ((n_inner > 1 && inner < dim) || (n_outer > 1 && outer < (n_inner - 1) * inner + dim))
        return H3FP4_ERR_SHAPE;
    return H3FP4_OK;
}

bool ranges_overlap(const Strided &a, const Strided &b, int64_t tokens, int64_t heads, int64_t dim)
{
    const auto bytes = [&](const Strided &x) { return 2 * ((tokens - 1) * x.token + (heads - 1) * x.head + dim); };
    const char *pa = static_cast<const char *>(a.p), *pb = static_cast<const char *>(b.p);
    return pa < pb + bytes(b) && pb < pa + bytes(a);
}

// Whether two outputs (check_strided_out) of the same strides have an element in common, as interleaved ones do not though
// their ranges overlap; of other strides, whether their ranges do.
bool rows_overlap(const Strided &a, const Strided &b, int64_t tokens, int64_t heads, int64_t dim)
{
    if (!ranges_overlap(a, b, tokens, heads, dim))
        return false;
    if ((tokens > 1 && a.token != b.token) || (heads > 1 && a.head != b.head))
        return true;
    const int64_t d = (static_cast<const char *>(b.p) - static_cast<const char *>(a.p)) / 2;   // 16-byte aligned, both
    const bool token_outer = heads == 1 || (tokens > 1 && a.token >= a.head);
    const int64_t inner = token_outer ? a.head : a.token, outer = token_outer ? a.token : a.head;
    const int64_t n_inner = token_outer ? heads : tokens, n_outer = token_outer ? tokens : heads;
    // Rows i outer + j inner apart, for i and j between the two: those nearest to -d.
    const int64_t i0 = n_outer > 1 ? -d / outer : 0;
    for (int64_t i = i0 - 2; i <= i0 + 2; ++i) {
        if (i <= -n_outer || i >= n_outer)
            continue;
        const int64_t rest = d + i * outer, j0 = n_inner > 1 ? -rest / inner : 0;
        for (int64_t j = j0 - 1; j <= j0 + 1; ++j)
            if (j > -n_inner && j < n_inner && rest + j * inner < dim && rest + j * inner > -dim)
                return true;
    }
    return false;
}

h3fp4_status make_rope(const h3fp4_rope *r, int64_t dim, int64_t tokens, h3fp4::RopeArgs *out)
{
    if (r == nullptr)
        return H3FP4_ERR_NULL;
    if (r->axes < 1 || r->axes > H3FP4_ROPE_MAX_AXES || r->ld_positions < r->axes ||
        r->ld_positions > (int64_t(1) << 30) || (r->inverse != 0 && r->inverse != 1))
        return H3FP4_ERR_SHAPE;
    int64_t total = 0;
    for (int i = 0; i < H3FP4_ROPE_MAX_AXES; ++i) {
        if (i < r->axes) {
            if (r->dims[i] < 0 || r->dims[i] % 2 != 0 || r->dims[i] > dim - total)
                return H3FP4_ERR_SHAPE;
            total += r->dims[i];
        }
        out->end[i] = static_cast<int32_t>(total);
    }
    if (r->layout != 0 && r->layout != 1)
        return H3FP4_ERR_UNSUPPORTED;
    if ((r->positions == nullptr || r->freqs == nullptr) && total != 0 && tokens != 0)
        return H3FP4_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(r->positions) & 3u) != 0 || (reinterpret_cast<uintptr_t>(r->freqs) & 7u) != 0)
        return H3FP4_ERR_ALIGN;
    out->positions = r->positions;
    out->ld_positions = r->ld_positions;
    out->freqs = r->freqs;
    out->pairs = static_cast<int32_t>(total / 2);
    out->layout = r->layout;
    out->inverse = r->inverse;
    return H3FP4_OK;
}

h3fp4_status check_cache(const h3fp4_kv_cache *c)
{
    if (c == nullptr)
        return H3FP4_ERR_NULL;
    if (c->num_pages < 0 || c->heads < 1 || c->heads > 65535 || int64_t(c->num_pages) * c->heads > INT32_MAX)
        return H3FP4_ERR_SHAPE;
    if ((c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128) ||
        (c->head_dim != 64 && c->head_dim != 128))
        return H3FP4_ERR_UNSUPPORTED;
    if (c->num_pages > 0 && (c->k_codes == nullptr || c->v_codes == nullptr || c->k_scale == nullptr || c->v_scale == nullptr))
        return H3FP4_ERR_NULL;
    if (!aligned16(c->k_codes) || !aligned16(c->v_codes) || (reinterpret_cast<uintptr_t>(c->k_scale) & 3u) != 0 ||
        (reinterpret_cast<uintptr_t>(c->v_scale) & 3u) != 0)
        return H3FP4_ERR_ALIGN;
    return H3FP4_OK;
}

h3fp4_status check_batch(const h3fp4_kv_batch *b, bool need_len, int64_t tokens)
{
    if (b == nullptr)
        return H3FP4_ERR_NULL;
    if (b->batch < 0 || b->batch > 65535 || b->max_tokens < 0 || b->max_tokens > 1000000 || b->ld_table < 0 ||
        b->ld_table > INT32_MAX || tokens < 0 || tokens > INT32_MAX)
        return H3FP4_ERR_SHAPE;
    if (b->batch > 0 && tokens > 0) {
        if (b->cu_tokens == nullptr || (need_len && b->len == nullptr) || (b->page_table == nullptr && b->ld_table > 0))
            return H3FP4_ERR_NULL;
        if (((reinterpret_cast<uintptr_t>(b->cu_tokens) | reinterpret_cast<uintptr_t>(b->len) |
              reinterpret_cast<uintptr_t>(b->page_table)) & 3u) != 0)
            return H3FP4_ERR_ALIGN;
    }
    return H3FP4_OK;
}

bool attention_sizes_ok(int64_t tokens, int32_t heads, int32_t kv_heads, int32_t head_dim, int32_t batch,
                        int32_t max_tokens, int32_t max_kv)
{
    return tokens >= 0 && tokens <= INT32_MAX && heads >= 1 && heads <= 65535 && kv_heads >= 1 &&
           heads % kv_heads == 0 && (head_dim == 64 || head_dim == 128) && batch >= 0 && batch <= 65535 &&
           max_tokens >= 0 && max_tokens <= 1000000 && max_kv >= 0 && max_kv <= (1 << 30);
}

}  // namespace

h3fp4_status h3fp4_rope_axes(const void *x_bf16, int64_t x_token_stride, int64_t x_head_stride, void *out_bf16,
                             int64_t out_token_stride, int64_t out_head_stride, int64_t tokens, int32_t heads,
                             int32_t head_dim, const h3fp4_rope *rope, void *stream)
{
    if (tokens < 0 || tokens > INT32_MAX || heads < 0 || heads > 65535 || head_dim < 8 || head_dim > 256 ||
        head_dim % 8 != 0)
        return H3FP4_ERR_SHAPE;
    h3fp4::RopeArgs r;
    h3fp4_status s = make_rope(rope, head_dim, tokens, &r);
    if (s != H3FP4_OK || tokens == 0 || heads == 0)
        return s;
    const Strided x{x_bf16, x_token_stride, x_head_stride}, out{out_bf16, out_token_stride, out_head_stride};
    if ((s = check_strided(x)) != H3FP4_OK || (s = check_strided_out(out, tokens, heads, head_dim)) != H3FP4_OK)
        return s;
    const bool same = x.p == out.p && x.token == out.token && x.head == out.head;
    if (!same && ranges_overlap(x, out, tokens, heads, head_dim))
        return H3FP4_ERR_UNSUPPORTED;
    return from_cuda(h3fp4::launch_rope(static_cast<const uint16_t *>(x_bf16), x.token, x.head,
                                        static_cast<uint16_t *>(out_bf16), out.token, out.head, tokens, heads, head_dim,
                                        r, as_stream(stream)));
}

h3fp4_status h3fp4_kv_cache_write(const h3fp4_kv_cache *cache, const h3fp4_kv_batch *batch, const void *k_bf16,
                                  int64_t k_token_stride, int64_t k_head_stride, const void *v_bf16,
                                  int64_t v_token_stride, int64_t v_head_stride, int64_t tokens,
                                  const h3fp4_rope *rope, void *stream)
{
    h3fp4_status s = check_cache(cache);
    if (s != H3FP4_OK || (s = check_batch(batch, true, tokens)) != H3FP4_OK)
        return s;
    h3fp4::RopeArgs r{};
    if (rope != nullptr && (s = make_rope(rope, cache->head_dim, tokens, &r)) != H3FP4_OK)
        return s;
    if (batch->batch == 0 || tokens == 0 || batch->max_tokens == 0)
        return H3FP4_OK;
    const Strided k{k_bf16, k_token_stride, k_head_stride}, v{v_bf16, v_token_stride, v_head_stride};
    if ((s = check_strided(k)) != H3FP4_OK || (s = check_strided(v)) != H3FP4_OK)
        return s;
    return from_cuda(h3fp4::launch_kv_write(*cache, *batch, static_cast<const uint16_t *>(k_bf16), k.token, k.head,
                                            static_cast<const uint16_t *>(v_bf16), v.token, v.head, tokens, r,
                                            as_stream(stream)));
}

h3fp4_status h3fp4_kv_cache_read(const h3fp4_kv_cache *cache, const h3fp4_kv_batch *batch, void *k_bf16,
                                 int64_t k_token_stride, int64_t k_head_stride, void *v_bf16, int64_t v_token_stride,
                                 int64_t v_head_stride, int64_t tokens, void *stream)
{
    h3fp4_status s = check_cache(cache);
    if (s != H3FP4_OK || (s = check_batch(batch, false, tokens)) != H3FP4_OK)
        return s;
    if (batch->batch == 0 || tokens == 0 || batch->max_tokens == 0)
        return H3FP4_OK;
    if (k_bf16 == nullptr && v_bf16 == nullptr)
        return H3FP4_ERR_NULL;
    const Strided k{k_bf16, k_token_stride, k_head_stride}, v{v_bf16, v_token_stride, v_head_stride};
    if ((k.p != nullptr && (s = check_strided_out(k, tokens, cache->heads, cache->head_dim)) != H3FP4_OK) ||
        (v.p != nullptr && (s = check_strided_out(v, tokens, cache->heads, cache->head_dim)) != H3FP4_OK))
        return s;
    if (k.p != nullptr && v.p != nullptr && rows_overlap(k, v, tokens, cache->heads, cache->head_dim))
        return H3FP4_ERR_UNSUPPORTED;
    return from_cuda(h3fp4::launch_kv_read(*cache, *batch, static_cast<uint16_t *>(k_bf16), k.token, k.head,
                                           static_cast<uint16_t *>(v_bf16), v.token, v.head, tokens,
                                           as_stream(stream)));
}

int64_t h3fp4_kv_attention_workspace(int64_t tokens, int32_t heads, int32_t kv_heads, int32_t head_dim, int32_t batch,
                                     int32_t max_tokens, int32_t max_kv)
{
    if (!attention_sizes_ok(tokens, heads, kv_heads, head_dim, batch, max_tokens, max_kv))
        return -1;
    return h3fp4::attention_workspace(h3fp4::AttnShape{tokens, heads, kv_heads, head_dim, batch, max_tokens, max_kv});
}

namespace {

// Checks of an attention call; *out is set where there is something to do.
h3fp4_status check_attention(const Strided &q, const Strided &out, float *lse, int64_t tokens, int32_t heads,
                             const h3fp4_kv_cache *cache, const h3fp4_kv_batch *batch, int32_t max_kv,
                             float softmax_scale, int32_t causal, int32_t window, const void *workspace,
                             int64_t workspace_bytes, std::optional<h3fp4::AttnArgs> *args)
{
    h3fp4_status s = check_cache(cache);
    if (s != H3FP4_OK || (s = check_batch(batch, true, tokens)) != H3FP4_OK)
        return s;
    if (!attention_sizes_ok(tokens, heads, cache->heads, cache->head_dim, batch->batch, batch->max_tokens, max_kv) ||
        window < 0 || (causal != 0 && causal != 1) || !(softmax_scale - softmax_scale == 0.0f))
        return H3FP4_ERR_SHAPE;
    if (batch->batch == 0 || tokens == 0 || batch->max_tokens == 0)
        return H3FP4_OK;
    if ((s = check_strided(q)) != H3FP4_OK ||
        (s = check_strided_out(out, tokens, heads, cache->head_dim)) != H3FP4_OK)
        return s;
    if (ranges_overlap(q, out, tokens, heads, cache->head_dim))
        return H3FP4_ERR_UNSUPPORTED;
    const int64_t need = h3fp4::attention_workspace(h3fp4::AttnShape{tokens, heads, cache->heads, cache->head_dim,
                                                                     batch->batch, batch->max_tokens, max_kv});
    if (need > 0 && workspace == nullptr)
        return H3FP4_ERR_NULL;
    if (need < 0 || workspace_bytes < need)
        return H3FP4_ERR_SHAPE;
    if (!aligned16(workspace) || (reinterpret_cast<uintptr_t>(lse) & 3u) != 0)
        return H3FP4_ERR_ALIGN;
    *args = h3fp4::AttnArgs{static_cast<const uint16_t *>(q.p), q.token, q.head,
                            static_cast<uint16_t *>(const_cast<void *>(out.p)), out.token, out.head, lse, tokens, heads,
                            *cache, *batch, max_kv, softmax_scale, causal,
                            window > max_kv ? 0 : window};   // a window past every position hides nothing
    return H3FP4_OK;
}

}  // namespace

h3fp4_status h3fp4_kv_attention(const void *q_bf16, int64_t q_token_stride, int64_t q_head_stride, void *out_bf16,
                                int64_t out_token_stride, int64_t out_head_stride, float *lse, int64_t tokens,
                                int32_t heads, const h3fp4_kv_cache *cache, const h3fp4_kv_batch *batch,
                                int32_t max_kv, float softmax_scale, int32_t causal, int32_t window, void *workspace,
                                int64_t workspace_bytes, void *stream)
{
    std::optional<h3fp4::AttnArgs> a;
    const h3fp4_status s = check_attention({q_bf16, q_token_stride, q_head_stride},
                                           {out_bf16, out_token_stride, out_head_stride}, lse, tokens, heads, cache, batch,
                                           max_kv, softmax_scale, causal, window, workspace, workspace_bytes, &a);
    return a ? from_cuda(h3fp4::launch_attention(*a, workspace, as_stream(stream))) : s;
}

h3fp4_status h3fp4_swizzle_scales(const uint8_t *sf_logical, int64_t rows, int64_t cols, int64_t ld,
                                  uint8_t *sf_out, void *stream)
{
    if (sf_logical == nullptr || sf_out == nullptr)
        return H3FP4_ERR_NULL;
    if (rows < 0 || cols <= 0 || cols % 4 != 0 || ld < cols || rows > INT32_MAX)
        return H3FP4_ERR_SHAPE;
    if (!aligned16(sf_out))
        return H3FP4_ERR_ALIGN;
    return from_cuda(h3fp4::launch_swizzle_scales(sf_logical, rows, cols, ld, sf_out, as_stream(stream)));
}

h3fp4_status h3fp4_diag_producer_barrier_timeout(const void *x_bf16, int64_t ldx, int64_t m, int64_t m_pad,
                                                 int64_t d, float *tensor_scale, uint32_t *scratch, uint8_t *qdata,
                                                 uint8_t *sfa, uint32_t limit_us, void *stream)
{
    if ((x_bf16 == nullptr && m != 0) || tensor_scale == nullptr || scratch == nullptr)
        return H3FP4_ERR_NULL;
    if (m < 0 || m > INT32_MAX || d <= 0 || d % 256 != 0 || d > (int64_t(1) << 24) || ldx < d || limit_us == 0 ||
        limit_us > 2000000u)
        return H3FP4_ERR_SHAPE;
    if (!aligned16(x_bf16) || ldx % 8 != 0)
        return H3FP4_ERR_ALIGN;
    h3fp4_status s = check_pack_outputs(m, m_pad, qdata, sfa);
    if (s != H3FP4_OK)
        return s;
    return from_cuda(h3fp4::launch_quantize_pack_barrier_timeout(
        static_cast<const uint16_t *>(x_bf16), ldx, m, m_pad, d, tensor_scale, scratch, qdata, sfa,
        static_cast<uint64_t>(limit_us) * 1000u, as_stream(stream)));
}

h3fp4_status h3fp4_diag_gemm_wait_timeout(const uint8_t *a_q, const uint8_t *a_sf, const float *a_tensor_scale,
                                          const uint8_t *b_q, const uint8_t *b_sf, const float *b_tensor_scale,
                                          void *c_bf16, int64_t ldc, int64_t m, int64_t m_pad, int64_t n, int64_t k,
                                          uint32_t limit_us, void *stream)
{
    h3fp4_gemm_config c;
    h3fp4_status s = check_gemm(a_q, a_sf, a_tensor_scale, b_q, b_sf, b_tensor_scale, c_bf16, ldc, m, m_pad, n, k,
                                nullptr, &c);
    if (s != H3FP4_OK)
        return s;
    if (limit_us == 0 || limit_us > 2000000u)
        return H3FP4_ERR_SHAPE;
    return h3fp4::launch_gemm_wait_timeout(a_q, a_sf, a_tensor_scale, b_q, b_sf, b_tensor_scale,
                                           static_cast<uint16_t *>(c_bf16), ldc, m, m_pad, n, k,
                                           static_cast<uint64_t>(limit_us) * 1000u, as_stream(stream));
}

h3fp4_status h3fp4_diag_attention_wait_timeout(const void *q_bf16, int64_t q_token_stride, int64_t q_head_stride,
                                               void *out_bf16, int64_t out_token_stride, int64_t out_head_stride,
                                               float *lse, int64_t tokens, int32_t heads, const h3fp4_kv_cache *cache,
                                               const h3fp4_kv_batch *batch, int32_t max_kv, void *workspace,
                                               int64_t workspace_bytes, uint32_t limit_us, void *stream)
{
    std::optional<h3fp4::AttnArgs> a;
    const h3fp4_status s = check_attention({q_bf16, q_token_stride, q_head_stride},
                                           {out_bf16, out_token_stride, out_head_stride}, lse, tokens, heads, cache, batch,
                                           max_kv, 1.0f, 0, 0, workspace, workspace_bytes, &a);
    if (s != H3FP4_OK || !a)
        return s;
    if (limit_us == 0 || limit_us > 2000000u)
        return H3FP4_ERR_SHAPE;
    if (!h3fp4::attention_timeout_ok(*a))
        return H3FP4_ERR_UNSUPPORTED;
    return from_cuda(h3fp4::launch_attention_wait_timeout(*a, workspace, static_cast<uint64_t>(limit_us) * 1000u,
                                                          as_stream(stream)));
}

h3fp4_status h3fp4_device_error(uint32_t *code)
{
    if (code == nullptr)
        return H3FP4_ERR_NULL;
    uint32_t kv = 0, attn = 0;
    const h3fp4_status s = h3fp4::read_device_error(code);
    if (s != H3FP4_OK)
        return s;
    if (h3fp4::read_kvcache_error(&kv) != cudaSuccess || h3fp4::read_attention_error(&attn) != cudaSuccess)
        return H3FP4_ERR_CUDA;
    *code |= kv | attn;
    return H3FP4_OK;
}

const char *h3fp4_status_string(h3fp4_status status)
{
    switch (status) {
    case H3FP4_OK: return "ok";
    case H3FP4_ERR_NULL: return "null pointer";
    case H3FP4_ERR_ALIGN: return "misaligned pointer or leading dimension";
    case H3FP4_ERR_SHAPE: return "invalid shape";
    case H3FP4_ERR_UNSUPPORTED: return "unsupported configuration";
    case H3FP4_ERR_CUDA: return "CUDA error";
    case H3FP4_ERR_DEVICE: return "device-side error";
    }
    return "unknown status";
}

const char *h3fp4_build_info(void)
{
    return "h3fp4 " H3FP4_VERSION " sm_103a (nvcc " H3FP4_STR(__CUDACC_VER_MAJOR__) "." H3FP4_STR(
        __CUDACC_VER_MINOR__) "." H3FP4_STR(__CUDACC_VER_BUILD__) ")";
}

}  // extern "C"

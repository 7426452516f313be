// launch.h -- internal launchers behind the C ABI (not exported).
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "h3fp4.h"

namespace h3fp4 {

// Row ranges of the modulation segments, passed to kernels by value.
struct SegTable {
    int32_t off[H3FP4_MAX_SEGMENTS + 1];
    int32_t nseg;
};

// Multiprocessor count of the current device (cached per device).
int sm_count();

cudaError_t launch_modulate_absmax(const uint16_t *x, int64_t ldx, int64_t m, int64_t d,
                                   const uint16_t *shift, const uint16_t *scale, int64_t ld_mod,
                                   const SegTable &seg, float *ts, uint32_t *scratch, cudaStream_t st);

cudaError_t launch_modulate_pack(const uint16_t *x, int64_t ldx, int64_t m, int64_t m_pad, int64_t d,
                                 const uint16_t *shift, const uint16_t *scale, int64_t ld_mod,
                                 const SegTable &seg, const float *ts, uint8_t *qdata, uint8_t *sf,
                                 cudaStream_t st);

cudaError_t launch_swiglu_pack(const uint16_t *gate, int64_t ldg, const uint16_t *up, int64_t ldu,
                               int64_t m, int64_t m_pad, int64_t f, float *ts, uint32_t *scratch,
                               uint8_t *qdata, uint8_t *sf, uint16_t *h, cudaStream_t st);

cudaError_t launch_modulate_produce(const uint16_t *x, int64_t ldx, int64_t m, int64_t m_pad, int64_t d,
                                    const uint16_t *shift, const uint16_t *scale, int64_t ld_mod, const SegTable &seg,
                                    float *ts, uint32_t *scratch, uint8_t *qdata, uint8_t *sf, cudaStream_t st);

cudaError_t read_producer_error(uint32_t *code);

cudaError_t launch_quantize_pack(const uint16_t *x, int64_t ldx, int64_t m, int64_t m_pad, int64_t d,
                                 float *ts, uint32_t *scratch, uint8_t *qdata, uint8_t *sf, cudaStream_t st);

cudaError_t launch_swizzle_scales(const uint8_t *src, int64_t rows, int64_t cols, int64_t ld,
                                  uint8_t *dst, cudaStream_t st);

// Gated residual epilogue of the GEMM: out = RN_bf16(residual + RN_bf16(gate_s * c)),
// gate [nseg, n] bf16 selected by the row segments.
struct GatedArgs {
    const uint16_t *gate;
    int64_t ld_gate;
    SegTable seg;
    const void *residual;
    int64_t ldr;
};

h3fp4_status launch_gemm(const uint8_t *a_q, const uint8_t *a_sf, const float *a_ts, const uint8_t *b_q,
                         const uint8_t *b_sf, const float *b_ts, uint16_t *c, int64_t ldc, int64_t m,
                         int64_t m_pad, int64_t n, int64_t k, const h3fp4_gemm_config &cfg, const GatedArgs *gated,
                         cudaStream_t st);

// Failure detection (diagnostics, not the hot path): the default GEMM with its
// operand loads withheld, so that every consumer wait runs out after wait_ns;
// the cooperative plain producer with a grid-barrier arrival target the grid
// cannot meet and a barrier limit of wait_ns.  Outputs are left untouched; the
// kernels record device error bits and return.
h3fp4_status launch_gemm_wait_timeout(const uint8_t *a_q, const uint8_t *a_sf, const float *a_ts,
                                      const uint8_t *b_q, const uint8_t *b_sf, const float *b_ts, uint16_t *c,
                                      int64_t ldc, int64_t m, int64_t m_pad, int64_t n, int64_t k, uint64_t wait_ns,
                                      cudaStream_t st);
cudaError_t launch_quantize_pack_barrier_timeout(const uint16_t *x, int64_t ldx, int64_t m, int64_t m_pad,
                                                int64_t d, float *ts, uint32_t *scratch, uint8_t *qdata, uint8_t *sf,
                                                uint64_t wait_ns, cudaStream_t st);

h3fp4_status read_device_error(uint32_t *code);

// Lets a kernel use this much dynamic shared memory: set on its first call on
// a device (threads that race on that set the same value).
template <auto kKernel>
cudaError_t allow_shared(int bytes)
{
    static std::atomic<uint64_t> done{0};   // a bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && (done.load(std::memory_order_relaxed) >> dev & 1) != 0))
        return e;
    e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64)
        done.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
    return e;
}

// ---------------------------------------------------------------------------
// Rotary positions, the 8-bit cache and its attention: arguments by value.
// ---------------------------------------------------------------------------
struct RopeArgs {
    const float *positions;
    int64_t ld_positions;
    const double *freqs;
    int32_t end[H3FP4_ROPE_MAX_AXES];   // first channel past each axis (unused axes: the total)
    int32_t pairs;                      // turned pairs; 0 = no rotation
    int32_t layout, inverse;
};

using KvCache = h3fp4_kv_cache;
using KvBatch = h3fp4_kv_batch;

cudaError_t launch_rope(const uint16_t *x, int64_t xt, int64_t xh, uint16_t *out, int64_t ot, int64_t oh,
                        int64_t tokens, int heads, int dim, const RopeArgs &r, cudaStream_t st);

cudaError_t launch_kv_write(const KvCache &cache, const KvBatch &batch, const uint16_t *k, int64_t kt, int64_t kh,
                            const uint16_t *v, int64_t vt, int64_t vh, int64_t tokens, const RopeArgs &rope,
                            cudaStream_t st);

cudaError_t launch_kv_read(const KvCache &cache, const KvBatch &batch, uint16_t *k, int64_t kt, int64_t kh,
                           uint16_t *v, int64_t vt, int64_t vh, int64_t tokens, cudaStream_t st);

struct AttnArgs {
    const uint16_t *q;
    int64_t qt, qh;        // strides of tokens and heads
    uint16_t *out;
    int64_t ot, oh;
    float *lse;
    int64_t tokens;
    int32_t heads;
    KvCache cache;
    KvBatch batch;
    int32_t max_kv;
    float scale;
    int32_t causal, window;
};

struct AttnShape {
    int64_t tokens;
    int32_t heads, kv_heads, head_dim, batch, max_tokens, max_kv;
    int32_t reach = 0;   // most keys that a query sees under a causal window; 0: all
};

int64_t attention_workspace(const AttnShape &s);
cudaError_t launch_attention(const AttnArgs &a, void *workspace, cudaStream_t st);

// Failure detection: few queries with copies that never complete.
bool attention_timeout_ok(const AttnArgs &a);
cudaError_t launch_attention_wait_timeout(const AttnArgs &a, void *workspace, uint64_t wait_ns, cudaStream_t st);

cudaError_t read_kvcache_error(uint32_t *code);
cudaError_t read_attention_error(uint32_t *code);

}  // namespace h3fp4

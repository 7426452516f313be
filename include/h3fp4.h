/*
 * h3fp4.h -- C ABI of the GB300 (sm_103a) modulation-fused NVFP4 activation
 * producer and block-scaled NVFP4 GEMM.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Every pointer is CALLER-OWNED DEVICE memory unless its comment says
 *    "host".  The library never allocates device memory and keeps no pointer
 *    after the call returns.  A pointer to an array with zero rows (the
 *    activation inputs when m == 0, the GEMM output when m == 0 or n == 0)
 *    may be NULL.
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *    Every call only enqueues work on that stream and returns; nothing
 *    synchronises the host.  Outputs are valid once the stream reaches them.
 *    The first call of an entry point on a device sets its kernels'
 *    attributes; after that, h3fp4_modulate_absmax, h3fp4_modulate_pack,
 *    h3fp4_swiglu_pack and h3fp4_gemm may be captured into a CUDA graph and
 *    replayed (the captured calls keep their pointers; new inputs are copied
 *    into the same buffers).
 *  - Arguments are checked on the host before anything is enqueued.  A failed
 *    check returns an error status and enqueues nothing.  A CUDA launch error
 *    returns H3FP4_ERR_CUDA (the CUDA error itself stays readable with
 *    cudaGetLastError()).  No entry point traps or aborts.
 *  - bf16 tensors are raw IEEE bfloat16 bit patterns (2 bytes), row-major,
 *    with the given leading dimension in ELEMENTS.
 *  - QDATA is packed E2M1, row-major [rows, width/2] bytes, element 2i in the
 *    low nibble of byte i and element 2i+1 in the high nibble.
 *  - Block scales (SFA / SFB) are E4M3 (bias 7, max 448, no infinities), one
 *    per 16 consecutive values of a row, stored in the block-scaled GEMM's
 *    scale layout: the logical [R, C] scale matrix (R = rows rounded up to a
 *    multiple of 128, C = width/16) is cut into 128 x 4 tiles stored
 *    tile-row-major as 512-byte atoms, and inside an atom the scale of row r,
 *    column c sits at byte (r % 32) * 16 + ((r % 128) / 32) * 4 + (c % 4).
 *    A scale buffer for `rows` rows therefore holds ceil(rows/128)*128 * C
 *    bytes.
 *
 * Numerics (fixed encoding rule; the source pages name the quantities but not
 * the reciprocal detail):
 *    y   = RN_bf16(RN_bf16(x * RN_bf16(scale + 1)) + shift)
 *    ts  = RN_f32(amax / 2688)                       (2688 = 6 * 448)
 *    bs  = E4M3_RNE_sat(RN_f32(block_amax / RN_f32(6 * ts)))   (0 if block_amax == 0)
 *    q   = E2M1_RNE_sat(RN_f32(y / RN_f32(dec(bs) * ts)))      (signed 0 if that product is 0)
 *    C   = RN_bf16(RN_f32(ts_a * ts_b) * sum_k a_k b_k)        (FP32 accumulation)
 * Non-finite inputs follow the same formulas in IEEE arithmetic: a NaN makes
 * its block maximum, amax and ts NaN, an infinity makes ts infinite; a NaN
 * quotient encodes as the E4M3 NaN code 0x7F and a NaN scale product, like a
 * zero one, gives zeros with y's signs.  So a tensor holding a NaN or an
 * infinity packs to signed-zero codes with scale 0x7F on its non-zero blocks
 * (0 on blocks whose quotient is 0), and any GEMM over it is NaN.
 */
#ifndef H3FP4_H
#define H3FP4_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define H3FP4_API __attribute__((visibility("default")))
#else
#define H3FP4_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum h3fp4_status {
    H3FP4_OK = 0,
    H3FP4_ERR_NULL = 1,        /* a required pointer is NULL */
    H3FP4_ERR_ALIGN = 2,       /* a pointer or leading dimension breaks the 16-byte rule */
    H3FP4_ERR_SHAPE = 3,       /* a size is negative, too large, or not a required multiple */
    H3FP4_ERR_UNSUPPORTED = 4, /* a configuration the library does not implement */
    H3FP4_ERR_CUDA = 5,        /* a CUDA call failed (see cudaGetLastError) */
    H3FP4_ERR_DEVICE = 6       /* a kernel recorded a device-side error (bounded wait ran out) */
} h3fp4_status;

/* Most modulation segments one call accepts. */
#define H3FP4_MAX_SEGMENTS 16

/*
 * h3fp4_modulate_absmax -- producer pass 1.
 * Source: "NVFP4 Modulation Producer Fusion", Dataflow (prototype step 1) and
 * Exactness Contract; "NVFP4 Streaming Design", Numerical Constraint items 1-2.
 *
 * Modulates every logical row of x (row r uses segment s, the one with
 * seg_row_offsets[s] <= r < seg_row_offsets[s+1]) without storing the result,
 * reduces one exact global max |y| over rows [0, m), and writes the FP32
 * tensor scale RN_f32(amax / 2688) to *tensor_scale.  A NaN anywhere in y
 * makes the tensor scale NaN.
 *
 *   x_bf16          [m, d] bf16, leading dimension ldx (>= d, multiple of 8), 16-byte aligned
 *   shift_bf16      [nseg, d] bf16, leading dimension ld_mod (>= d, multiple of 8), 16-byte aligned
 *   scale_bf16      [nseg, d] bf16, same layout as shift
 *   seg_row_offsets HOST array of nseg + 1 int32: 0 = off[0] <= off[1] <= ... <= off[nseg] = m
 *   nseg            1 .. H3FP4_MAX_SEGMENTS
 *   tensor_scale    1 float (output)
 *   scratch         2 uint32 words of device scratch (contents on entry are ignored; the
 *                   call clears them on the stream).  Two calls that overlap on the GPU
 *                   must not share it.
 *   d               multiple of 256; m >= 0 (m == 0 gives tensor scale 0)
 */
H3FP4_API h3fp4_status h3fp4_modulate_absmax(const void *x_bf16, int64_t ldx, int64_t m, int64_t d,
                                   const void *shift_bf16, const void *scale_bf16, int64_t ld_mod,
                                   const int32_t *seg_row_offsets, int32_t nseg,
                                   float *tensor_scale, uint32_t *scratch, void *stream);

/*
 * h3fp4_modulate_pack -- producer pass 2.
 * Source: "NVFP4 Modulation Producer Fusion", Dataflow (prototype step 2);
 * "NVFP4 Streaming Design", Numerical Constraint items 3-4; "FC2 NVFP4 Library
 * Scheduling", Exact Operation (zero-row padding to the descriptor M).
 *
 * Re-derives y exactly as pass 1 does and writes QDATA and SFA for rows
 * [0, m_pad).  Rows m <= r < m_pad get zero QDATA bytes; every scale of a row
 * r >= m (up to ceil(m_pad/128)*128) is 0.  Every byte of both buffers is
 * written.
 *
 *   tensor_scale  1 float (input, normally the output of pass 1)
 *   qdata         [m_pad, d/2] bytes, 16-byte aligned
 *   sfa           ceil(m_pad/128)*128 * d/16 bytes in the scale layout, 16-byte aligned
 *   m <= m_pad; other arguments as for h3fp4_modulate_absmax.
 */
H3FP4_API h3fp4_status h3fp4_modulate_pack(const void *x_bf16, int64_t ldx, int64_t m, int64_t m_pad,
                                 int64_t d, const void *shift_bf16, const void *scale_bf16,
                                 int64_t ld_mod, const int32_t *seg_row_offsets, int32_t nseg,
                                 const float *tensor_scale, uint8_t *qdata, uint8_t *sfa,
                                 void *stream);

/*
 * h3fp4_modulate_produce -- h3fp4_modulate_absmax followed by
 * h3fp4_modulate_pack in ONE cooperative launch.
 * Source: "NVFP4 Streaming Design", P2 (a single-launch cooperative producer:
 * pass 1 and pass 2 around a grid barrier, with a bounded wait).
 *
 * Same arguments and results as the two calls (tensor_scale is written and
 * also used by the pack).  Every CTA of the co-resident grid reduces its
 * pass-1 tiles, arrives on a grid barrier in `scratch` and packs its pass-2
 * tiles once all have arrived; the barrier gives up after 2 s, reporting
 * bit 8 through h3fp4_device_error instead of hanging.
 */
H3FP4_API h3fp4_status h3fp4_modulate_produce(const void *x_bf16, int64_t ldx, int64_t m, int64_t m_pad,
                                    int64_t d, const void *shift_bf16, const void *scale_bf16,
                                    int64_t ld_mod, const int32_t *seg_row_offsets, int32_t nseg,
                                    float *tensor_scale, uint32_t *scratch, uint8_t *qdata,
                                    uint8_t *sfa, void *stream);

/*
 * h3fp4_swiglu_pack -- SwiGLU-fused producer (both passes, in one cooperative launch).
 * Source: "FC2 NVFP4 Library Scheduling", Exact Operation and Current Baseline
 * (exact BF16 SwiGLU fused into NVFP4 production of the FC2 input).
 *
 * h = RN_bf16(silu_bf16(gate) * up) with silu_bf16 the correctly rounded bf16
 * of g / (1 + e^-g); then the global absmax -> tensor scale and the pack of h,
 * exactly as the modulation producer does for y.
 *
 *   gate_bf16, up_bf16  [m, f] bf16, leading dimensions ldg / ldu (multiples of 8), 16-byte aligned
 *   f                   multiple of 256
 *   tensor_scale        1 float (output)
 *   scratch             2 uint32 words (as for h3fp4_modulate_absmax)
 *   qdata, sfa          as for h3fp4_modulate_pack with d = f
 *   h_workspace         NULL, or [m, f] bf16 (leading dimension f) that pass 1 fills with h
 *                       so that pass 2 reads h instead of recomputing it
 */
H3FP4_API h3fp4_status h3fp4_swiglu_pack(const void *gate_bf16, int64_t ldg, const void *up_bf16,
                               int64_t ldu, int64_t m, int64_t m_pad, int64_t f,
                               float *tensor_scale, uint32_t *scratch, uint8_t *qdata,
                               uint8_t *sfa, void *h_workspace, void *stream);

/*
 * h3fp4_quantize_pack -- NVFP4 producer of an activation that needs no fused
 * transform (both passes, in one cooperative launch).
 * Source: "NVFP4 Modulation Producer Fusion", Change Summary (the same two-pass
 * producer: global absmax -> FP32 tensor scale, then E4M3 block scales and
 * E2M1 codes); "NVFP4 Streaming Design", P0 and P2 (the attention-output
 * projection is one of the four H3 projections, its input quantized by the
 * same rules without the modulation).
 *
 * amax = max |x| over the m logical rows, ts = RN_f32(amax / 2688), then the
 * pack of x exactly as h3fp4_modulate_pack packs y.
 *
 *   x_bf16        [m, d] bf16, leading dimension ldx (multiple of 8), 16-byte aligned
 *   d             multiple of 256
 *   tensor_scale  1 float (output)
 *   scratch       2 uint32 words (as for h3fp4_modulate_absmax)
 *   qdata, sfa    as for h3fp4_modulate_pack
 */
H3FP4_API h3fp4_status h3fp4_quantize_pack(const void *x_bf16, int64_t ldx, int64_t m, int64_t m_pad,
                                 int64_t d, float *tensor_scale, uint32_t *scratch, uint8_t *qdata,
                                 uint8_t *sfa, void *stream);

/* Tuning knobs of the GEMM; pass NULL for the defaults. */
typedef struct h3fp4_gemm_config {
    /* N-group A-tile reuse factor: the persistent schedule walks the output
     * tiles (256 columns wide) in groups of n_group N-tiles x all M-tiles, N
     * fastest, so each A row block serves n_group consecutive output tiles
     * while it is L2-resident (0 = kernel default: the default kernel takes
     * the fewest near-equal groups whose B tiles total at most ~27.5 MB, the
     * others 28; values above the number of N-tiles are clamped). */
    int32_t n_group;
    int32_t stages;    /* reserved, must be 0 (the pipeline depth is fixed per kernel) */
    /* GEMM kernel: 0 = library default (currently 4), 1 = one CTA per 128 x 256 output tile
     * (4-stage ring, scale warps stage the scales in TMEM), 4 = CTA pairs on
     * two SMs per 256 x 256 tile (tcgen05 cta_group::2, each SM loads its own
     * half of A and of B; 5-stage ring) whose leader copies the scales into
     * TMEM with tcgen05.cp from two warps of their own.  Other values:
     * H3FP4_ERR_UNSUPPORTED. */
    int32_t cta_pair;
    int32_t reserved;  /* must be 0 */
} h3fp4_gemm_config;

/*
 * h3fp4_gemm -- block-scaled NVFP4 GEMM with the alpha epilogue.
 * Source: "NVFP4 Streaming Design", Available Foundation (E2M1 A/B, E4M3
 * scales, FP32 accumulation, BF16 output) and P0 (alpha = activation tensor
 * scale x weight tensor scale applied before the BF16 conversion); "FC2 NVFP4
 * Library Scheduling", Exact Operation (row-major activation [M,K] times
 * weight [N,K] to row-major BF16 [M,N], alpha from device pointers, logical
 * rows sliced from the padded descriptor M).
 *
 * C[i, j] = RN_bf16(RN_f32(*a_tensor_scale * *b_tensor_scale) * acc[i, j]),
 * acc = FP32 accumulation over k of e2m1(a) e4m3(sfa) e2m1(b) e4m3(sfb).
 * Only rows i < m and columns j < n are written.
 *
 *   a_q   [m_pad, k/2] bytes (activation QDATA), 16-byte aligned
 *   a_sf  ceil(m_pad/128)*128 * k/16 bytes, scale layout, 16-byte aligned
 *   b_q   [n, k/2] bytes (weight QDATA), 16-byte aligned
 *   b_sf  ceil(n/128)*128 * k/16 bytes, scale layout, 16-byte aligned
 *   a_tensor_scale, b_tensor_scale   1 float each
 *   c_bf16  [m, n] bf16 output with leading dimension ldc (>= n, multiple of 8), 16-byte aligned
 *   k multiple of 256; n multiple of 128; 0 <= m <= m_pad; m_pad multiple of 16
 */
H3FP4_API h3fp4_status h3fp4_gemm(const uint8_t *a_q, const uint8_t *a_sf, const float *a_tensor_scale,
                        const uint8_t *b_q, const uint8_t *b_sf, const float *b_tensor_scale,
                        void *c_bf16, int64_t ldc, int64_t m, int64_t m_pad, int64_t n, int64_t k,
                        const h3fp4_gemm_config *cfg, void *stream);

/*
 * h3fp4_gemm_gated_residual -- h3fp4_gemm with the gated residual epilogue.
 * Source: "NVFP4 Streaming Design", P4: Exact Epilogue (after the owned GEMM,
 * the explicit BF16 conversion, gate multiply, residual add and final BF16
 * rounding sequence), for the projections whose output is added to the
 * residual stream through an AdaLN gate (attention output, FC2).
 *
 * out[i, j] = RN_bf16(residual[i, j] + RN_bf16(gate[s(i), j] * c[i, j]))
 * with c[i, j] the value h3fp4_gemm would write and s(i) the segment of row i
 * (seg_row_offsets as for h3fp4_modulate_absmax: host array of nseg + 1
 * non-decreasing offsets, [0] = 0, [nseg] = m).  Only rows i < m and columns
 * j < n are written.
 *
 *   gate_bf16      [nseg, n] bf16, leading dimension ld_gate (>= n, multiple of 8), 16-byte aligned
 *   residual_bf16  [m, n] bf16, leading dimension ldr (>= n, multiple of 8), 16-byte aligned
 *   out_bf16       [m, n] bf16, leading dimension ldo; either the residual itself (same pointer and
 *                  leading dimension: updated in place) or not overlapping it (else H3FP4_ERR_UNSUPPORTED)
 *   other arguments as for h3fp4_gemm
 */
H3FP4_API h3fp4_status h3fp4_gemm_gated_residual(
    const uint8_t *a_q, const uint8_t *a_sf, const float *a_tensor_scale, const uint8_t *b_q, const uint8_t *b_sf,
    const float *b_tensor_scale, const void *gate_bf16, int64_t ld_gate, const int32_t *seg_row_offsets, int32_t nseg,
    const void *residual_bf16, int64_t ldr, void *out_bf16, int64_t ldo, int64_t m, int64_t m_pad, int64_t n,
    int64_t k, const h3fp4_gemm_config *cfg, void *stream);

/*
 * ---------------------------------------------------------------------------
 * Attention between the QKV and the attention-output projections: rotary
 * positions with several axes, an 8-bit key/value cache in pages, and the
 * attention that reads it.  No counterpart on the source pages, which stop at
 * the linears; arithmetic and layouts are defined here.
 * ---------------------------------------------------------------------------
 *
 * h3fp4_rope -- rotary positions along up to 4 axes (time, height, width, ...).
 *
 * The first dims[0] channels of a head turn with the position on axis 0, the
 * next dims[1] with axis 1, and so on; channels past sum(dims) are copied.
 * Pair j of axis a (j < dims[a]/2) takes the angle phi = position * frequency,
 * with the frequency of that pair in radians per unit of position, and
 *     a' = RN_bf16(a cos(phi) - b sin(phi)),  b' = RN_bf16(a sin(phi) + b cos(phi))
 * in FP32 before the rounding.  The angle is reduced to a fraction of a turn
 * without rounding error, so that the result keeps FP32 accuracy at any
 * position a float holds exactly.  Non-finite positions or frequencies, or
 * |position * frequency| >= 2^24 turns, are outside the definition: their
 * results are unspecified.
 * inverse = 1 turns by -phi: the inverse map and, the map being orthogonal,
 * also the gradient of the forward one.
 */
#define H3FP4_ROPE_MAX_AXES 4
typedef struct h3fp4_rope {
    const float *positions;     /* device [tokens, axes], leading dimension ld_positions (>= axes) */
    int64_t ld_positions;
    const double *freqs;        /* device [sum(dims)/2]: the pairs of axis 0, then of axis 1, ... */
    int32_t axes;               /* 1 .. H3FP4_ROPE_MAX_AXES */
    int32_t dims[H3FP4_ROPE_MAX_AXES]; /* channels of each axis: even, >= 0, their sum <= the head's channels */
    int32_t layout;             /* within an axis' channels, pair j is 0: (2j, 2j + 1); 1: (j, j + dims/2) */
    int32_t inverse;            /* 0 or 1 */
} h3fp4_rope;

/*
 * h3fp4_rope_axes -- out = x with every head of every token turned.
 *
 *   x_bf16, out_bf16  [tokens, heads, head_dim] bf16, the channels contiguous; strides of tokens and
 *                     heads in elements (multiples of 8, not negative), 16-byte aligned.  out either is x
 *                     (same pointer and strides: in place) or does not overlap it (the two address ranges
 *                     from first to last element; else H3FP4_ERR_UNSUPPORTED).  Queries and keys in the
 *                     rows of a QKV projection are one call with heads = 2 H.  Strides: at most 2^30.
 *   head_dim          multiple of 8, 8 .. 256
 */
H3FP4_API h3fp4_status h3fp4_rope_axes(const void *x_bf16, int64_t x_token_stride, int64_t x_head_stride,
                                       void *out_bf16, int64_t out_token_stride, int64_t out_head_stride,
                                       int64_t tokens, int32_t heads, int32_t head_dim, const h3fp4_rope *rope,
                                       void *stream);

/*
 * h3fp4_norm_rope -- per-head RMS norm of queries and keys, and their rotation,
 * in one pass over each.
 *
 * For every token and head, with w the side's weight:
 *     r = 1 / sqrt(mean(x^2) + eps),  z = x r w,  out = RN_bf16(z turned as by h3fp4_rope_axes)
 * in FP32 before the one rounding.  Rows of any finite size are in range, and
 * weights of up to 2^77 (x meets w before r); a row with an infinity gives 0,
 * and NaN in the infinity's pair; one with a NaN gives NaN.
 *
 *   q, k       the two sides; either may be NULL (or have no heads).  x and out are [tokens, heads, head_dim]
 *              bf16, strides as for h3fp4_rope_axes.  out either is its own x (same pointer and strides: in place)
 *              or has no element in common with either side's x or the other out (else H3FP4_ERR_UNSUPPORTED): of
 *              the same strides they may be interleaved, as queries and keys in a QKV projection's rows are, of
 *              others their ranges are apart
 *   weight     device [head_dim], shared by the side's heads; bf16 (weight_f32 0) or float (1).  NULL: ones
 *   head_dim   multiple of 8, 8 .. 256
 *   eps        2^-100 .. 2^20
 *   rope       NULL: no rotation.  inverse must be 0
 */
typedef struct h3fp4_norm_heads {
    const void *x;
    int64_t x_token_stride, x_head_stride;
    void *out;
    int64_t out_token_stride, out_head_stride;
    const void *weight;
    int32_t heads;              /* 0 .. 65535 */
    int32_t weight_f32;         /* 0 or 1 */
} h3fp4_norm_heads;

H3FP4_API h3fp4_status h3fp4_norm_rope(const h3fp4_norm_heads *q, const h3fp4_norm_heads *k, int64_t tokens,
                                       int32_t head_dim, float eps, const h3fp4_rope *rope, void *stream);

/*
 * h3fp4_norm_rope_backward -- gradients of h3fp4_norm_rope from those of its
 * outputs, dy; nothing of the forward pass is kept but its inputs.
 *
 * With g = dy turned back and r as above:
 *     dx = RN_bf16(r (w g - x r^2 mean(w g x))),  dweight[c] = sum of g[c] x[c] r over the side's tokens and heads
 * Products w g are in range up to 2^115.  dweight is written, not added to, in
 * FP32 sums of a fixed order (the same bits every time on a device); zeros where
 * there are no tokens or heads.
 *
 *   dy, x, dx  [tokens, heads, head_dim] bf16, strides as for h3fp4_rope_axes.  dx either is its side's dy or x
 *              (same pointer and strides) or has no element in common with any of the call's arrays, as above
 *   weight     as in the forward call
 *   dweight    device float [head_dim], 4-byte aligned; NULL: not wanted
 *   workspace  h3fp4_norm_rope_backward_workspace bytes of device scratch, 16-byte aligned (contents on entry are
 *              ignored; two calls that overlap on the GPU must not share it); may be NULL where no dweight is wanted
 *   other arguments as for h3fp4_norm_rope
 */
typedef struct h3fp4_norm_grads {
    const void *dy;
    int64_t dy_token_stride, dy_head_stride;
    const void *x;
    int64_t x_token_stride, x_head_stride;
    void *dx;
    int64_t dx_token_stride, dx_head_stride;
    const void *weight;
    float *dweight;
    int32_t heads;
    int32_t weight_f32;
} h3fp4_norm_grads;

H3FP4_API h3fp4_status h3fp4_norm_rope_backward(const h3fp4_norm_grads *q, const h3fp4_norm_grads *k, int64_t tokens,
                                                int32_t head_dim, float eps, const h3fp4_rope *rope, void *workspace,
                                                int64_t workspace_bytes, void *stream);

/* Bytes of workspace that h3fp4_norm_rope_backward wants on the current device (-1 for a head_dim it refuses). */
H3FP4_API int64_t h3fp4_norm_rope_backward_workspace(int32_t head_dim);

/*
 * h3fp4_kv_cache -- keys and values in E4M3 (bias 7, max 448), in pages of
 * page_size tokens, with one FP32 scale per page and head for the keys and
 * one for the values: a value is code * scale.
 *
 *   codes   [num_pages, heads, page_size, head_dim] bytes, contiguous, 16-byte aligned
 *   scales  [num_pages, heads] float, contiguous
 *   page_size 16, 32, 64 or 128;  head_dim 64 or 128;  num_pages * heads below 2^31
 *
 * A page table names each sequence's pages: position p of sequence b is token
 * p % page_size of page page_table[b * ld_table + p / page_size].  A page may
 * appear in several places as long as no call writes it for more than one.
 */
typedef struct h3fp4_kv_cache {
    uint8_t *k_codes, *v_codes;
    float *k_scale, *v_scale;
    int32_t num_pages, page_size, heads, head_dim;
} h3fp4_kv_cache;

/*
 * h3fp4_kv_batch -- the sequences of a call.  Tokens of all sequences are
 * packed: those of sequence b are rows cu_tokens[b] .. cu_tokens[b+1] - 1 of
 * the call's token arrays, max_tokens the most that any sequence has.  The
 * arrays are in DEVICE memory (they may change between replays of a captured
 * call); what they hold is checked by the kernels: an entry that is out of
 * range (a page outside the cache or past the table, rows outside the token
 * arrays, more tokens than max_tokens) is not followed, and bit 512 is
 * reported through h3fp4_device_error.  What such a sequence's outputs hold is
 * then unspecified.  Of a sequence without tokens in the call neither the
 * length nor the pages are looked at.
 */
typedef struct h3fp4_kv_batch {
    const int32_t *page_table;  /* device [batch, ld_table] */
    int64_t ld_table;           /* pages a sequence's row of the table has room for */
    const int32_t *len;         /* device [batch]: meaning at each call */
    const int32_t *cu_tokens;   /* device [batch + 1] */
    int32_t batch;              /* 0 .. 65535 */
    int32_t max_tokens;         /* 0 .. 1,000,000 */
} h3fp4_kv_batch;

/*
 * h3fp4_kv_cache_write -- quantises new keys and values into the cache.
 *
 * len[b] is the number of tokens that sequence b holds before the call; its
 * new tokens take the positions from len[b] on.  For each page and head with
 * new tokens, for keys and values each:
 *     e = ceil(log2(amax / 448)) held to [-40, 119] (amax = 0: -40), amax over the page's new values
 *     scale = 2^e, or the page's scale so far if that is larger and the page holds earlier tokens
 *     code = E4M3_RNE_sat(x / scale)
 * Where the scale grows, the page's earlier codes are rounded to it (a shift
 * by a power of two: exact but for codes that become subnormal).  Powers of
 * two keep that repeated rounding harmless, and code * scale exact in bf16.  A
 * NaN or infinite element is stored as the E4M3 NaN 0x7F and does not count
 * for amax.  Pages' tokens past the new ones keep their bytes.
 *
 *   k_bf16, v_bf16  [tokens, heads, head_dim] bf16, strides as for h3fp4_rope_axes
 *   rope            NULL, or positions of the new tokens: keys are turned first, with the bf16 result
 *                   of h3fp4_rope_axes
 */
H3FP4_API h3fp4_status h3fp4_kv_cache_write(const h3fp4_kv_cache *cache, const h3fp4_kv_batch *batch,
                                            const void *k_bf16, int64_t k_token_stride, int64_t k_head_stride,
                                            const void *v_bf16, int64_t v_token_stride, int64_t v_head_stride,
                                            int64_t tokens, const h3fp4_rope *rope, void *stream);

/*
 * h3fp4_kv_cache_read -- the cache's keys and values as bf16,
 * RN_bf16(code * scale).
 *
 * len[b] is the first position of sequence b that is read (NULL: 0 for every
 * sequence), its number of tokens cu_tokens[b+1] - cu_tokens[b].
 *
 *   k_bf16, v_bf16  [tokens, heads, head_dim] bf16 outputs, strides as for h3fp4_rope_axes; one of the
 *                   two may be NULL.  They have no element in common (else H3FP4_ERR_UNSUPPORTED): of
 *                   the same strides they may be interleaved, of others their ranges are apart
 */
H3FP4_API h3fp4_status h3fp4_kv_cache_read(const h3fp4_kv_cache *cache, const h3fp4_kv_batch *batch, void *k_bf16,
                                           int64_t k_token_stride, int64_t k_head_stride, void *v_bf16,
                                           int64_t v_token_stride, int64_t v_head_stride, int64_t tokens,
                                           void *stream);

/*
 * h3fp4_kv_attention -- attention of new queries over the cache.
 *
 * len[b] is the number of keys of sequence b, those of the new tokens
 * included; query i of its n tokens stands at position len[b] - n + i.  A
 * query sees the positions j < len[b] with
 *     j <= its own position          if causal, and
 *     j >  its own position - window if window > 0.
 * For each query and head h (which reads cache head h / (heads / cache heads)):
 *     s_j = softmax_scale * q . k_j,  out = RN_bf16(sum_j exp(s_j) v_j / sum_j exp(s_j)),
 *     lse = log(sum_j exp(s_j))
 * with sums, the softmax and its statistics in FP32.  The products take the
 * stored codes exactly; q is scaled by a power of two per row and exact in
 * FP16 but for channels below 2^-28 of the row's largest, and the weights
 * exp(s_j - max) enter the second product rounded to FP16: by 2^-11 down to
 * 2^-21 of the largest (a weight counts here times its page's value scale),
 * to a multiple of 2^-31 of it below that.  A query that sees
 * nothing gets out = 0 and lse = -infinity.  Positions that a query does not
 * see have no effect on it, whatever their codes hold, and pages of which no
 * query sees anything are not looked at, whatever the table holds for them.
 *
 *   q_bf16, out_bf16  [tokens, heads, head_dim] bf16, strides as for h3fp4_rope_axes, no overlap
 *   lse               NULL, or [tokens, heads] float, contiguous
 *   heads             a multiple of the cache's heads, at most 65535
 *   max_kv            the most keys that any sequence has (sizes the launch; longer ones are
 *                     reported as out of range); at most 2^30
 *   softmax_scale     finite; scales of the cache's pages lie in [2^-60, 2^120] (those that a write sets do).
 *                     Scores have FP32's accuracy where softmax_scale times the row's largest channel is
 *                     0 or 2^-100 at least; past FP32's range they are infinities
 *   workspace         h3fp4_kv_attention_workspace bytes of device scratch, 16-byte aligned (contents on
 *                     entry are ignored; two calls that overlap on the GPU must not share it); may be NULL
 *                     where that is 0
 */
H3FP4_API h3fp4_status h3fp4_kv_attention(const void *q_bf16, int64_t q_token_stride, int64_t q_head_stride,
                                          void *out_bf16, int64_t out_token_stride, int64_t out_head_stride,
                                          float *lse, int64_t tokens, int32_t heads, const h3fp4_kv_cache *cache,
                                          const h3fp4_kv_batch *batch, int32_t max_kv, float softmax_scale,
                                          int32_t causal, int32_t window, void *workspace, int64_t workspace_bytes,
                                          void *stream);

/* Bytes of workspace that h3fp4_kv_attention wants for these sizes (host only; -1 for sizes it refuses). */
H3FP4_API int64_t h3fp4_kv_attention_workspace(int64_t tokens, int32_t heads, int32_t kv_heads, int32_t head_dim,
                                               int32_t batch, int32_t max_tokens, int32_t max_kv);

/*
 * h3fp4_kv_attention_sinks -- h3fp4_kv_attention whose first tokens stay visible
 * under a sliding window: a query sees the positions j < len[b] with
 *     j <= its own position                            if causal, and
 *     j > its own position - window, or j < sinks      if window > 0.
 * Pages that lie wholly between the two are not looked at, whatever the table
 * holds for them, so that they may serve other sequences: a bounded number is
 * in use however long the sequence is.  Positions, and the table's row, go on
 * counting from its beginning.
 *
 *   sinks      0 .. 2^30 (0, or no window: h3fp4_kv_attention)
 *   workspace  as for h3fp4_kv_attention
 */
H3FP4_API h3fp4_status h3fp4_kv_attention_sinks(const void *q_bf16, int64_t q_token_stride, int64_t q_head_stride,
                                                void *out_bf16, int64_t out_token_stride, int64_t out_head_stride,
                                                float *lse, int64_t tokens, int32_t heads, const h3fp4_kv_cache *cache,
                                                const h3fp4_kv_batch *batch, int32_t max_kv, float softmax_scale,
                                                int32_t causal, int32_t window, int32_t sinks, void *workspace,
                                                int64_t workspace_bytes, void *stream);

/*
 * h3fp4_kv_attention_shared -- attention of sequences that share prefixes,
 * whose codes are read once for all of a group's queries.
 *
 * `prefix` holds a row of the page table for each group of sequences: len[g]
 * keys, all of which every query of tokens prefix.cu_tokens[g] ..
 * prefix.cu_tokens[g+1] - 1 sees (a group's tokens follow one another, and the
 * groups).  `batch` holds the sequences' own keys, as for h3fp4_kv_attention:
 * positions, lengths and pages count from the prefix's end, so that a prefix
 * may end inside a page.  A token's output is the softmax over its prefix and
 * what it sees of its own keys, out and lse as for h3fp4_kv_attention; tokens
 * of no group have no prefix, groups may be empty, and prefixes too.  The two
 * halves are joined from FP32 means and logarithms.  Rows outside the
 * sequences are left as they were, and so are those of a group whose length or
 * rows are out of range (or of a sequence's): reported, joined to nothing.
 *
 *   prefix      batch: the groups; max_tokens: the most tokens of a group
 *   max_prefix  the most keys of a prefix; at most 2^30
 *   workspace   h3fp4_kv_attention_shared_workspace bytes of device scratch, 16-byte aligned (contents on entry
 *               are ignored; two calls that overlap on the GPU must not share it)
 *   other arguments as for h3fp4_kv_attention
 */
H3FP4_API h3fp4_status h3fp4_kv_attention_shared(const void *q_bf16, int64_t q_token_stride, int64_t q_head_stride,
                                                 void *out_bf16, int64_t out_token_stride, int64_t out_head_stride,
                                                 float *lse, int64_t tokens, int32_t heads, const h3fp4_kv_cache *cache,
                                                 const h3fp4_kv_batch *prefix, int32_t max_prefix,
                                                 const h3fp4_kv_batch *batch, int32_t max_kv, float softmax_scale,
                                                 int32_t causal, void *workspace, int64_t workspace_bytes, void *stream);

/* Bytes of workspace that h3fp4_kv_attention_shared wants for these sizes (host only; -1 for sizes it refuses). */
H3FP4_API int64_t h3fp4_kv_attention_shared_workspace(int64_t tokens, int32_t heads, int32_t kv_heads, int32_t head_dim,
                                                      int32_t groups, int32_t max_group_tokens, int32_t max_prefix,
                                                      int32_t batch, int32_t max_tokens, int32_t max_kv);

/*
 * h3fp4_kv_tables -- what the cache and attention calls want to know of a
 * batch, from its requests' lengths, without the host: offsets and lengths,
 * pages for the new tokens from a list of free ones, and each token's place.
 *
 * Sequence b holds held[b] tokens and gets count[b] new ones.  In the order of
 * the sequences:
 *     cu_tokens[b + 1] = count[0] + ... + count[b],   kv_len[b] = held[b] + count[b],
 *     page_table[b, p] = the next of free_pages, for ceil(held[b] / page_size) <= p < ceil(kv_len[b] / page_size),
 * the first taken being free_pages[*free_at] and *free_at_out = *free_at + those
 * taken.  (The list is read forwards only: pages that are given up come back
 * by a new list, or a new place in one.)
 * New token i of sequence b, at position held[b] + i, is row
 * cu_tokens[b] + i of
 *     slots     page_table[b, position / page_size] * page_size + position % page_size
 *     positions the position (float, as h3fp4_rope takes them)
 * and rows past the last token hold -1 in both.  Other entries of the table
 * stay as they were.  (cu_tokens, kv_len) are an h3fp4_kv_batch's cu_tokens
 * and len for attention, (cu_tokens, held) for h3fp4_kv_cache_write.
 *
 * Reported as bit 512 of h3fp4_device_error: a sequence whose held or count is
 * negative, whose count is more than max_tokens or whose pages are more than
 * ld_table (it gets nothing: no tokens, kv_len 0); a free list that runs out
 * or whose place is negative (what lies outside it counts as taken up to its
 * end, so that no page is taken twice), or a page number outside [0, num_pages) in it or in the entry of a page that
 * the sequence has begun (the table gets -1 for it, unless it was there; the
 * tokens' slots are -1); more tokens than the rows of slots (those are not
 * written; cu_tokens stops at 2^31 - 1).
 *
 *   held, count   device [batch]
 *   page_table    device [batch, ld_table], read and written
 *   free_pages    device [num_free]; free_at, free_at_out: one each, not the same (a call never changes what it reads,
 *                 but for the table's entries past the tokens held)
 *   cu_tokens     device [batch + 1]; kv_len device [batch]; slots device int64 [tokens]; positions device [tokens];
 *                 slots and positions may be NULL.  No output overlaps an input or another output
 *   batch         0 .. 65535; max_tokens 0 .. 1,000,000; tokens 0 .. 2^31 - 1; page_size 16, 32, 64 or 128
 */
typedef struct h3fp4_kv_requests {
    const int32_t *held, *count;
    int32_t *page_table;
    int64_t ld_table;
    const int32_t *free_pages;
    const int32_t *free_at;
    int32_t *free_at_out;
    int32_t *cu_tokens, *kv_len;
    int64_t *slots;
    float *positions;
    int64_t tokens;             /* rows of slots and positions */
    int32_t batch, max_tokens, num_free, num_pages, page_size;
} h3fp4_kv_requests;

H3FP4_API h3fp4_status h3fp4_kv_tables(const h3fp4_kv_requests *requests, void *stream);

/*
 * h3fp4_swizzle_scales -- helper for preparing weights: copies a LOGICAL
 * row-major E4M3 scale matrix [rows, cols] (leading dimension ld bytes) into
 * the scale layout above, padding rows up to a multiple of 128 with zeros.
 * Not part of the hot path (weights are prepared once).
 *
 *   cols multiple of 4; out holds ceil(rows/128)*128 * cols bytes, 16-byte aligned
 */
H3FP4_API h3fp4_status h3fp4_swizzle_scales(const uint8_t *sf_logical, int64_t rows, int64_t cols,
                                  int64_t ld, uint8_t *sf_out, void *stream);

/*
 * h3fp4_swiglu_pack_noalloc -- h3fp4_swiglu_pack for callers that cannot
 * allocate device memory.  No counterpart on the source pages.
 *
 * Some callers have no device allocator at hand when they call in (a plugin
 * running inside another framework's operator, a serving loop that must not
 * allocate after warm-up), so they cannot pass the scratch words or the h
 * workspace.  This entry point computes exactly what h3fp4_swiglu_pack
 * computes (same tensor scale, QDATA and SFA bytes) with its scratch in a
 * static device array owned by the library: 256 bytes of counters plus room
 * for H3FP4_NOALLOC_MAX_ELEMENTS bf16 values of h (8 MiB in all), held by
 * every GPU that loads the library until the process exits.  It calls no
 * cudaMalloc, cudaFree or allocating library routine.
 *
 *   Arguments as for h3fp4_swiglu_pack, without scratch and h_workspace.
 *   m * f must not exceed H3FP4_NOALLOC_MAX_ELEMENTS (else H3FP4_ERR_SHAPE,
 *   nothing enqueued).
 *
 * The first call on a device looks up the array's device address (with that
 * device current) and may load the library's device code; make that first
 * call before any stream capture.  The address is kept for the life of the
 * process's context on that device: after cudaDeviceReset, do not call this
 * entry point again in that process.  All calls share the array and it keeps the
 * last call's contents (each call clears its counters and rewrites h before
 * reading it); calls whose GPU work overlaps race on it and must be
 * serialised by the caller.
 */
#define H3FP4_NOALLOC_MAX_ELEMENTS (1 << 22)
H3FP4_API h3fp4_status h3fp4_swiglu_pack_noalloc(const void *gate_bf16, int64_t ldg, const void *up_bf16,
                                                 int64_t ldu, int64_t m, int64_t m_pad, int64_t f,
                                                 float *tensor_scale, uint8_t *qdata, uint8_t *sfa,
                                                 void *stream);

/*
 * h3fp4_device_error -- reads and clears the device-side error word of the
 * current device (synchronous).  Kernels whose pipeline waits give up after
 * their time limit (2 s) record a nonzero code there instead of hanging, and
 * return.  Bits: GEMM waits 1 (a free stage), 2 (operands landed), 4 (a
 * finished accumulator), 8 (a drained accumulator), 16 (scale atoms landed);
 * 256 the cooperative producer's grid barrier; 512 an entry of a page table
 * or length array out of range, 1,024 a pipeline wait (attention calls).
 * Returns H3FP4_OK and stores the word in *code (0 = no error).
 */
H3FP4_API h3fp4_status h3fp4_device_error(uint32_t *code);

/*
 * Failure detection -- diagnostics, not part of the hot path.  No counterpart
 * on the source pages beyond the bounded waits themselves ("NVFP4 Streaming
 * Design", P2: a cooperative producer around a grid barrier with a bounded
 * wait).  Each call runs one of the library's kernels with a wait that cannot
 * be satisfied and a limit of limit_us microseconds (1 .. 2,000,000, else
 * H3FP4_ERR_SHAPE), so that a caller can check that a wait which runs out
 * ends the kernel with an error code instead of a hang, and that the device
 * stays usable afterwards.
 *
 * h3fp4_diag_producer_barrier_timeout -- the cooperative plain producer
 * (h3fp4_quantize_pack's kernel, same arguments and checks) with its grid
 * barrier's arrival target one above the grid size: every CTA gives up after
 * limit_us, records bit 256 and returns.  tensor_scale, qdata and sfa are not
 * written; pass 1 reads x.
 *
 * h3fp4_diag_gemm_wait_timeout -- the default GEMM kernel (same arguments
 * and checks as h3fp4_gemm, default configuration) with its operand loads
 * withheld: the scale-copy, MMA and epilogue warps' waits run out after
 * limit_us and record bits 16, 2 and 4.  c_bf16 is not written and no
 * operand is read.
 *
 * h3fp4_diag_attention_wait_timeout -- the attention kernel of few queries
 * (arguments and checks of h3fp4_kv_attention, every key seen, a scale of 1;
 * 128 channels, at most 8 query rows a cache head, else H3FP4_ERR_UNSUPPORTED)
 * with its copies of the codes announced larger than they are: the first wait
 * of each warp runs out after limit_us, as do those for the copies still on
 * their way, and the call ends after about three times limit_us with bit 1,024,
 * however many keys there are.  out_bf16 and lse are not written.
 */
H3FP4_API h3fp4_status h3fp4_diag_producer_barrier_timeout(const void *x_bf16, int64_t ldx, int64_t m,
                                                           int64_t m_pad, int64_t d, float *tensor_scale,
                                                           uint32_t *scratch, uint8_t *qdata, uint8_t *sfa,
                                                           uint32_t limit_us, void *stream);
H3FP4_API h3fp4_status h3fp4_diag_gemm_wait_timeout(const uint8_t *a_q, const uint8_t *a_sf,
                                                    const float *a_tensor_scale, const uint8_t *b_q,
                                                    const uint8_t *b_sf, const float *b_tensor_scale, void *c_bf16,
                                                    int64_t ldc, int64_t m, int64_t m_pad, int64_t n, int64_t k,
                                                    uint32_t limit_us, void *stream);
H3FP4_API h3fp4_status h3fp4_diag_attention_wait_timeout(const void *q_bf16, int64_t q_token_stride,
                                                         int64_t q_head_stride, void *out_bf16,
                                                         int64_t out_token_stride, int64_t out_head_stride, float *lse,
                                                         int64_t tokens, int32_t heads, const h3fp4_kv_cache *cache,
                                                         const h3fp4_kv_batch *batch, int32_t max_kv, void *workspace,
                                                         int64_t workspace_bytes, uint32_t limit_us, void *stream);

/* Human-readable name of a status code (static string). */
H3FP4_API const char *h3fp4_status_string(h3fp4_status status);

/* Build description: version, target architecture, compiler. (static string) */
H3FP4_API const char *h3fp4_build_info(void);

#ifdef __cplusplus
}
#endif

#endif /* H3FP4_H */

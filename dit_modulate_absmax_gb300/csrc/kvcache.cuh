// kvcache.cuh -- the 8-bit key/value cache as the kernels see it: page
// lookup with range checks, and conversions between E4M3 and wider formats.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "launch.h"

namespace h3fp4 {

constexpr uint32_t ERR_KV_RANGE = 1u << 9;   // an entry of a page table or length array out of range

// Rows and lengths of one sequence of a call.
struct KvSequence {
    int64_t row;    // first row in the packed token arrays
    int n;          // its tokens in this call
    int len;        // len[b] (0 without a length array)
    bool ok;        // rows and counts in range (without tokens in this call nothing of it is looked at)
};

__device__ __forceinline__ KvSequence kv_sequence(const KvBatch &bt, int b, int64_t tokens)
{
    KvSequence s;
    s.row = bt.cu_tokens[b];
    s.n = bt.cu_tokens[b + 1] - bt.cu_tokens[b];
    s.len = bt.len != nullptr ? bt.len[b] : 0;
    s.ok = s.n == 0 || (s.row >= 0 && s.n > 0 && s.n <= bt.max_tokens && s.row + s.n <= tokens && s.len >= 0);
    return s;
}

// The two E4M3 codes in the low 16 bits as halves (exact; 0x7F and 0xFF give NaN).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t c)
{
    uint32_t r;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(r) : "r"(c));
    return r;
}

// Four codes as two pairs of halves.
__device__ __forceinline__ uint2 e4m3x4_to_f16x4(uint32_t c)
{
    uint2 r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
        : "=r"(r.x), "=r"(r.y)
        : "r"(c));
    return r;
}

__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t c)
{
    const uint32_t h = e4m3x2_to_f16x2(c);
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// Codes of lo (bits 0-7) and hi (bits 8-15): nearest even, saturating, NaN -> 0x7F.
__device__ __forceinline__ uint32_t floats_to_e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

}  // namespace h3fp4

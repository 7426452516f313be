// norm_rope.cuh -- arguments of the per-head norms with rotation, by value.
#pragma once

#include "launch.h"

namespace h3fp4 {

// Queries or keys: [tokens, heads, dim] with strides of tokens and heads.
struct NormSide {
    const uint16_t *x;
    int64_t xt, xh;
    uint16_t *out;
    int64_t ot, oh;
    const void *weight;   // [dim], nullptr: ones
    int32_t heads, wide;  // wide: the weight is FP32, else bf16
};

struct NormGradSide {
    const uint16_t *dy;
    int64_t gt, gh;
    const uint16_t *x;
    int64_t xt, xh;
    uint16_t *dx;
    int64_t ot, oh;
    const void *weight;
    float *dweight;       // [dim], nullptr: not wanted
    int32_t heads, wide;
};

cudaError_t launch_norm_rope(const NormSide &q, const NormSide &k, int64_t tokens, int dim, float eps, const RopeArgs &r, cudaStream_t st);
int64_t norm_grad_workspace(int dim);
cudaError_t launch_norm_rope_grad(const NormGradSide &q, const NormGradSide &k, int64_t tokens, int dim, float eps, const RopeArgs &r,
                                  void *workspace, cudaStream_t st);

}  // namespace h3fp4

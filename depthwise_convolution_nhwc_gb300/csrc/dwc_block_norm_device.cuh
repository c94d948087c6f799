// dwc_block_norm_device.cuh -- what the block norm's kernels share.
#pragma once

#include "dwc_norm_device.cuh"

namespace dwc {

// act(v) and, where asked for, its derivative (act: 0 none, 1 sigmoid, 2 silu).
__device__ __forceinline__ float gate_of(float v, int act, float* slope = nullptr) {
    if (act == 0) {
        if (slope != nullptr) *slope = 1.f;
        return v;
    }
    if (slope == nullptr) return act == 1 ? sigmoid(v) : silu(v);
    const float s = sigmoid(v);
    *slope = act == 1 ? s * (1.f - s) : silu_slope(v, s);
    return act == 1 ? s : v * s;
}

// The same of 8 values in pairs, one branch for all.
__device__ __forceinline__ void gate8(float2 (&v)[4], int act) {
    if (act == 0) return;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 s = sigmoid2(v[j]);
        v[j] = act == 1 ? s : __fmul2_rn(v[j], s);
    }
}
__device__ __forceinline__ void gate8(float2 (&v)[4], float2 (&slope)[4], int act) {
    if (act == 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) slope[j] = both(1.f);
    } else if (act == 1) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = sigmoid2(v[j]);
            slope[j] = __fmul2_rn(v[j], make_float2(1.f - v[j].x, 1.f - v[j].y));
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 s = sigmoid2(v[j]);
            v[j] = __fmul2_rn(v[j], s);
            slope[j] = __fadd2_rn(s, __ffma2_rn(v[j], make_float2(-s.x, -s.y), v[j]));
        }
    }
}

// Gradients of the parameters from `count` partial rows [sum t xhat | sum dy zhat].
cudaError_t launch_block_norm_params(const BlockNorm& p, int count);

}  // namespace dwc

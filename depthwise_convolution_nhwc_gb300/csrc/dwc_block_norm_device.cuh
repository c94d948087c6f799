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

// Gradients of the parameters from `count` partial rows [sum t xhat | sum dy zhat].
cudaError_t launch_block_norm_params(const BlockNorm& p, int count);

}  // namespace dwc

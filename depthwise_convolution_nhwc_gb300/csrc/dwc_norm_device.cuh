// dwc_norm_device.cuh -- device-side parts shared by the norm and dropout kernels.
#pragma once

#include "dwc_device.cuh"
#include "dwc_norm_host.h"

namespace dwc {

// Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3",
// SC 2011): 10 rounds of two 32 x 32 -> 64 bit products and exclusive-ors on a 128-bit counter
// with a 64-bit key.  One block serves 8 elements, 16 bits each.  The kernels it feeds are bound
// by memory and the products run at a fraction of the issue rate, so bits are what it must not
// waste: dropout of 134M bf16 values took 111 us with 32 bits a value, 88 us with 16 (a plain
// copy 86 us).  The price is that p is held to a multiple of 2^-16.
__device__ __forceinline__ uint4 philox4x32_10(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3,
                                               uint32_t k0, uint32_t k1) {
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = static_cast<uint64_t>(c0) * 0xD2511F53u;
        const uint64_t b = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
        c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ k0;
        c1 = static_cast<uint32_t>(b);
        c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ k1;
        c3 = static_cast<uint32_t>(a);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(c0, c1, c2, c3);
}

// Dropout as a kernel holds it: the counter's high words are the call's offset plus the step
// that the caller may keep on the device.
struct DropState {
    uint32_t threshold, k0, k1, o0, o1;
    float scale;
    __device__ __forceinline__ void init(const Dropout& d) {
        threshold = d.threshold;
        k0 = d.k0;
        k1 = d.k1;
        scale = d.scale;
        const uint64_t o = d.offset + (d.step != nullptr && d.threshold != 0 ? *d.step : 0ull);
        o0 = static_cast<uint32_t>(o);
        o1 = static_cast<uint32_t>(o >> 32);
    }
    // the 8 draws of elements 8 * block .. 8 * block + 7, two to a word
    __device__ __forceinline__ uint4 draw(uint64_t block) const {
        return philox4x32_10(static_cast<uint32_t>(block), static_cast<uint32_t>(block >> 32), o0, o1, k0, k1);
    }
    // one value; the comparison selects, so a dropped infinity or NaN gives 0
    __device__ __forceinline__ float apply(float v, uint32_t h) const { return h >= threshold ? v * scale : 0.f; }
    __device__ __forceinline__ float one(float v, uint64_t i) const {
        const uint4 b = draw(i >> 3);
        const uint32_t j = static_cast<uint32_t>(i) & 7u;
        const uint32_t w = j < 4 ? (j < 2 ? b.x : b.y) : (j < 6 ? b.z : b.w);
        return apply(v, (j & 1u) ? w >> 16 : w & 0xffffu);
    }
};

// A parameter (gamma, beta) of any of the three types; null stands for `absent`.
__device__ __forceinline__ float load_param(const void* p, int type, int c, float absent) {
    if (p == nullptr) return absent;
    if (type == kF32) return static_cast<const float*>(p)[c];
    if (type == kBF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[c]);
    return __half2float(static_cast<const __half*>(p)[c]);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}

}  // namespace dwc

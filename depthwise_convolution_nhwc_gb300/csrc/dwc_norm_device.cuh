// dwc_norm_device.cuh -- device-side parts shared by the norm and dropout kernels.
#pragma once

#include <type_traits>

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
    uint32_t threshold, below, k0, k1, o0, o1;
    float scale;
    __device__ __forceinline__ void init(const Dropout& d) {
        threshold = d.threshold;
        below = (d.threshold << 16) - 1u;   // (65536 gives 2^32 - 1: nothing lies above it)
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
    // one value and its draw in the high half of `h` (h >> 16 >= threshold, threshold > 0); the
    // comparison selects, so a dropped infinity or NaN gives 0
    __device__ __forceinline__ float apply(float v, uint32_t h) const { return h > below ? v * scale : 0.f; }
    __device__ __forceinline__ float one(float v, uint64_t i) const {
        const uint4 b = draw(i >> 3);
        const uint32_t j = static_cast<uint32_t>(i) & 7u;
        const uint32_t w = j < 4 ? (j < 2 ? b.x : b.y) : (j < 6 ? b.z : b.w);
        return apply(v, (j & 1u) ? w : w << 16);
    }
};

// A parameter (gamma, beta) of any of the three types; null stands for `absent`.
__device__ __forceinline__ float load_param(const void* p, int type, int c, float absent) {
    if (p == nullptr) return absent;
    if (type == kF32) return static_cast<const float*>(p)[c];
    if (type == kBF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[c]);
    return __half2float(static_cast<const __half*>(p)[c]);
}

// 2^v and 1 / v by the approximations of one instruction (2 ulp, 1 ulp), and through them 1 / (1 + exp(-v)) and v / (1 +
// exp(-v)).  The argument's scaling by log2(e) costs a relative error of 2^-23 |v| of the exponential, which counts
// only where the exponential does; the full-range expf and division in their place made gates as dear as
// everything else of a memory-bound kernel.
__device__ __forceinline__ float exp2_fast(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float rcp_fast(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float sigmoid(float v) { return rcp_fast(1.f + exp2_fast(v * -kLog2e)); }
__device__ __forceinline__ float silu(float v) { return v * sigmoid(v); }
// d silu / d v, from sigmoid(v)
__device__ __forceinline__ float silu_slope(float v, float s) { return fmaf(v * s, 1.f - s, s); }
// two of each
__device__ __forceinline__ float2 sigmoid2(float2 v) {
    const float2 t = __fmul2_rn(v, make_float2(-kLog2e, -kLog2e));
    const float2 w = __fadd2_rn(make_float2(exp2_fast(t.x), exp2_fast(t.y)), make_float2(1.f, 1.f));
    return make_float2(rcp_fast(w.x), rcp_fast(w.y));
}
__device__ __forceinline__ float2 silu2(float2 v) { return __fmul2_rn(v, sigmoid2(v)); }
__device__ __forceinline__ float2 silu_slope2(float2 v) {
    const float2 s = sigmoid2(v), vs = __fmul2_rn(v, s);
    return __fadd2_rn(s, __ffma2_rn(vs, make_float2(-s.x, -s.y), vs));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}

// ---- vectors of 8 elements ---------------------------------------------------------------
// 16 bytes of a 16-bit type, 32 bytes of fp32 (one 256-bit access, new with sm_100; two 16-byte
// ones would each touch half of every sector).  In registers: four fp32 pairs, for the packed
// fp32x2 arithmetic.
template <typename T>
struct Vec8 {  // 16-bit types
    uint4 u;
    __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(const T* p) { u = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void set(int j, T v) { reinterpret_cast<T*>(&u)[j] = v; }
    __device__ __forceinline__ void widen(float2 (&f)[4]) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (std::is_same<T, __nv_bfloat16>::value)
                f[k] = make_float2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
            else
                f[k] = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
        }
    }
    __device__ static __forceinline__ void store(T* p, const float2 (&f)[4]) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                const __nv_bfloat162 h = __float22bfloat162_rn(f[k]);
                w[k] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
                const __half2 h = __float22half2_rn(f[k]);
                w[k] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

template <>
struct Vec8<float> {
    float v[8];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.f;
    }
    __device__ __forceinline__ void load(const float* p) {
        asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                     : "l"(p)
                     : "memory");
    }
    __device__ __forceinline__ void set(int j, float x) { v[j] = x; }
    __device__ __forceinline__ void widen(float2 (&f)[4]) const {
#pragma unroll
        for (int k = 0; k < 4; ++k) f[k] = make_float2(v[2 * k], v[2 * k + 1]);
    }
    __device__ static __forceinline__ void store(float* p, const float2 (&f)[4]) {
        asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(f[0].x), "f"(f[0].y),
                     "f"(f[1].x), "f"(f[1].y), "f"(f[2].x), "f"(f[2].y), "f"(f[3].x), "f"(f[3].y)
                     : "memory");
    }
};

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Whether elements col .. col + 7 all belong to a row of C; where a row does not start at a
// vector boundary its first and last vector hang over (col may be negative).
__device__ __forceinline__ bool inside(int col, int C) { return col >= 0 && col + 8 <= C; }
__device__ __forceinline__ bool in_row(int c, int C) { return static_cast<unsigned>(c) < static_cast<unsigned>(C); }

// Elements beside the row are set to 0.
__device__ __forceinline__ void mask8(float2 (&f)[4], int col, int C) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (!in_row(col + 2 * k, C)) f[k].x = 0.f;
        if (!in_row(col + 2 * k + 1, C)) f[k].y = 0.f;
    }
}

// Store of a vector: only the row's own elements.  `whole`: the warp has no vector that hangs over.
template <typename T>
__device__ __forceinline__ void store_row8(T* row, const float2 (&f)[4], int col, int C, bool whole) {
    if (whole || inside(col, C)) {
        Vec8<T>::store(row + col, f);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (in_row(col + 2 * k, C)) store_out(row + col + 2 * k, f[k].x);
            if (in_row(col + 2 * k + 1, C)) store_out(row + col + 2 * k + 1, f[k].y);
        }
    }
}

// The dropout of 8 consecutive elements whose first index is 8 * block.
__device__ __forceinline__ void drop8(const DropState& d, float2 (&f)[4], uint64_t block) {
    const uint4 b = d.draw(block);
    const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        f[k].x = d.apply(f[k].x, w[k] << 16);
        f[k].y = d.apply(f[k].y, w[k]);
    }
}

}  // namespace dwc

// dwc_dropout.cu -- dropout of dense tensors and of rows with an aligned stride, 8 elements per access.
//
// y = keep ? x * scale : 0, the mask drawn in registers (one Philox block per 8 elements, see
// dwc_norm_device.cuh).  Bound by memory: x is read once and y written once; the generator's 20
// wide products per block run beside the copies.  Each thread takes kVecs vectors, a CTA's width
// apart, whose loads are in flight together.
#include <algorithm>

#include "dwc_norm_device.cuh"

namespace dwc {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 4;

// kStrided: rows of `row_vecs` vectors, ld elements apart in x (dense in y); the vector's place costs a
// division, which the copies nearly hide: bf16 8192 x 8192 of 16384 channels takes 54 us, dense 50 us, and
// the general kernel, one element at a time, 300 us on the strided rows (each with a flushed L2).
template <typename T, bool kStrided>
__global__ void __launch_bounds__(kThreads) dropout_vec_kernel(const T* x, T* y, long long n, long long ld, int row_vecs,
                                                               Dropout d) {
    pdl_trigger();
    pdl_wait();
    DropState drop;
    drop.init(d);
    const long long vecs = n / 8;
    const long long first = static_cast<long long>(blockIdx.x) * (kThreads * kVecs) + threadIdx.x;
    Vec8<T> raw[kVecs];
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
        const long long i = first + k * kThreads;
        raw[k].zero();
        if (i >= vecs) continue;
        if constexpr (kStrided) {
            const long long r = i / row_vecs;
            raw[k].load(x + r * ld + 8 * (i - r * row_vecs));
        } else {
            raw[k].load(x + 8 * i);
        }
    }
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
        const long long i = first + k * kThreads;
        if (i >= vecs) break;
        float2 f[4];
        raw[k].widen(f);
        if (drop.threshold != 0) drop8(drop, f, static_cast<uint64_t>(i));
        Vec8<T>::store(y + 8 * i, f);
    }
    // the last n % 8 elements
    if (!kStrided && blockIdx.x == 0 && threadIdx.x < n - 8 * vecs) {
        const long long i = 8 * vecs + threadIdx.x;
        const float v = to_f32(x[i]);
        store_out(y + i, drop.threshold != 0 ? drop.one(v, i) : v);
    }
}

template <typename T>
cudaError_t dropout_t(const DropoutCall& p) {
    const long long n = p.rows * p.C;
    const long long grid = std::max(1LL, (n / 8 + kThreads * kVecs - 1) / (kThreads * kVecs));
    if (grid > 0x7fffffffLL) return cudaErrorNotSupported;
    const bool strided = p.ld_x != p.C && p.rows > 1;
    if (strided && p.C % 8 != 0) return cudaErrorNotSupported;
    return launch_pdl(strided ? dropout_vec_kernel<T, true> : dropout_vec_kernel<T, false>,
                      dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, p.stream, static_cast<const T*>(p.x),
                      static_cast<T*>(p.y), n, p.ld_x, std::max(1, p.C / 8), p.drop);
}

}  // namespace

cudaError_t launch_dropout_vec(const DropoutCall& p) {
    switch (p.type) {
        case kF32: return dropout_t<float>(p);
        case kBF16: return dropout_t<__nv_bfloat16>(p);
        default: return dropout_t<__half>(p);
    }
}

}  // namespace dwc

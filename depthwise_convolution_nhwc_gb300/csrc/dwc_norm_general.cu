// dwc_norm_general.cu -- layer norm, its residual form and dropout for any row stride,
// alignment and channel count: one CTA per row, one element per thread at a time.
#include <algorithm>

#include "dwc_norm_device.cuh"

namespace dwc {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Sums of two values over the CTA, for every thread.  `red` holds one pair a warp; the first barrier keeps
// a call's pairs from being written while an earlier call's are still read.
__device__ __forceinline__ float2 cta_sum(float2 v, float2* red) {
    v.x = warp_sum(v.x);
    v.y = warp_sum(v.y);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        s.x += red[w].x;
        s.y += red[w].y;
    }
    return s;
}

// One row per CTA.  The fp32 row is kept in shared memory where it fits (`staged`; each thread
// reads back only what it wrote) and formed again from the inputs in each of the three passes
// where it does not.  Mean first, then the squares of the differences: no cancellation.
template <typename TS, typename TB, bool kAdd>
__global__ void __launch_bounds__(kThreads) norm_fwd_general_kernel(NormFwd p, int staged) {
    extern __shared__ float row_buf[];
    __shared__ float2 red[kWarps];
    pdl_trigger();
    pdl_wait();
    DropState drop;
    if (kAdd) drop.init(p.drop);
    const int C = p.C;
    const float inv = 1.f / static_cast<float>(C);
    for (long long r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const TS* in = static_cast<const TS*>(p.in) + r * p.ld_in;
        const TB* x = static_cast<const TB*>(p.x) + r * p.ld_x;
        const uint64_t first = static_cast<uint64_t>(r) * C;
        auto value = [&](int c) {
            float v = to_f32(in[c]);
            if (kAdd) {
                const float b = to_f32(x[c]);
                v += drop.threshold != 0 ? drop.one(b, first + c) : b;
            }
            return v;
        };
        float2 s = make_float2(0.f, 0.f);
        for (int c = threadIdx.x; c < C; c += kThreads) {
            const float v = value(c);
            if (staged) row_buf[c] = v;
            s.x += v;
        }
        const float mean = cta_sum(s, red).x * inv;
        s.x = 0.f;
        for (int c = threadIdx.x; c < C; c += kThreads) {
            const float d = (staged ? row_buf[c] : value(c)) - mean;
            s.x = fmaf(d, d, s.x);
        }
        const float rstd = 1.f / sqrtf(cta_sum(s, red).x * inv + p.eps);
        TB* y = static_cast<TB*>(p.y) + first;
        TS* z = static_cast<TS*>(p.z) + first;
        for (int c = threadIdx.x; c < C; c += kThreads) {
            const float v = staged ? row_buf[c] : value(c);
            // (z may be the stream itself: this thread has read the element for the last time)
            if (kAdd) store_out(z + c, v);
            store_out(y + c, fmaf((v - mean) * rstd, load_param(p.gamma, p.param_type, c, 1.f),
                                  load_param(p.beta, p.param_type, c, 0.f)));
        }
        if (threadIdx.x == 0) {
            if (p.mean != nullptr) p.mean[r] = mean;
            if (p.rstd != nullptr) p.rstd[r] = rstd;
        }
    }
}

// One row per CTA at a time, two passes over dy and z (the second from L1 or L2).  Every CTA adds
// the parameter gradients of its rows into its own row of partial sums; a column belongs to one
// thread, so the additions have a fixed order.
template <typename TS, typename TB>
__global__ void __launch_bounds__(kThreads) norm_bwd_general_kernel(NormBwd p) {
    __shared__ float2 red[kWarps];
    pdl_trigger();
    pdl_wait();
    DropState drop;
    drop.init(p.drop);
    const int C = p.C;
    const float inv = 1.f / static_cast<float>(C);
    float* part = p.partial == nullptr ? nullptr : p.partial + static_cast<size_t>(blockIdx.x) * 2 * C;
    bool first_row = true;
    for (long long r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const TB* dy = static_cast<const TB*>(p.dy) + r * p.ld_dy;
        const TS* z = static_cast<const TS*>(p.z) + r * p.ld_z;
        const TS* dz = p.dz == nullptr ? nullptr : static_cast<const TS*>(p.dz) + r * p.ld_dz;
        const uint64_t first = static_cast<uint64_t>(r) * C;
        const float mean = p.mean[r], rstd = p.rstd[r];
        float2 s = make_float2(0.f, 0.f);
        for (int c = threadIdx.x; c < C; c += kThreads) {
            const float g = to_f32(dy[c]);
            const float a = g * load_param(p.gamma, p.param_type, c, 1.f);
            const float xhat = (to_f32(z[c]) - mean) * rstd;
            s.x += a;
            s.y = fmaf(a, xhat, s.y);
            if (part != nullptr) {
                const float t = g * xhat;
                part[c] = first_row ? t : part[c] + t;
                part[C + c] = first_row ? g : part[C + c] + g;
            }
        }
        s = cta_sum(s, red);
        const float c1 = s.x * inv, c2 = s.y * inv;
        TS* ds = static_cast<TS*>(p.d_stream) + first;
        TB* db = p.d_branch == nullptr ? nullptr : static_cast<TB*>(p.d_branch) + first;
        for (int c = threadIdx.x; c < C; c += kThreads) {
            const float a = to_f32(dy[c]) * load_param(p.gamma, p.param_type, c, 1.f);
            const float xhat = (to_f32(z[c]) - mean) * rstd;
            float g = rstd * (a - c1 - xhat * c2);
            if (dz != nullptr) g += to_f32(dz[c]);
            store_out(ds + c, g);
            if (db != nullptr) store_out(db + c, drop.threshold != 0 ? drop.one(g, first + c) : g);
        }
        first_row = false;
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) dropout_general_kernel(DropoutCall p) {
    pdl_trigger();
    pdl_wait();
    DropState drop;
    drop.init(p.drop);
    const long long n = p.rows * p.C;
    const long long step = static_cast<long long>(gridDim.x) * kThreads;
    for (long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; i < n; i += step) {
        const long long r = i / p.C;
        const float v = to_f32(static_cast<const T*>(p.x)[r * p.ld_x + (i - r * p.C)]);
        store_out(static_cast<T*>(p.y) + i, drop.threshold != 0 ? drop.one(v, i) : v);
    }
}

// Column sums of the partial rows: a CTA takes kWidth columns, each thread every (1024 / kWidth)-th row of
// one, 8 loads in flight, and a warp adds the threads' sums of a column.  A fixed order, whatever the
// timing.  The kernel is bound by the latency of its loads: 8 columns (a sector) to a CTA where there
// are few of them (bf16 200704 x 128 backward 29.1 us, 30.3 with 32), 32 where that would be more CTAs than two to an SM.
// (`part` is not __restrict__: that would promise data unchanged for as long as the kernel runs, and the
// row kernel may still write it when this one starts.)
constexpr int kSumThreads = 1024;

template <int kWidth>
__global__ void __launch_bounds__(kSumThreads) norm_param_sum_kernel(const float* part, int count, int C,
                                                                     float* dgamma, float* dbeta) {
    constexpr int kSlots = kSumThreads / kWidth;
    __shared__ float sums[kSlots][kWidth + 1];
    pdl_trigger();
    const int col = threadIdx.x % kWidth, slot = threadIdx.x / kWidth;
    const long long j = static_cast<long long>(blockIdx.x) * kWidth + col;
    const size_t step = static_cast<size_t>(2) * C;
    float s = 0.f;
    pdl_wait();
    if (j < 2LL * C) {
        const float* from = part + j;
        for (int k = slot; k < count; k += 8 * kSlots) {
            float t[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) t[i] = k + kSlots * i < count ? from[(k + kSlots * i) * step] : 0.f;
            s += ((t[0] + t[1]) + (t[2] + t[3])) + ((t[4] + t[5]) + (t[6] + t[7]));
        }
    }
    sums[slot][col] = s;
    __syncthreads();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (warp >= kWidth) return;
    s = 0.f;
#pragma unroll
    for (int i = lane; i < kSlots; i += 32) s += sums[i][warp];
    s = warp_sum(s);
    const long long o = static_cast<long long>(blockIdx.x) * kWidth + warp;
    if (lane != 0 || o >= 2LL * C) return;
    float* out = o < C ? dgamma : dbeta;
    if (out != nullptr) out[o < C ? o : o - C] = s;
}

template <int kWidth>
cudaError_t param_sum(const float* partial, int count, int C, float* dgamma, float* dbeta, cudaStream_t stream) {
    const unsigned blocks = static_cast<unsigned>((2LL * C + kWidth - 1) / kWidth);
    return launch_pdl(norm_param_sum_kernel<kWidth>, dim3(blocks), dim3(kSumThreads), 0, stream, partial, count, C, dgamma,
                      dbeta);
}

template <typename TS, typename TB, bool kAdd>
cudaError_t fwd_t(const NormFwd& p) {
    static DeviceOnce once;
    const int staged = static_cast<size_t>(p.C) * sizeof(float) <= 96 * 1024;
    const size_t smem = staged ? static_cast<size_t>(p.C) * sizeof(float) : 0;
    const cudaError_t err = opt_in_smem(norm_fwd_general_kernel<TS, TB, kAdd>, once, 96 * 1024);
    if (err != cudaSuccess) return err;
    const long long cap = static_cast<long long>(device_info().sm_count) * 64;
    return launch_pdl(norm_fwd_general_kernel<TS, TB, kAdd>, dim3(static_cast<unsigned>(std::min(p.rows, cap))),
                      dim3(kThreads), smem, p.stream, p, staged);
}

template <typename TS, typename TB>
cudaError_t fwd_s(const NormFwd& p) {
    return p.x != nullptr ? fwd_t<TS, TB, true>(p) : fwd_t<TS, TB, false>(p);
}

template <typename TS, typename TB>
cudaError_t bwd_t(const NormBwd& p) {
    const int parts = norm_bwd_partials(p.rows, p.C);
    const cudaError_t err = launch_pdl(norm_bwd_general_kernel<TS, TB>, dim3(static_cast<unsigned>(parts)),
                                       dim3(kThreads), 0, p.stream, p);
    if (err != cudaSuccess || p.partial == nullptr) return err;
    return launch_norm_param_sum(p.partial, parts, p.C, p.dgamma, p.dbeta, p.stream);
}

template <typename T>
cudaError_t dropout_t(const DropoutCall& p) {
    const long long cap = static_cast<long long>(device_info().sm_count) * 64;
    const long long want = (p.rows * p.C + kThreads - 1) / kThreads;
    return launch_pdl(dropout_general_kernel<T>, dim3(static_cast<unsigned>(std::min(want, cap))), dim3(kThreads), 0,
                      p.stream, p);
}

}  // namespace

// Partial rows: four CTAs per SM for short rows, two for long ones, and at most 2^25 columns in
// all (256 MB) for very wide rows.
int norm_bwd_partials(long long rows, int C) {
    const long long by_size = std::max<long long>(1, (1LL << 25) / C);
    return static_cast<int>(std::min({rows, (C <= 1024 ? 4LL : 2LL) * device_info().sm_count, by_size}));
}

#define DWC_BY_PAIR(fn, p)                                                                        \
    if ((p).stream_type == kF32 && (p).branch_type == kF32) return fn<float, float>(p);           \
    if ((p).stream_type == kF32 && (p).branch_type == kBF16) return fn<float, __nv_bfloat16>(p);  \
    if ((p).stream_type == kF32 && (p).branch_type == kF16) return fn<float, __half>(p);          \
    if ((p).stream_type == kBF16) return fn<__nv_bfloat16, __nv_bfloat16>(p);                     \
    return fn<__half, __half>(p);

cudaError_t launch_norm_fwd_general(const NormFwd& p) { DWC_BY_PAIR(fwd_s, p) }
cudaError_t launch_norm_bwd_general(const NormBwd& p) { DWC_BY_PAIR(bwd_t, p) }

cudaError_t launch_dropout_general(const DropoutCall& p) {
    switch (p.type) {
        case kF32: return dropout_t<float>(p);
        case kBF16: return dropout_t<__nv_bfloat16>(p);
        default: return dropout_t<__half>(p);
    }
}

cudaError_t launch_norm_param_sum(const float* partial, int count, int C, float* dgamma, float* dbeta,
                                  cudaStream_t stream) {
    if (2LL * C <= 8LL * 2 * device_info().sm_count) return param_sum<8>(partial, count, C, dgamma, dbeta, stream);
    return param_sum<32>(partial, count, C, dgamma, dbeta, stream);
}

}  // namespace dwc

// dwc_block_norm.cu -- the norms on either side of a residual connection with its gate and scales,
// forward and backward.
//
//     n = x rstd_post gamma_post,  z = alpha res + scale act(gate) n,  y = z rstd_pre gamma_pre
//
// General kernels: any row stride, alignment and channel count; one CTA per row, one element per
// thread at a time.
#include <algorithm>

#include "dwc_block_norm_device.cuh"

namespace dwc {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ float cta_sum(float v, float* red) {
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += red[w];
    return s;
}

template <typename TS, typename TB>
__global__ void __launch_bounds__(kThreads) block_norm_fwd_general_kernel(BlockNorm p) {
    __shared__ float red[kWarps];
    pdl_trigger();
    pdl_wait();
    const int C = p.C;
    const float inv = 1.f / static_cast<float>(C);
    for (long long r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const TB* x = static_cast<const TB*>(p.x) + r * p.ld_x;
        const TB* gate = p.gate == nullptr ? nullptr : static_cast<const TB*>(p.gate) + r * p.ld_gate;
        const TS* res = static_cast<const TS*>(p.res) + r * p.ld_res;
        TS* z = static_cast<TS*>(p.z) + r * C;
        TB* y = static_cast<TB*>(p.y) + r * C;
        float s = 0.f;
        for (int c = threadIdx.x; c < C; c += kThreads) {
            const float v = to_f32(x[c]);
            s = fmaf(v, v, s);
        }
        const float post = 1.f / sqrtf(fmaf(cta_sum(s, red), inv, p.eps));
        const auto sum = [&](int c) {
            float m = to_f32(x[c]) * post * load_param(p.gamma_post, p.param_type, c, 1.f);
            if (gate != nullptr) m *= gate_of(to_f32(gate[c]), p.act);
            return fmaf(p.alpha, to_f32(res[c]), load_param(p.scale, p.param_type, c, 1.f) * m);
        };
        s = 0.f;
        for (int c = threadIdx.x; c < C; c += kThreads) {
            const float v = sum(c);
            s = fmaf(v, v, s);
        }
        const float pre = 1.f / sqrtf(fmaf(cta_sum(s, red), inv, p.eps));
        for (int c = threadIdx.x; c < C; c += kThreads) {
            const float v = sum(c);     // (outputs may be inputs: this thread has read the element for the last time)
            store_out(z + c, v);
            store_out(y + c, v * pre * load_param(p.gamma_pre, p.param_type, c, 1.f));
        }
        if (threadIdx.x == 0) {
            if (p.rstd_post_out != nullptr) p.rstd_post_out[r] = post;
            if (p.rstd_pre_out != nullptr) p.rstd_pre_out[r] = pre;
        }
    }
}

template <typename TS, typename TB>
__global__ void __launch_bounds__(kThreads) block_norm_bwd_general_kernel(BlockNorm p) {
    __shared__ float red[kWarps];
    pdl_trigger();
    pdl_wait();
    const int C = p.C;
    const float inv = 1.f / static_cast<float>(C);
    float* part = p.partial == nullptr ? nullptr : p.partial + static_cast<size_t>(blockIdx.x) * 2 * C;
    bool first_row = true;
    for (long long r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const TB* dy = static_cast<const TB*>(p.dy) + r * p.ld_dy;
        const TS* dz = p.dz == nullptr ? nullptr : static_cast<const TS*>(p.dz) + r * p.ld_dz;
        const TB* x = static_cast<const TB*>(p.x) + r * p.ld_x;
        const TS* z = static_cast<const TS*>(p.z_in) + r * p.ld_z;
        const TB* gate = p.gate == nullptr ? nullptr : static_cast<const TB*>(p.gate) + r * p.ld_gate;
        const float post = p.rstd_post[r], pre = p.rstd_pre[r];
        float s = 0.f;
        for (int c = threadIdx.x; c < C; c += kThreads)
            s = fmaf(to_f32(dy[c]) * load_param(p.gamma_pre, p.param_type, c, 1.f), to_f32(z[c]) * pre, s);
        const float m_pre = cta_sum(s, red) * inv;
        const auto stream = [&](int c) {
            const float a = to_f32(dy[c]) * load_param(p.gamma_pre, p.param_type, c, 1.f);
            const float g = pre * (a - to_f32(z[c]) * pre * m_pre);
            return dz != nullptr ? g + to_f32(dz[c]) : g;
        };
        s = 0.f;
        for (int c = threadIdx.x; c < C; c += kThreads) {
            const float g = stream(c), xhat = to_f32(x[c]) * post, gamma = load_param(p.gamma_post, p.param_type, c, 1.f);
            const float act = gate != nullptr ? gate_of(to_f32(gate[c]), p.act) : 1.f;
            const float t = g * act;
            s = fmaf(load_param(p.scale, p.param_type, c, 1.f) * gamma * t, xhat, s);
            if (part != nullptr) {
                const float v[2] = {t * xhat, to_f32(dy[c]) * (to_f32(z[c]) * pre)};
#pragma unroll
                for (int i = 0; i < 2; ++i) part[i * static_cast<size_t>(C) + c] = first_row ? v[i] : part[i * static_cast<size_t>(C) + c] + v[i];
            }
        }
        const float m_post = cta_sum(s, red) * inv;
        for (int c = threadIdx.x; c < C; c += kThreads) {
            const float g = stream(c), xhat = to_f32(x[c]) * post, gamma = load_param(p.gamma_post, p.param_type, c, 1.f);
            const float scaled = load_param(p.scale, p.param_type, c, 1.f) * g;
            float slope = 0.f;
            const float act = gate != nullptr ? gate_of(to_f32(gate[c]), p.act, &slope) : 1.f;
            store_out(static_cast<TB*>(p.dx) + r * C + c, post * fmaf(-xhat, m_post, scaled * act * gamma));
            store_out(static_cast<TS*>(p.dres) + r * C + c, p.alpha * g);
            if (p.dgate != nullptr) store_out(static_cast<TB*>(p.dgate) + r * C + c, scaled * (xhat * gamma) * slope);
        }
        first_row = false;
    }
}

// Column sums of the partial rows: a CTA takes kWidth columns of both sums, each thread every
// (1024 / kWidth)-th row, 8 loads in flight.  A fixed order, whatever the timing.
constexpr int kSumThreads = 1024;
template <int kWidth>
__global__ void __launch_bounds__(kSumThreads) block_norm_param_kernel(BlockNorm p, int count) {
    constexpr int kSlots = kSumThreads / kWidth;
    __shared__ float sums[kSlots][kWidth + 1];
    pdl_trigger();
    const int col = threadIdx.x % kWidth, slot = threadIdx.x / kWidth, C = p.C;
    const long long j = static_cast<long long>(blockIdx.x) * kWidth + col;
    const size_t step = static_cast<size_t>(2) * C;
    float s = 0.f;
    pdl_wait();
    if (j < 2LL * C) {
        const float* from = p.partial + j;
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
    const int c = static_cast<int>(o < C ? o : o - C);
    if (o >= C) {
        if (p.grads[1] != nullptr) p.grads[1][c] = s;
        return;
    }
    if (p.grads[0] != nullptr) p.grads[0][c] = load_param(p.scale, p.param_type, c, 1.f) * s;
    if (p.grads[2] != nullptr) p.grads[2][c] = load_param(p.gamma_post, p.param_type, c, 1.f) * s;
}

template <typename TS, typename TB>
cudaError_t fwd_t(const BlockNorm& p) {
    const long long cap = static_cast<long long>(device_info().sm_count) * 64;
    return launch_pdl(block_norm_fwd_general_kernel<TS, TB>, dim3(static_cast<unsigned>(std::min(p.rows, cap))), dim3(kThreads), 0,
                      p.stream, p);
}

template <typename TS, typename TB>
cudaError_t bwd_t(const BlockNorm& p) {
    const int parts = block_norm_partials(p.rows, p.C);
    const cudaError_t err = launch_pdl(block_norm_bwd_general_kernel<TS, TB>, dim3(static_cast<unsigned>(parts)), dim3(kThreads), 0,
                                       p.stream, p);
    return err != cudaSuccess || p.partial == nullptr ? err : launch_block_norm_params(p, parts);
}

}  // namespace

// Partial rows: two CTAs per SM, and at most 2^25 columns in all (256 MB) for very wide rows.
int block_norm_partials(long long rows, int C) {
    const long long by_size = std::max<long long>(1, (1LL << 25) / C);
    return static_cast<int>(std::min({rows, 4LL * device_info().sm_count, by_size}));
}

#define DWC_BY_PAIR(fn, p)                                                                        \
    if ((p).stream_type == kF32 && (p).branch_type == kF32) return fn<float, float>(p);           \
    if ((p).stream_type == kF32 && (p).branch_type == kBF16) return fn<float, __nv_bfloat16>(p);  \
    if ((p).stream_type == kF32 && (p).branch_type == kF16) return fn<float, __half>(p);          \
    if ((p).stream_type == kBF16) return fn<__nv_bfloat16, __nv_bfloat16>(p);                     \
    return fn<__half, __half>(p);

cudaError_t launch_block_norm_fwd_general(const BlockNorm& p) { DWC_BY_PAIR(fwd_t, p) }
cudaError_t launch_block_norm_bwd_general(const BlockNorm& p) { DWC_BY_PAIR(bwd_t, p) }

cudaError_t launch_block_norm_params(const BlockNorm& p, int count) {
    const auto launch = [&](auto kern, int width) {
        return launch_pdl(kern, dim3(static_cast<unsigned>((2LL * p.C + width - 1) / width)), dim3(kSumThreads), 0, p.stream, p, count);
    };
    if (2LL * p.C <= 8LL * 2 * device_info().sm_count) return launch(block_norm_param_kernel<8>, 8);
    return launch(block_norm_param_kernel<32>, 32);
}

}  // namespace dwc

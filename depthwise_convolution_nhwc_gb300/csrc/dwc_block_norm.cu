// dwc_block_norm.cu -- the norms on either side of a residual connection with its gate and scales,
// forward and backward, for any row stride, alignment and channel count; the sum of partial parameter gradients.
//
//     n = x rstd_post gamma_post,  z = alpha res + scale act(gate) n,  y = z rstd_pre gamma_pre
//
// One CTA per row, which is read in three passes (the second and third from L1 or L2): 8 elements to an
// access where every tensor allows it (rows too wide for the kernels of dwc_block_norm_rows.cuh), else one.
#include <algorithm>

#include "dwc_block_norm_device.cuh"

namespace dwc {
namespace {

constexpr int kThreads = 256;          // several CTAs to an SM
constexpr int kWideThreads = 1024;     // one, with its columns' sums in shared memory
constexpr size_t kWideSmem = 200 * 1024;

template <int kThreads>
__device__ __forceinline__ float cta_sum(float v, float* red) {
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) s += red[w];
    return s;
}

// V adjacent fp32 values (1 or 8).
template <int V>
struct Some {
    float v[V];
};
template <int V, typename T>
__device__ __forceinline__ Some<V> get(const T* p) {
    Some<V> f;
    if constexpr (V == 1) {
        f.v[0] = to_f32(*p);
    } else {
        Vec8<T> raw;
        float2 g[4];
        raw.load(p);
        raw.widen(g);
#pragma unroll
        for (int j = 0; j < 4; ++j) f.v[2 * j] = g[j].x, f.v[2 * j + 1] = g[j].y;
    }
    return f;
}
template <int V, typename T>
__device__ __forceinline__ void put(T* p, const Some<V>& f) {
    if constexpr (V == 1) {
        store_out(p, f.v[0]);
    } else {
        float2 g[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) g[j] = make_float2(f.v[2 * j], f.v[2 * j + 1]);
        Vec8<T>::store(p, g);
    }
}
template <int V>
__device__ __forceinline__ Some<V> param(const void* p, int type, int c) {
    Some<V> f;
    if (p == nullptr) {
#pragma unroll
        for (int j = 0; j < V; ++j) f.v[j] = 1.f;
        return f;
    }
    if (type == kF32) return get<V>(static_cast<const float*>(p) + c);
    if (type == kBF16) return get<V>(static_cast<const __nv_bfloat16*>(p) + c);
    return get<V>(static_cast<const __half*>(p) + c);
}

template <typename TS, typename TB, int V>
__global__ void __launch_bounds__(kThreads) block_norm_fwd_general_kernel(BlockNorm p) {
    __shared__ float red[kThreads / 32];
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
        for (int c = threadIdx.x * V; c < C; c += kThreads * V) {
            const Some<V> f = get<V>(x + c);
#pragma unroll
            for (int j = 0; j < V; ++j) s = fmaf(f.v[j], f.v[j], s);
        }
        const float post = 1.f / sqrtf(fmaf(cta_sum<kThreads>(s, red), inv, p.eps));
        const auto sum = [&](int c) {
            Some<V> f = get<V>(x + c);
            const Some<V> t = get<V>(res + c), gamma = param<V>(p.gamma_post, p.param_type, c), scale = param<V>(p.scale, p.param_type, c);
            if (gate != nullptr) {
                const Some<V> g = get<V>(gate + c);
#pragma unroll
                for (int j = 0; j < V; ++j) f.v[j] = fmaf(p.alpha, t.v[j], scale.v[j] * (f.v[j] * post * gamma.v[j] * gate_of(g.v[j], p.act)));
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) f.v[j] = fmaf(p.alpha, t.v[j], scale.v[j] * (f.v[j] * post * gamma.v[j]));
            }
            return f;
        };
        s = 0.f;
        for (int c = threadIdx.x * V; c < C; c += kThreads * V) {
            const Some<V> f = sum(c);
#pragma unroll
            for (int j = 0; j < V; ++j) s = fmaf(f.v[j], f.v[j], s);
        }
        const float pre = 1.f / sqrtf(fmaf(cta_sum<kThreads>(s, red), inv, p.eps));
        for (int c = threadIdx.x * V; c < C; c += kThreads * V) {
            Some<V> f = sum(c);     // (outputs may be inputs: this thread has read the elements for the last time)
            put(z + c, f);
            const Some<V> gamma = param<V>(p.gamma_pre, p.param_type, c);
#pragma unroll
            for (int j = 0; j < V; ++j) f.v[j] = f.v[j] * pre * gamma.v[j];
            put(y + c, f);
        }
        if (threadIdx.x == 0) {
            if (p.rstd_post_out != nullptr) p.rstd_post_out[r] = post;
            if (p.rstd_pre_out != nullptr) p.rstd_pre_out[r] = pre;
        }
    }
}

// Every CTA adds the parameter gradients of its rows into its own row of partial sums [sum t xhat | sum dy zhat]; a column
// belongs to one thread, so the additions have a fixed order.  NT is kWideThreads: the sums wait in shared memory until the
// end (fp32 stream, bf16 branches, 2048 x 16384: 442 us with the sums read and written in memory every row).
template <typename TS, typename TB, int V, int NT>
__global__ void __launch_bounds__(NT) block_norm_bwd_general_kernel(BlockNorm p) {
    extern __shared__ __align__(16) float sums[];
    __shared__ float red[NT / 32];
    pdl_trigger();
    pdl_wait();
    const int C = p.C;
    const float inv = 1.f / static_cast<float>(C);
    float* const row_out = p.partial == nullptr ? nullptr : p.partial + static_cast<size_t>(blockIdx.x) * 2 * C;
    float* const part = row_out == nullptr || NT == kThreads ? row_out : sums;
    bool first_row = true;
    for (long long r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const TB* dy = static_cast<const TB*>(p.dy) + r * p.ld_dy;
        const TS* dz = p.dz == nullptr ? nullptr : static_cast<const TS*>(p.dz) + r * p.ld_dz;
        const TB* x = static_cast<const TB*>(p.x) + r * p.ld_x;
        const TS* z = static_cast<const TS*>(p.z_in) + r * p.ld_z;
        const TB* gate = p.gate == nullptr ? nullptr : static_cast<const TB*>(p.gate) + r * p.ld_gate;
        const float post = p.rstd_post[r], pre = p.rstd_pre[r];
        float s = 0.f;
        for (int c = threadIdx.x * V; c < C; c += NT * V) {
            const Some<V> d = get<V>(dy + c), f = get<V>(z + c), gamma = param<V>(p.gamma_pre, p.param_type, c);
#pragma unroll
            for (int j = 0; j < V; ++j) s = fmaf(d.v[j] * gamma.v[j], f.v[j] * pre, s);
        }
        const float m_pre = cta_sum<NT>(s, red) * inv;
        // g, the gradient that reaches the stream's sum; `hat`: dy zhat
        const auto stream = [&](int c, Some<V>& hat) {
            Some<V> g = get<V>(dy + c);
            const Some<V> f = get<V>(z + c), gamma = param<V>(p.gamma_pre, p.param_type, c);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                hat.v[j] = g.v[j] * (f.v[j] * pre);
                g.v[j] = pre * (g.v[j] * gamma.v[j] - f.v[j] * pre * m_pre);
            }
            if (dz != nullptr) {
                const Some<V> e = get<V>(dz + c);
#pragma unroll
                for (int j = 0; j < V; ++j) g.v[j] += e.v[j];
            }
            return g;
        };
        s = 0.f;
        for (int c = threadIdx.x * V; c < C; c += NT * V) {
            Some<V> hat, g = stream(c, hat), xhat = get<V>(x + c);
            const Some<V> gamma = param<V>(p.gamma_post, p.param_type, c), scale = param<V>(p.scale, p.param_type, c);
            if (gate != nullptr) {
                const Some<V> f = get<V>(gate + c);
#pragma unroll
                for (int j = 0; j < V; ++j) g.v[j] *= gate_of(f.v[j], p.act);
            }
#pragma unroll
            for (int j = 0; j < V; ++j) {
                xhat.v[j] *= post;
                s = fmaf(scale.v[j] * gamma.v[j] * g.v[j], xhat.v[j], s);
            }
            if (part != nullptr) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    part[c + j] = first_row ? g.v[j] * xhat.v[j] : part[c + j] + g.v[j] * xhat.v[j];
                    part[C + c + j] = first_row ? hat.v[j] : part[C + c + j] + hat.v[j];
                }
            }
        }
        const float m_post = cta_sum<NT>(s, red) * inv;
        for (int c = threadIdx.x * V; c < C; c += NT * V) {
            Some<V> hat, g = stream(c, hat), xhat = get<V>(x + c), act, slope;
            const Some<V> gamma = param<V>(p.gamma_post, p.param_type, c), scale = param<V>(p.scale, p.param_type, c);
#pragma unroll
            for (int j = 0; j < V; ++j) act.v[j] = 1.f, slope.v[j] = 0.f;
            if (gate != nullptr) {
                const Some<V> f = get<V>(gate + c);
#pragma unroll
                for (int j = 0; j < V; ++j) act.v[j] = gate_of(f.v[j], p.act, &slope.v[j]);
            }
            Some<V> o;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                xhat.v[j] *= post;
                o.v[j] = p.alpha * g.v[j];
                g.v[j] *= scale.v[j];
                slope.v[j] *= g.v[j] * (xhat.v[j] * gamma.v[j]);
                act.v[j] = post * fmaf(-xhat.v[j], m_post, g.v[j] * act.v[j] * gamma.v[j]);
            }
            put(static_cast<TB*>(p.dx) + r * C + c, act);
            put(static_cast<TS*>(p.dres) + r * C + c, o);
            if (p.dgate != nullptr) put(static_cast<TB*>(p.dgate) + r * C + c, slope);
        }
        first_row = false;
    }
    if (NT == kThreads || part == nullptr) return;
    for (int c = threadIdx.x * V; c < C; c += NT * V)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            row_out[c + j] = sums[c + j];
            row_out[C + c + j] = sums[C + c + j];
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

// Whether 8 elements of every row can be read or written at once from any multiple of 8.
bool vectors_of(const BlockNorm& p, bool backward) {
    if (p.C % 8 != 0) return false;
    const auto fits = [&](const void* t, int type, long long ld) {
        return t == nullptr || (reinterpret_cast<uintptr_t>(t) % (8 * elem_bytes(type)) == 0 && (p.rows == 1 || ld % 8 == 0));
    };
    const int ts = p.stream_type, tb = p.branch_type, tp = p.param_type;
    if (!fits(p.x, tb, p.ld_x) || !fits(p.gate, tb, p.ld_gate) || !fits(p.gamma_post, tp, 0) || !fits(p.gamma_pre, tp, 0) || !fits(p.scale, tp, 0))
        return false;
    if (!backward) return fits(p.res, ts, p.ld_res) && fits(p.z, ts, 0) && fits(p.y, tb, 0);
    return fits(p.dy, tb, p.ld_dy) && fits(p.dz, ts, p.ld_dz) && fits(p.z_in, ts, p.ld_z) && fits(p.dx, tb, 0) && fits(p.dres, ts, 0) &&
           fits(p.dgate, tb, 0);
}

template <typename TS, typename TB>
cudaError_t fwd_t(const BlockNorm& p) {
    const long long cap = static_cast<long long>(device_info().sm_count) * 64;
    return launch_pdl(vectors_of(p, false) ? block_norm_fwd_general_kernel<TS, TB, 8> : block_norm_fwd_general_kernel<TS, TB, 1>,
                      dim3(static_cast<unsigned>(std::min(p.rows, cap))), dim3(kThreads), 0, p.stream, p);
}

template <typename TS, typename TB, int V>
cudaError_t bwd_v(const BlockNorm& p) {
    int parts = block_norm_partials(p.rows, p.C);
    const size_t bytes = static_cast<size_t>(p.C) * 2 * sizeof(float);
    cudaError_t err;
    if (bytes <= kWideSmem && p.C >= kWideThreads) {
        static DeviceOnce once;
        err = opt_in_smem(block_norm_bwd_general_kernel<TS, TB, V, kWideThreads>, once, kWideSmem);
        if (err != cudaSuccess) return err;
        parts = std::min(parts, device_info().sm_count);
        err = launch_pdl(block_norm_bwd_general_kernel<TS, TB, V, kWideThreads>, dim3(static_cast<unsigned>(parts)), dim3(kWideThreads), bytes,
                         p.stream, p);
    } else {
        err = launch_pdl(block_norm_bwd_general_kernel<TS, TB, V, kThreads>, dim3(static_cast<unsigned>(parts)), dim3(kThreads), 0, p.stream, p);
    }
    return err != cudaSuccess || p.partial == nullptr ? err : launch_block_norm_params(p, parts);
}

template <typename TS, typename TB>
cudaError_t bwd_t(const BlockNorm& p) {
    return vectors_of(p, true) ? bwd_v<TS, TB, 8>(p) : bwd_v<TS, TB, 1>(p);
}

}  // namespace

// Partial rows: four CTAs per SM, and at most 2^25 columns in all (256 MB) for very wide rows.
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

// dwc_scan_step.cu -- selective scan of one position for each of several sequences, states updated in
// place.
//
// Bound by memory: the fp32 states are read and written once (8 N bytes a channel; everything else
// is a few bytes).  A lane has four adjacent states of a channel; the lanes of a channel add up y.
#include <algorithm>

#include "dwc_scan.cuh"

namespace dwc {
namespace scan {
namespace {

constexpr int kStepThreads = 256;

// kVec: N is a multiple of 4 and the states and A are aligned to 16 bytes.
template <typename T, int L, bool kVec>
__global__ void __launch_bounds__(kStepThreads) scan_step_kernel(Scan p, float* states, long long state_stride) {
    pdl_trigger();
    pdl_wait();
    const int C = p.C, N = p.N;
    const long long i = static_cast<long long>(blockIdx.x) * kStepThreads + threadIdx.x;
    const int at = static_cast<int>(i / (static_cast<long long>(C) * L));
    const bool live = at < p.seqs.count;     // (the last CTA's other threads go along for the exchanges)
    const int s = live ? at : 0;
    const int rest = static_cast<int>(i - static_cast<long long>(at) * C * L), ch = rest / L, n0 = rest % L * 4;
    const int g = ch / (C / p.G);
    float* state = states + s * state_stride + static_cast<long long>(ch) * N;
    const float* a = p.A + static_cast<long long>(ch) * N;
    const T *b = static_cast<const T*>(p.b.p) + s * p.b.seq + g * N, *c = static_cast<const T*>(p.c.p) + s * p.c.seq + g * N;
    float h[4], an[4];
    if (kVec) {
        if (n0 < N) {
            const float4 v = *reinterpret_cast<const float4*>(state + n0), w = *reinterpret_cast<const float4*>(a + n0);
            h[0] = v.x, h[1] = v.y, h[2] = v.z, h[3] = v.w;
            an[0] = w.x, an[1] = w.y, an[2] = w.z, an[3] = w.w;
        }
    } else {
        get_states(h, state, n0, N);
        get_states(an, a, n0, N);
    }
    const float u = to_f32(static_cast<const T*>(p.u.p)[s * p.u.seq + ch]);
    float delta = to_f32(static_cast<const T*>(p.dt.p)[s * p.dt.seq + ch]) + (p.dt_bias != nullptr ? p.dt_bias[ch] : 0.f);
    if (p.softplus) delta = softplus(delta);
    const float in = delta * u;
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (n0 + j >= N) continue;
        h[j] = fmaf(exp2_fast(delta * (an[j] * kLog2e)), h[j], in * to_f32(b[n0 + j]));
        sum = fmaf(to_f32(c[n0 + j]), h[j], sum);
    }
    if (!live) {
    } else if (kVec) {
        if (n0 < N) *reinterpret_cast<float4*>(state + n0) = make_float4(h[0], h[1], h[2], h[3]);
    } else {
        put_states(state, h, n0, N);
    }
#pragma unroll
    for (int m = L / 2; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    if (!live || rest % L != 0) return;
    if (p.D != nullptr) sum = fmaf(p.D[ch], u, sum);
    if (p.z.p != nullptr) sum *= silu(to_f32(static_cast<const T*>(p.z.p)[s * p.z.seq + ch]));
    store_out(static_cast<T*>(p.y) + static_cast<long long>(s) * C + ch, sum);
}

template <typename T, int L>
cudaError_t step_l(const Scan& p, float* state, long long state_stride) {
    const long long grid = (static_cast<long long>(p.seqs.count) * p.C * L + kStepThreads - 1) / kStepThreads;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const auto off = [](const void* t) { return reinterpret_cast<uintptr_t>(t) % 16 != 0; };
    const bool vec = p.N % 4 == 0 && state_stride % 4 == 0 && !off(state) && !off(p.A);
    return launch_pdl(vec ? scan_step_kernel<T, L, true> : scan_step_kernel<T, L, false>, dim3(static_cast<unsigned>(grid)),
                      dim3(kStepThreads), 0, p.stream, p, state, state_stride);
}

template <typename T>
cudaError_t step_t(const Scan& p, float* state, long long state_stride) {
    if (p.N <= 4) return step_l<T, 1>(p, state, state_stride);
    if (p.N <= 8) return step_l<T, 2>(p, state, state_stride);
    if (p.N <= 16) return step_l<T, 4>(p, state, state_stride);
    if (p.N <= 32) return step_l<T, 8>(p, state, state_stride);
    if (p.N <= 64) return step_l<T, 16>(p, state, state_stride);
    return step_l<T, 32>(p, state, state_stride);
}

}  // namespace
}  // namespace scan

cudaError_t launch_scan_step(const Scan& p, float* state, long long state_stride) {
    switch (p.type) {
        case kF32: return scan::step_t<float>(p, state, state_stride);
        case kBF16: return scan::step_t<__nv_bfloat16>(p, state, state_stride);
        default: return scan::step_t<__half>(p, state, state_stride);
    }
}

namespace {

// Positions to a chunk.  A batch whose sequences fill `enough` CTAs of the `resident` that the GPU holds together
// stays whole (packed sequences differ in length: those up to twice the mean do); else there are as many chunks
// as make one round of CTAs, 64 positions at least.
long long span_of(const Seqs& s, long long blocks, long long resident, long long enough) {
    if (s.count == 0 || s.length == 0) return 1 << 20;
    const long long rows = seq_rows(s);
    long long span;
    if (s.count * blocks >= enough) {
        span = s.offsets != nullptr ? 2 * (rows / s.count) : s.length;
    } else if (s.offsets != nullptr) {
        span = rows * blocks / resident;
    } else {
        const long long each = std::max<long long>(1, resident / (s.count * blocks));
        span = (s.length + each - 1) / each;
    }
    return std::max<long long>(64, (span + 15) / 16 * 16);
}

}  // namespace

long long scan_fwd_span(const Scan& p) {
    const long long resident = 640LL / scan::fwd_threads(p.N) * device_info().sm_count;
    return span_of(p.seqs, scan::channel_blocks(p, scan::fwd_channels(p.N)), resident, resident / 3);
}
long long scan_bwd_span(const Scan& p) {
    const long long resident = (p.N <= 64 ? scan::BwdShape<4>::kResident : scan::BwdShape<32>::kResident) * static_cast<long long>(device_info().sm_count);
    return span_of(p.seqs, scan::channel_blocks(p, scan::bwd_channels(p.N)), resident, resident / 2);
}
size_t scan_fwd_workspace_floats(const Scan& p) {
    const scan::FwdSpace s(p);
    return static_cast<size_t>(s.ends + s.sums);
}
size_t scan_bwd_workspace_floats(const Scan& p) {
    const scan::BwdSpace s(p);
    return static_cast<size_t>(s.bc + s.params + s.ends + s.sums);
}

}  // namespace dwc

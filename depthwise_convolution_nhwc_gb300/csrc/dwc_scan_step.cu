// dwc_scan_step.cu -- selective scan of one position for each of several sequences, states updated in
// place; how the sequences of the other passes are cut into chunks.
//
// Bound by memory: the fp32 states are read and written once (8 N bytes a channel; everything else
// is a few bytes).  A lane has four adjacent states of a channel, of kSeqs sequences whose loads are in flight
// together; the lanes of a channel add up y.
#include <algorithm>

#include "dwc_scan.cuh"

namespace dwc {
namespace scan {
namespace {

constexpr int kStepThreads = 128;

// Four adjacent states of B or C (zeros past the last): one load of 4 values where kVec.
template <typename T, bool kVec>
__device__ __forceinline__ Four four_of(const T* p, int n0, int N) {
    Four f;
    if constexpr (kVec) {
        f.clear();
        if (n0 >= N) return f;
        if constexpr (sizeof(T) == 4) {
            f.load(p + n0);
        } else {
            const uint2 w = *reinterpret_cast<const uint2*>(p + n0);
            f.v[0] = Elem<T>::load_pair(reinterpret_cast<const T*>(&w.x)), f.v[1] = Elem<T>::load_pair(reinterpret_cast<const T*>(&w.y));
        }
    } else {
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = n0 + j < N ? to_f32(p[n0 + j]) : 0.f;
        f.v[0] = make_float2(v[0], v[1]), f.v[1] = make_float2(v[2], v[3]);
    }
    return f;
}

// kVec: N is a multiple of 4, the states and A are aligned to 16 bytes, B and C to four values.
template <typename T, int L, bool kVec, int kSeqs>
__global__ void __launch_bounds__(kStepThreads) scan_step_kernel(Scan p, float* states, long long state_stride) {
    pdl_trigger();
    pdl_wait();
    const int C = p.C, N = p.N, groups = (p.seqs.count + kSeqs - 1) / kSeqs;
    const long long i = static_cast<long long>(blockIdx.x) * kStepThreads + threadIdx.x;
    const int at = static_cast<int>(i / (static_cast<long long>(C) * L));
    const bool live = at < groups;           // (the last CTA's other threads go along for the exchanges)
    const int first = live ? at * kSeqs : 0;
    const int rest = static_cast<int>(i - static_cast<long long>(at) * C * L), ch = rest / L, n0 = rest % L * 4;
    const int g = ch / (C / p.G);
    Four h[kSeqs], b[kSeqs], c[kSeqs], a2;
    float u[kSeqs], dt[kSeqs], z[kSeqs];
    a2.get4(p.A + static_cast<long long>(ch) * N, n0, 0, N, kVec);
    a2.to_rates();
    const float bias = p.dt_bias != nullptr ? p.dt_bias[ch] : 0.f, skip = p.D != nullptr ? p.D[ch] : 0.f;
#pragma unroll
    for (int q = 0; q < kSeqs; ++q) {
        const int s = min(first + q, p.seqs.count - 1);
        h[q].get4(states + s * state_stride + static_cast<long long>(ch) * N, n0, 0, N, kVec);
        b[q] = four_of<T, kVec>(static_cast<const T*>(p.b.p) + s * p.b.seq + g * N, n0, N);
        c[q] = four_of<T, kVec>(static_cast<const T*>(p.c.p) + s * p.c.seq + g * N, n0, N);
        u[q] = to_f32(static_cast<const T*>(p.u.p)[s * p.u.seq + ch]);
        dt[q] = to_f32(static_cast<const T*>(p.dt.p)[s * p.dt.seq + ch]);
        z[q] = p.z.p != nullptr ? to_f32(static_cast<const T*>(p.z.p)[s * p.z.seq + ch]) : 0.f;
    }
#pragma unroll
    for (int q = 0; q < kSeqs; ++q) {
        const int s = first + q;
        float delta = dt[q] + bias;
        if (p.softplus) delta = softplus(delta);
        const float in = delta * u[q];
        float2 sum2 = both(0.f);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            h[q].v[j] = __ffma2_rn(both(in), b[q].v[j], __fmul2_rn(decay_of(delta, a2.v[j]), h[q].v[j]));
            sum2 = __ffma2_rn(c[q].v[j], h[q].v[j], sum2);
        }
        float sum = sum2.x + sum2.y;
#pragma unroll
        for (int m = L / 2; m > 0; m >>= 1) sum += from_lane(sum, m);
        if (!live || s >= p.seqs.count) continue;       // (no exchange below)
        h[q].put4(states + s * state_stride + static_cast<long long>(ch) * N, n0, N, kVec);
        if (rest % L != 0) continue;
        sum = fmaf(skip, u[q], sum);
        if (p.z.p != nullptr) sum *= silu(z[q]);
        store_out(static_cast<T*>(p.y) + static_cast<long long>(s) * C + ch, sum);
    }
}

template <typename T, int L, bool kVec, int kSeqs>
cudaError_t step_s(const Scan& p, float* state, long long state_stride) {
    const long long groups = (p.seqs.count + kSeqs - 1) / kSeqs;
    const long long grid = (groups * p.C * L + kStepThreads - 1) / kStepThreads;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    return launch_pdl(scan_step_kernel<T, L, kVec, kSeqs>, dim3(static_cast<unsigned>(grid)), dim3(kStepThreads), 0, p.stream, p, state,
                      state_stride);
}

template <typename T, int L>
cudaError_t step_l(const Scan& p, float* state, long long state_stride) {
    const auto off = [](const void* t, size_t a) { return reinterpret_cast<uintptr_t>(t) % a != 0; };
    const auto four = [&](const RowsView& v) { return !off(v.p, 4 * sizeof(T)) && (p.seqs.count <= 1 || v.seq % 4 == 0); };
    const bool vec = p.N % 4 == 0 && (p.seqs.count <= 1 || state_stride % 4 == 0) && !off(state, 16) && !off(p.A, 16) && four(p.b) && four(p.c);
    if (!vec) return step_s<T, L, false, 1>(p, state, state_stride);
    // several sequences to a thread once that leaves every SM 1024 threads
    const bool many = static_cast<long long>(p.seqs.count) * p.C * L >= 4LL * 1024 * device_info().sm_count;
    return many ? step_s<T, L, true, 4>(p, state, state_stride) : step_s<T, L, true, 1>(p, state, state_stride);
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
    const long long blocks = scan::channel_blocks(p, scan::bwd_channels(p.N));
    const long long span = span_of(p.seqs, blocks, resident, resident / 2), most = scan::most_partial_rows(p);
    if (seq_rows(p.seqs) <= most) return span;
    // Partial rows for some of the positions at a time, of pieces that fill half of the GPU then: sequences of a batch stay
    // whole where that holds, and no piece takes more than half of them.
    const long long fill = std::min(most, 2 * most * blocks / resident);
    if (p.seqs.offsets == nullptr && span >= p.seqs.length && p.seqs.length <= fill) return span;
    return std::max<long long>(64, std::min(span, fill / 2 / 16 * 16));
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

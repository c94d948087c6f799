// dwc_scan.cuh -- selective scan along sequences, forward and backward.
//
//     h[t, n] = exp(delta[t] A[n]) h[t-1, n] + delta[t] u[t] B[t, n]
//     y[t]    = (sum_n C[t, n] h[t, n] + D u[t]) silu(z[t])
//
// L lanes serve a pair of channels, four states of each to a lane, and walk along the positions with
// the states in registers.  Tiles of 16 positions are brought in by the whole CTA: per channel and position delta
// and u, once, as fp32 in shared memory, and B and C widened.
//
// Measured (bf16, 16 states, device time): forward of one sequence of 16384 positions and 2048 channels, in chunks, 119 + 6 + 178 us
// (its bytes would take 40), of 8 sequences of 2048 positions and 4096 channels with what the backward pass needs 432 us,
// backward 1455 us (both: 158).  More states, call to call, forward and backward: 32 0.75 + 3.2 ms, 64 1.57 + 7.6, 128 2.7 + 15.1,
// where the partial rows of dB and dC (4.3 and 8.6 GB, written and read once) are a sixth of the backward pass.
//
// Errors: decays are the hardware's exponential, off by up to 2 ulp, of an argument rounded twice, and slow states remember many
// of them.  Of packed fp32 3005 x 1002 with 11 states dA is off by 1.07e-6 (of its norm), the same formulas in PyTorch by 0.69e-6,
// these kernels with correctly rounded decays by 0.29e-6; a softplus of full precision changes nothing (1.06e-6).
//
// What bounds it: per state and position 4 packed operations (2 cycles a warp for a pair of states), an exponential (4
// cycles a warp) and what shared memory hands to the lanes, 128 bytes a cycle for the whole SM, broadcast or not: a lane
// that had one channel took 8 bytes of B and C a state, twice the time of the arithmetic (16-byte loads count four
// times).  Hence two channels to a lane.
#pragma once

#include <algorithm>

#include "dwc_seq_device.cuh"

namespace dwc {
namespace scan {

constexpr int kTile = kScanTile, kStep = 4;       // positions of a tile, and that go through together

// log(1 + exp(v)) = max(v, 0) + log(1 + e), e = exp(-|v|): the logarithm as 2 atanh(s), s = e / (2 + e) <= 1/3, whose odd
// series is s + s^3 P(s^2) with P of degree 3 by Chebyshev interpolation on [0, 1/9] (relative error 1.6e-8): relative
// errors stay near 2^-22 however small e is.  (A NaN stays one: fmaxf would drop it.)
__device__ __forceinline__ float2 softplus2(float2 v, float2* slope = nullptr) {
    const float2 e = make_float2(exp2_fast(fabsf(v.x) * -kLog2e), exp2_fast(fabsf(v.y) * -kLog2e));
    const float2 w = __fadd2_rn(e, both(2.f));
    const float2 s = __fmul2_rn(e, make_float2(rcp_fast(w.x), rcp_fast(w.y))), q = __fmul2_rn(s, s);
    float2 p = __ffma2_rn(both(0.13433775305747986f), q, both(0.14116978645324707f));
    p = __ffma2_rn(p, q, both(0.2000383585691452f));
    p = __ffma2_rn(p, q, both(0.33333319425582886f));
    const float2 t = __fadd2_rn(s, s);
    if (slope != nullptr) {         // 1 / (1 + exp(-v)) = 1 / (1 + e), or e / (1 + e) where v < 0
        const float2 o = __fadd2_rn(e, both(1.f)), r = make_float2(rcp_fast(o.x), rcp_fast(o.y));
        *slope = make_float2(v.x < 0.f ? e.x * r.x : r.x, v.y < 0.f ? e.y * r.y : r.y);
    }
    return __fadd2_rn(make_float2(v.x < 0.f ? 0.f : v.x, v.y < 0.f ? 0.f : v.y), __ffma2_rn(__fmul2_rn(t, q), p, t));
}
__device__ __forceinline__ float softplus(float v) { return softplus2(both(v)).x; }

__device__ __forceinline__ float from_lane(float v, int mask) { return __shfl_xor_sync(0xffffffffu, v, mask); }

// Places in shared memory, such that neither the threads that write vectors of 8 channels or states nor the lanes that
// read a channel's or four states' values meet in the banks, and that a position adds a constant to an address.
// Two values per position and channel: units of two channels (16 bytes) change places among four, rows 64 bytes longer.
template <int kChannels>
struct StepAt {
    static constexpr int kRow = kChannels + 8, kSize = kTile * kRow;
    static __device__ __forceinline__ int at(int t, int ch) { return t * kRow + ((((ch >> 1) ^ (ch >> 3 & 3)) << 1) | (ch & 1)); }
};
// One value per position and channel: rows 8 bytes longer.
template <int kChannels>
struct ValueAt {
    static constexpr int kRow = kChannels + 2, kSize = kTile * kRow;
    static __device__ __forceinline__ int at(int t, int ch) { return t * kRow + ch; }
};
// Rows of NP states: 16 bytes more after every 128.  The position is w * kStep + q.
template <int NP>
struct RowAt {
    static constexpr int U = NP / 4, kSize = kTile * U / 8 * 9 * 4;
    static __device__ __forceinline__ int at(int w, int q, int n) {
        const int more = U >= 8 ? (w * kStep + q) * (U / 8) : U == 4 ? w * (kStep / 2) + (q >> 1) : w;
        return ((w * kStep + q) * U + more + (n >> 2) + (U > 8 ? n >> 5 : 0)) * 4 + (n & 3);
    }
};
static_assert(kStep == 4, "RowAt");

// Sums over the lanes 2, 4, ... L / 2 apart of a channel pair's L, of kStep values each.  The lanes part the values among
// themselves: of two neighbouring positions' values a lane keeps one, then (from 8 lanes on) of the two pairs'.
template <int L>
struct Parts {
    static constexpr int kHeld = L >= 4 ? 2 : 4, kMine = L >= 8 ? 1 : kHeld;
    static __device__ __forceinline__ float either(float low, float high, int mask, int sub) {
        const bool upper = (sub & mask) != 0;
        return (upper ? high : low) + from_lane(upper ? low : high, mask);
    }
    static __device__ __forceinline__ void finish(float (&v)[kHeld], int sub) {
        if constexpr (L >= 8) v[0] = either(v[0], v[1], 4, sub);
#pragma unroll
        for (int m = 8; m < L; m *= 2) v[0] += from_lane(v[0], m);
    }
    // position of a lane's i-th value
    static __device__ __forceinline__ int position(int i, int sub) {
        return L < 4 ? i : (L >= 8 ? (sub >> 1 & 2) : 2 * i) + (sub >> 1 & 1);
    }
    static __device__ __forceinline__ bool owner(int sub) { return L <= 8 || sub < 8; }      // (others hold copies)
};

// Index among `saved` of the state in front of tile `tile` of a sequence.
__device__ __forceinline__ long long saved_slot(const Seqs& q, const Piece& r, long long tile) {
    if (q.offsets != nullptr) return r.base / kScanTile + r.s + tile;
    const long long n = q.length == 0 ? 1 : (q.length + kScanTile - 1) / kScanTile;
    return r.s * n + tile;
}

// What a CTA works on: `channels` channels of one group from `c`, of which `width` exist.
struct Block {
    int g, c, width;
};
__device__ __forceinline__ Block block_of(const Scan& p, int block, int channels) {
    const int per = p.C / p.G, blocks = (per + channels - 1) / channels;
    Block b;
    b.g = block / blocks;
    const int at = (block - b.g * blocks) * channels;
    b.c = b.g * per + at;
    b.width = min(channels, per - at);
    return b;
}

// B or C of a tile: vectors of 8 states, padded with zeros.
template <typename T, int NP, int kThreads>
struct StateRows {
    static constexpr int kRows = kTile, kVecs = NP / 8, kEach = (kRows * kVecs + kThreads - 1) / kThreads;
    Vec8<T> raw[kEach];
    __device__ __forceinline__ void fetch(const T* base, const RowsView& v, long long t0, long long end, int N) {
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int i = threadIdx.x + k * kThreads, t = i / kVecs, col = i % kVecs * 8;
            if (i < kRows * kVecs && t0 + t < end) load8(raw[k], base + (t0 + t) * v.row + col, N - col, v.vec && N % 8 == 0 && col < N);
            else raw[k].zero();
        }
    }
    // each four states in 1, 2 or 4 orders: n, n ^ 2 (two orders); n, n ^ 1, n ^ 2, n ^ 3 (four)
    template <int kOrders>
    __device__ __forceinline__ void spread(float* to) const {
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int i = threadIdx.x + k * kThreads;
            if (i >= kRows * kVecs) continue;
            float2 f[4];
            raw[k].widen(f);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                float* at = to + RowAt<NP>::at(i / kVecs / kStep, i / kVecs % kStep, i % kVecs * 8 + 4 * q);
                const float v[4] = {f[2 * q].x, f[2 * q].y, f[2 * q + 1].x, f[2 * q + 1].y};
#pragma unroll
                for (int o = 0; o < kOrders; ++o) {
                    const int m = kOrders == 2 ? 2 * o : o;
                    *reinterpret_cast<float4*>(at + o * RowAt<NP>::kSize) = make_float4(v[m], v[1 ^ m], v[2 ^ m], v[3 ^ m]);
                }
            }
        }
    }
};

// A log2(e), kept finite: no decay is 0 times infinity.  Positions past a sequence's end, whose delta is 0, leave every state
// alone, and a state that keeps nothing (A of minus infinity, or past -2.36e38, whose product is infinite) has derivatives of 0.
// (A NaN stays one.)
__device__ __forceinline__ float rate_of(float a) {
    float v;
    asm("min.NaN.f32 %0, %1, 0f7F7FFFFF;\n\tmax.NaN.f32 %0, %0, 0fFF7FFFFF;" : "=f"(v) : "f"(a * kLog2e));
    return v;
}

// Values of four states in a lane's order (n ^ perm).
struct Four {
    float2 v[2];
    // (`four`: the number of states is a multiple of 4 and the array aligned to 16 bytes)
    __device__ __forceinline__ void get4(const float* from, int n0, int perm, int states, bool four) {
        if (!four) {
            get(from, n0, perm, states);
            return;
        }
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
        if (from != nullptr && n0 < states) f = *reinterpret_cast<const float4*>(from + n0);
        if (perm & 2) f = make_float4(f.z, f.w, f.x, f.y);
        if (perm & 1) f = make_float4(f.y, f.x, f.w, f.z);
        v[0] = make_float2(f.x, f.y), v[1] = make_float2(f.z, f.w);
    }
    // (in the states' own order)
    __device__ __forceinline__ void put4(float* to, int n0, int states, bool four) const {
        if (!four) put(to, n0, 0, states);
        else if (n0 < states) *reinterpret_cast<float4*>(to + n0) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    }
    __device__ __forceinline__ void get(const float* from, int n0, int perm, int states) {
        float f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = n0 + (i ^ perm);
            f[i] = from != nullptr && n < states ? from[n] : 0.f;
        }
        v[0] = make_float2(f[0], f[1]), v[1] = make_float2(f[2], f[3]);
    }
    __device__ __forceinline__ void put(float* to, int n0, int perm, int states) const {
        const float f[4] = {v[0].x, v[0].y, v[1].x, v[1].y};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = n0 + (i ^ perm);
            if (n < states) to[n] = f[i];
        }
    }
    __device__ __forceinline__ void load(const float* from) {
        const float4 f = *reinterpret_cast<const float4*>(from);
        v[0] = make_float2(f.x, f.y), v[1] = make_float2(f.z, f.w);
    }
    __device__ __forceinline__ void to_rates() {
#pragma unroll
        for (int i = 0; i < 2; ++i) v[i] = make_float2(rate_of(v[i].x), rate_of(v[i].y));
    }
    __device__ __forceinline__ void clear() { v[0] = v[1] = both(0.f); }
};

// exp(delta A) of two states, from their rates
__device__ __forceinline__ float2 decay_of(float delta, float2 a2) {
    const float2 e = __fmul2_rn(both(delta), a2);
    return make_float2(exp2_fast(e.x), exp2_fast(e.y));
}

// delta of two channels, and its derivative by dt
__device__ __forceinline__ float2 delta_of(float2 raw, float2 bias, bool plus, bool in, float2* slope = nullptr) {
    const float2 v = __fadd2_rn(raw, bias);
    if (slope != nullptr) *slope = both(1.f);
    const float2 d = plus ? softplus2(v, slope) : v;
    return in ? d : both(0.f);      // positions past the end leave the states alone
}

// -------------------------------------------------------------------------------- forward

template <int L>
struct FwdShape {
    // (small CTAs spread evenly: 8 sequences of 4096 channels are 1024 CTAs of 64 threads, about 7 to an SM)
    static constexpr int kThreads = L == 32 ? 128 : 64, kResident = 640 / kThreads;       // CTAs to an SM: 96 registers a thread
    static constexpr int kChannels = 2 * kThreads / L, NP = 4 * L;
};

// Sequences that are too few to fill the GPU are cut into chunks of p.span positions.  kStates: the first of
// three kernels, which walks every chunk but a sequence's last from a state of zero and keeps the
// state at its end (`ends`, [slot][C][N]) and the sum of delta (`sums`, [slot][C]); the chunks are then joined,
// h = exp(A sum delta) h + end, and the second walk begins each chunk with the state in front of it.
template <typename T, int L, bool kStates>
__global__ void __launch_bounds__(FwdShape<L>::kThreads, FwdShape<L>::kResident) scan_fwd_kernel(Scan p, int blocks, float* ends, float* sums) {
    using S = FwdShape<L>;
    constexpr int kThreads = S::kThreads, kChannels = S::kChannels, kColumns = kChannels / 8, NP = S::NP, W = 32 / L;
    constexpr int kEach = (kTile * kColumns + kThreads - 1) / kThreads;      // vectors of a tile to a thread
    using Step = StepAt<kChannels>;
    using Value = ValueAt<kChannels>;
    using Row = RowAt<NP>;
    __shared__ __align__(16) float2 step[Step::kSize];    // delta, u
    __shared__ __align__(16) float bs[Row::kSize], cs[kStates ? 4 : Row::kSize], ys[kStates ? 4 : Value::kSize];
    __shared__ __align__(16) float bias[kChannels], skip[kChannels];
    pdl_trigger();
    pdl_wait();
    const long long slot = blockIdx.x / blocks;
    const Block k = block_of(p, static_cast<int>(blockIdx.x - slot * blocks), kChannels);
    const Piece r = find_piece(p.seqs, slot, p.span);
    if (!r.some || (kStates && r.last)) return;
    const int C = p.C, N = p.N;
    const T *u = view_at<T>(p.u, p.seqs, r) + k.c, *dt = view_at<T>(p.dt, p.seqs, r) + k.c;
    const T* z = kStates || p.z.p == nullptr ? nullptr : view_at<T>(p.z, p.seqs, r) + k.c;
    const T *b = view_at<T>(p.b, p.seqs, r) + k.g * N, *c = view_at<T>(p.c, p.seqs, r) + k.g * N;
    T* y = static_cast<T*>(p.y) + dense_row(p.seqs, r) * C + k.c;
    const bool even = (C / p.G) % 8 == 0, four = N % 4 == 0 && reinterpret_cast<uintptr_t>(p.saved) % 16 == 0;
    for (int i = threadIdx.x; i < kChannels; i += kThreads) {
        bias[i] = i < k.width && p.dt_bias != nullptr ? p.dt_bias[k.c + i] : 0.f;
        skip[i] = i < k.width && p.D != nullptr ? p.D[k.c + i] : 0.f;
    }
    // this lane's channels within the block (odd lanes hold them the other way round) and states
    const int lane = threadIdx.x & 31, sub = lane % L, n0 = sub * 4;
    const int pair = (static_cast<int>(threadIdx.x >> 5) * W + lane / L) * 2;
    const int ch[2] = {pair + (sub & 1), pair + 1 - (sub & 1)};
    const long long wide = static_cast<long long>(C) * N;
    Four a2[2], h[2];
    float total[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const bool serves = ch[j] < k.width;
        const long long at = static_cast<long long>(k.c + ch[j]) * N;
        a2[j].get(serves ? p.A + at : nullptr, n0, 0, N);
        a2[j].to_rates();
        if (kStates) h[j].clear();
        else if (ends != nullptr) h[j].get(serves ? ends + slot * wide + at : nullptr, n0, 0, N);
        else h[j].get(serves && p.state != nullptr ? p.state + r.s * wide + at : nullptr, n0, 0, N);
    }

    Vec8<T> ru[kEach], rz[kEach], rdt[kEach];
    StateRows<T, NP, kThreads> rb, rc;
    const auto row_of = [](int i) { return (static_cast<int>(threadIdx.x) + i * kThreads) / kColumns; };
    const int col = threadIdx.x % kColumns * 8, left = k.width - col;            // (kColumns divides the threads)
    const bool vec_u = p.u.vec && even && left >= 8, vec_dt = p.dt.vec && even && left >= 8, vec_z = p.z.vec && even && left >= 8;
    const bool vec_y = even && left >= 8 && reinterpret_cast<uintptr_t>(p.y) % (8 * sizeof(T)) == 0;
    auto fetch = [&](long long t0) {
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int row = row_of(i);
            ru[i].zero(), rdt[i].zero();
            if (row >= kTile || t0 + row >= r.end) continue;
            load8(ru[i], u + (t0 + row) * p.u.row + col, left, vec_u);
            load8(rdt[i], dt + (t0 + row) * p.dt.row + col, left, vec_dt);
        }
        rb.fetch(b, p.b, t0, r.end, N);
        if (!kStates) rc.fetch(c, p.c, t0, r.end, N);
    };
    fetch(r.first);
    __syncthreads();
    for (long long t0 = r.first; t0 < r.end; t0 += kTile) {
        Vec8<T> keep[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int row = row_of(i);
            keep[i] = ru[i];
            if (row >= kTile) continue;
            float2 fu[4], fd[4];
            ru[i].widen(fu);
            rdt[i].widen(fd);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 d = delta_of(fd[j], *reinterpret_cast<const float2*>(&bias[col + 2 * j]), p.softplus, t0 + row < r.end);
                *reinterpret_cast<float4*>(&step[Step::at(row, col + 2 * j)]) = make_float4(d.x, fu[j].x, d.y, fu[j].y);
            }
        }
        rb.template spread<1>(bs);
        if constexpr (!kStates) rc.template spread<1>(cs);
        __syncthreads();
        if constexpr (!kStates) {
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                rz[i].zero();
                if (z != nullptr && row_of(i) < kTile && t0 + row_of(i) < r.end)
                    load8(rz[i], z + (t0 + row_of(i)) * p.z.row + col, left, vec_z);
            }
            if (p.saved != nullptr) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    if (ch[j] < k.width)
                        h[j].put4(p.saved + saved_slot(p.seqs, r, t0 / kScanTile) * wide + static_cast<long long>(k.c + ch[j]) * N, n0, N, four);
            }
        }
        if (t0 + kTile < r.end) fetch(t0 + kTile);
#pragma unroll
        for (int t = 0; t < kTile; t += kStep) {
            // (decays and inputs of all four positions first: they wait for nothing, the states only for them)
            float part[Parts<L>::kHeld], last = 0.f, in[kStep][2];
            float2 a[kStep][2][2];
#pragma unroll
            for (int q = 0; q < kStep; ++q)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float2 s = step[Step::at(t + q, ch[j])];
                    in[q][j] = s.x * s.y;
                    if (kStates) total[j] += s.x;
#pragma unroll
                    for (int i = 0; i < 2; ++i) a[q][j][i] = decay_of(s.x, a2[j].v[i]);
                }
#pragma unroll
            for (int q = 0; q < kStep; ++q) {
                Four fb, fc;
                fb.load(&bs[Row::at(t / kStep, q, n0)]);
                if constexpr (!kStates) fc.load(&cs[Row::at(t / kStep, q, n0)]);
                float sum[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float2 x = both(0.f);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        h[j].v[i] = __ffma2_rn(both(in[q][j]), fb.v[i], __fmul2_rn(a[q][j][i], h[j].v[i]));
                        if constexpr (!kStates) x = __ffma2_rn(fc.v[i], h[j].v[i], x);
                    }
                    sum[j] = x.x + x.y;
                }
                if constexpr (!kStates) {
                    // (the partner's other channel is this lane's first)
                    const float v = sum[0] + from_lane(sum[1], 1);
                    if constexpr (L < 4) part[q] = v;
                    else if (q % 2 == 0) last = v;
                    else part[q / 2] = Parts<L>::either(last, v, 2, sub);
                }
            }
            if constexpr (!kStates) {
                Parts<L>::finish(part, sub);
                if (Parts<L>::owner(sub)) {
#pragma unroll
                    for (int i = 0; i < Parts<L>::kMine; ++i) ys[Value::at(t + Parts<L>::position(i, sub), ch[0])] = part[i];
                }
            }
        }
        __syncthreads();
        if constexpr (!kStates) {
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int row = row_of(i);
                if (row >= kTile || t0 + row >= r.end || col >= k.width) continue;
                float2 fu[4], fz[4], f[4];
                keep[i].widen(fu);
                rz[i].widen(fz);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 o = *reinterpret_cast<const float2*>(&skip[col + 2 * j]);
                    f[j] = __ffma2_rn(o, fu[j], *reinterpret_cast<const float2*>(&ys[Value::at(row, col + 2 * j)]));
                    if (z != nullptr) f[j] = __fmul2_rn(f[j], silu2(fz[j]));
                }
                store8(y + (t0 + row) * C + col, f, left, vec_y);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if (ch[j] >= k.width) continue;
        const long long at = static_cast<long long>(k.c + ch[j]) * N;
        if (kStates) {
            h[j].put(ends + slot * wide + at, n0, 0, N);
            if (sub == 0) sums[slot * C + k.c + ch[j]] = total[j];
        } else if (r.last && p.final_state != nullptr) {
            h[j].put(p.final_state + r.s * wide + at, n0, 0, N);
        }
    }
}

// What a chunk leaves of the state in front of it, 2^x (x: the sum of delta times the rate), as two factors: 2^x may leave fp32's
// range where its product with a state does not.  Past 2^+-120 each is the root, the growing one (A > 0, delta < 0) held to 2^127,
// so that a state of zero stays zero however much it would grow and every other normal one is infinite past 2^254.
// (Factors, since they do not wait for the state: a test of it in between cost packed sequences 6 us of 203.)
__device__ __forceinline__ float2 chunk_factors(float x) {
    const bool far = fabsf(x) > 120.f;
    const float f = exp2_fast(far ? fminf(0.5f * x, 127.f) : x);
    return make_float2(f, far ? f : 1.f);
}

// The states in front of every chunk, in place of those at their ends: a thread per sequence, channel and state.
// Eight chunks' values are on their way together.
template <bool kBackward>
__global__ void __launch_bounds__(256) scan_join_kernel(Scan p, float* ends, const float* sums, const float* from) {
    pdl_trigger();
    pdl_wait();
    const int C = p.C, N = p.N;
    const long long width = static_cast<long long>(C) * N, i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    const int s = static_cast<int>(i / width);
    if (s >= p.seqs.count) return;
    const long long j = i - s * width, c = j / N;
    long long first, n;          // the sequence's slots
    if (p.seqs.offsets != nullptr) {
        const long long at = seq_offset(p.seqs, s), end = seq_offset(p.seqs, s + 1);
        first = at / p.span + s;
        n = end > at ? (end - at + p.span - 1) / p.span : 1;
    } else {
        n = p.seqs.length == 0 ? 1 : (p.seqs.length + p.span - 1) / p.span;
        first = s * n;
    }
    const float a2 = rate_of(p.A[j]);
    float h = from != nullptr ? from[i] : 0.f;
    constexpr int U = 8;
    for (long long k = 0; k < n; k += U) {
        float e[U];
        float2 f[U];
#pragma unroll
        for (int q = 0; q < U; ++q) {
            // (the last chunk's end is not needed, nor formed)
            const bool in = k + q < n - 1;
            const long long slot = first + (kBackward ? n - 1 - k - q : k + q);
            e[q] = in ? ends[slot * width + j] : 0.f;
            f[q].x = in ? sums[slot * C + c] : 0.f;
        }
#pragma unroll
        for (int q = 0; q < U; ++q) f[q] = chunk_factors(f[q].x * a2);
#pragma unroll
        for (int q = 0; q < U; ++q) {
            if (k + q >= n) break;
            const long long slot = first + (kBackward ? n - 1 - k - q : k + q);
            ends[slot * width + j] = h;
            h = fmaf(f[q].x, f[q].y * h, e[q]);
        }
    }
}

// ------------------------------------------------------------------------------- backward

// The first of the backward pass's kernels where sequences are cut into chunks: what reaches the
// position in front of a chunk from within it, dh = g C + carry, carry = exp(delta A) dh (`ends`), and the sum
// of delta.  Every chunk but a sequence's first is walked, from its end.
template <typename T, int L>
__global__ void __launch_bounds__(FwdShape<L>::kThreads, FwdShape<L>::kResident) scan_adjoint_kernel(Scan p, int blocks, float* ends, float* sums) {
    using S = FwdShape<L>;
    constexpr int kThreads = S::kThreads, kChannels = S::kChannels, kColumns = kChannels / 8, NP = S::NP, W = 32 / L;
    constexpr int kEach = (kTile * kColumns + kThreads - 1) / kThreads;
    using Step = StepAt<kChannels>;
    using Row = RowAt<NP>;
    __shared__ __align__(16) float2 step[Step::kSize];    // delta, g
    __shared__ __align__(16) float cs[Row::kSize];
    __shared__ __align__(16) float bias[kChannels];
    pdl_trigger();
    pdl_wait();
    const long long slot = blockIdx.x / blocks;
    const Block k = block_of(p, static_cast<int>(blockIdx.x - slot * blocks), kChannels);
    const Piece r = find_piece(p.seqs, slot, p.span);
    if (!r.some || r.index == 0) return;
    const int C = p.C, N = p.N;
    const T *dt = view_at<T>(p.dt, p.seqs, r) + k.c, *dy = view_at<T>(p.dy, p.seqs, r) + k.c;
    const T* z = p.z.p == nullptr ? nullptr : view_at<T>(p.z, p.seqs, r) + k.c;
    const T* c = view_at<T>(p.c, p.seqs, r) + k.g * N;
    const bool even = (C / p.G) % 8 == 0;
    for (int i = threadIdx.x; i < kChannels; i += kThreads)
        bias[i] = i < k.width && p.dt_bias != nullptr ? p.dt_bias[k.c + i] : 0.f;
    const int lane = threadIdx.x & 31, sub = lane % L, n0 = sub * 4;
    const int ch = (static_cast<int>(threadIdx.x >> 5) * W + lane / L) * 2;
    Four a2[2], carry[2];
    float total[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        a2[j].get(ch + j < k.width ? p.A + static_cast<long long>(k.c + ch + j) * N : nullptr, n0, 0, N);
        a2[j].to_rates();
        carry[j].clear();
    }
    const auto row_of = [](int i) { return (static_cast<int>(threadIdx.x) + i * kThreads) / kColumns; };
    const int col = threadIdx.x % kColumns * 8, left = k.width - col;
    const bool vec_dt = p.dt.vec && even && left >= 8, vec_dy = p.dy.vec && even && left >= 8, vec_z = p.z.vec && even && left >= 8;
    Vec8<T> rdt[kEach], rdy[kEach], rz[kEach];
    StateRows<T, NP, kThreads> rc;
    auto fetch = [&](long long t0) {
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int row = row_of(i);
            rdt[i].zero(), rdy[i].zero(), rz[i].zero();
            if (row >= kTile || t0 + row >= r.end) continue;
            load8(rdt[i], dt + (t0 + row) * p.dt.row + col, left, vec_dt);
            load8(rdy[i], dy + (t0 + row) * p.dy.row + col, left, vec_dy);
            if (z != nullptr) load8(rz[i], z + (t0 + row) * p.z.row + col, left, vec_z);
        }
        rc.fetch(c, p.c, t0, r.end, N);
    };
    const long long tiles = (r.end - r.first + kTile - 1) / kTile;
    fetch(r.first + (tiles - 1) * kTile);
    for (long long tile = tiles - 1; tile >= 0; --tile) {
        const long long t0 = r.first + tile * kTile;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int row = row_of(i);
            if (row >= kTile) continue;
            float2 fd[4], fy[4], fz[4];
            rdt[i].widen(fd);
            rdy[i].widen(fy);
            rz[i].widen(fz);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 d = delta_of(fd[j], *reinterpret_cast<const float2*>(&bias[col + 2 * j]), p.softplus, t0 + row < r.end);
                if (z != nullptr) fy[j] = __fmul2_rn(fy[j], silu2(fz[j]));
                *reinterpret_cast<float4*>(&step[Step::at(row, col + 2 * j)]) = make_float4(d.x, fy[j].x, d.y, fy[j].y);
            }
        }
        rc.template spread<1>(cs);
        __syncthreads();
        if (tile > 0) fetch(t0 - kTile);
#pragma unroll 4
        for (int t = kTile - 1; t >= 0; --t) {
            Four fc;
            fc.load(&cs[Row::at(t / kStep, t % kStep, n0)]);
            const float4 s = *reinterpret_cast<const float4*>(&step[Step::at(t, ch)]);
            const float delta[2] = {s.x, s.z}, g[2] = {s.y, s.w};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    carry[j].v[i] = __fmul2_rn(decay_of(delta[j], a2[j].v[i]), __ffma2_rn(both(g[j]), fc.v[i], carry[j].v[i]));
                total[j] += delta[j];
            }
        }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if (ch + j >= k.width) continue;
        carry[j].put(ends + (slot * C + k.c + ch + j) * N, n0, 0, N);
        if (sub == 0) sums[slot * C + k.c + ch + j] = total[j];
    }
}

// Tiles of 16 positions from the last to the first.  From the state in front of a tile (kept by the
// forward pass) the states in front of every 4th position are formed again (`front`); then, 4 positions
// at a time from the last, a h[t-1] and a of each, in registers, and the gradients going back:
//     dh = g C + carry,  carry = a dh  (g: the gradient of the sum over the states and D u)
//     dC = sum_c g h,  dB = sum_c dh delta u,  dA += dh a h[t-1] delta
//     into = sum_n dh B,  decay = sum_n dh a h[t-1] A,  du = into delta + D g,  ddelta = into u + decay
// Bound by the instructions and their latency (27 a state and position, at 0.55 a cycle with three to four warps a
// scheduler; shared memory hands out values in 60 % of the cycles): 10 packed operations on a pair of states going back, 1.75
// times 3 and two exponentials to form the states again, the rest exchanges between lanes, register pairs for
// scalars and what each position and channel takes once.  So a lane has two channels and four states of each: dB and dC are added over its channels before they leave it, and lanes part the sums
// among themselves without selecting what to send.  For that a lane holds its four states in the
// order n ^ perm, so that the upper pair is always what the partner keeps (B and C lie in shared
// memory in each of the orders), and odd lanes hold their two channels the other way round.
template <int L>
struct BwdShape {
    static constexpr int kLanes = 32 / L;                  // lanes of a warp that share states
    static constexpr int kOrders = kLanes >= 4 ? 4 : kLanes;
    // (small CTAs, seven to an SM at 128 registers a thread: 8 sequences of 4096 channels are 1024 of them, one round of 1064;
    // of 128 threads they were 512, three or four to an SM, and took a quarter longer)
    static constexpr int kThreads = L == 32 ? 128 : 64, kResident = L == 32 ? 3 : 7;
    static constexpr int kChannels = 2 * kThreads / L, NP = 4 * L, kWarps = kThreads / 32;
    static constexpr int kColumns = kChannels / 8, kEach = (kTile * kColumns + kThreads - 1) / kThreads;
    // dB and dC of kStep positions take the place of the states in front of them where they fit
    static constexpr bool kShared = kStep * 2 * NP <= 8 * 32;
    static constexpr size_t kFloats = 2 * StepAt<kChannels>::kSize + ValueAt<kChannels>::kSize + 2 * kOrders * RowAt<NP>::kSize + kTile / kStep * 8 * kThreads +
                                      (kShared ? 0 : kWarps * kTile * 2 * NP) + 2 * kChannels + 8 * kThreads + kEach * 16 * kThreads;
    // place of dB (0) or dC (1) of position t and state n among `front` or the sums
    static __device__ __forceinline__ int place(int warp, int t, int which, int n) {
        if constexpr (kShared) {
            const int at = (t % kStep * 2 + which) * NP + n;
            return (t / kStep * 8 + at / 32) * kThreads + warp * 32 + at % 32;
        }
        return ((warp * kTile + t) * 2 + which) * NP + n;
    }
};

// Of the pieces those that one launch works on: the first row of each is one of `from` .. `to` - 1, their slots begin with
// `slot`, and `rows` rows from `from` on have partial rows of dB and dC.
struct Window {
    long long from, to, slot, rows;
    __device__ __forceinline__ bool has(const Seqs& q, const Piece& r) const {
        const long long row = dense_row(q, r) + r.first;
        return row >= from && row < to;
    }
};

template <typename T, int L>
__global__ void __launch_bounds__(BwdShape<L>::kThreads, BwdShape<L>::kResident)
    scan_bwd_kernel(Scan p, int blocks, Window window, const float* carries, float* part_bc, float* part_p) {
    using S = BwdShape<L>;
    constexpr int kThreads = S::kThreads, kChannels = S::kChannels, kColumns = S::kColumns, NP = S::NP, W = S::kLanes;
    constexpr int kOrders = S::kOrders, kEach = S::kEach;
    extern __shared__ __align__(16) float smem[];
    using Step = StepAt<kChannels>;
    using Value = ValueAt<kChannels>;
    using Row = RowAt<NP>;
    float2* const step = reinterpret_cast<float2*>(smem);      // delta, u; then du, ddelta
    float* const bs = smem + 2 * Step::kSize;                  // in each order
    float* const cs = bs + kOrders * Row::kSize;
    float* front = cs + kOrders * Row::kSize;
    float* sums = S::kShared ? front : front + kTile / kStep * 8 * kThreads;       // dB and dC of every warp
    float* bias = front + kTile / kStep * 8 * kThreads + (S::kShared ? 0 : S::kWarps * kTile * 2 * NP);
    float* skip = bias + kChannels;
    float4* sum_bias = reinterpret_cast<float4*>(skip + kChannels) + threadIdx.x;         // (two of them, kThreads apart)
    // of this thread's vectors the derivatives of delta by dt, and dy silu'(z)
    float4* stash = reinterpret_cast<float4*>(skip + kChannels + 8 * kThreads) + threadIdx.x;
    float* const gs = skip + kChannels + 8 * kThreads + kEach * 16 * kThreads;   // g; then the sum over the states and D u
    front += threadIdx.x;
    pdl_trigger();
    pdl_wait();
    const long long slot = blockIdx.x / blocks;          // (of the window's)
    const int block = static_cast<int>(blockIdx.x - slot * blocks);
    Block k = block_of(p, block, kChannels);
    Piece r = find_piece(p.seqs, window.slot + slot, p.span);
    // (a piece of another launch's: nothing to walk or to write)
    if (r.some && !window.has(p.seqs, r)) k.width = 0, r.some = false;
    const int C = p.C, N = p.N;
    const bool even = (C / p.G) % 8 == 0;
    const long long dense = r.some ? dense_row(p.seqs, r) : 0;
    // (where the tensors begin: in shared memory, since registers are what the walk has too few of, and spilled ones come
    // back from L2, which the shared memory leaves no L1 in front of)
    __shared__ struct {
        const T *u, *dt, *z, *dy, *b, *c;
        T *du, *ddt, *dz;
        float* rows;
        const float* saved;
    } at_;
    const bool gated = p.z.p != nullptr;
    if (threadIdx.x == 0) {
        at_.u = view_at<T>(p.u, p.seqs, r) + k.c;
        at_.dt = view_at<T>(p.dt, p.seqs, r) + k.c;
        at_.z = gated ? view_at<T>(p.z, p.seqs, r) + k.c : nullptr;
        at_.dy = view_at<T>(p.dy, p.seqs, r) + k.c;
        at_.b = view_at<T>(p.b, p.seqs, r) + k.g * N;
        at_.c = view_at<T>(p.c, p.seqs, r) + k.g * N;
        const long long o = dense * C + k.c;
        at_.du = static_cast<T*>(p.du) + o;
        at_.ddt = static_cast<T*>(p.ddt) + o;
        at_.dz = static_cast<T*>(p.dz) + o;
        at_.rows = part_bc + (block * window.rows + dense - window.from) * 2 * N;
        at_.saved = p.saved + (saved_slot(p.seqs, r, 0) * C + k.c) * N;
    }
    __syncthreads();
    const volatile auto& at = at_;
    for (int i = threadIdx.x; i < kChannels; i += kThreads) {
        bias[i] = i < k.width && p.dt_bias != nullptr ? p.dt_bias[k.c + i] : 0.f;
        skip[i] = i < k.width && p.D != nullptr ? p.D[k.c + i] : 0.f;
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % L, cl = lane / L, n0 = sub * 4;
    const int perm = (W >= 2 && (cl & (W / 2)) ? 2 : 0) | (W >= 4 && (cl & (W / 4)) ? 1 : 0);
    const int order = W >= 4 ? perm : perm >> 1;
    // this lane's channels within the block
    const int pair = (warp * W + cl) * 2;
    const int ch[2] = {pair + (sub & 1), pair + 1 - (sub & 1)};
    Four a2[2], da[2], carry[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const bool serves = ch[j] < k.width;
        const long long mine = static_cast<long long>(k.c + ch[j]) * N, wide = static_cast<long long>(C) * N;
        a2[j].get(serves ? p.A + mine : nullptr, n0, perm, N);
        a2[j].to_rates();
        da[j].clear();
        if (carries != nullptr) carry[j].get(serves && r.some ? carries + slot * wide + mine : nullptr, n0, perm, N);
        else carry[j].get(serves && r.some && p.dfinal != nullptr ? p.dfinal + r.s * wide + mine : nullptr, n0, perm, N);
    }
    float sum_d = 0.f;
    sum_bias[0] = sum_bias[kThreads] = make_float4(0.f, 0.f, 0.f, 0.f);
    const auto row_of = [](int i) { return (static_cast<int>(threadIdx.x) + i * kThreads) / kColumns; };
    const int col = threadIdx.x % kColumns * 8, left = k.width - col;            // (kColumns divides the threads)
    const bool eight = even && left >= 8, four = N % 4 == 0 && reinterpret_cast<uintptr_t>(p.saved) % 16 == 0;
    const auto aligned = [&](const void* t) { return eight && reinterpret_cast<uintptr_t>(t) % (8 * sizeof(T)) == 0; };
    // whether this thread's vectors take one access each: u, dt, z, dy, du, ddt, dz
    const unsigned whole = (p.u.vec && eight ? 1u : 0u) | (p.dt.vec && eight ? 2u : 0u) | (p.z.vec && eight ? 4u : 0u) |
                           (p.dy.vec && eight ? 8u : 0u) | (aligned(p.du) ? 16u : 0u) | (aligned(p.ddt) ? 32u : 0u) |
                           (aligned(p.dz) ? 64u : 0u);

    // (positions are 32-bit numbers)
    const int begin = static_cast<int>(r.first), end = r.some ? static_cast<int>(r.end) : begin;
    for (int t0 = begin + (end - begin - 1) / kTile * kTile; t0 >= begin && t0 < end; t0 -= kTile) {
        Vec8<T> ru[kEach], rdt[kEach], rz[kEach], rdy[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int row = row_of(i);
            ru[i].zero(), rdt[i].zero(), rz[i].zero(), rdy[i].zero();
            if (row >= kTile || left <= 0) continue;
            const long long t = t0 + row;
            if (t < end) {
                load8(ru[i], at.u + t * p.u.row + col, left, (whole & 1) != 0);
                load8(rdt[i], at.dt + t * p.dt.row + col, left, (whole & 2) != 0);
                load8(rdy[i], at.dy + t * p.dy.row + col, left, (whole & 8) != 0);
                if (gated) load8(rz[i], at.z + t * p.z.row + col, left, (whole & 4) != 0);
            }
            if (t0 > begin) {         // (the tile in front of this one: a whole one)
                prefetch_l2(at.u + (t - kTile) * p.u.row + col);
                prefetch_l2(at.dt + (t - kTile) * p.dt.row + col);
                prefetch_l2(at.dy + (t - kTile) * p.dy.row + col);
                if (gated) prefetch_l2(at.z + (t - kTile) * p.z.row + col);
            }
        }
        StateRows<T, NP, kThreads> rb, rc;
        rb.fetch(at.b, p.b, t0, end, N);
        rc.fetch(at.c, p.c, t0, end, N);
        Four h[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float* from = at.saved + (static_cast<long long>(t0 / kScanTile) * C + ch[j]) * N;
            h[j].get4(ch[j] < k.width ? from : nullptr, n0, perm, N, four);
            if (t0 > begin && ch[j] < k.width && n0 < N) prefetch_l2(from - static_cast<long long>(C) * N + n0);
        }
        __syncthreads();            // the last tile's sums have been read
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int row = row_of(i);
            if (row >= kTile) continue;
            float2 fu[4], fd[4], fz[4], fy[4];
            ru[i].widen(fu);
            rdt[i].widen(fd);
            rz[i].widen(fz);
            rdy[i].widen(fy);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float2 slope;
                const float2 d = delta_of(fd[j], *reinterpret_cast<const float2*>(&bias[col + 2 * j]), p.softplus, t0 + row < end, &slope);
                fd[j] = slope;
                if (gated) {
                    const float2 s = sigmoid2(fz[j]), zs = __fmul2_rn(fz[j], s);
                    fz[j] = __fmul2_rn(fy[j], __fadd2_rn(s, __ffma2_rn(zs, make_float2(-s.x, -s.y), zs)));
                    fy[j] = __fmul2_rn(fy[j], zs);
                }
                *reinterpret_cast<float4*>(&step[Step::at(row, col + 2 * j)]) = make_float4(d.x, fu[j].x, d.y, fu[j].y);
                *reinterpret_cast<float2*>(&gs[Value::at(row, col + 2 * j)]) = fy[j];
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                stash[(4 * i + j) * kThreads] = make_float4(fd[2 * j].x, fd[2 * j].y, fd[2 * j + 1].x, fd[2 * j + 1].y);
                stash[(4 * i + 2 + j) * kThreads] = make_float4(fz[2 * j].x, fz[2 * j].y, fz[2 * j + 1].x, fz[2 * j + 1].y);
            }
        }
        rb.template spread<kOrders>(bs);
        rc.template spread<kOrders>(cs);
        __syncthreads();
#pragma unroll 1
        for (int w = 0; w < kTile / kStep; ++w) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                front[(w * 8 + j * 4 + 0) * kThreads] = h[j].v[0].x, front[(w * 8 + j * 4 + 1) * kThreads] = h[j].v[0].y;
                front[(w * 8 + j * 4 + 2) * kThreads] = h[j].v[1].x, front[(w * 8 + j * 4 + 3) * kThreads] = h[j].v[1].y;
            }
            if (w == kTile / kStep - 1) break;
#pragma unroll
            for (int q = 0; q < kStep; ++q) {
                const int t = w * kStep + q;
                Four fb;
                fb.load(bs + (order * Row::kSize + Row::at(w, q, n0)));
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float2 s = step[Step::at(t, ch[j])];
                    const float in = s.x * s.y;
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        h[j].v[i] = __ffma2_rn(both(in), fb.v[i], __fmul2_rn(decay_of(s.x, a2[j].v[i]), h[j].v[i]));
                }
            }
        }
#pragma unroll 1
        for (int w = kTile / kStep - 1; w >= 0; --w) {
            float2 held[kStep][2][2], decay[kStep][2][2];       // a h[t-1], a
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                h[j].v[0] = make_float2(front[(w * 8 + j * 4 + 0) * kThreads], front[(w * 8 + j * 4 + 1) * kThreads]);
                h[j].v[1] = make_float2(front[(w * 8 + j * 4 + 2) * kThreads], front[(w * 8 + j * 4 + 3) * kThreads]);
            }
            __syncwarp();       // (their place is taken by dB and dC)
#pragma unroll
            for (int q = 0; q < kStep; ++q) {
                const int t = w * kStep + q;
                Four fb;
                fb.load(bs + (order * Row::kSize + Row::at(w, q, n0)));
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float2 s = step[Step::at(t, ch[j])];
                    const float in = s.x * s.y;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        decay[q][j][i] = decay_of(s.x, a2[j].v[i]);
                        held[q][j][i] = __fmul2_rn(decay[q][j][i], h[j].v[i]);
                        if (q + 1 < kStep) h[j].v[i] = __ffma2_rn(both(in), fb.v[i], held[q][j][i]);
                    }
                }
            }
            float into[Parts<L>::kHeld], decays[Parts<L>::kHeld], ys[Parts<L>::kHeld], last[3];
#pragma unroll
            for (int q = kStep - 1; q >= 0; --q) {
                const int t = w * kStep + q;
                Four fb, fc;
                fb.load(bs + (order * Row::kSize + Row::at(w, q, n0)));
                fc.load(cs + (order * Row::kSize + Row::at(w, q, n0)));
                float2 vb[2] = {both(0.f), both(0.f)}, vc[2] = {both(0.f), both(0.f)};
                float s1[2], s2[2], s3[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float2 s = step[Step::at(t, ch[j])];
                    const float g = gs[Value::at(t, ch[j])], in = s.x * s.y;
                    float2 x1 = both(0.f), x2 = both(0.f), x3 = both(0.f);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 dh = __ffma2_rn(both(g), fc.v[i], carry[j].v[i]);
                        const float2 now = __ffma2_rn(both(in), fb.v[i], held[q][j][i]);
                        const float2 x = __fmul2_rn(dh, held[q][j][i]);
                        vb[i] = __ffma2_rn(dh, both(in), vb[i]);
                        vc[i] = __ffma2_rn(both(g), now, vc[i]);
                        x1 = __ffma2_rn(dh, fb.v[i], x1);
                        x2 = __ffma2_rn(x, a2[j].v[i], x2);
                        x3 = __ffma2_rn(fc.v[i], now, x3);
                        da[j].v[i] = __ffma2_rn(x, both(s.x), da[j].v[i]);
                        carry[j].v[i] = __fmul2_rn(dh, decay[q][j][i]);
                    }
                    s1[j] = x1.x + x1.y, s2[j] = x2.x + x2.y, s3[j] = x3.x + x3.y;
                }
                // over the states, first step: the partner's other channel is this lane's first
                const float x1 = s1[0] + from_lane(s1[1], 1), x2 = s2[0] + from_lane(s2[1], 1), x3 = s3[0] + from_lane(s3[1], 1);
                if constexpr (L < 4) {
                    into[q] = x1, decays[q] = x2, ys[q] = x3;
                } else if (q % 2 != 0) {
                    last[0] = x1, last[1] = x2, last[2] = x3;
                } else {
                    into[q / 2] = Parts<L>::either(x1, last[0], 2, sub);
                    decays[q / 2] = Parts<L>::either(x2, last[1], 2, sub);
                    ys[q / 2] = Parts<L>::either(x3, last[2], 2, sub);
                }
                // over the warp's channels
                if constexpr (W >= 2) {
                    vb[0] = make_float2(vb[0].x + from_lane(vb[1].x, W / 2 * L), vb[0].y + from_lane(vb[1].y, W / 2 * L));
                    vc[0] = make_float2(vc[0].x + from_lane(vc[1].x, W / 2 * L), vc[0].y + from_lane(vc[1].y, W / 2 * L));
                }
                if constexpr (W >= 4) {
                    vb[0].x += from_lane(vb[0].y, W / 4 * L);
                    vc[0].x += from_lane(vc[0].y, W / 4 * L);
                }
                const auto give = [&](int which, int n, float v) { sums[S::place(warp, t, which, n0 + n)] = v; };
                if constexpr (W >= 8) {
                    const bool which = (cl & (W / 8)) != 0;
                    float v = (which ? vc[0].x : vb[0].x) + from_lane(which ? vb[0].x : vc[0].x, W / 8 * L);
                    if constexpr (W >= 16) v += from_lane(v, W / 16 * L);
                    if (W < 16 || (cl & (W / 16)) == 0) give(which, perm, v);
                } else {
                    give(0, perm, vb[0].x), give(1, perm, vc[0].x);
                    if constexpr (W <= 2) give(0, 1 ^ perm, vb[0].y), give(1, 1 ^ perm, vc[0].y);
                    if constexpr (W == 1) {
                        give(0, 2, vb[1].x), give(0, 3, vb[1].y);
                        give(1, 2, vc[1].x), give(1, 3, vc[1].y);
                    }
                }
            }
            // over the states
            Parts<L>::finish(into, sub);
            Parts<L>::finish(decays, sub);
            Parts<L>::finish(ys, sub);
            __syncwarp();       // all lanes have read these positions
            if (Parts<L>::owner(sub)) {
#pragma unroll
                for (int q = 0; q < Parts<L>::kMine; ++q) {
                    const int t = w * kStep + Parts<L>::position(q, sub);
                    const float2 s = step[Step::at(t, ch[0])];
                    const float g = gs[Value::at(t, ch[0])];
                    sum_d = fmaf(g, s.y, sum_d);
                    step[Step::at(t, ch[0])] = make_float2(fmaf(into[q], s.x, skip[ch[0]] * g), fmaf(into[q], s.y, decays[q] * 0.6931471805599453f));
                    gs[Value::at(t, ch[0])] = fmaf(skip[ch[0]], s.y, ys[q]);
                }
            }
        }
        __syncthreads();
        // dB and dC of the CTA's channels
        float* rows = at.rows + static_cast<long long>(t0) * 2 * N;
        const int here = min(end - t0, kTile);
#pragma unroll
        for (int i = 0; i < kTile * 2 * NP / kThreads; ++i) {
            const int j = (threadIdx.x + i * kThreads) % (2 * NP), t = (threadIdx.x + i * kThreads) / (2 * NP), n = j % NP;
            if (n >= N || t >= here) continue;
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < S::kWarps; ++w) s += sums[S::place(w, t, j / NP, n)];
            rows[(2 * t + j / NP) * N + n] = s;
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int row = row_of(i);
            if (row >= kTile || t0 + row >= end || col >= k.width) continue;
            float2 du[4], ddt[4], dz[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float4 s = *reinterpret_cast<const float4*>(&step[Step::at(row, col + 2 * j)]);
                const float4 slope = stash[(4 * i + j / 2) * kThreads], z = stash[(4 * i + 2 + j / 2) * kThreads];
                du[j] = make_float2(s.x, s.z);
                ddt[j] = __fmul2_rn(make_float2(s.y, s.w), j % 2 ? make_float2(slope.z, slope.w) : make_float2(slope.x, slope.y));
                dz[j] = __fmul2_rn(j % 2 ? make_float2(z.z, z.w) : make_float2(z.x, z.y),
                                   *reinterpret_cast<const float2*>(&gs[Value::at(row, col + 2 * j)]));
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float4 s = sum_bias[j * kThreads];
                s.x += ddt[2 * j].x, s.y += ddt[2 * j].y, s.z += ddt[2 * j + 1].x, s.w += ddt[2 * j + 1].y;
                sum_bias[j * kThreads] = s;
            }
            const long long o = static_cast<long long>(t0 + row) * C + col;
            store8(at.du + o, du, left, (whole & 16) != 0);
            store8(at.ddt + o, ddt, left, (whole & 32) != 0);
            if (gated) store8(at.dz + o, dz, left, (whole & 64) != 0);
        }
    }
    // this chunk's rows of parameter gradients: C x N of dA, C of dD, C of the bias's
    float* part = part_p + slot * C * (N + 2);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        if (ch[j] >= k.width) continue;
        const long long at = static_cast<long long>(k.c + ch[j]) * N;
        if (r.some && r.index == 0 && p.dstate != nullptr) carry[j].put(p.dstate + static_cast<long long>(r.s) * C * N + at, n0, perm, N);
        da[j].put(part + at, n0, perm, N);
    }
    __syncthreads();
    // over the threads of a column, and over the lanes that had a channel first
    float* red = smem;
    constexpr int kRows = kThreads / kColumns;
    constexpr int kStride = kChannels + 4;      // (rows of 8 columns apart: fewer conflicts)
#pragma unroll
    for (int j = 0; j < 2; ++j)
        *reinterpret_cast<float4*>(&red[static_cast<int>(threadIdx.x) / kColumns * kStride + col + 4 * j]) = sum_bias[j * kThreads];
    __syncthreads();
    float* mine = part + static_cast<long long>(C) * N + k.c;
    for (int i = threadIdx.x; i < k.width; i += kThreads) {
        float s = 0.f;
        for (int q = 0; q < kRows; ++q) s += red[q * kStride + i];
        mine[C + i] = s;
    }
    __syncthreads();
    red[threadIdx.x] = sum_d;
    __syncthreads();
    for (int i = threadIdx.x; i < k.width; i += kThreads) {
        const int lanes = i / 2 * L + (i & 1);      // the first lane whose first channel is i
        float s = 0.f;
        for (int q = 0; q < L; q += 2) s += red[lanes + q];
        mine[i] = s;
    }
}

// The first row of the piece that a row belongs to.
__device__ __forceinline__ long long piece_row(const Seqs& q, long long row, long long span) {
    long long base;
    if (q.offsets == nullptr) {
        base = row / q.length * q.length;
    } else {
        int lo = 0, hi = q.count - 1;           // the last sequence that does not begin behind the row
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (seq_offset(q, mid) <= row) lo = mid;
            else hi = mid - 1;
        }
        base = seq_offset(q, lo);
    }
    return base + (row - base) / span * span;
}

// dB and dC from the partial rows of a group's blocks.  (`some`: the window leaves pieces to other launches.)
template <typename T>
__global__ void __launch_bounds__(256) scan_bc_kernel(Scan p, const float* part, int per_group, Window window, bool some) {
    pdl_trigger();
    pdl_wait();
    const int N = p.N, G = p.G;
    const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x, at = i / (G * 2 * N), row = window.from + at;
    if (at >= window.rows || row >= seq_rows_device(p.seqs)) return;
    const int j = static_cast<int>(i - at * G * 2 * N), g = j / (2 * N), which = (j - g * 2 * N) / N, n = j % N;
    if (p.seqs.offsets != nullptr && (row < seq_offset(p.seqs, 0) || row >= seq_offset(p.seqs, p.seqs.count))) return;
    if (some) {
        const long long first = piece_row(p.seqs, row, p.span);
        if (first < window.from || first >= window.to) return;
    }
    const float* from = part + (static_cast<long long>(g) * per_group * window.rows + at) * 2 * N + which * N + n;
    const long long step = window.rows * 2 * N;
    float s = 0.f;
    int k = 0;
    for (; k + 8 <= per_group; k += 8) {
        float t[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = from[(k + i) * step];
        s += ((t[0] + t[1]) + (t[2] + t[3])) + ((t[4] + t[5]) + (t[6] + t[7]));
    }
    for (; k < per_group; ++k) s += from[k * step];
    store_out(static_cast<T*>(which == 0 ? p.db : p.dc) + (row * G + g) * N + n, s);
}

// ---------------------------------------------------------------------------------- host

inline int channel_blocks(const Scan& p, int channels) { return p.G * ((p.C / p.G + channels - 1) / channels); }

// Lanes to a pair of channels, four states of each to a lane.
inline int lanes_of(int N) { return N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : N <= 64 ? 16 : 32; }
#define DWC_SCAN_BY_LANES(N, call)   \
    switch (lanes_of(N)) {           \
        case 2: return call(2);      \
        case 4: return call(4);      \
        case 8: return call(8);      \
        case 16: return call(16);    \
        default: return call(32);    \
    }
inline int fwd_channels(int N) {
#define DWC_CHANNELS(L) (FwdShape<L>::kChannels)
    DWC_SCAN_BY_LANES(N, DWC_CHANNELS)
#undef DWC_CHANNELS
}
inline int fwd_threads(int N) { return N <= 64 ? FwdShape<4>::kThreads : FwdShape<32>::kThreads; }
inline int bwd_channels(int N) {
#define DWC_CHANNELS(L) (BwdShape<L>::kChannels)
    DWC_SCAN_BY_LANES(N, DWC_CHANNELS)
#undef DWC_CHANNELS
}

// The workspaces, in floats.
struct FwdSpace {
    long long ends = 0, sums = 0;      // with chunks only
    explicit FwdSpace(const Scan& p) {
        if (p.span >= p.seqs.length) return;
        sums = seq_slots(p.seqs, p.span) * p.C;
        ends = sums * p.N;
    }
};
// Every block of channels has its own partial rows of dB and dC, 2 N floats a position, which with 33 states and more are
// 2 N bytes a position and channel, many times the tensors themselves.  They are held to what the forward pass keeps of the
// states, or to 8 GB where that is less: past it ranges of rows take turns, each with a launch of its own (bf16, 4096 channels:
// 16 x 2048, 128 states 30.1 ms, with 16 GB 30.1; 8 x 8192, 64 states 32.1, with 16 GB 30.5; 1 x 65536, 64 states 38.7 and 38.2).
constexpr long long kMostPartial = 1LL << 31;       // floats
inline long long most_partial_rows(const Scan& p) {
    const long long each = static_cast<long long>(channel_blocks(p, bwd_channels(p.N))) * 2 * p.N;
    return std::max(kMostPartial, seq_slots(p.seqs, kScanTile) * p.C * p.N) / each;
}
struct BwdSpace {
    long long window, rows;            // rows whose pieces one launch takes, and rows that those pieces reach
    long long bc, params, ends = 0, sums = 0;
    explicit BwdSpace(const Scan& p) {
        const long long slots = seq_slots(p.seqs, p.span), C = p.C, most = most_partial_rows(p);
        window = rows = seq_rows(p.seqs);
        if (rows > most) {
            // (pieces that are whole sequences of a batch end where the next begins, others go past the window)
            const bool whole = p.seqs.offsets == nullptr && p.span >= p.seqs.length;
            window = whole ? std::max(1LL, most / p.seqs.length) * p.seqs.length : std::max(p.span, most - p.span);
            rows = whole ? window : window + p.span;
        }
        bc = static_cast<long long>(channel_blocks(p, bwd_channels(p.N))) * rows * 2 * p.N;
        params = slots * C * (p.N + 2);
        if (p.span >= p.seqs.length) return;
        sums = slots * C;
        ends = sums * p.N;
    }
};

template <bool kBackward>
cudaError_t launch_join(const Scan& p, float* ends, const float* sums, const float* from) {
    const long long grid = (static_cast<long long>(p.seqs.count) * p.C * p.N + 255) / 256;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    return launch_pdl(scan_join_kernel<kBackward>, dim3(static_cast<unsigned>(grid)), dim3(256), 0, p.stream, p, ends, sums, from);
}

template <typename T, int L>
cudaError_t fwd_t(const Scan& p) {
    using S = FwdShape<L>;
    const int blocks = channel_blocks(p, S::kChannels);
    const long long grid = seq_slots(p.seqs, p.span) * blocks;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const FwdSpace space(p);
    float *ends = space.ends > 0 ? p.workspace : nullptr, *sums = p.workspace + space.ends;
    const dim3 ctas(static_cast<unsigned>(grid)), threads(S::kThreads);
    if (ends != nullptr) {
        cudaError_t err = launch_pdl(scan_fwd_kernel<T, L, true>, ctas, threads, 0, p.stream, p, blocks, ends, sums);
        if (err == cudaSuccess) err = launch_join<false>(p, ends, sums, p.state);
        if (err != cudaSuccess) return err;
    }
    return launch_pdl(scan_fwd_kernel<T, L, false>, ctas, threads, 0, p.stream, p, blocks, ends, sums);
}

template <typename T, int L>
cudaError_t adjoint_t(const Scan& p, float* ends, float* sums) {
    using S = FwdShape<L>;
    const int blocks = channel_blocks(p, S::kChannels);
    const long long grid = seq_slots(p.seqs, p.span) * blocks;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const cudaError_t err = launch_pdl(scan_adjoint_kernel<T, L>, dim3(static_cast<unsigned>(grid)), dim3(S::kThreads), 0, p.stream,
                                       p, blocks, ends, sums);
    return err != cudaSuccess ? err : launch_join<true>(p, ends, sums, p.dfinal);
}

template <typename T, int L>
cudaError_t bwd_t(const Scan& p) {
    using S = BwdShape<L>;
    constexpr size_t smem = S::kFloats * sizeof(float);
    const int blocks = channel_blocks(p, S::kChannels);
    const long long slots = seq_slots(p.seqs, p.span), rows = seq_rows(p.seqs), C = p.C;
    const BwdSpace space(p);
    float *bc = p.workspace, *params = bc + space.bc, *ends = params + space.params;
    const long long sums = (space.rows * p.G * 2 * p.N + 255) / 256;
    static DeviceOnce once;
    cudaError_t err = opt_in_smem(scan_bwd_kernel<T, L>, once, static_cast<int>(smem));
    if (err == cudaSuccess && space.ends > 0) err = adjoint_t<T, L>(p, ends, ends + space.ends);
    const bool some = space.window < rows;
    // (no rows: the pieces of empty sequences)
    for (long long from = 0; err == cudaSuccess && (from == 0 || from < rows); from += space.window) {
        const bool last = !some || from + space.window >= rows;
        Window w{from, last ? INT64_MAX : from + space.window, 0, space.rows};
        long long end = slots;
        if (some && p.seqs.offsets != nullptr) {
            // piece k of sequence s, slot offset / span + s + k, has its first row, offset + k span, in slot - s spans
            w.slot = from / p.span;
            if (!last) end = (w.to - 1) / p.span + p.seqs.count;
        } else if (some) {
            const long long n = (p.seqs.length + p.span - 1) / p.span;         // of each sequence
            w.slot = from / p.seqs.length * n;
            if (!last) end = ((w.to - 1) / p.seqs.length + 1) * n;
        }
        const long long grid = (end - w.slot) * blocks;
        if (grid > 0x7fffffffLL || sums > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
        err = launch_pdl(scan_bwd_kernel<T, L>, dim3(static_cast<unsigned>(grid)), dim3(S::kThreads), smem, p.stream, p, blocks, w,
                         static_cast<const float*>(space.ends > 0 ? ends + w.slot * C * p.N : nullptr), bc,
                         params + w.slot * C * (p.N + 2));
        if (err == cudaSuccess && sums > 0)
            err = launch_pdl(scan_bc_kernel<T>, dim3(static_cast<unsigned>(sums)), dim3(256), 0, p.stream, p,
                             static_cast<const float*>(bc), blocks / p.G, w, some);
        if (!some) break;
    }
    if (err == cudaSuccess) err = launch_row_sum(params, slots, C * (p.N + 2), {p.dA, p.dD, p.ddt_bias}, {C * p.N, C, C}, p.stream);
    return err;
}

template <typename T>
cudaError_t fwd(const Scan& p) {
#define DWC_FWD(L) (fwd_t<T, L>(p))
    DWC_SCAN_BY_LANES(p.N, DWC_FWD)
#undef DWC_FWD
}

template <typename T>
cudaError_t bwd(const Scan& p) {
#define DWC_BWD(L) (bwd_t<T, L>(p))
    DWC_SCAN_BY_LANES(p.N, DWC_BWD)
#undef DWC_BWD
}

}  // namespace scan
}  // namespace dwc

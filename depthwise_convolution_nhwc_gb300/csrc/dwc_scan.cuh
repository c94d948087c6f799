// dwc_scan.cuh -- selective scan along sequences, forward and backward.
//
//     h[t, n] = exp(delta[t] A[n]) h[t-1, n] + delta[t] u[t] B[t, n]
//     y[t]    = (sum_n C[t, n] h[t, n] + D u[t]) silu(z[t])
//
// L lanes serve a channel, NS states each, and walk along the positions with the states in registers.
// Tiles of 32 positions are brought in by the whole CTA: per channel and position delta and
// delta * u, once, as fp32 in shared memory, and B and C widened.  The sums over the states are
// parted among the lanes: L positions together, each lane ends with one of them.
#pragma once

#include <algorithm>

#include "dwc_seq_device.cuh"

namespace dwc {
namespace scan {

constexpr int kThreads = 128;
constexpr int kTile = 32;

// log(1 + e) for e in [0, 1] as 2 atanh(s), s = e / (2 + e) <= 1/3: the odd series up to s^15, whose
// rest is below 2 s^17 / 17 < 1e-9 of it; relative errors stay near 2^-23 however small e is.
__device__ __forceinline__ float log1p_unit(float e) {
    const float s = __fdividef(e, 2.f + e), q = s * s;
    float p = 1.f / 15.f;
    p = fmaf(p, q, 1.f / 13.f);
    p = fmaf(p, q, 1.f / 11.f);
    p = fmaf(p, q, 1.f / 9.f);
    p = fmaf(p, q, 1.f / 7.f);
    p = fmaf(p, q, 1.f / 5.f);
    p = fmaf(p, q, 1.f / 3.f);
    const float t = s + s;
    return fmaf(t * q, p, t);
}
// (a NaN stays one: fmaxf would drop it)
__device__ __forceinline__ float softplus(float v) { return (v < 0.f ? 0.f : v) + log1p_unit(exp2_fast(fabsf(v) * -kLog2e)); }

// The sum over the L lanes of a channel of v[sub], for lane `sub`: halves are exchanged, then quarters.
template <int L>
__device__ __forceinline__ float parted(float (&v)[L], int sub) {
#pragma unroll
    for (int m = L / 2; m > 0; m >>= 1) {
        const bool upper = (sub & m) != 0;
#pragma unroll
        for (int i = 0; i < m; ++i) {
            const float keep = upper ? v[m + i] : v[i], send = upper ? v[i] : v[m + i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, m);
        }
    }
    return v[0];
}

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

template <int N>
__device__ __forceinline__ void put_states(float* to, const float (&h)[N], int n0, int states) {
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (n0 + i < states) to[n0 + i] = h[i];
}
template <int N>
__device__ __forceinline__ void get_states(float (&h)[N], const float* from, int n0, int states) {
#pragma unroll
    for (int i = 0; i < N; ++i) h[i] = from != nullptr && n0 + i < states ? from[n0 + i] : 0.f;
}

// B or C of a tile: vectors of 8 states, padded with zeros.
template <typename T, int NP, int kRows = kTile>
struct StateRows {
    static constexpr int kVecs = (NP + 7) / 8, kEach = (kRows * kVecs + kThreads - 1) / kThreads;
    Vec8<T> raw[kEach];
    __device__ __forceinline__ void fetch(const T* base, const RowsView& v, long long t0, long long end, int N) {
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int i = threadIdx.x + k * kThreads, t = i / kVecs, col = i % kVecs * 8;
            if (i < kRows * kVecs && t0 + t < end) load8(raw[k], base + (t0 + t) * v.row, col, N, v.vec && N % 8 == 0);
            else raw[k].zero();
        }
    }
    __device__ __forceinline__ void spread(float (*to)[NP]) const {
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int i = threadIdx.x + k * kThreads;
            if (i >= kRows * kVecs) continue;
            float2 f[4];
            raw[k].widen(f);
            float4* o = reinterpret_cast<float4*>(&to[i / kVecs][i % kVecs * 8]);
            o[0] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
            o[1] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
        }
    }
    // each four states in 1, 2 or 4 orders: n, n ^ 2 (two orders); n, n ^ 1, n ^ 2, n ^ 3 (four)
    template <int kOrders>
    __device__ __forceinline__ void spread(float (*to)[kRows][NP]) const {
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int i = threadIdx.x + k * kThreads;
            if (i >= kRows * kVecs) continue;
            float2 f[4];
            raw[k].widen(f);
#pragma unroll
            for (int o = 0; o < kOrders; ++o) {
                const int m = kOrders == 2 ? 2 * o : o;
                float4* at = reinterpret_cast<float4*>(&to[o][i / kVecs][i % kVecs * 8]);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const float v[4] = {f[2 * q].x, f[2 * q].y, f[2 * q + 1].x, f[2 * q + 1].y};
                    at[q] = make_float4(v[m], v[1 ^ m], v[2 ^ m], v[3 ^ m]);
                }
            }
        }
    }
};

template <int N>
__device__ __forceinline__ void row_values(float (&v)[N], const float* from) {
    static_assert(N % 2 == 0, "pairs");
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const float4 f = *reinterpret_cast<const float4*>(from + i);
            v[i] = f.x, v[i + 1] = f.y, v[i + 2] = f.z, v[i + 3] = f.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const float2 f = *reinterpret_cast<const float2*>(from + i);
            v[i] = f.x, v[i + 1] = f.y;
        }
    }
}

template <int N>
__device__ __forceinline__ void row_pairs(float2 (&v)[N], const float* from) {
    float f[2 * N];
    row_values(f, from);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = make_float2(f[2 * i], f[2 * i + 1]);
}

// -------------------------------------------------------------------------------- forward

// Sequences that are too few to fill the GPU are cut into chunks of p.span positions.  kStates: the first of
// three kernels, which walks every chunk but a sequence's last from a state of zero and keeps the
// state at its end (`ends`, [slot][C][N]) and the sum of delta (`sums`, [slot][C]); the chunks are then joined,
// h = exp(A sum delta) h + end, and the second walk begins each chunk with the state in front of it.
template <typename T, int NS, int L, bool kStates>
__global__ void __launch_bounds__(kThreads, L == 16 ? 3 : 6) scan_fwd_kernel(Scan p, int blocks, float* ends, float* sums) {
    constexpr int kChannels = kThreads / L, kColumns = kChannels / 8, NP = NS * L;
    constexpr int kEach = (kTile * kColumns + kThreads - 1) / kThreads;      // vectors of a tile to a thread
    __shared__ __align__(16) float2 step[kTile][kChannels];    // delta, delta * u
    __shared__ __align__(16) float bs[kTile][NP], cs[kStates ? 1 : kTile][NP], ys[kStates ? 1 : kTile][kChannels];
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
    const bool even = (C / p.G) % 8 == 0, vec_y = even && reinterpret_cast<uintptr_t>(p.y) % (8 * sizeof(T)) == 0;
    for (int i = threadIdx.x; i < kChannels; i += kThreads) {
        bias[i] = i < k.width && p.dt_bias != nullptr ? p.dt_bias[k.c + i] : 0.f;
        skip[i] = i < k.width && p.D != nullptr ? p.D[k.c + i] : 0.f;
    }
    // as a server of a channel's states
    const int ch = threadIdx.x / L, sub = threadIdx.x % L, n0 = sub * NS;
    const bool serves = ch < k.width;
    const long long mine = (static_cast<long long>(r.s) * C + k.c + ch) * N, here = (slot * C + k.c + ch) * N;
    float a2[NS], h[NS], total = 0.f;
    get_states(a2, serves ? p.A + static_cast<long long>(k.c + ch) * N : nullptr, n0, N);
#pragma unroll
    for (int i = 0; i < NS; ++i) a2[i] *= kLog2e;
    if (kStates) get_states(h, nullptr, n0, N);
    else if (ends != nullptr) get_states(h, serves ? ends + here : nullptr, n0, N);
    else get_states(h, serves && p.state != nullptr ? p.state + mine : nullptr, n0, N);

    Vec8<T> ru[kEach], rz[kEach], rdt[kEach];
    StateRows<T, NP> rb, rc;
    const auto row_of = [](int i) { return (static_cast<int>(threadIdx.x) + i * kThreads) / kColumns; };
    const auto col_of = [](int i) { return (static_cast<int>(threadIdx.x) + i * kThreads) % kColumns * 8; };
    auto fetch = [&](long long t0) {
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int row = row_of(i), col = col_of(i);
            ru[i].zero(), rdt[i].zero();
            if (row >= kTile || t0 + row >= r.end) continue;
            load8(ru[i], u + (t0 + row) * p.u.row, col, k.width, p.u.vec && even);
            load8(rdt[i], dt + (t0 + row) * p.dt.row, col, k.width, p.dt.vec && even);
        }
        rb.fetch(b, p.b, t0, r.end, N);
        if (!kStates) rc.fetch(c, p.c, t0, r.end, N);
    };
    fetch(r.first);
    __syncthreads();
    for (long long t0 = r.first; t0 < r.end; t0 += kTile) {
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int row = row_of(i), col = col_of(i);
            if (row >= kTile) continue;
            float2 fu[4], fd[4];
            ru[i].widen(fu);
            rdt[i].widen(fd);
            const bool in = t0 + row < r.end;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 o = *reinterpret_cast<const float2*>(&bias[col + 2 * j]);
                float d0 = fd[j].x + o.x, d1 = fd[j].y + o.y;
                if (p.softplus) d0 = softplus(d0), d1 = softplus(d1);
                if (!in) d0 = d1 = 0.f;        // positions past the end leave the states alone
                *reinterpret_cast<float4*>(&step[row][col + 2 * j]) = make_float4(d0, d0 * fu[j].x, d1, d1 * fu[j].y);
            }
        }
        rb.spread(bs);
        if (!kStates) rc.spread(cs);
        __syncthreads();
        Vec8<T> keep[kEach];
        if (!kStates) {
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                keep[i] = ru[i];
                rz[i].zero();
                if (z != nullptr && row_of(i) < kTile && t0 + row_of(i) < r.end)
                    load8(rz[i], z + (t0 + row_of(i)) * p.z.row, col_of(i), k.width, p.z.vec && even);
            }
        }
        if (t0 + kTile < r.end) fetch(t0 + kTile);
#pragma unroll 1
        for (int t = 0; t < kTile; t += L) {
            if (!kStates && p.saved != nullptr && t % kScanTile == 0 && serves && (t == 0 || t0 + t < r.end))
                put_states(p.saved + (saved_slot(p.seqs, r, (t0 + t) / kScanTile) * C + k.c + ch) * N, h, n0, N);
            float part[L];
#pragma unroll
            for (int q = 0; q < L; ++q) {
                const float2 s = step[t + q][ch];
                float2 fb[NS / 2], fc[NS / 2], sum = both(0.f);
                row_pairs(fb, &bs[t + q][n0]);
                if (!kStates) row_pairs(fc, &cs[t + q][n0]);
#pragma unroll
                for (int i = 0; i < NS / 2; ++i) {
                    float2 a = __fmul2_rn(both(s.x), make_float2(a2[2 * i], a2[2 * i + 1])), hh = make_float2(h[2 * i], h[2 * i + 1]);
                    a = make_float2(exp2_fast(a.x), exp2_fast(a.y));
                    hh = __ffma2_rn(both(s.y), fb[i], __fmul2_rn(a, hh));
                    h[2 * i] = hh.x, h[2 * i + 1] = hh.y;
                    if (!kStates) sum = __ffma2_rn(fc[i], hh, sum);
                }
                if (kStates) total += s.x;
                part[q] = sum.x + sum.y;
            }
            if (!kStates) ys[t + sub][ch] = parted<L>(part, sub);
        }
        __syncthreads();
        if constexpr (!kStates) {
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int row = row_of(i), col = col_of(i);
                if (row >= kTile || t0 + row >= r.end || col >= k.width) continue;
                float2 fu[4], fz[4], f[4];
                keep[i].widen(fu);
                rz[i].widen(fz);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 o = *reinterpret_cast<const float2*>(&skip[col + 2 * j]);
                    f[j] = __ffma2_rn(o, fu[j], *reinterpret_cast<const float2*>(&ys[row][col + 2 * j]));
                    if (z != nullptr) f[j] = __fmul2_rn(f[j], make_float2(silu(fz[j].x), silu(fz[j].y)));
                }
                store8(y + (t0 + row) * C, f, col, k.width, vec_y);
            }
        }
    }
    if (!serves) return;
    if (kStates) {
        put_states(ends + here, h, n0, N);
        if (sub == 0) sums[slot * C + k.c + ch] = total;
    } else if (r.last && p.final_state != nullptr) {
        put_states(p.final_state + mine, h, n0, N);
    }
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
    const float a2 = p.A[j] * kLog2e;
    float h = from != nullptr ? from[i] : 0.f;
    constexpr int U = 8;
    for (long long k = 0; k < n; k += U) {
        float e[U], d[U];
#pragma unroll
        for (int q = 0; q < U; ++q) {
            // (the last chunk's end is not needed, nor formed)
            const bool in = k + q < n - 1;
            const long long slot = first + (kBackward ? n - 1 - k - q : k + q);
            e[q] = in ? ends[slot * width + j] : 0.f;
            d[q] = in ? sums[slot * C + c] : 0.f;
        }
#pragma unroll
        for (int q = 0; q < U; ++q) {
            if (k + q >= n) break;
            const long long slot = first + (kBackward ? n - 1 - k - q : k + q);
            ends[slot * width + j] = h;
            h = fmaf(exp2_fast(d[q] * a2), h, e[q]);
        }
    }
}

// ------------------------------------------------------------------------------- backward

// The first of the backward pass's kernels where sequences are cut into chunks: what reaches the
// position in front of a chunk from within it, dh = g C + carry, carry = exp(delta A) dh (`ends`), and the sum
// of delta.  Every chunk but a sequence's first is walked, from its end.
template <typename T, int NS, int L>
__global__ void __launch_bounds__(kThreads, 6) scan_adjoint_kernel(Scan p, int blocks, float* ends, float* sums) {
    constexpr int kChannels = kThreads / L, kColumns = kChannels / 8, NP = NS * L;
    constexpr int kEach = (kTile * kColumns + kThreads - 1) / kThreads;
    __shared__ __align__(16) float2 step[kTile][kChannels];    // delta, g
    __shared__ __align__(16) float cs[kTile][NP];
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
    const int ch = threadIdx.x / L, sub = threadIdx.x % L, n0 = sub * NS;
    const bool serves = ch < k.width;
    float a2[NS], carry[NS], total = 0.f;
    get_states(a2, serves ? p.A + static_cast<long long>(k.c + ch) * N : nullptr, n0, N);
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        a2[i] *= kLog2e;
        carry[i] = 0.f;
    }
    const auto row_of = [](int i) { return (static_cast<int>(threadIdx.x) + i * kThreads) / kColumns; };
    const auto col_of = [](int i) { return (static_cast<int>(threadIdx.x) + i * kThreads) % kColumns * 8; };
    Vec8<T> rdt[kEach], rdy[kEach], rz[kEach];
    StateRows<T, NP> rc;
    auto fetch = [&](long long t0) {
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int row = row_of(i), col = col_of(i);
            rdt[i].zero(), rdy[i].zero(), rz[i].zero();
            if (row >= kTile || t0 + row >= r.end) continue;
            load8(rdt[i], dt + (t0 + row) * p.dt.row, col, k.width, p.dt.vec && even);
            load8(rdy[i], dy + (t0 + row) * p.dy.row, col, k.width, p.dy.vec && even);
            if (z != nullptr) load8(rz[i], z + (t0 + row) * p.z.row, col, k.width, p.z.vec && even);
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
            const int row = row_of(i), col = col_of(i);
            if (row >= kTile) continue;
            float2 fd[4], fy[4], fz[4];
            rdt[i].widen(fd);
            rdy[i].widen(fy);
            rz[i].widen(fz);
            const bool in = t0 + row < r.end;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 o = *reinterpret_cast<const float2*>(&bias[col + 2 * j]);
                float d0 = fd[j].x + o.x, d1 = fd[j].y + o.y;
                if (p.softplus) d0 = softplus(d0), d1 = softplus(d1);
                if (!in) d0 = d1 = 0.f;
                if (z != nullptr) fy[j] = __fmul2_rn(fy[j], make_float2(silu(fz[j].x), silu(fz[j].y)));
                *reinterpret_cast<float4*>(&step[row][col + 2 * j]) = make_float4(d0, fy[j].x, d1, fy[j].y);
            }
        }
        rc.spread(cs);
        __syncthreads();
        if (tile > 0) fetch(t0 - kTile);
#pragma unroll 4
        for (int t = kTile - 1; t >= 0; --t) {
            const float2 s = step[t][ch];
            float2 fc[NS / 2];
            row_pairs(fc, &cs[t][n0]);
#pragma unroll
            for (int i = 0; i < NS / 2; ++i) {
                float2 a = __fmul2_rn(both(s.x), make_float2(a2[2 * i], a2[2 * i + 1]));
                a = make_float2(exp2_fast(a.x), exp2_fast(a.y));
                const float2 dh = __ffma2_rn(both(s.y), fc[i], make_float2(carry[2 * i], carry[2 * i + 1]));
                a = __fmul2_rn(a, dh);
                carry[2 * i] = a.x, carry[2 * i + 1] = a.y;
            }
            total += s.x;
        }
    }
    if (!serves) return;
    put_states(ends + (slot * C + k.c + ch) * N, carry, n0, N);
    if (sub == 0) sums[slot * C + k.c + ch] = total;
}

// Tiles of 16 positions from the last to the first.  From the state in front of a tile (kept by the
// forward pass) the states in front of every 4th position are formed again (`front`); then, 4 positions
// at a time from the last, a h[t-1] and a of each, in registers, and the gradients going back:
//     dh = g C + carry,  carry = a dh  (g: the gradient of the sum over the states and D u)
//     dC = sum_c g h,  dB = sum_c dh delta u,  dA += dh a h[t-1] delta
//     into = sum_n dh B,  decay = sum_n dh a h[t-1] A,  du = into delta + D g,  ddelta = into u + decay
// Bound by the exchanges between lanes as much as by the arithmetic (10 packed operations on a pair of states
// going back, 1.75 times 3 and two exponentials to form the states again), so a lane has two channels and four
// states of each: dB and dC are added over its channels before they leave it, and lanes part the sums
// among themselves without selecting what to send.  For that a lane holds its four states in the
// order n ^ perm, so that the upper pair is always what the partner keeps (B and C lie in shared
// memory in each of the orders), and odd lanes hold their two channels the other way round.
constexpr int kBwdTile = kScanTile, kBwdStep = 4;

// Values of four states in a lane's order.
struct Four {
    float2 v[2];
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
};

template <int L>
struct BwdShape {
    static constexpr int kLanes = 32 / L;                  // lanes of a warp that share states
    static constexpr int kOrders = kLanes >= 4 ? 4 : kLanes;
    static constexpr int kChannels = 2 * kThreads / L, NP = 4 * L, kWarps = kThreads / 32;
    static constexpr size_t kFloats = kBwdTile * kChannels * 3 + 2 * kOrders * kBwdTile * NP +
                                      kBwdTile / kBwdStep * 8 * kThreads + kWarps * kBwdTile * 2 * NP + 2 * kChannels;
};

__device__ __forceinline__ float from_lane(float v, int mask) { return __shfl_xor_sync(0xffffffffu, v, mask); }

template <typename T, int L>
__global__ void __launch_bounds__(kThreads, 3) scan_bwd_kernel(Scan p, int blocks, const float* carries, float* part_bc, float* part_p) {
    using S = BwdShape<L>;
    constexpr int kChannels = S::kChannels, kColumns = kChannels / 8, NP = S::NP, W = S::kLanes, kOrders = S::kOrders;
    constexpr int kEach = (kBwdTile * kColumns + kThreads - 1) / kThreads;
    extern __shared__ __align__(16) float smem[];
    float2 (*step)[kChannels] = reinterpret_cast<float2 (*)[kChannels]>(smem);      // delta, u; then du, ddelta
    float (*gs)[kChannels] = reinterpret_cast<float (*)[kChannels]>(step + kBwdTile);       // g; then the sum over the states
    float (*bs)[kBwdTile][NP] = reinterpret_cast<float (*)[kBwdTile][NP]>(gs + kBwdTile);
    float (*cs)[kBwdTile][NP] = bs + kOrders;
    float* front = reinterpret_cast<float*>(cs + kOrders);
    float* sums = front + kBwdTile / kBwdStep * 8 * kThreads;       // warps x positions x (dB, dC)
    float* bias = sums + S::kWarps * kBwdTile * 2 * NP;
    float* skip = bias + kChannels;
    front += threadIdx.x;
    pdl_trigger();
    pdl_wait();
    const long long slot = blockIdx.x / blocks;
    const int block = static_cast<int>(blockIdx.x - slot * blocks);
    const Block k = block_of(p, block, kChannels);
    const Piece r = find_piece(p.seqs, slot, p.span);
    const int C = p.C, N = p.N;
    const bool even = (C / p.G) % 8 == 0;
    const long long dense = r.some ? dense_row(p.seqs, r) : 0;
    const auto aligned = [&](const void* t) { return even && reinterpret_cast<uintptr_t>(t) % (8 * sizeof(T)) == 0; };
    const T *u = view_at<T>(p.u, p.seqs, r) + k.c, *dt = view_at<T>(p.dt, p.seqs, r) + k.c, *dy = view_at<T>(p.dy, p.seqs, r) + k.c;
    const T* z = p.z.p == nullptr ? nullptr : view_at<T>(p.z, p.seqs, r) + k.c;
    const T *b = view_at<T>(p.b, p.seqs, r) + k.g * N, *c = view_at<T>(p.c, p.seqs, r) + k.g * N;
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
        const long long at = static_cast<long long>(k.c + ch[j]) * N, wide = static_cast<long long>(C) * N;
        a2[j].get(serves ? p.A + at : nullptr, n0, perm, N);
        if (carries != nullptr) carry[j].get(serves && r.some ? carries + slot * wide + at : nullptr, n0, perm, N);
        else carry[j].get(serves && r.some && p.dfinal != nullptr ? p.dfinal + r.s * wide + at : nullptr, n0, perm, N);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            a2[j].v[i] = __fmul2_rn(a2[j].v[i], both(kLog2e));
            da[j].v[i] = both(0.f);
        }
    }
    float sum_d = 0.f, sum_bias[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) sum_bias[j] = 0.f;
    const auto row_of = [](int i) { return (static_cast<int>(threadIdx.x) + i * kThreads) / kColumns; };
    const int col = threadIdx.x % kColumns * 8;            // (kColumns divides the threads)

    const long long tiles = r.some ? (r.end - r.first + kBwdTile - 1) / kBwdTile : 0;
    for (long long tile = tiles - 1; tile >= 0; --tile) {
        const long long t0 = r.first + tile * kBwdTile;
        Vec8<T> ru[kEach], rdt[kEach], rz[kEach], rdy[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int row = row_of(i);
            ru[i].zero(), rdt[i].zero(), rz[i].zero(), rdy[i].zero();
            if (row >= kBwdTile || t0 + row >= r.end || col >= k.width) continue;
            load8(ru[i], u + (t0 + row) * p.u.row, col, k.width, p.u.vec && even);
            load8(rdt[i], dt + (t0 + row) * p.dt.row, col, k.width, p.dt.vec && even);
            load8(rdy[i], dy + (t0 + row) * p.dy.row, col, k.width, p.dy.vec && even);
            if (z != nullptr) load8(rz[i], z + (t0 + row) * p.z.row, col, k.width, p.z.vec && even);
        }
        StateRows<T, NP, kBwdTile> rb, rc;
        rb.fetch(b, p.b, t0, r.end, N);
        rc.fetch(c, p.c, t0, r.end, N);
        Four h[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
            h[j].get(ch[j] < k.width ? p.saved + (saved_slot(p.seqs, r, t0 / kScanTile) * C + k.c + ch[j]) * N : nullptr, n0, perm, N);
        __syncthreads();            // the last tile's sums have been read
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int row = row_of(i);
            if (row >= kBwdTile) continue;
            float2 fu[4], fd[4], fz[4], fy[4];
            ru[i].widen(fu);
            rdt[i].widen(fd);
            rz[i].widen(fz);
            rdy[i].widen(fy);
            const bool in = t0 + row < r.end;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 o = *reinterpret_cast<const float2*>(&bias[col + 2 * j]);
                float d0 = fd[j].x + o.x, d1 = fd[j].y + o.y;
                if (p.softplus) d0 = softplus(d0), d1 = softplus(d1);
                if (!in) d0 = d1 = 0.f;        // positions past the end change nothing
                if (z != nullptr) fy[j] = __fmul2_rn(fy[j], make_float2(silu(fz[j].x), silu(fz[j].y)));
                *reinterpret_cast<float4*>(&step[row][col + 2 * j]) = make_float4(d0, fu[j].x, d1, fu[j].y);
                *reinterpret_cast<float2*>(&gs[row][col + 2 * j]) = fy[j];
            }
        }
        rb.template spread<kOrders>(bs);
        rc.template spread<kOrders>(cs);
        __syncthreads();
#pragma unroll 1
        for (int w = 0; w < kBwdTile / kBwdStep; ++w) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                front[(w * 8 + j * 4 + 0) * kThreads] = h[j].v[0].x, front[(w * 8 + j * 4 + 1) * kThreads] = h[j].v[0].y;
                front[(w * 8 + j * 4 + 2) * kThreads] = h[j].v[1].x, front[(w * 8 + j * 4 + 3) * kThreads] = h[j].v[1].y;
            }
            if (w == kBwdTile / kBwdStep - 1) break;
#pragma unroll
            for (int q = 0; q < kBwdStep; ++q) {
                const int t = w * kBwdStep + q;
                const float4 fb = *reinterpret_cast<const float4*>(&bs[order][t][n0]);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float2 s = step[t][ch[j]];
                    const float in = s.x * s.y;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 e = __fmul2_rn(both(s.x), a2[j].v[i]);
                        const float2 a = make_float2(exp2_fast(e.x), exp2_fast(e.y));
                        h[j].v[i] = __ffma2_rn(both(in), i == 0 ? make_float2(fb.x, fb.y) : make_float2(fb.z, fb.w),
                                               __fmul2_rn(a, h[j].v[i]));
                    }
                }
            }
        }
#pragma unroll 1
        for (int w = kBwdTile / kBwdStep - 1; w >= 0; --w) {
            float2 held[kBwdStep][2][2], decay[kBwdStep][2][2];       // a h[t-1], a
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                h[j].v[0] = make_float2(front[(w * 8 + j * 4 + 0) * kThreads], front[(w * 8 + j * 4 + 1) * kThreads]);
                h[j].v[1] = make_float2(front[(w * 8 + j * 4 + 2) * kThreads], front[(w * 8 + j * 4 + 3) * kThreads]);
            }
#pragma unroll
            for (int q = 0; q < kBwdStep; ++q) {
                const int t = w * kBwdStep + q;
                const float4 fb = *reinterpret_cast<const float4*>(&bs[order][t][n0]);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float2 s = step[t][ch[j]];
                    const float in = s.x * s.y;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 e = __fmul2_rn(both(s.x), a2[j].v[i]);
                        decay[q][j][i] = make_float2(exp2_fast(e.x), exp2_fast(e.y));
                        held[q][j][i] = __fmul2_rn(decay[q][j][i], h[j].v[i]);
                        if (q + 1 < kBwdStep)
                            h[j].v[i] = __ffma2_rn(both(in), i == 0 ? make_float2(fb.x, fb.y) : make_float2(fb.z, fb.w), held[q][j][i]);
                    }
                }
            }
            float into[kBwdStep], decays[kBwdStep], ys[kBwdStep];
#pragma unroll
            for (int q = kBwdStep - 1; q >= 0; --q) {
                const int t = w * kBwdStep + q;
                const float4 b4 = *reinterpret_cast<const float4*>(&bs[order][t][n0]);
                const float4 c4 = *reinterpret_cast<const float4*>(&cs[order][t][n0]);
                const float2 fb[2] = {make_float2(b4.x, b4.y), make_float2(b4.z, b4.w)};
                const float2 fc[2] = {make_float2(c4.x, c4.y), make_float2(c4.z, c4.w)};
                float2 vb[2] = {both(0.f), both(0.f)}, vc[2] = {both(0.f), both(0.f)};
                float s1[2], s2[2], s3[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float2 s = step[t][ch[j]];
                    const float g = gs[t][ch[j]], in = s.x * s.y;
                    float2 x1 = both(0.f), x2 = both(0.f), x3 = both(0.f);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 dh = __ffma2_rn(both(g), fc[i], carry[j].v[i]);
                        const float2 now = __ffma2_rn(both(in), fb[i], held[q][j][i]);
                        const float2 x = __fmul2_rn(dh, held[q][j][i]);
                        vb[i] = __ffma2_rn(dh, both(in), vb[i]);
                        vc[i] = __ffma2_rn(both(g), now, vc[i]);
                        x1 = __ffma2_rn(dh, fb[i], x1);
                        x2 = __ffma2_rn(x, a2[j].v[i], x2);
                        x3 = __ffma2_rn(fc[i], now, x3);
                        da[j].v[i] = __ffma2_rn(x, both(s.x), da[j].v[i]);
                        carry[j].v[i] = __fmul2_rn(dh, decay[q][j][i]);
                    }
                    s1[j] = x1.x + x1.y, s2[j] = x2.x + x2.y, s3[j] = x3.x + x3.y;
                }
                // over the states, first step: the partner's other channel is this lane's first
                into[q] = s1[0] + from_lane(s1[1], 1);
                decays[q] = s2[0] + from_lane(s2[1], 1);
                ys[q] = s3[0] + from_lane(s3[1], 1);
                // over the warp's channels
                float* to = sums + (warp * kBwdTile + t) * 2 * NP;
                if constexpr (W >= 2) {
                    vb[0] = make_float2(vb[0].x + from_lane(vb[1].x, W / 2 * L), vb[0].y + from_lane(vb[1].y, W / 2 * L));
                    vc[0] = make_float2(vc[0].x + from_lane(vc[1].x, W / 2 * L), vc[0].y + from_lane(vc[1].y, W / 2 * L));
                }
                if constexpr (W >= 4) {
                    vb[0].x += from_lane(vb[0].y, W / 4 * L);
                    vc[0].x += from_lane(vc[0].y, W / 4 * L);
                }
                if constexpr (W >= 8) {
                    const bool which = (cl & (W / 8)) != 0;
                    float v = (which ? vc[0].x : vb[0].x) + from_lane(which ? vb[0].x : vc[0].x, W / 8 * L);
                    if constexpr (W >= 16) v += from_lane(v, W / 16 * L);
                    if (W < 16 || (cl & (W / 16)) == 0) to[(which ? NP : 0) + n0 + perm] = v;
                } else if constexpr (W == 4) {
                    to[n0 + perm] = vb[0].x;
                    to[NP + n0 + perm] = vc[0].x;
                } else if constexpr (W == 2) {
                    to[n0 + perm] = vb[0].x, to[n0 + (1 ^ perm)] = vb[0].y;
                    to[NP + n0 + perm] = vc[0].x, to[NP + n0 + (1 ^ perm)] = vc[0].y;
                } else {
                    *reinterpret_cast<float4*>(to + n0) = make_float4(vb[0].x, vb[0].y, vb[1].x, vb[1].y);
                    *reinterpret_cast<float4*>(to + NP + n0) = make_float4(vc[0].x, vc[0].y, vc[1].x, vc[1].y);
                }
            }
            // over the states: the lanes part the positions among themselves
            constexpr int kParts = L >= 8 ? 4 : L / 2, kMine = kBwdStep / kParts;
            int first = 0;
            if constexpr (L >= 4) {
                const bool upper = (sub & 2) != 0;
                first = upper ? 2 : 0;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    into[q] = (upper ? into[q + 2] : into[q]) + from_lane(upper ? into[q] : into[q + 2], 2);
                    decays[q] = (upper ? decays[q + 2] : decays[q]) + from_lane(upper ? decays[q] : decays[q + 2], 2);
                    ys[q] = (upper ? ys[q + 2] : ys[q]) + from_lane(upper ? ys[q] : ys[q + 2], 2);
                }
            }
            if constexpr (L >= 8) {
                const bool upper = (sub & 4) != 0;
                first += upper ? 1 : 0;
                into[0] = (upper ? into[1] : into[0]) + from_lane(upper ? into[0] : into[1], 4);
                decays[0] = (upper ? decays[1] : decays[0]) + from_lane(upper ? decays[0] : decays[1], 4);
                ys[0] = (upper ? ys[1] : ys[0]) + from_lane(upper ? ys[0] : ys[1], 4);
            }
#pragma unroll
            for (int m = 8; m < L; m *= 2) {
                into[0] += from_lane(into[0], m);
                decays[0] += from_lane(decays[0], m);
                ys[0] += from_lane(ys[0], m);
            }
            __syncwarp();       // all lanes have read these positions
            if (L < 16 || sub < 8) {
#pragma unroll
                for (int q = 0; q < kMine; ++q) {
                    const int t = w * kBwdStep + first + q;
                    const float2 s = step[t][ch[0]];
                    const float g = gs[t][ch[0]];
                    sum_d = fmaf(g, s.y, sum_d);
                    step[t][ch[0]] = make_float2(fmaf(into[q], s.x, skip[ch[0]] * g), fmaf(into[q], s.y, decays[q] * 0.6931471805599453f));
                    gs[t][ch[0]] = ys[q];
                }
            }
        }
        __syncthreads();
        // dB and dC of the CTA's channels
        for (int i = threadIdx.x; i < kBwdTile * 2 * NP; i += kThreads) {
            const int t = i / (2 * NP), j = i % (2 * NP), which = j / NP, n = j % NP;
            if (n >= N || t0 + t >= r.end) continue;
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < S::kWarps; ++w) s += sums[(w * kBwdTile + t) * 2 * NP + j];
            part_bc[((block * seq_rows_device(p.seqs) + dense + t0 + t) * 2 + which) * N + n] = s;
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int row = row_of(i);
            if (row >= kBwdTile || t0 + row >= r.end || col >= k.width) continue;
            float2 fu[4], fd[4], fz[4], fy[4], du[4], ddt[4], dz[4];
            ru[i].widen(fu);
            rdt[i].widen(fd);
            rz[i].widen(fz);
            rdy[i].widen(fy);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float4 s = *reinterpret_cast<const float4*>(&step[row][col + 2 * j]);
                du[j] = make_float2(s.x, s.z);
                ddt[j] = make_float2(s.y, s.w);
                if (p.softplus) {
                    const float2 o = *reinterpret_cast<const float2*>(&bias[col + 2 * j]);
                    ddt[j] = __fmul2_rn(ddt[j], make_float2(sigmoid(fd[j].x + o.x), sigmoid(fd[j].y + o.y)));
                }
                sum_bias[2 * j] += ddt[j].x;
                sum_bias[2 * j + 1] += ddt[j].y;
                if (z != nullptr) {
                    const float2 sum = __ffma2_rn(*reinterpret_cast<const float2*>(&skip[col + 2 * j]), fu[j],
                                                  *reinterpret_cast<const float2*>(&gs[row][col + 2 * j]));
                    dz[j] = __fmul2_rn(__fmul2_rn(fy[j], sum), make_float2(silu_slope(fz[j].x, sigmoid(fz[j].x)),
                                                                           silu_slope(fz[j].y, sigmoid(fz[j].y))));
                }
            }
            const long long o = (dense + t0 + row) * C + k.c;
            store8(static_cast<T*>(p.du) + o, du, col, k.width, aligned(p.du));
            store8(static_cast<T*>(p.ddt) + o, ddt, col, k.width, aligned(p.ddt));
            if (z != nullptr) store8(static_cast<T*>(p.dz) + o, dz, col, k.width, aligned(p.dz));
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
    for (int j = 0; j < 8; ++j) red[static_cast<int>(threadIdx.x) / kColumns * kStride + col + j] = sum_bias[j];
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

// dB and dC from the partial rows of a group's blocks.
template <typename T>
__global__ void __launch_bounds__(256) scan_bc_kernel(Scan p, const float* part, int per_group, long long rows) {
    pdl_trigger();
    pdl_wait();
    const int N = p.N, G = p.G;
    const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= rows * G * 2 * N) return;
    const long long row = i / (G * 2 * N);
    const int j = static_cast<int>(i - row * G * 2 * N), g = j / (2 * N), which = (j - g * 2 * N) / N, n = j % N;
    if (p.seqs.offsets != nullptr && (row < seq_offset(p.seqs, 0) || row >= seq_offset(p.seqs, p.seqs.count))) return;
    float s = 0.f;
    for (int k = 0; k < per_group; ++k) s += part[((static_cast<long long>(g) * per_group + k) * rows + row) * 2 * N + which * N + n];
    store_out(static_cast<T*>(which == 0 ? p.db : p.dc) + (row * G + g) * N + n, s);
}

// ---------------------------------------------------------------------------------- host

inline int channel_blocks(const Scan& p, int channels) { return p.G * ((p.C / p.G + channels - 1) / channels); }

// Forward: states to a lane and lanes to a channel, by the number of states.
#define DWC_SCAN_FWD_SHAPE(N, call)                 \
    if ((N) <= 8) return call(2, 4);                \
    if ((N) <= 16) return call(4, 4);               \
    if ((N) <= 32) return call(8, 4);               \
    if ((N) <= 64) return call(8, 8);               \
    return call(8, 16);
inline int fwd_channels(int N) {
#define DWC_CHANNELS(NS, L) (kThreads / (L))
    DWC_SCAN_FWD_SHAPE(N, DWC_CHANNELS)
#undef DWC_CHANNELS
}
inline int bwd_lanes(int N) { return N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : N <= 64 ? 16 : 32; }

// The workspaces, in floats.
struct FwdSpace {
    long long ends = 0, sums = 0;      // with chunks only
    explicit FwdSpace(const Scan& p) {
        if (p.span >= p.seqs.length) return;
        sums = seq_slots(p.seqs, p.span) * p.C;
        ends = sums * p.N;
    }
};
struct BwdSpace {
    long long bc, params, ends = 0, sums = 0;
    explicit BwdSpace(const Scan& p) {
        const long long slots = seq_slots(p.seqs, p.span), C = p.C;
        bc = static_cast<long long>(channel_blocks(p, 2 * kThreads / bwd_lanes(p.N))) * seq_rows(p.seqs) * 2 * p.N;
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

template <typename T, int NS, int L>
cudaError_t fwd_t(const Scan& p) {
    const int blocks = channel_blocks(p, kThreads / L);
    const long long grid = seq_slots(p.seqs, p.span) * blocks;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const FwdSpace space(p);
    float *ends = space.ends > 0 ? p.workspace : nullptr, *sums = p.workspace + space.ends;
    if (ends != nullptr) {
        cudaError_t err = launch_pdl(scan_fwd_kernel<T, NS, L, true>, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, p.stream,
                                     p, blocks, ends, sums);
        if (err == cudaSuccess) err = launch_join<false>(p, ends, sums, p.state);
        if (err != cudaSuccess) return err;
    }
    return launch_pdl(scan_fwd_kernel<T, NS, L, false>, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, p.stream, p, blocks,
                      ends, sums);
}

template <typename T, int NS, int L>
cudaError_t adjoint_t(const Scan& p, float* ends, float* sums) {
    const int blocks = channel_blocks(p, kThreads / L);
    const long long grid = seq_slots(p.seqs, p.span) * blocks;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const cudaError_t err = launch_pdl(scan_adjoint_kernel<T, NS, L>, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, p.stream,
                                       p, blocks, ends, sums);
    return err != cudaSuccess ? err : launch_join<true>(p, ends, sums, p.dfinal);
}
template <typename T>
cudaError_t adjoint(const Scan& p, float* ends, float* sums) {
#define DWC_ADJOINT(NS, L) (adjoint_t<T, NS, L>(p, ends, sums))
    DWC_SCAN_FWD_SHAPE(p.N, DWC_ADJOINT)
#undef DWC_ADJOINT
}

template <typename T, int L>
cudaError_t bwd_t(const Scan& p) {
    using S = BwdShape<L>;
    constexpr size_t smem = S::kFloats * sizeof(float);
    const int blocks = channel_blocks(p, S::kChannels);
    const long long slots = seq_slots(p.seqs, p.span), grid = slots * blocks, rows = seq_rows(p.seqs), C = p.C;
    const long long sums = (rows * p.G * 2 * p.N + 255) / 256;
    if (grid > 0x7fffffffLL || sums > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const BwdSpace space(p);
    float *bc = p.workspace, *params = bc + space.bc, *ends = params + space.params;
    static DeviceOnce once;
    cudaError_t err = opt_in_smem(scan_bwd_kernel<T, L>, once, static_cast<int>(smem));
    if (err == cudaSuccess && space.ends > 0) err = adjoint<T>(p, ends, ends + space.ends);
    if (err == cudaSuccess)
        err = launch_pdl(scan_bwd_kernel<T, L>, dim3(static_cast<unsigned>(grid)), dim3(kThreads), smem, p.stream, p, blocks,
                         static_cast<const float*>(space.ends > 0 ? ends : nullptr), bc, params);
    if (err == cudaSuccess && sums > 0)
        err = launch_pdl(scan_bc_kernel<T>, dim3(static_cast<unsigned>(sums)), dim3(256), 0, p.stream, p,
                         static_cast<const float*>(bc), blocks / p.G, rows);
    if (err == cudaSuccess) err = launch_row_sum(params, slots, C * (p.N + 2), {p.dA, p.dD, p.ddt_bias}, {C * p.N, C, C}, p.stream);
    return err;
}

template <typename T>
cudaError_t fwd(const Scan& p) {
#define DWC_FWD(NS, L) (fwd_t<T, NS, L>(p))
    DWC_SCAN_FWD_SHAPE(p.N, DWC_FWD)
#undef DWC_FWD
}

template <typename T>
cudaError_t bwd(const Scan& p) {
    switch (bwd_lanes(p.N)) {
        case 2: return bwd_t<T, 2>(p);
        case 4: return bwd_t<T, 4>(p);
        case 8: return bwd_t<T, 8>(p);
        case 16: return bwd_t<T, 16>(p);
        default: return bwd_t<T, 32>(p);
    }
}

}  // namespace scan
}  // namespace dwc

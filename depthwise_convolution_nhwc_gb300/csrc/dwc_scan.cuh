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
constexpr int kTile = kScanTile;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_fast(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

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
__device__ __forceinline__ float softplus(float v) { return (v < 0.f ? 0.f : v) + log1p_unit(expf(-fabsf(v))); }

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
    if (q.offsets != nullptr) return r.base / kTile + r.s + tile;
    const long long n = q.length == 0 ? 1 : (q.length + kTile - 1) / kTile;
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

// Raw vectors of 8 channels of a tile: thread i holds position i / (channels / 8), columns 8 * (i % ...).
template <typename T, int L>
struct Tile {
    static constexpr int kChannels = kThreads / L, kColumns = kChannels / 8;
    static constexpr int kActive = kTile * kColumns;       // threads that hold a vector (at most all)
    static_assert(kActive <= kThreads, "one vector a thread");
};

// B and C of a tile: vectors of 8 states, padded with zeros.
template <typename T, int NP>
struct StateRows {
    static constexpr int kVecs = NP / 8, kEach = (kTile * kVecs + kThreads - 1) / kThreads;
    Vec8<T> raw[kEach];
    __device__ __forceinline__ void fetch(const T* base, const RowsView& v, long long t0, long long end, int N) {
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int i = threadIdx.x + k * kThreads, t = i / kVecs, col = i % kVecs * 8;
            if (i < kTile * kVecs && t0 + t < end) load8(raw[k], base + (t0 + t) * v.row, col, N, v.vec && N % 8 == 0);
            else raw[k].zero();
        }
    }
    __device__ __forceinline__ void spread(float (*to)[NP]) const {
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int i = threadIdx.x + k * kThreads;
            if (i >= kTile * kVecs) continue;
            float2 f[4];
            raw[k].widen(f);
            float4* o = reinterpret_cast<float4*>(&to[i / kVecs][i % kVecs * 8]);
            o[0] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
            o[1] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
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

// -------------------------------------------------------------------------------- forward

template <typename T, int NS, int L>
__global__ void __launch_bounds__(kThreads) scan_fwd_kernel(Scan p, int blocks) {
    constexpr int kChannels = Tile<T, L>::kChannels, kColumns = Tile<T, L>::kColumns, NP = NS * L;
    __shared__ __align__(16) float2 step[kTile][kChannels];    // delta, delta * u
    __shared__ __align__(16) float bs[kTile][NP], cs[kTile][NP], ys[kTile][kChannels];
    pdl_trigger();
    pdl_wait();
    const long long slot = blockIdx.x / blocks;
    const Block k = block_of(p, static_cast<int>(blockIdx.x - slot * blocks), kChannels);
    const Piece r = find_piece(p.seqs, slot, p.seqs.length + 1);
    if (!r.some) return;
    const int C = p.C, N = p.N;
    const T *u = view_at<T>(p.u, p.seqs, r) + k.c, *dt = view_at<T>(p.dt, p.seqs, r) + k.c;
    const T* z = p.z.p == nullptr ? nullptr : view_at<T>(p.z, p.seqs, r) + k.c;
    const T *b = view_at<T>(p.b, p.seqs, r) + k.g * N, *c = view_at<T>(p.c, p.seqs, r) + k.g * N;
    T* y = static_cast<T*>(p.y) + dense_row(p.seqs, r) * C + k.c;
    const bool even = (C / p.G) % 8 == 0, vec_y = even && reinterpret_cast<uintptr_t>(p.y) % (8 * sizeof(T)) == 0;

    // as a holder of vectors
    const int row = threadIdx.x / kColumns, col = threadIdx.x % kColumns * 8;
    const bool holder = row < kTile && col < k.width;
    float bias[8], skip[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const bool in = holder && col + j < k.width;
        bias[j] = in && p.dt_bias != nullptr ? p.dt_bias[k.c + col + j] : 0.f;
        skip[j] = in && p.D != nullptr ? p.D[k.c + col + j] : 0.f;
    }
    // as a server of a channel's states
    const int ch = threadIdx.x / L, sub = threadIdx.x % L, n0 = sub * NS;
    const bool serves = ch < k.width;
    const long long mine = (static_cast<long long>(r.s) * C + k.c + ch) * N;
    float a2[NS], h[NS];
    get_states(a2, serves ? p.A + static_cast<long long>(k.c + ch) * N : nullptr, n0, N);
#pragma unroll
    for (int i = 0; i < NS; ++i) a2[i] *= kLog2e;
    get_states(h, serves && p.state != nullptr ? p.state + mine : nullptr, n0, N);

    Vec8<T> ru, rdt, rz, nu, ndt, nz;
    StateRows<T, NP> nb, nc;
    auto fetch = [&](long long t0) {
        nu.zero(), ndt.zero(), nz.zero();
        if (holder && t0 + row < r.end) {
            load8(nu, u + (t0 + row) * p.u.row, col, k.width, p.u.vec && even);
            load8(ndt, dt + (t0 + row) * p.dt.row, col, k.width, p.dt.vec && even);
            if (z != nullptr) load8(nz, z + (t0 + row) * p.z.row, col, k.width, p.z.vec && even);
        }
        nb.fetch(b, p.b, t0, r.end, N);
        nc.fetch(c, p.c, t0, r.end, N);
    };
    fetch(r.first);
    for (long long t0 = r.first; t0 < r.end; t0 += kTile) {
        ru = nu, rdt = ndt, rz = nz;
        if (row < kTile) {
            float2 fu[4], fd[4];
            ru.widen(fu);
            rdt.widen(fd);
            const bool in = t0 + row < r.end;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float d0 = fd[j].x + bias[2 * j], d1 = fd[j].y + bias[2 * j + 1];
                if (p.softplus) d0 = softplus(d0), d1 = softplus(d1);
                if (!in) d0 = d1 = 0.f;        // positions past the end leave the states alone
                step[row][col + 2 * j] = make_float2(d0, d0 * fu[j].x);
                step[row][col + 2 * j + 1] = make_float2(d1, d1 * fu[j].y);
            }
        }
        nb.spread(bs);
        nc.spread(cs);
        __syncthreads();
        if (t0 + kTile < r.end) fetch(t0 + kTile);
        if (p.saved != nullptr && serves)
            put_states(p.saved + (saved_slot(p.seqs, r, t0 / kTile) * C + k.c + ch) * N, h, n0, N);
#pragma unroll 1
        for (int t = 0; t < kTile; t += L) {
            float sums[L];
#pragma unroll
            for (int q = 0; q < L; ++q) {
                const float2 s = step[t + q][ch];
                float fb[NS], fc[NS];
                row_values(fb, &bs[t + q][n0]);
                row_values(fc, &cs[t + q][n0]);
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    h[i] = fmaf(exp2_fast(s.x * a2[i]), h[i], s.y * fb[i]);
                    sum = fmaf(fc[i], h[i], sum);
                }
                sums[q] = sum;
            }
            const float sum = parted<L>(sums, sub);
            ys[t + sub][ch] = sum;
        }
        __syncthreads();
        if (holder && t0 + row < r.end) {
            float2 fu[4], fz[4], f[4];
            ru.widen(fu);
            rz.widen(fz);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f[j].x = fmaf(skip[2 * j], fu[j].x, ys[row][col + 2 * j]);
                f[j].y = fmaf(skip[2 * j + 1], fu[j].y, ys[row][col + 2 * j + 1]);
                if (z != nullptr) {
                    f[j].x *= silu(fz[j].x);
                    f[j].y *= silu(fz[j].y);
                }
            }
            store8(y + (t0 + row) * C, f, col, k.width, vec_y);
        }
    }
    if (r.last && p.final_state != nullptr && serves) put_states(p.final_state + mine, h, n0, N);
}

// ------------------------------------------------------------------------------- backward

// Tiles from the last to the first.  From the state in front of a tile (kept by the forward pass)
// the states at every SB-th position are formed again; then, SB positions at a time from the last,
// a h[t-1] and a of each of them, in registers, and the gradients going back:
//     dh = g C + carry,  carry = a dh  (g: the gradient of the sum over the states and D u)
//     dC = sum_c g h,  dB = sum_c dh delta u,  dA += dh a h[t-1] delta
//     into = sum_n dh B,  decay = sum_n dh a h[t-1] A,  du = into delta + D g,  ddelta = into u + decay
// The sums of dB and dC over a CTA's channels go to partial rows, one per block of channels.
template <typename T, int NS, int L, int SB>
__global__ void __launch_bounds__(kThreads) scan_bwd_kernel(Scan p, int blocks, float* part_bc, float* part_a, float* part_d,
                                                            float* part_bias) {
    constexpr int kChannels = Tile<T, L>::kChannels, kColumns = Tile<T, L>::kColumns, NP = NS * L;
    constexpr int kWarps = kThreads / 32, kLanes = 32 / L;      // channels of a warp
    static_assert(SB % L == 0 || L % SB == 0, "parts");
    constexpr int kPart = SB < L ? SB : L;
    extern __shared__ __align__(16) float smem[];
    float2 (*step)[kChannels] = reinterpret_cast<float2 (*)[kChannels]>(smem);
    float (*bs)[NP] = reinterpret_cast<float (*)[NP]>(smem + kTile * kChannels * 2);
    float (*cs)[NP] = bs + kTile;
    float (*gs)[kChannels] = reinterpret_cast<float (*)[kChannels]>(cs + kTile);
    float (*into_s)[kChannels] = gs + kTile;
    float (*decay_s)[kChannels] = into_s + kTile;
    float (*ys)[kChannels] = decay_s + kTile;
    float* sums = reinterpret_cast<float*>(ys + kTile);        // warps x positions x (dB, dC)
    float* front = sums + kWarps * kTile * 2 * NP + threadIdx.x;    // states in front of every SB-th position
    pdl_trigger();
    pdl_wait();
    const long long slot = blockIdx.x / blocks;
    const int block = static_cast<int>(blockIdx.x - slot * blocks);
    const Block k = block_of(p, block, kChannels);
    const Piece r = find_piece(p.seqs, slot, p.seqs.length + 1);
    const int C = p.C, N = p.N;
    const bool even = (C / p.G) % 8 == 0;
    const long long dense = r.some ? dense_row(p.seqs, r) : 0;
    const auto aligned = [&](const void* t) { return even && reinterpret_cast<uintptr_t>(t) % (8 * sizeof(T)) == 0; };
    const T *u = view_at<T>(p.u, p.seqs, r) + k.c, *dt = view_at<T>(p.dt, p.seqs, r) + k.c, *dy = view_at<T>(p.dy, p.seqs, r) + k.c;
    const T* z = p.z.p == nullptr ? nullptr : view_at<T>(p.z, p.seqs, r) + k.c;
    const T *b = view_at<T>(p.b, p.seqs, r) + k.g * N, *c = view_at<T>(p.c, p.seqs, r) + k.g * N;

    const int row = threadIdx.x / kColumns, col = threadIdx.x % kColumns * 8;
    const bool holder = row < kTile && col < k.width;
    float bias[8], skip[8], sum_d[8], sum_bias[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const bool in = holder && col + j < k.width;
        bias[j] = in && p.dt_bias != nullptr ? p.dt_bias[k.c + col + j] : 0.f;
        skip[j] = in && p.D != nullptr ? p.D[k.c + col + j] : 0.f;
        sum_d[j] = sum_bias[j] = 0.f;
    }
    const int ch = threadIdx.x / L, sub = threadIdx.x % L, n0 = sub * NS;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool serves = ch < k.width;
    const long long mine = (static_cast<long long>(r.s) * C + k.c + ch) * N;
    float a2[NS], an[NS], carry[NS], da[NS];
    get_states(an, serves ? p.A + static_cast<long long>(k.c + ch) * N : nullptr, n0, N);
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        a2[i] = an[i] * kLog2e;
        da[i] = 0.f;
    }
    get_states(carry, serves && r.some && p.dfinal != nullptr ? p.dfinal + mine : nullptr, n0, N);

    const long long tiles = r.some ? (r.end - r.first + kTile - 1) / kTile : 0;
    for (long long tile = tiles - 1; tile >= 0; --tile) {
        const long long t0 = r.first + tile * kTile;
        const bool in = t0 + row < r.end;
        Vec8<T> ru, rdt, rz, rdy;
        ru.zero(), rdt.zero(), rz.zero(), rdy.zero();
        StateRows<T, NP> rb, rc;
        if (holder && in) {
            load8(ru, u + (t0 + row) * p.u.row, col, k.width, p.u.vec && even);
            load8(rdt, dt + (t0 + row) * p.dt.row, col, k.width, p.dt.vec && even);
            load8(rdy, dy + (t0 + row) * p.dy.row, col, k.width, p.dy.vec && even);
            if (z != nullptr) load8(rz, z + (t0 + row) * p.z.row, col, k.width, p.z.vec && even);
        }
        rb.fetch(b, p.b, t0, r.end, N);
        rc.fetch(c, p.c, t0, r.end, N);
        float h[NS];
        get_states(h, serves ? p.saved + (saved_slot(p.seqs, r, t0 / kTile) * C + k.c + ch) * N : nullptr, n0, N);
        __syncthreads();            // the last tile's sums have been read
        if (row < kTile) {
            float2 fu[4], fd[4], fz[4], fy[4];
            ru.widen(fu);
            rdt.widen(fd);
            rz.widen(fz);
            rdy.widen(fy);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float d0 = fd[j].x + bias[2 * j], d1 = fd[j].y + bias[2 * j + 1];
                if (p.softplus) d0 = softplus(d0), d1 = softplus(d1);
                if (!in) d0 = d1 = 0.f;
                step[row][col + 2 * j] = make_float2(d0, d0 * fu[j].x);
                step[row][col + 2 * j + 1] = make_float2(d1, d1 * fu[j].y);
                gs[row][col + 2 * j] = z != nullptr ? fy[j].x * silu(fz[j].x) : fy[j].x;
                gs[row][col + 2 * j + 1] = z != nullptr ? fy[j].y * silu(fz[j].y) : fy[j].y;
            }
        }
        rb.spread(bs);
        rc.spread(cs);
        __syncthreads();
#pragma unroll 1
        for (int w = 0; w < kTile / SB; ++w) {
#pragma unroll
            for (int i = 0; i < NS; ++i) front[(w * NS + i) * kThreads] = h[i];
            if (w == kTile / SB - 1) break;
#pragma unroll
            for (int q = 0; q < SB; ++q) {
                const float2 s = step[w * SB + q][ch];
                float fb[NS];
                row_values(fb, &bs[w * SB + q][n0]);
#pragma unroll
                for (int i = 0; i < NS; ++i) h[i] = fmaf(exp2_fast(s.x * a2[i]), h[i], s.y * fb[i]);
            }
        }
#pragma unroll 1
        for (int w = kTile / SB - 1; w >= 0; --w) {
            float held[SB][NS], decay[SB][NS];       // a h[t-1], a
#pragma unroll
            for (int i = 0; i < NS; ++i) h[i] = front[(w * NS + i) * kThreads];
#pragma unroll
            for (int q = 0; q < SB; ++q) {
                const float2 s = step[w * SB + q][ch];
                float fb[NS];
                row_values(fb, &bs[w * SB + q][n0]);
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    decay[q][i] = exp2_fast(s.x * a2[i]);
                    held[q][i] = decay[q][i] * h[i];
                    h[i] = fmaf(s.y, fb[i], held[q][i]);
                }
            }
            float s1[SB], s2[SB], s3[SB];
#pragma unroll
            for (int q = SB - 1; q >= 0; --q) {
                const int t = w * SB + q;
                const float2 s = step[t][ch];
                const float g = gs[t][ch];
                float fb[NS], fc[NS], v[2 * NS];
                row_values(fb, &bs[t][n0]);
                row_values(fc, &cs[t][n0]);
                s1[q] = s2[q] = s3[q] = 0.f;
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    const float dh = fmaf(g, fc[i], carry[i]);
                    const float now = fmaf(s.y, fb[i], held[q][i]);
                    const float x = dh * held[q][i];
                    v[i] = dh * s.y;
                    v[NS + i] = g * now;
                    s1[q] = fmaf(dh, fb[i], s1[q]);
                    s2[q] = fmaf(x, an[i], s2[q]);
                    s3[q] = fmaf(fc[i], now, s3[q]);
                    da[i] = fmaf(x, s.x, da[i]);
                    carry[i] = dh * decay[q][i];
                }
                // over the warp's channels: lanes of the same states part the 2 NS values among themselves
                int m = kLanes / 2, at_v = 0;
                constexpr int kV = 2 * NS;
#pragma unroll
                for (int half = kV / 2; half > 0 && m > 0; half >>= 1, m >>= 1) {
                    const bool upper = (lane / L & m) != 0;
                    if (upper) at_v += half;
#pragma unroll
                    for (int i = 0; i < half; ++i) {
                        const float keep = upper ? v[half + i] : v[i], send = upper ? v[i] : v[half + i];
                        v[i] = keep + __shfl_xor_sync(0xffffffffu, send, m * L);
                    }
                }
                constexpr int kHeld = kV > kLanes ? kV / kLanes : 1;        // values left to a lane
                if constexpr (kLanes > kV) {
#pragma unroll
                    for (; m > 0; m >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], m * L);
                }
#pragma unroll
                for (int i = 0; i < kHeld; ++i) {
                    const int j = at_v + i, which = j / NS, n = n0 + j % NS;
                    if (kLanes <= kV || (lane / L) % (kLanes / kV > 0 ? kLanes / kV : 1) == 0)
                        sums[((warp * kTile + t) * 2 + which) * NP + n] = v[i];
                }
            }
#pragma unroll
            for (int q = 0; q < SB; q += kPart) {
                float v1[L], v2[L], v3[L];
#pragma unroll
                for (int i = 0; i < L; ++i) {
                    v1[i] = i < kPart ? s1[q + (i < kPart ? i : 0)] : 0.f;
                    v2[i] = i < kPart ? s2[q + (i < kPart ? i : 0)] : 0.f;
                    v3[i] = i < kPart ? s3[q + (i < kPart ? i : 0)] : 0.f;
                }
                const float x1 = parted<L>(v1, sub), x2 = parted<L>(v2, sub), x3 = parted<L>(v3, sub);
                if (sub < kPart) {
                    into_s[w * SB + q + sub][ch] = x1;
                    decay_s[w * SB + q + sub][ch] = x2;
                    ys[w * SB + q + sub][ch] = x3;
                }
            }
        }
        __syncthreads();
        // dB and dC of the CTA's channels
        for (int i = threadIdx.x; i < kTile * 2 * N; i += kThreads) {
            const int t = i / (2 * N), j = i - t * 2 * N, which = j / N, n = j - which * N;
            if (t0 + t >= r.end) break;
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) s += sums[((w * kTile + t) * 2 + which) * NP + n];
            part_bc[(block * seq_rows_device(p.seqs) + dense + t0 + t) * 2 * N + j] = s;
        }
        if (holder && in) {
            float2 fu[4], fd[4], fz[4], fy[4], du[4], ddt[4], dz[4];
            ru.widen(fu);
            rdt.widen(fd);
            rz.widen(fz);
            rdy.widen(fy);
            const auto finish = [&](int j, float uu, float raw, float zz, float dyy, float& o_u, float& o_dt, float& o_z) {
                const float g = gs[row][col + j], into = into_s[row][col + j], delta = step[row][col + j].x;
                o_u = fmaf(into, delta, skip[j] * g);
                float d = fmaf(into, uu, decay_s[row][col + j]);
                if (p.softplus) d *= sigmoid(raw + bias[j]);
                o_dt = d;
                sum_d[j] = fmaf(g, uu, sum_d[j]);
                sum_bias[j] += d;
                if (z != nullptr) o_z = dyy * fmaf(skip[j], uu, ys[row][col + j]) * silu_slope(zz, sigmoid(zz));
            };
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                finish(2 * j, fu[j].x, fd[j].x, fz[j].x, fy[j].x, du[j].x, ddt[j].x, dz[j].x);
                finish(2 * j + 1, fu[j].y, fd[j].y, fz[j].y, fy[j].y, du[j].y, ddt[j].y, dz[j].y);
            }
            const long long o = (dense + t0 + row) * C + k.c;
            store8(static_cast<T*>(p.du) + o, du, col, k.width, aligned(p.du));
            store8(static_cast<T*>(p.ddt) + o, ddt, col, k.width, aligned(p.ddt));
            if (z != nullptr) store8(static_cast<T*>(p.dz) + o, dz, col, k.width, aligned(p.dz));
        }
    }
    if (serves) {
        if (r.some && p.dstate != nullptr) put_states(p.dstate + mine, carry, n0, N);
        put_states(part_a + (slot * C + k.c + ch) * N, da, n0, N);
    }
    // over the threads of a column
    __syncthreads();
    float* red = smem;
    if (row < kTile) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            red[(row * kChannels + col + j) * 2] = sum_d[j];
            red[(row * kChannels + col + j) * 2 + 1] = sum_bias[j];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < k.width * 2; i += kThreads) {
        float s = 0.f;
        for (int q = 0; q < kTile; ++q) s += red[q * kChannels * 2 + i];
        (i % 2 == 0 ? part_d : part_bias)[slot * C + k.c + i / 2] = s;
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

// Lanes to a channel by the number of states.
inline int lanes_of(int N) { return N <= 32 ? 4 : N <= 64 ? 8 : 16; }

template <typename T, int NS, int L>
cudaError_t fwd_t(const Scan& p) {
    const int blocks = channel_blocks(p, kThreads / L);
    const long long grid = seq_slots(p.seqs, p.seqs.length + 1) * blocks;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    return launch_pdl(scan_fwd_kernel<T, NS, L>, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, p.stream, p, blocks);
}

// The backward pass's workspace, in floats: partial dB and dC, dA, dD and the bias's gradient.
struct Partials {
    long long bc, a, d, total;
    explicit Partials(const Scan& p) {
        const long long slots = seq_slots(p.seqs, p.seqs.length + 1), C = p.C;
        bc = static_cast<long long>(channel_blocks(p, kThreads / lanes_of(p.N))) * seq_rows(p.seqs) * 2 * p.N;
        a = slots * C * p.N;
        d = slots * C;
        total = bc + a + 2 * d;
    }
};

template <typename T, int NS, int L, int SB>
cudaError_t bwd_t(const Scan& p) {
    constexpr int kChannels = kThreads / L, NP = NS * L;
    constexpr size_t smem = sizeof(float) * (kTile * kChannels * 6 + kTile * NP * 2 + kThreads / 32 * kTile * 2 * NP + kTile / SB * NS * kThreads);
    const int blocks = channel_blocks(p, kChannels);
    const long long slots = seq_slots(p.seqs, p.seqs.length + 1), grid = slots * blocks, rows = seq_rows(p.seqs);
    const Partials part(p);
    float *bc = p.workspace, *a = bc + part.bc, *d = a + part.a, *bias = d + part.d;
    static DeviceOnce once;
    cudaError_t err = opt_in_smem(scan_bwd_kernel<T, NS, L, SB>, once, static_cast<int>(smem));
    if (err != cudaSuccess) return err;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    err = launch_pdl(scan_bwd_kernel<T, NS, L, SB>, dim3(static_cast<unsigned>(grid)), dim3(kThreads), smem, p.stream, p, blocks,
                     bc, a, d, bias);
    const long long sums = (rows * p.G * 2 * p.N + 255) / 256;
    if (sums > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    if (err == cudaSuccess && sums > 0)
        err = launch_pdl(scan_bc_kernel<T>, dim3(static_cast<unsigned>(sums)), dim3(256), 0, p.stream, p,
                         static_cast<const float*>(bc), blocks / p.G, rows);
    const long long C = p.C;
    if (err == cudaSuccess) err = launch_row_sum(a, slots, C * p.N, C * p.N, p.dA, p.stream);
    if (err == cudaSuccess) err = launch_row_sum(d, slots, C, C, p.dD, p.stream);
    if (err == cudaSuccess) err = launch_row_sum(bias, slots, C, C, p.ddt_bias, p.stream);
    return err;
}

template <typename T>
cudaError_t fwd(const Scan& p) {
    if (p.N <= 8) return fwd_t<T, 2, 4>(p);
    if (p.N <= 16) return fwd_t<T, 4, 4>(p);
    if (p.N <= 32) return fwd_t<T, 8, 4>(p);
    if (p.N <= 64) return fwd_t<T, 8, 8>(p);
    return fwd_t<T, 8, 16>(p);
}

template <typename T>
cudaError_t bwd(const Scan& p) {
    if (p.N <= 8) return bwd_t<T, 2, 4, 8>(p);
    if (p.N <= 16) return bwd_t<T, 4, 4, 8>(p);
    if (p.N <= 32) return bwd_t<T, 8, 4, 4>(p);
    if (p.N <= 64) return bwd_t<T, 8, 8, 4>(p);
    return bwd_t<T, 8, 16, 4>(p);
}

}  // namespace scan
}  // namespace dwc

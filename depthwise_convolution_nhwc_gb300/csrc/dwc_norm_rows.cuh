// dwc_norm_rows.cuh -- layer norm and its residual form, forward and backward, on rows of up to
// 16384 channels held by a group of threads.
//
// Both passes are bound by memory: a row is read once, reduced in registers or shared memory and
// written once, 8 elements per access.  A group of threads serves one row:
//   rows of up to 8, 16 and 32 vectors: G = 8, 16, 32 lanes, one vector each; up to 64 and 128
//   vectors: a warp with 2 and 4; longer rows (up to 4 vectors x 512 threads): several warps.
//
// Alignment.  A dense row of C channels starts (row * C) mod 8 elements past a vector boundary, and
// so does every tensor of the call if its base is aligned and its row stride is congruent to C
// modulo 8.  The group works on the vectors of the address, shifted against the row by that
// amount; the first and last one may hang over and are masked (kAligned: C is a multiple of 8
// and nothing is).  Groups advance by a multiple of 8 rows, so a group's shift never changes:
// its columns (parameters, gradient sums) stay its own.  The dropout's blocks of 8 elements
// coincide with these vectors.
#pragma once

#include <algorithm>

#include "dwc_norm_device.cuh"

namespace dwc {
namespace norm {

constexpr int kRowVecs = 4;              // vectors per thread where several warps serve a row
constexpr int kWarpCta = 256;            // threads of a CTA whose warps or lane groups serve rows
constexpr int kMaxCta = 512;             // threads of a CTA otherwise: 128 registers each
constexpr int kDynamicSmem = 225 * 1024;

// Vectors that the longest-shifted row of C channels touches.
inline int row_vectors(int C) {
    int g = 8;                            // gcd(C, 8): the shifts are its multiples
    while (C % g != 0) g /= 2;
    return (C + (8 - g) + 7) / 8;
}

// Sum over the G lanes of a group.
template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int m = G / 2; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}

// Elements that warp `warp` of a group of `threads` threads holds of a row.
__device__ __forceinline__ int warp_columns(int warp, int threads, int shift, int C) {
    int n = 0;
#pragma unroll
    for (int k = 0; k < kRowVecs; ++k) {
        const int lo = max(0, (k * threads + warp * 32) * 8 - shift);
        const int hi = min(C, (k * threads + warp * 32 + 32) * 8 - shift);
        n += max(0, hi - lo);
    }
    return n;
}

// Where a group finds 8 consecutive parameters in fp32: the caller's own fp32 array where the
// vectors line up with it, else a copy in shared memory laid out along the group's shifted
// vectors (written once per group, read for every row).
struct ParamSource {
    const float* p = nullptr;            // indexed by column + shift
    bool present = false;
    __device__ __forceinline__ void get(float2 (&f)[4], int at, float absent) const {
        if (!present) {
#pragma unroll
            for (int k = 0; k < 4; ++k) f[k] = both(absent);
            return;
        }
        const float4 a = *reinterpret_cast<const float4*>(p + at), b = *reinterpret_cast<const float4*>(p + at + 4);
        f[0] = make_float2(a.x, a.y), f[1] = make_float2(a.z, a.w);
        f[2] = make_float2(b.x, b.y), f[3] = make_float2(b.z, b.w);
    }
};

__device__ __forceinline__ float shifted_param(const void* p, int type, int c, int C, float absent) {
    return in_row(c, C) ? load_param(p, type, c, absent) : 0.f;
}

// ------------------------------------------------------------------------------- forward
//
// Row statistics: each warp (or lane group) takes the mean of its own elements, then the sum of
// squares about it, and the warps of a group are merged by their counts (Chan, Golub and LeVeque,
// "Updating formulae and a pairwise algorithm for computing sample variances", 1979): one
// barrier per row, and no cancellation however far the mean lies from zero.

// Elements col .. col + 7: a whole vector where it lies within [low, room) of the row's start (the
// tensor's extent: neighbouring rows' elements are masked after), else the row's own elements.
template <bool kAligned, typename T>
__device__ __forceinline__ void load_row8(Vec8<T>& v, const T* row, int col, int C, int low, int room) {
    if (kAligned || (col >= low && col + 8 <= room)) {
        v.load(row + col);
    } else {
        v.zero();
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (in_row(col + j, C)) v.set(j, row[col + j]);
    }
}

// G > 0: lanes of a row's group, NV vectors a lane, U rows at a time (their loads in flight
// together); G == 0: the CTA serves a row.  `staged`: parameters go through shared memory.
template <typename TS, typename TB, bool kAdd, bool kAligned, int G, int NV, int U>
__global__ void __launch_bounds__(G > 0 ? kWarpCta : kMaxCta) norm_fwd_rows_kernel(NormFwd p, int staged) {
    extern __shared__ __align__(16) float smem[];
    __shared__ float2 merge[2][32];
    constexpr bool kCta = G == 0;
    constexpr int GW = kCta ? 32 : G;                              // lanes that reduce by shuffles
    const int width = kCta ? blockDim.x : G;                       // threads of a group
    const int lane = kCta ? threadIdx.x : threadIdx.x % GW;
    const int local = kCta ? 0 : threadIdx.x / GW;                 // group within the CTA
    const int per_cta = kCta ? 1 : kWarpCta / GW;
    const int groups = gridDim.x * per_cta;
    const int group = blockIdx.x * per_cta + local;
    const int C = p.C;
    const int shift = kAligned ? 0 : static_cast<int>((static_cast<long long>(group) * C) & 7);
    const float inv = 1.f / static_cast<float>(C);
    // (an update in place overwrites the neighbouring rows: then only the row's own elements are read)
    const bool whole = !kAdd || p.z != p.in;
    const int low = whole ? -8 : 0;
    pdl_trigger();
    pdl_wait();
    DropState drop;
    if (kAdd) drop.init(p.drop);

    // parameters: registers for one vector a lane, else read (or staged) per use
    float2 gam[4], bet[4];
    ParamSource gsrc, bsrc;
    if constexpr (NV == 1) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int c = lane * 8 + 2 * k - shift;
            gam[k] = make_float2(shifted_param(p.gamma, p.param_type, c, C, 1.f), shifted_param(p.gamma, p.param_type, c + 1, C, 1.f));
            bet[k] = make_float2(shifted_param(p.beta, p.param_type, c, C, 0.f), shifted_param(p.beta, p.param_type, c + 1, C, 0.f));
        }
    } else {
        gsrc.present = staged || p.gamma != nullptr;
        bsrc.present = staged || p.beta != nullptr;
        gsrc.p = static_cast<const float*>(p.gamma);
        bsrc.p = static_cast<const float*>(p.beta);
        if (staged) {
            const int span = width * NV * 8;
            float* g = smem + local * 2 * span;
            for (int i = lane; i < span; i += width) {
                g[i] = shifted_param(p.gamma, p.param_type, i - shift, C, 1.f);
                g[span + i] = shifted_param(p.beta, p.param_type, i - shift, C, 0.f);
            }
            gsrc.p = g;
            bsrc.p = g + span;
            if (kCta) __syncthreads(); else __syncwarp();
        }
    }
    // elements of this thread's warp or group, and (lane l) of warp l of the CTA
    const int mine = kCta ? warp_columns(threadIdx.x >> 5, width, shift, C) : C;
    const int peer = kCta && (threadIdx.x & 31) < (width >> 5) ? warp_columns(threadIdx.x & 31, width, shift, C) : 0;
    const float mine_inv = mine > 0 ? 1.f / static_cast<float>(mine) : 0.f;
    int parity = 0;

    // (the lane groups of a warp stay together: the warp goes on while its first group has a row)
    const int in_warp = kCta ? 0 : local % (32 / GW);
    for (long long r0 = group; r0 - in_warp < p.rows; r0 += static_cast<long long>(groups) * U) {
        Vec8<TS> raw[U][NV];
        Vec8<TB> branch[kAdd ? U : 1][kAdd ? NV : 1];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long r = r0 + static_cast<long long>(u) * groups;
            // elements from the row's start to the tensor's end, at least
            const int room = kAligned ? 0 : whole ? static_cast<int>(min((p.rows - r) * C, 1LL << 30)) : C;
            const TS* in = static_cast<const TS*>(p.in) + r * p.ld_in;
            const TB* x = static_cast<const TB*>(p.x) + r * p.ld_x;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int col = (k * width + lane) * 8 - shift;
                raw[u][k].zero();
                if constexpr (kAdd) branch[u][k].zero();
                if (r < p.rows && col < C) {
                    load_row8<kAligned>(raw[u][k], in, col, C, low, room);
                    if constexpr (kAdd) load_row8<kAligned>(branch[u][k], x, col, C, low, room);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long r = r0 + static_cast<long long>(u) * groups;
            const bool live = r < p.rows;
            float2 v[NV][4], s2 = both(0.f);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int col = (k * width + lane) * 8 - shift;
                raw[u][k].widen(v[k]);
                if constexpr (kAdd) {
                    float2 b[4];
                    branch[u][k].widen(b);
                    if (drop.threshold != 0 && live && col < C)
                        drop8(drop, b, static_cast<uint64_t>(r * C + col) >> 3);
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[k][j] = __fadd2_rn(v[k][j], b[j]);
                    if (live && col < C) store_row8<kAligned>(static_cast<TS*>(p.z) + r * C, v[k], col, C);
                }
                if (!kAligned && !inside(col, C)) mask8(v[k], col, C);
#pragma unroll
                for (int j = 0; j < 4; ++j) s2 = __fadd2_rn(s2, v[k][j]);
            }
            float mean = group_sum<GW>(s2.x + s2.y) * mine_inv;
            float2 q2 = both(0.f);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int col = (k * width + lane) * 8 - shift;
                if (col >= C) continue;
                float2 d[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) d[j] = __fadd2_rn(v[k][j], both(-mean));
                if (!kAligned && !inside(col, C)) mask8(d, col, C);
#pragma unroll
                for (int j = 0; j < 4; ++j) q2 = __ffma2_rn(d[j], d[j], q2);
            }
            float q = group_sum<GW>(q2.x + q2.y);
            if (kCta) {
                const int w = threadIdx.x & 31;
                if (w == 0) merge[parity][threadIdx.x >> 5] = make_float2(mean, q);
                __syncthreads();
                const float2 m = w < (width >> 5) ? merge[parity][w] : make_float2(0.f, 0.f);
                parity ^= 1;
                const float n = static_cast<float>(peer);
                mean = warp_sum(n * m.x) * inv;
                const float d = m.x - mean;
                q = warp_sum(peer > 0 ? fmaf(n * d, d, m.y) : 0.f);
            }
            const float rstd = 1.f / sqrtf(q * inv + p.eps);
            if (!live) continue;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int at = (k * width + lane) * 8, col = at - shift;
                if (col >= C) continue;
                if constexpr (NV > 1) {
                    gsrc.get(gam, at, 1.f);
                    bsrc.get(bet, at, 0.f);
                }
                float2 y[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 xhat = __fmul2_rn(__fadd2_rn(v[k][j], both(-mean)), both(rstd));
                    y[j] = __ffma2_rn(xhat, gam[j], bet[j]);
                }
                store_row8<kAligned>(static_cast<TB*>(p.y) + r * C, y, col, C);
            }
            if (lane == 0) {
                if (p.mean != nullptr) p.mean[r] = mean;
                if (p.rstd != nullptr) p.rstd[r] = rstd;
            }
        }
    }
}

// ------------------------------------------------------------------------------ backward

// Asynchronous copies of one row's tensors into the thread group's own part of shared memory.
// Each thread holds 8 elements of every vector slot: one 16-byte granule of a 16-bit type or two of
// fp32, of which the lanes of a warp copy consecutive ones (whole sectors).  A warp's granules stay
// in the tensor's order, so each copy fills 512 contiguous bytes; the fp32 reads then meet in
// banks two by two, which costs little: with the halves of the vectors parted into two planes
// (no conflicts) the copies themselves were the limit, 238 us instead of 185 for 16384 x 4096 with
// an fp32 stream.  Vectors past the row's end are filled with zeros (a copy of no bytes), so the
// arithmetic needs no branches.  Granules that hang over the row's ends are copied whole while
// they stay inside the tensor (the reader masks the neighbouring rows' elements); at the
// tensor's very end single elements are stored instead.
__device__ __forceinline__ void copy16(void* dst, const void* src, bool some) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(some ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <bool kAligned, typename T>
__device__ __forceinline__ void copy_granule(uint4* dst, const T* row, int col, int C, int room) {
    constexpr int n = 16 / sizeof(T);
    const bool some = col < C;
    if (kAligned || !some || col + n <= room) {
        copy16(dst, row + (some ? col : 0), some);
    } else {
        T* to = reinterpret_cast<T*>(dst);
#pragma unroll
        for (int j = 0; j < n; ++j)
            if (in_row(col + j, C)) to[j] = row[col + j];
    }
}

// One vector slot of the lanes of a (sub-)warp of GW lanes: `slot` is the thread's own first granule,
// `col` its first element.
template <bool kAligned, typename T, int GW>
__device__ __forceinline__ void copy_slot(uint4* slot, const T* row, int lane, int col, int C, int room) {
    if constexpr (sizeof(T) == 2) {
        copy_granule<kAligned>(slot, row, col, C, room);
    } else {
        const int first = col - 4 * lane;       // this lane's granule of the group's 2 * GW
        copy_granule<kAligned>(slot - lane, row, first, C, room);
        copy_granule<kAligned>(slot - lane + GW, row, first + 4 * GW, C, room);
    }
}

template <typename T>
__device__ __forceinline__ void read_slot(float2 (&f)[4], const uint4* slot) {
    if constexpr (sizeof(T) == 2) {
        Vec8<T> v;
        v.u = *slot;
        v.widen(f);
    } else {
        const float4 a = reinterpret_cast<const float4*>(slot)[0], b = reinterpret_cast<const float4*>(slot)[1];
        f[0] = make_float2(a.x, a.y), f[1] = make_float2(a.z, a.w);
        f[2] = make_float2(b.x, b.y), f[3] = make_float2(b.z, b.w);
    }
}

// CTAs per SM that the register budget allows: 80 registers a thread for one vector, 128 for 2 and
// 4, of which 16 a vector hold the gradient sums and 8 gamma.
constexpr int bwd_min_ctas(int G, int NV) { return G == 0 ? 1 : NV == 1 ? 3 : 2; }

// Barrier of one group of `threads` threads (a multiple of 32) of the CTA.
__device__ __forceinline__ void group_barrier(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Sums of 2 R values over the GW lanes of a group, R = 1 or 2: the lanes part the values among
// themselves (halves, then quarters), so that log2(GW) steps serve all.  Lanes lane / (GW / 2R) == q
// return sum q of v[0], v[1], ...
template <int GW, int R>
__device__ __forceinline__ float parted_sum(const float (&v)[2 * R], int lane) {
    float a = v[0], b = v[1];
    int m = GW / 2;
    if constexpr (R == 2) {
        const bool upper = (lane & m) != 0;
        const float c = upper ? v[0] : v[2], d = upper ? v[1] : v[3];
        a = (upper ? v[2] : v[0]) + __shfl_xor_sync(0xffffffffu, c, m);
        b = (upper ? v[3] : v[1]) + __shfl_xor_sync(0xffffffffu, d, m);
        m /= 2;
    }
    const bool upper = (lane & m) != 0;
    float t = (upper ? b : a) + __shfl_xor_sync(0xffffffffu, upper ? a : b, m);
#pragma unroll
    for (m /= 2; m > 0; m >>= 1) t += __shfl_xor_sync(0xffffffffu, t, m);
    return t;
}

// Each thread keeps the sums of dy * xhat and dy of its columns in registers over all rows of its
// group; at the end the groups of a CTA are added in order and the CTA writes one row of partial
// sums.  The sums (and gamma, up to two vectors a thread) take the registers, so the rows wait in
// shared memory, S times R rows per group, and are read twice there (before and after a row's
// two means are known).  R rows go through together: one reduction and one barrier for both,
// and two independent chains of latencies.  G == 0: groups of `group_threads` threads, several
// to a CTA where they are short: one CTA per SM, so that there are few rows of partial sums.
// kAdd: the residual form (dz, a branch gradient, dropout).
template <typename TS, typename TB, bool kAdd, bool kAligned, int G, int NV, int R, int S>
__global__ void __launch_bounds__(G > 0 ? kWarpCta : kMaxCta, bwd_min_ctas(G, NV))
norm_bwd_rows_kernel(NormBwd p, int staged, int group_threads) {
    extern __shared__ __align__(16) float smem[];
    __shared__ float merge[2][2 * R][kMaxCta / 32];
    constexpr bool kCta = G == 0;                  // several warps serve a row
    constexpr bool kHeld = NV <= 2;                // gamma stays in registers
    constexpr int GW = kCta ? 32 : G;              // lanes whose vectors are adjacent
    constexpr int kBranch = sizeof(TB) / 2, kStream = sizeof(TS) / 2;  // granules of a slot
    const int threads = kCta ? blockDim.x : kWarpCta;
    const int width = kCta ? group_threads : G;
    const int local = threadIdx.x / width;         // group within the CTA
    const int lane = threadIdx.x - local * width;
    const int sub = threadIdx.x % GW;
    const int per_cta = threads / width;
    const int groups = gridDim.x * per_cta;
    const int group = blockIdx.x * per_cta + local;
    const int C = p.C;
    const int shift = kAligned ? 0 : static_cast<int>((static_cast<long long>(group) * C) & 7);
    const float inv = 1.f / static_cast<float>(C);
    const bool has_dz = kAdd && p.dz != nullptr;
    const bool has_branch = kAdd && p.d_branch != nullptr;
    // shared memory: stage, row, then slot (dy, z, dz of each vector), then thread
    const int z_at = NV * kBranch * threads, dz_at = z_at + NV * kStream * threads;
    const int row_granules = dz_at + (has_dz ? NV * kStream * threads : 0);
    uint4* const slots = reinterpret_cast<uint4*>(smem);
    const int mine_b = threadIdx.x * kBranch, mine_s = threadIdx.x * kStream;   // this thread's granules of a slot
    pdl_trigger();
    pdl_wait();
    DropState drop;
    if (kAdd) drop.init(p.drop);

    auto fetch = [&](int stage, long long r0) {
#pragma unroll
        for (int u = 0; u < R; ++u) {
            const long long r = r0 + static_cast<long long>(u) * groups;
            if (r >= p.rows) continue;
            // elements from the row's start to the tensor's end, at least
            const int room = kAligned ? 0 : static_cast<int>(min((p.rows - r) * C, 1LL << 30));
            uint4* to = slots + (stage * R + u) * row_granules;
            const TB* dy = static_cast<const TB*>(p.dy) + r * p.ld_dy;
            const TS* z = static_cast<const TS*>(p.z) + r * p.ld_z;
            const TS* dz = has_dz ? static_cast<const TS*>(p.dz) + r * p.ld_dz : nullptr;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int col = (k * width + lane) * 8 - shift;
                copy_slot<kAligned, TB, GW>(to + k * kBranch * threads + mine_b, dy, sub, col, C, room);
                copy_slot<kAligned, TS, GW>(to + z_at + k * kStream * threads + mine_s, z, sub, col, C, room);
            }
            if (has_dz) {
#pragma unroll
                for (int k = 0; k < NV; ++k)
                    copy_slot<kAligned, TS, GW>(to + dz_at + k * kStream * threads + mine_s, dz, sub,
                                                (k * width + lane) * 8 - shift, C, room);
            }
        }
        copy_commit();
    };
#pragma unroll
    for (int i = 0; i < S; ++i) fetch(i, group + static_cast<long long>(i) * R * groups);

    // gamma: registers for one or two vectors a thread, else the caller's array (aligned fp32) or a
    // copy along the shifted vectors, read per use
    float2 gam[kHeld ? NV : 1][4];
    const float* gsrc = static_cast<const float*>(p.gamma);
    int last = C - 8;                               // the last whole vector there
    if constexpr (kHeld) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = (k * width + lane) * 8 + 2 * j - shift;
                gam[k][j] = make_float2(shifted_param(p.gamma, p.param_type, c, C, 1.f),
                                        shifted_param(p.gamma, p.param_type, c + 1, C, 1.f));
            }
    } else if (staged) {
        const int span = width * NV * 8;
        float* g = smem + S * R * row_granules * 4 + local * span;
        for (int i = lane; i < span; i += width) g[i] = shifted_param(p.gamma, p.param_type, i - shift, C, 1.f);
        gsrc = g;
        last = span - 8;
        if (kCta) group_barrier(1 + local, width); else __syncwarp();
    }
    auto gamma_of = [&](int k) -> const float2(&)[4] {
        if constexpr (kHeld) {
            return gam[k];
        } else {
            const float* g = gsrc + min((k * width + lane) * 8, last);
            const float4 a = *reinterpret_cast<const float4*>(g), b = *reinterpret_cast<const float4*>(g + 4);
            gam[0][0] = make_float2(a.x, a.y), gam[0][1] = make_float2(a.z, a.w);
            gam[0][2] = make_float2(b.x, b.y), gam[0][3] = make_float2(b.z, b.w);
            return gam[0];
        }
    };
    float2 sum_g[NV][4], sum_b[NV][4];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) sum_g[k][j] = sum_b[k][j] = both(0.f);
    int parity = 0, stage = 0;
    float next_mean[R], next_rstd[R];
    auto fetch_stats = [&](long long r0) {
#pragma unroll
        for (int u = 0; u < R; ++u) {
            const long long r = r0 + static_cast<long long>(u) * groups;
            next_mean[u] = r < p.rows ? p.mean[r] : 0.f;
            next_rstd[u] = r < p.rows ? p.rstd[r] : 0.f;
        }
    };
    fetch_stats(group);

    const long long step = static_cast<long long>(R) * groups;
    const int in_warp = kCta ? 0 : local % (32 / GW);
    for (long long r0 = group; r0 - in_warp < p.rows; r0 += step) {
        float mean[R], rstd[R];
#pragma unroll
        for (int u = 0; u < R; ++u) {
            mean[u] = next_mean[u];
            rstd[u] = next_rstd[u];
        }
        fetch_stats(r0 + step);
        copy_wait<S - 1>();
        __syncwarp();
        const uint4* from = slots + stage * R * row_granules;
        float s[2 * R];
#pragma unroll
        for (int u = 0; u < R; ++u) {
            float2 s1 = both(0.f), s2 = both(0.f);
            // (no barrier and no shuffle in here: a warp's groups may enter apart)
            if (r0 + static_cast<long long>(u) * groups < p.rows) {
                const uint4* row = from + u * row_granules;
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    float2 f[4], x[4];
                    read_slot<TB>(f, row + k * kBranch * threads + mine_b);
                    read_slot<TS>(x, row + z_at + k * kStream * threads + mine_s);
                    const float2(&gk)[4] = gamma_of(k);
                    if constexpr (!kAligned) {
                        const int col = (k * width + lane) * 8 - shift;
                        if (!inside(col, C)) {
                            mask8(f, col, C);
                            mask8(x, col, C);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 xhat = __fmul2_rn(__fadd2_rn(x[j], both(-mean[u])), both(rstd[u]));
                        const float2 a = __fmul2_rn(f[j], gk[j]);
                        s1 = __fadd2_rn(s1, a);
                        s2 = __ffma2_rn(a, xhat, s2);
                        sum_g[k][j] = __ffma2_rn(f[j], xhat, sum_g[k][j]);
                        sum_b[k][j] = __fadd2_rn(sum_b[k][j], f[j]);
                    }
                }
            }
            s[2 * u] = s1.x + s1.y;
            s[2 * u + 1] = s2.x + s2.y;
        }
        constexpr int kPart = GW / (2 * R);   // lanes that hold one of the sums
        float t = parted_sum<GW, R>(s, sub);
        if constexpr (kCta) {
            // the warps' sums: lane l of every warp takes sum l / kPart of warps l % kPart, ...
            if (sub % kPart == 0) merge[parity][sub / kPart][threadIdx.x >> 5] = t;
            group_barrier(1 + local, width);
            const int warps = width >> 5, first = local * warps;
            t = 0.f;
            for (int w = sub % kPart; w < warps; w += kPart) t += merge[parity][sub / kPart][first + w];
#pragma unroll
            for (int m = kPart / 2; m > 0; m >>= 1) t += __shfl_xor_sync(0xffffffffu, t, m);
            parity ^= 1;
        }
#pragma unroll
        for (int q = 0; q < 2 * R; ++q) s[q] = __shfl_sync(0xffffffffu, t, q * kPart, GW);
#pragma unroll
        for (int u = 0; u < R; ++u) {
            const long long r = r0 + static_cast<long long>(u) * groups;
            if (r >= p.rows) continue;        // (no barrier and no shuffle below)
            // dx = rstd (a - c1 - xhat c2) = rstd a - k1 - (x - mean) k2
            const float k1 = rstd[u] * s[2 * u] * inv, k2 = rstd[u] * rstd[u] * s[2 * u + 1] * inv;
            const uint4* row = from + u * row_granules;
            TS* ds = static_cast<TS*>(p.d_stream) + r * C;
            TB* db = has_branch ? static_cast<TB*>(p.d_branch) + r * C : nullptr;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int col = (k * width + lane) * 8 - shift;
                float2 f[4], x[4], g[4];
                read_slot<TB>(f, row + k * kBranch * threads + mine_b);
                read_slot<TS>(x, row + z_at + k * kStream * threads + mine_s);
                const float2(&gk)[4] = gamma_of(k);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 a = __ffma2_rn(__fmul2_rn(f[j], gk[j]), both(rstd[u]), both(-k1));
                    g[j] = __ffma2_rn(__fadd2_rn(x[j], both(-mean[u])), both(-k2), a);
                }
                if (has_dz) {
                    read_slot<TS>(x, row + dz_at + k * kStream * threads + mine_s);
#pragma unroll
                    for (int j = 0; j < 4; ++j) g[j] = __fadd2_rn(g[j], x[j]);
                }
                if (col < C) {
                    store_row8<kAligned>(ds, g, col, C);
                    if (has_branch) {
                        if (drop.threshold != 0) drop8(drop, g, static_cast<uint64_t>(r * C + col) >> 3);
                        store_row8<kAligned>(db, g, col, C);
                    }
                }
            }
        }
        __syncwarp();   // all lanes have read the stage
        fetch(stage, r0 + S * step);
        if (++stage == S) stage = 0;
    }
    copy_wait<0>();
    if (p.partial == nullptr) return;
    float* part = p.partial + static_cast<size_t>(blockIdx.x) * 2 * C;
    const bool combine = per_cta > 1;
    if (combine) __syncthreads();   // no group reads its rows or parameters any more
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int col = (k * width + lane) * 8 - shift;
        float* to = combine ? smem + local * 2 * C : part;   // the groups' sums, [group][2][C]
        if (kAligned) {
            if (col >= C) continue;
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
                const float2 *g = &sum_g[k][j], *b = &sum_b[k][j];
                *reinterpret_cast<float4*>(to + col + 2 * j) = make_float4(g[0].x, g[0].y, g[1].x, g[1].y);
                *reinterpret_cast<float4*>(to + C + col + 2 * j) = make_float4(b[0].x, b[0].y, b[1].x, b[1].y);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = col + j;
                if (!in_row(c, C)) continue;
                to[c] = j & 1 ? sum_g[k][j / 2].y : sum_g[k][j / 2].x;
                to[C + c] = j & 1 ? sum_b[k][j / 2].y : sum_b[k][j / 2].x;
            }
        }
    }
    if (!combine) return;
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * C; i += threads) {
        float t = 0.f;
        for (int g = 0; g < per_cta; ++g) t += smem[g * 2 * C + i];
        part[i] = t;
    }
}

// ------------------------------------------------------------------------------- launches

// What a launch needs to know of its kernel, asked from the runtime once per kernel.
struct KernelFacts {
    DeviceOnce smem;
    std::atomic<int> regs{0};
    template <class K>
    int registers(K kern) {
        int r = regs.load(std::memory_order_relaxed);
        if (r == 0) {
            r = kernel_regs(kern, 128);
            regs.store(r, std::memory_order_relaxed);
        }
        return r;
    }
};

// CTAs for `want` of them: at most what the SMs hold together, in eights (a group's rows are a
// multiple of 8 apart, see the head of this file).
inline long long persistent_grid(long long want, size_t smem, int threads, int regs) {
    const long long all = static_cast<long long>(device_info().sm_count) * resident_ctas(smem, threads, regs);
    return std::min(want, std::max(8LL, all / 8 * 8));
}

inline bool params_line_up(const void* gamma, const void* beta, int type, int C) {
    return C % 8 == 0 && (type == kF32 || (gamma == nullptr && beta == nullptr)) &&
           (reinterpret_cast<uintptr_t>(gamma) | reinterpret_cast<uintptr_t>(beta)) % 16 == 0;
}

template <typename TS, typename TB, bool kAdd, bool kAligned, int G, int NV, int U>
cudaError_t fwd_launch(const NormFwd& p, int vectors) {
    auto kern = norm_fwd_rows_kernel<TS, TB, kAdd, kAligned, G, NV, U>;
    const int threads = G > 0 ? kWarpCta : (vectors + NV * 32 - 1) / (NV * 32) * 32;
    const int per_cta = G > 0 ? kWarpCta / G : 1;
    const int staged = NV > 1 && !params_line_up(p.gamma, p.beta, p.param_type, p.C);
    const size_t bytes = staged ? static_cast<size_t>(threads) * NV * 8 * 2 * sizeof(float) : 0;
    static KernelFacts facts;
    const cudaError_t err = opt_in_smem(kern, facts.smem, kDynamicSmem);
    if (err != cudaSuccess) return err;
    const long long grid = persistent_grid((p.rows + per_cta - 1) / per_cta, bytes, threads, facts.registers(kern));
    return launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(threads), bytes, p.stream, p, staged);
}

// Groups of `width` threads in a CTA: several only once there is a row for every SM.
inline int row_groups(long long rows, int width) {
    return static_cast<int>(std::max(1LL, std::min<long long>(kMaxCta / width, rows / device_info().sm_count)));
}

// Bytes a thread's vector slots take per stage.
template <typename TS, typename TB>
size_t slot_bytes(const NormBwd& p) {
    return 8 * (sizeof(TB) + sizeof(TS) * (p.dz != nullptr ? 2 : 1));
}

template <typename TS, typename TB, bool kAdd, bool kAligned, int G, int NV, int R, int S>
cudaError_t bwd_launch(const NormBwd& p, int vectors) {
    auto kern = norm_bwd_rows_kernel<TS, TB, kAdd, kAligned, G, NV, R, S>;
    const int width = G > 0 ? G : (vectors + NV * 32 - 1) / (NV * 32) * 32;
    const int per_cta = G > 0 ? kWarpCta / G : row_groups(p.rows, width);
    const int threads = width * per_cta;
    const int staged = NV > 2 && (p.gamma == nullptr || !params_line_up(p.gamma, nullptr, p.param_type, p.C));
    size_t bytes = (S * R * slot_bytes<TS, TB>(p) + (staged ? 8 * sizeof(float) : 0)) * NV * threads;
    if (per_cta > 1 && p.partial != nullptr)
        bytes = std::max(bytes, static_cast<size_t>(per_cta) * 2 * p.C * sizeof(float));
    if (bytes > kDynamicSmem) return cudaErrorNotSupported;
    static KernelFacts facts;
    cudaError_t err = opt_in_smem(kern, facts.smem, kDynamicSmem);
    if (err != cudaSuccess) return err;
    long long want = (p.rows + per_cta - 1) / per_cta;
    if (p.partial != nullptr) want = std::min<long long>(want, norm_bwd_partials(p.rows, p.C));
    const long long grid = persistent_grid(want, bytes, threads, facts.registers(kern));
    err = launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(threads), bytes, p.stream, p, staged, width);
    if (err != cudaSuccess || p.partial == nullptr) return err;
    return launch_norm_param_sum(p.partial, static_cast<int>(grid), p.C, p.dgamma, p.dbeta, p.stream);
}

template <typename TS, typename TB, bool kAdd, bool kAligned>
cudaError_t fwd_rows_a(const NormFwd& p) {
    const int v = row_vectors(p.C);
    if (v <= 8) return fwd_launch<TS, TB, kAdd, kAligned, 8, 1, 4>(p, v);
    if (v <= 16) return fwd_launch<TS, TB, kAdd, kAligned, 16, 1, 4>(p, v);
    if (v <= 32) return fwd_launch<TS, TB, kAdd, kAligned, 32, 1, 4>(p, v);
    if (v <= 64) return fwd_launch<TS, TB, kAdd, kAligned, 32, 2, 2>(p, v);
    if (v <= 128) return fwd_launch<TS, TB, kAdd, kAligned, 32, 4, 1>(p, v);
    if (v <= kMaxCta * kRowVecs) return fwd_launch<TS, TB, kAdd, kAligned, 0, kRowVecs, 1>(p, v);
    return cudaErrorNotSupported;
}

template <typename TS, typename TB, bool kAdd>
cudaError_t fwd_rows(const NormFwd& p) {
    return p.C % 8 == 0 ? fwd_rows_a<TS, TB, kAdd, true>(p) : fwd_rows_a<TS, TB, kAdd, false>(p);
}

template <typename TS, typename TB, bool kAdd, bool kAligned>
cudaError_t bwd_rows_a(const NormBwd& p) {
    const int v = row_vectors(p.C);
    if (v <= 8) return bwd_launch<TS, TB, kAdd, kAligned, 8, 1, 2, 1>(p, v);
    if (v <= 16) return bwd_launch<TS, TB, kAdd, kAligned, 16, 1, 2, 1>(p, v);
    if (v <= 32) return bwd_launch<TS, TB, kAdd, kAligned, 32, 1, 2, 1>(p, v);
    if (v <= 64) return bwd_launch<TS, TB, kAdd, kAligned, 32, 2, 2, 1>(p, v);
    // two stages of two rows where they fit in shared memory, else one (of one row for the widest,
    // and not even that for fp32 rows near 16384 with all three tensors and staged parameters)
    cudaError_t err = cudaErrorNotSupported;
    if (v <= kMaxCta * 2) {
        err = bwd_launch<TS, TB, kAdd, kAligned, 0, 2, 2, 2>(p, v);
        if (err == cudaErrorNotSupported) err = bwd_launch<TS, TB, kAdd, kAligned, 0, 2, 1, 2>(p, v);
    } else if (v <= kMaxCta * 4) {
        err = bwd_launch<TS, TB, kAdd, kAligned, 0, 4, 1, 1>(p, v);
    }
    return err;
}

template <typename TS, typename TB, bool kAdd>
cudaError_t bwd_rows(const NormBwd& p) {
    return p.C % 8 == 0 ? bwd_rows_a<TS, TB, kAdd, true>(p) : bwd_rows_a<TS, TB, kAdd, false>(p);
}

}  // namespace norm
}  // namespace dwc

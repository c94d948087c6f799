// dwc_norm_rows.cuh -- layer norm and its residual form, forward and backward, on rows of up to
// 16384 channels held by a group of threads.
//
// Both passes are bound by memory: a row is read once, reduced in registers or shared memory and
// written once, 8 elements per access.  A group of threads serves one row:
//   rows of up to 8, 16 and 32 vectors: G = 8, 16, 32 lanes, one vector each; up to 64 vectors: a
//   warp with 2; longer rows: several warps, 2 vectors a thread and above 1024 vectors 4 (up to
//   512 threads).
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

constexpr int kWarpCta = 256;            // threads of a CTA whose warps or lane groups serve rows
constexpr int kMaxCta = 512;             // threads of a CTA otherwise: 128 registers each
constexpr int kDynamicSmem = 225 * 1024;

// Vectors that the longest-shifted row of C channels touches.
inline int row_vectors(int C) {
    int g = 8;                            // gcd(C, 8): the shifts are its multiples
    while (C % g != 0) g /= 2;
    return (C + (8 - g) + 7) / 8;
}

// Elements that warp `warp` of a group of `threads` threads with `vecs` vectors each holds of a row.
__device__ __forceinline__ int warp_columns(int warp, int threads, int vecs, int shift, int C) {
    int n = 0;
    for (int k = 0; k < vecs; ++k) {
        const int lo = max(0, (k * threads + warp * 32) * 8 - shift);
        const int hi = min(C, (k * threads + warp * 32 + 32) * 8 - shift);
        n += max(0, hi - lo);
    }
    return n;
}

__device__ __forceinline__ float shifted_param(const void* p, int type, int c, int C, float absent) {
    return in_row(c, C) ? load_param(p, type, c, absent) : 0.f;
}

// Gamma or beta of a thread's vectors.  Up to two vectors a thread they stay in registers; beyond
// that they are read per use, from the caller's array where that is fp32 and lines up with the
// vectors, else from a copy in shared memory laid out along the group's shifted vectors.
template <int NV>
struct Params {
    static constexpr bool kHeld = NV <= 2;
    float2 f[kHeld ? NV : 1][4];
    const float* from;
    int last;                             // the last vector that may be read there
    __device__ __forceinline__ void hold(const void* p, int type, int C, int lane, int width, int shift, float absent) {
        if constexpr (kHeld) {
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int c = (k * width + lane) * 8 + 2 * j - shift;
                    f[k][j] = make_float2(shifted_param(p, type, c, C, absent), shifted_param(p, type, c + 1, C, absent));
                }
        } else {
            from = static_cast<const float*>(p);
            last = C - 8;
        }
    }
    // (the caller synchronises the group before the first use)
    __device__ __forceinline__ void stage(float* to, const void* p, int type, int C, int lane, int width, int shift,
                                          float absent) {
        const int span = width * NV * 8;
        for (int i = lane; i < span; i += width) to[i] = shifted_param(p, type, i - shift, C, absent);
        from = to;
        last = span - 8;
    }
    __device__ __forceinline__ const float2 (&get(int at, int k))[4] {
        if constexpr (kHeld) {
            return f[k];
        } else {
            const float* g = from + min(at, last);
            const float4 a = *reinterpret_cast<const float4*>(g), b = *reinterpret_cast<const float4*>(g + 4);
            f[0][0] = make_float2(a.x, a.y), f[0][1] = make_float2(a.z, a.w);
            f[0][2] = make_float2(b.x, b.y), f[0][3] = make_float2(b.z, b.w);
            return f[0];
        }
    }
};

// Asynchronous copies of one row's tensors into the thread group's own part of shared memory.
// Each thread holds 8 elements of every vector slot: one 16-byte granule of a 16-bit type or two of
// fp32, of which the lanes of a warp copy consecutive ones (whole sectors).  A warp's granules stay
// in the tensor's order, so each copy fills 512 contiguous bytes; the fp32 reads then meet in
// banks two by two, which costs little: with the halves of the vectors parted into two planes
// (no conflicts) the copies themselves were the limit, 238 us instead of 185 for 16384 x 4096 with
// an fp32 stream.  Vectors past the row's end are filled with zeros (a copy of no bytes), so the
// arithmetic needs no branches.  Granules that hang over the row's ends are copied whole while
// they stay within [low, room) of the row's start, the tensor's extent (the reader masks the
// neighbouring rows' elements); beyond it, at the tensor's very end, single elements are stored.
__device__ __forceinline__ void copy16(void* dst, const void* src, bool some) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(some ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <bool kAligned, typename T>
__device__ __forceinline__ void copy_granule(uint4* dst, const T* row, int col, int C, int low, int room) {
    constexpr int n = 16 / sizeof(T);
    const bool some = col < C;
    if (kAligned || !some || (col >= low && col + n <= room)) {
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
__device__ __forceinline__ void copy_slot(uint4* slot, const T* row, int lane, int col, int C, int low, int room) {
    if constexpr (sizeof(T) == 2) {
        copy_granule<kAligned>(slot, row, col, C, low, room);
    } else {
        const int first = col - 4 * lane;       // this lane's granule of the group's 2 * GW
        copy_granule<kAligned>(slot - lane, row, first, C, low, room);
        copy_granule<kAligned>(slot - lane + GW, row, first + 4 * GW, C, low, room);
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

// Barrier of one group of `threads` threads (a multiple of 32) of the CTA.
__device__ __forceinline__ void group_barrier(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Sums of N = 1, 2 or 4 values over the GW lanes of a group: the lanes part the values among
// themselves (halves, then quarters), so that N - 1 + log2(GW / N) exchanges serve all.  Lanes
// with lane / (GW / N) == q return sum q.
template <int GW, int N>
__device__ __forceinline__ float parted_sum(const float (&v)[N], int lane) {
    static_assert(N == 1 || N == 2 || N == 4, "parts");
    float t;
    if constexpr (N == 1) {
        t = v[0];
    } else {
        const bool upper = (lane & (GW / 2)) != 0;
        float half[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i)
            half[i] = (upper ? v[N / 2 + i] : v[i]) + __shfl_xor_sync(0xffffffffu, upper ? v[i] : v[N / 2 + i], GW / 2);
        if constexpr (N == 2) {
            t = half[0];
        } else {
            const bool odd = (lane & (GW / 4)) != 0;
            t = (odd ? half[1] : half[0]) + __shfl_xor_sync(0xffffffffu, odd ? half[0] : half[1], GW / 4);
        }
    }
#pragma unroll
    for (int m = GW / (2 * N); m > 0; m >>= 1) t += __shfl_xor_sync(0xffffffffu, t, m);
    return t;
}

// ------------------------------------------------------------------------------- forward

// CTAs per SM that the register budget allows: 80 registers a thread for one vector, 128 for more.
constexpr int fwd_min_ctas(int G, int NV) { return G == 0 ? 1 : NV == 1 ? 3 : 2; }

// Rows wait in shared memory, S times R of them per group, and R rows go through together (one
// barrier for both, two independent chains of latencies); their values then stay in registers
// until y is written.  G == 0: groups of `group_threads` threads, several to a CTA.
//
// Row statistics: each warp (or lane group) takes the mean of its own elements, then the sum of
// squares about it, and the warps of a group are merged by their counts (Chan, Golub and LeVeque,
// "Updating formulae and a pairwise algorithm for computing sample variances", 1979): one
// barrier per R rows, and no cancellation however far the mean lies from zero.
template <typename TS, typename TB, bool kAdd, bool kAligned, int G, int NV, int R, int S>
__global__ void __launch_bounds__(G > 0 ? kWarpCta : kMaxCta, fwd_min_ctas(G, NV))
norm_fwd_rows_kernel(NormFwd p, int staged, int group_threads) {
    extern __shared__ __align__(16) float smem[];
    __shared__ float2 merge[2][R][kMaxCta / 32];
    constexpr bool kCta = G == 0;                  // several warps serve a row
    constexpr int GW = kCta ? 32 : G;              // lanes whose vectors are adjacent
    constexpr int kPart = GW / R;                  // lanes that hold one row's sums
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
    // (an update in place overwrites the neighbouring rows: then only the row's own elements are read)
    const bool whole = !kAdd || p.z != p.in;
    const int low = whole ? -8 : 0;
    // shared memory: stage, row, then slot (the stream's vectors, the branch's), then thread
    const int x_at = NV * kStream * threads;
    const int row_granules = x_at + (kAdd ? NV * kBranch * threads : 0);
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
            const int room = kAligned ? 0 : whole ? static_cast<int>(min((p.rows - r) * C, 1LL << 30)) : C;
            uint4* to = slots + (stage * R + u) * row_granules;
            const TS* in = static_cast<const TS*>(p.in) + r * p.ld_in;
            const TB* x = static_cast<const TB*>(p.x) + r * p.ld_x;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int col = (k * width + lane) * 8 - shift;
                copy_slot<kAligned, TS, GW>(to + k * kStream * threads + mine_s, in, sub, col, C, low, room);
                if (kAdd) copy_slot<kAligned, TB, GW>(to + x_at + k * kBranch * threads + mine_b, x, sub, col, C, low, room);
            }
        }
        copy_commit();
    };
#pragma unroll
    for (int i = 0; i < S; ++i) fetch(i, group + static_cast<long long>(i) * R * groups);

    Params<NV> gamma, beta;
    gamma.hold(p.gamma, p.param_type, C, lane, width, shift, 1.f);
    beta.hold(p.beta, p.param_type, C, lane, width, shift, 0.f);
    if (NV > 2 && staged) {
        float* to = smem + S * R * row_granules * 4 + local * width * NV * 16;
        gamma.stage(to, p.gamma, p.param_type, C, lane, width, shift, 1.f);
        beta.stage(to + width * NV * 8, p.beta, p.param_type, C, lane, width, shift, 0.f);
        if (kCta) group_barrier(1 + local, width); else __syncwarp();
    }
    // elements of this thread's warp or group, and of the warp whose sums this lane merges
    const int warps = width >> 5, first_warp = local * warps;
    const int mine = kCta ? warp_columns(lane >> 5, width, NV, shift, C) : C;
    const int peer = kCta && sub % kPart < warps ? warp_columns(sub % kPart, width, NV, shift, C) : 0;
    const float mine_inv = mine > 0 ? 1.f / static_cast<float>(mine) : 0.f;
    int parity = 0, stage = 0;

    const long long step = static_cast<long long>(R) * groups;
    // (the lane groups of a warp stay together: the warp goes on while its first group has a row, and
    // all its lanes run the loop's barriers and shuffles)
    const int in_warp = kCta ? 0 : local % (32 / GW);
    for (long long r0 = group; r0 - in_warp < p.rows; r0 += step) {
        copy_wait<S - 1>();
        __syncwarp();
        const uint4* from = slots + stage * R * row_granules;
        float2 v[R][NV][4];
        float s[R], mean[R], rstd[R];
#pragma unroll
        for (int u = 0; u < R; ++u) {
            const long long r = r0 + static_cast<long long>(u) * groups;
            const bool live = r < p.rows;
            const uint4* row = from + u * row_granules;
            float2 s2 = both(0.f);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int col = (k * width + lane) * 8 - shift;
                read_slot<TS>(v[u][k], row + k * kStream * threads + mine_s);
                if constexpr (kAdd) {
                    float2 b[4];
                    read_slot<TB>(b, row + x_at + k * kBranch * threads + mine_b);
                    if (drop.threshold != 0) drop8(drop, b, static_cast<uint64_t>(r * C + col) >> 3);
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[u][k][j] = __fadd2_rn(v[u][k][j], b[j]);
                    if (live && col < C) store_row8<kAligned>(static_cast<TS*>(p.z) + r * C, v[u][k], col, C);
                }
                if (!kAligned && !inside(col, C)) mask8(v[u][k], col, C);
#pragma unroll
                for (int j = 0; j < 4; ++j) s2 = __fadd2_rn(s2, v[u][k][j]);
            }
            s[u] = s2.x + s2.y;
        }
        // the stage is read: the rows S steps on take it
        __syncwarp();
        fetch(stage, r0 + S * step);
        if (++stage == S) stage = 0;

        float t = parted_sum<GW, R>(s, sub);
#pragma unroll
        for (int u = 0; u < R; ++u) mean[u] = __shfl_sync(0xffffffffu, t, u * kPart, GW) * mine_inv;
#pragma unroll
        for (int u = 0; u < R; ++u) {
            float2 q2 = both(0.f);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int col = (k * width + lane) * 8 - shift;
                float2 d[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) d[j] = __fadd2_rn(v[u][k][j], both(-mean[u]));
                if (!inside(col, C)) mask8(d, col, C);
#pragma unroll
                for (int j = 0; j < 4; ++j) q2 = __ffma2_rn(d[j], d[j], q2);
            }
            s[u] = q2.x + q2.y;
        }
        t = parted_sum<GW, R>(s, sub);
        float m = mean[0];
        if constexpr (R == 2) m = sub < kPart ? mean[0] : mean[1];
        if constexpr (kCta) {
            // lane l merges row l / kPart over the group's warps, warp l % kPart
            if (sub % kPart == 0) merge[parity][sub / kPart][threadIdx.x >> 5] = make_float2(m, t);
            group_barrier(1 + local, width);
            const int w = sub % kPart;
            const float2 e = w < warps ? merge[parity][sub / kPart][first_warp + w] : make_float2(0.f, 0.f);
            parity ^= 1;
            const float n = static_cast<float>(peer);
            m = n * e.x;
#pragma unroll
            for (int x = kPart / 2; x > 0; x >>= 1) m += __shfl_xor_sync(0xffffffffu, m, x);
            m *= inv;
            const float d = e.x - m;
            t = peer > 0 ? fmaf(n * d, d, e.y) : 0.f;
#pragma unroll
            for (int x = kPart / 2; x > 0; x >>= 1) t += __shfl_xor_sync(0xffffffffu, t, x);
        }
        t = 1.f / sqrtf(t * inv + p.eps);
#pragma unroll
        for (int u = 0; u < R; ++u) {
            mean[u] = __shfl_sync(0xffffffffu, m, u * kPart, GW);
            rstd[u] = __shfl_sync(0xffffffffu, t, u * kPart, GW);
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int at = (k * width + lane) * 8, col = at - shift;
            const float2(&g)[4] = gamma.get(at, k);
            const float2(&b)[4] = beta.get(at, k);
#pragma unroll
            for (int u = 0; u < R; ++u) {
                const long long r = r0 + static_cast<long long>(u) * groups;
                float2 y[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 xhat = __fmul2_rn(__fadd2_rn(v[u][k][j], both(-mean[u])), both(rstd[u]));
                    y[j] = __ffma2_rn(xhat, g[j], b[j]);
                }
                if (r < p.rows && col < C) store_row8<kAligned>(static_cast<TB*>(p.y) + r * C, y, col, C);
            }
        }
        if (lane == 0) {
#pragma unroll
            for (int u = 0; u < R; ++u) {
                const long long r = r0 + static_cast<long long>(u) * groups;
                if (r >= p.rows) continue;
                if (p.mean != nullptr) p.mean[r] = mean[u];
                if (p.rstd != nullptr) p.rstd[r] = rstd[u];
            }
        }
    }
    copy_wait<0>();
}

// ------------------------------------------------------------------------------ backward

// CTAs per SM that the register budget allows: 80 registers a thread for one vector, 128 for 2 and
// 4, of which 16 a vector hold the gradient sums and 8 gamma.
constexpr int bwd_min_ctas(int G, int NV) { return G == 0 ? 1 : NV == 1 ? 3 : 2; }

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
                copy_slot<kAligned, TB, GW>(to + k * kBranch * threads + mine_b, dy, sub, col, C, -8, room);
                copy_slot<kAligned, TS, GW>(to + z_at + k * kStream * threads + mine_s, z, sub, col, C, -8, room);
            }
            if (has_dz) {
#pragma unroll
                for (int k = 0; k < NV; ++k)
                    copy_slot<kAligned, TS, GW>(to + dz_at + k * kStream * threads + mine_s, dz, sub,
                                                (k * width + lane) * 8 - shift, C, -8, room);
            }
        }
        copy_commit();
    };
#pragma unroll
    for (int i = 0; i < S; ++i) fetch(i, group + static_cast<long long>(i) * R * groups);

    Params<NV> gamma;
    gamma.hold(p.gamma, p.param_type, C, lane, width, shift, 1.f);
    if (NV > 2 && staged) {
        gamma.stage(smem + S * R * row_granules * 4 + local * width * NV * 8, p.gamma, p.param_type, C, lane, width,
                    shift, 1.f);
        if (kCta) group_barrier(1 + local, width); else __syncwarp();
    }
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
                    const float2(&gk)[4] = gamma.get((k * width + lane) * 8, k);
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
        float t = parted_sum<GW, 2 * R>(s, sub);
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
                const float2(&gk)[4] = gamma.get((k * width + lane) * 8, k);
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

// Groups of `width` threads in a CTA: several only once there is a row for every SM.
inline int row_groups(long long rows, int width) {
    return static_cast<int>(std::max(1LL, std::min<long long>(kMaxCta / width, rows / device_info().sm_count)));
}

template <typename TS, typename TB, bool kAdd, bool kAligned, int G, int NV, int R, int S>
cudaError_t fwd_launch(const NormFwd& p, int vectors) {
    auto kern = norm_fwd_rows_kernel<TS, TB, kAdd, kAligned, G, NV, R, S>;
    const int width = G > 0 ? G : (vectors + NV * 32 - 1) / (NV * 32) * 32;
    const int per_cta = G > 0 ? kWarpCta / G : row_groups(p.rows, width);
    const int threads = width * per_cta;
    const int staged = NV > 2 && (p.gamma == nullptr || p.beta == nullptr ||
                                  !params_line_up(p.gamma, p.beta, p.param_type, p.C));
    const size_t slot = 8 * (sizeof(TS) + (kAdd ? sizeof(TB) : 0));
    const size_t bytes = (S * R * slot + (staged ? 16 * sizeof(float) : 0)) * NV * threads;
    if (bytes > kDynamicSmem) return cudaErrorNotSupported;
    static KernelFacts facts;
    const cudaError_t err = opt_in_smem(kern, facts.smem, kDynamicSmem);
    if (err != cudaSuccess) return err;
    const long long grid = persistent_grid((p.rows + per_cta - 1) / per_cta, bytes, threads, facts.registers(kern));
    return launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(threads), bytes, p.stream, p, staged, width);
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
    if (v <= 8) return fwd_launch<TS, TB, kAdd, kAligned, 8, 1, 2, 2>(p, v);
    if (v <= 16) return fwd_launch<TS, TB, kAdd, kAligned, 16, 1, 2, 2>(p, v);
    if (v <= 32) return fwd_launch<TS, TB, kAdd, kAligned, 32, 1, 2, 2>(p, v);
    if (v <= 64) return fwd_launch<TS, TB, kAdd, kAligned, 32, 2, 2, 1>(p, v);
    // two stages of two rows where they fit in shared memory, else of one row; the widest rows in one
    // stage (and not at all as fp32 with an fp32 branch and staged parameters)
    cudaError_t err = cudaErrorNotSupported;
    if (v <= kMaxCta * 2) {
        err = fwd_launch<TS, TB, kAdd, kAligned, 0, 2, 2, 2>(p, v);
        if (err == cudaErrorNotSupported) err = fwd_launch<TS, TB, kAdd, kAligned, 0, 2, 1, 2>(p, v);
    } else if (v <= kMaxCta * 4) {
        err = fwd_launch<TS, TB, kAdd, kAligned, 0, 4, 1, 2>(p, v);
        if (err == cudaErrorNotSupported) err = fwd_launch<TS, TB, kAdd, kAligned, 0, 4, 1, 1>(p, v);
    }
    return err;
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
        err = bwd_launch<TS, TB, kAdd, kAligned, 0, 4, 1, 2>(p, v);
        if (err == cudaErrorNotSupported) err = bwd_launch<TS, TB, kAdd, kAligned, 0, 4, 1, 1>(p, v);
    }
    return err;
}

template <typename TS, typename TB, bool kAdd>
cudaError_t bwd_rows(const NormBwd& p) {
    return p.C % 8 == 0 ? bwd_rows_a<TS, TB, kAdd, true>(p) : bwd_rows_a<TS, TB, kAdd, false>(p);
}

}  // namespace norm
}  // namespace dwc

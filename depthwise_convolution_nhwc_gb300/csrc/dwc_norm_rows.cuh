// dwc_norm_rows.cuh -- layer norm and its residual form on rows held in registers.
//
// Both passes are bound by memory: a row is read once into registers (8 elements per access),
// reduced there and written once.  A group of G threads serves one row:
//   rows of up to 8, 16 and 32 vectors: G = 8, 16, 32 lanes, one vector each; up to 64 and 128
//   vectors: a warp with 2 and 4; longer rows (up to 4 vectors x 512 threads): a whole CTA.
//
// Alignment.  A dense row of C channels starts (row * C) mod 8 elements past a vector boundary, and
// so does every tensor of the call if its base is aligned and its row stride is congruent to C
// modulo 8.  The group works on the vectors of the address, shifted against the row by that
// amount; the first and last one may hang over and are masked.  Groups advance by a multiple of 8
// rows, so a group's shift never changes: its columns (parameters, gradient sums) stay its own.
// The dropout's blocks of 8 elements coincide with these vectors.
//
// Row statistics: each warp (or lane group) takes the mean of its own elements, then the sum of
// squares about it, and the warps of a CTA are merged by their counts (Chan, Golub and LeVeque,
// "Updating formulae and a pairwise algorithm for computing sample variances", 1979): one
// barrier per row, and no cancellation however far the mean lies from zero.
#pragma once

#include <algorithm>

#include "dwc_norm_device.cuh"

namespace dwc {
namespace norm {

constexpr int kCtaVecs = 4;          // vectors per thread where a CTA serves a row
constexpr int kWarpCta = 256;        // threads of a CTA whose warps or lane groups serve rows
constexpr int kDynamicSmem = 225 * 1024;
constexpr int kMaxCta = 512;         // threads of a CTA that serves a row: 128 registers each

// Vectors that the longest-shifted row of C channels touches.
inline int row_vectors(int C) {
    int g = 8;                        // gcd(C, 8): the shifts are its multiples
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

// Columns of [first, first + 32 * 8) shifted vectors of a warp, summed over its vectors.
__device__ __forceinline__ int warp_columns(int warp, int threads, int shift, int C) {
    int n = 0;
#pragma unroll
    for (int k = 0; k < kCtaVecs; ++k) {
        const int lo = max(0, (k * threads + warp * 32) * 8 - shift);
        const int hi = min(C, (k * threads + warp * 32 + 32) * 8 - shift);
        n += max(0, hi - lo);
    }
    return n;
}

// Where a group finds 8 consecutive parameters in fp32: the caller's own fp32 array where the
// vectors line up with it, else a copy of it in shared memory that is laid out along the
// group's shifted vectors (written once per group, read for every row).
struct ParamSource {
    const float* p = nullptr;        // indexed by column + shift
    bool present = false;
    __device__ __forceinline__ void get(float (&f)[8], int at, float absent) const {
        if (!present) {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = absent;
            return;
        }
        const float4 a = *reinterpret_cast<const float4*>(p + at), b = *reinterpret_cast<const float4*>(p + at + 4);
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    }
};

// ------------------------------------------------------------------------------- forward

// G > 0: lanes of a row's group, NV vectors a lane, U rows at a time (their loads in flight
// together); G == 0: the CTA serves a row.  `staged`: parameters go through shared memory.
template <typename TS, typename TB, bool kAdd, int G, int NV, int U>
__global__ void __launch_bounds__(G > 0 ? kWarpCta : kMaxCta) norm_fwd_rows_kernel(NormFwd p, int staged) {
    extern __shared__ __align__(16) float smem[];
    __shared__ float2 merge[2][32];
    constexpr bool kCta = G == 0;
    const int width = kCta ? blockDim.x : G;                       // threads of a group
    const int lane = kCta ? threadIdx.x : threadIdx.x % (kCta ? 1 : G);
    const int local = kCta ? 0 : threadIdx.x / width;              // group within the CTA
    const int per_cta = kCta ? 1 : kWarpCta / width;
    const long long groups = static_cast<long long>(gridDim.x) * per_cta;
    const long long group = static_cast<long long>(blockIdx.x) * per_cta + local;
    const int C = p.C;
    const int shift = static_cast<int>((group * C) & 7);
    const float inv = 1.f / static_cast<float>(C);
    pdl_trigger();
    pdl_wait();
    DropState drop;
    if (kAdd) drop.init(p.drop);

    // parameters: registers for one vector a lane, else read (or staged) per use
    float gam[8], bet[8];
    ParamSource gsrc, bsrc;
    if constexpr (NV == 1) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = lane * 8 + j - shift;
            const bool in = static_cast<unsigned>(c) < static_cast<unsigned>(C);
            gam[j] = in ? load_param(p.gamma, p.param_type, c, 1.f) : 0.f;
            bet[j] = in ? load_param(p.beta, p.param_type, c, 0.f) : 0.f;
        }
    } else {
        gsrc.present = staged || p.gamma != nullptr;
        bsrc.present = staged || p.beta != nullptr;
        gsrc.p = static_cast<const float*>(p.gamma);
        bsrc.p = static_cast<const float*>(p.beta);
        if (staged) {
            const int span = width * NV * 8;
            float* g = smem + static_cast<size_t>(local) * 2 * span;
            for (int i = lane; i < span; i += width) {
                const int c = i - shift;
                const bool in = static_cast<unsigned>(c) < static_cast<unsigned>(C);
                g[i] = in ? load_param(p.gamma, p.param_type, c, 1.f) : 0.f;
                g[span + i] = in ? load_param(p.beta, p.param_type, c, 0.f) : 0.f;
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
    const int in_warp = kCta ? 0 : local % (32 / (kCta ? 32 : G));
    for (long long r0 = group; r0 - in_warp < p.rows; r0 += groups * U) {
        Vec8<TS> raw[U][NV];
        Vec8<TB> branch[kAdd ? U : 1][kAdd ? NV : 1];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long r = r0 + u * groups;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int col = (k * width + lane) * 8 - shift;
                raw[u][k].zero();
                if (kAdd) branch[u][k].zero();
                if (r < p.rows && col < C) {
                    load_row8(raw[u][k], static_cast<const TS*>(p.in) + r * p.ld_in, col, C);
                    if (kAdd) load_row8(branch[u][k], static_cast<const TB*>(p.x) + r * p.ld_x, col, C);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long r = r0 + u * groups;
            const bool live = r < p.rows;
            float v[NV][8];
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int col = (k * width + lane) * 8 - shift;
                raw[u][k].widen(v[k]);
                if (kAdd) {
                    float b[8];
                    branch[u][k].widen(b);
                    if (drop.threshold != 0 && live && col < C)
                        drop8(drop, b, static_cast<uint64_t>(r * C + col) >> 3);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[k][j] += b[j];
                    if (live && col < C) store_row8(static_cast<TS*>(p.z) + r * C, v[k], col, C);
                }
                // (elements beside the row are 0: their inputs read as 0, and 0 is dropped or kept as 0)
#pragma unroll
                for (int j = 0; j < 8; ++j) s += v[k][j];
            }
            float mean = (kCta ? warp_sum(s) : group_sum<kCta ? 32 : G>(s)) * mine_inv;
            float q = 0.f;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int col = (k * width + lane) * 8 - shift;
                if (inside(col, C)) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float d = v[k][j] - mean;
                        q = fmaf(d, d, q);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float d = static_cast<unsigned>(col + j) < static_cast<unsigned>(C) ? v[k][j] - mean : 0.f;
                        q = fmaf(d, d, q);
                    }
                }
            }
            q = kCta ? warp_sum(q) : group_sum<kCta ? 32 : G>(q);
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
                float y[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] = fmaf((v[k][j] - mean) * rstd, gam[j], bet[j]);
                store_row8(static_cast<TB*>(p.y) + r * C, y, col, C);
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
// Each thread holds 8 elements of every vector slot; a slot is one 16-byte granule of a 16-bit
// type or two of fp32.  For fp32 the lanes of a warp copy consecutive granules (whole sectors)
// and the two halves of a vector land in two planes, so both sides are free of bank conflicts.
// Granules that hang over the row's ends are copied whole while they stay inside the tensor
// (the reader masks the neighbouring rows' elements); at the tensor's very end single elements
// are stored instead.
__device__ __forceinline__ void copy16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <typename T>
__device__ __forceinline__ void copy_granule(uint4* dst, const T* row, int col, int C, int room) {
    constexpr int n = 16 / sizeof(T);
    if (col >= C) return;
    if (col + n <= room) {
        copy16(dst, row + col);
    } else {
        T* to = reinterpret_cast<T*>(dst);
#pragma unroll
        for (int j = 0; j < n; ++j)
            if (static_cast<unsigned>(col + j) < static_cast<unsigned>(C)) to[j] = row[col + j];
    }
}

// One vector slot of the lanes of a (sub-)warp of GW lanes: `slot` is the thread's own granule of
// the slot's first plane, `col` its first element, `plane` granules lie between two planes.
template <typename T, int GW>
__device__ __forceinline__ void copy_slot(uint4* slot, int plane, const T* row, int lane, int col, int C, int room) {
    if constexpr (sizeof(T) == 2) {
        copy_granule(slot, row, col, C, room);
    } else {
        uint4* base = slot - lane + (lane & 1) * plane + (lane >> 1);
        const int first = col - 4 * lane;       // this lane's granule of the group's 2 * GW
        copy_granule(base, row, first, C, room);
        copy_granule(base + GW / 2, row, first + 4 * GW, C, room);
    }
}

template <typename T>
__device__ __forceinline__ void read_slot(float (&f)[8], const uint4* slot, int plane) {
    if constexpr (sizeof(T) == 2) {
        Vec8<T> v;
        v.u = *slot;
        v.widen(f);
    } else {
        const float4 a = *reinterpret_cast<const float4*>(slot), b = *reinterpret_cast<const float4*>(slot + plane);
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    }
}

__device__ __forceinline__ void mask8(float (&f)[8], int col, int C) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (static_cast<unsigned>(col + j) >= static_cast<unsigned>(C)) f[j] = 0.f;
}

// CTAs per SM that the register budget allows: 80 registers a thread for one vector, 128 for 2 and
// 4, of which 16 a vector hold the gradient sums.
constexpr int bwd_min_ctas(int G, int NV) { return G == 0 ? 1 : NV == 1 ? 3 : 2; }

// Barrier of one group of `threads` threads (a multiple of 32) of the CTA.
__device__ __forceinline__ void group_barrier(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Each thread keeps the sums of dy * xhat and dy of its columns in registers over all rows of its
// group; at the end the groups of a CTA are added in order and the CTA writes one row of partial
// sums.  The sums take the registers, so the rows wait in shared memory, S of them per group, and
// are read twice there (before and after the row's two means are known).  G == 0: groups of
// `group_threads` threads, several to a CTA where they are short: one CTA per SM, so that there
// are few rows of partial sums.
template <typename TS, typename TB, int G, int NV, int S>
__global__ void __launch_bounds__(G > 0 ? kWarpCta : kMaxCta, bwd_min_ctas(G, NV))
norm_bwd_rows_kernel(NormBwd p, int staged, int group_threads) {
    extern __shared__ __align__(16) float smem[];
    __shared__ float2 merge[2][kMaxCta / 32];
    constexpr bool kCta = G == 0;                  // several warps serve a row
    constexpr int GW = kCta ? 32 : G;              // lanes whose vectors are adjacent
    constexpr int kBranch = sizeof(TB) / 2, kStream = sizeof(TS) / 2;  // planes of a slot
    const int threads = kCta ? blockDim.x : kWarpCta;
    const int width = kCta ? group_threads : G;
    const int local = threadIdx.x / width;         // group within the CTA
    const int lane = threadIdx.x - local * width;
    const int sub = threadIdx.x % GW;
    const int per_cta = threads / width;
    const int first_warp = local * width / 32;
    const int groups = gridDim.x * per_cta;
    const int group = blockIdx.x * per_cta + local;
    const int C = p.C;
    const int shift = static_cast<int>((static_cast<long long>(group) * C) & 7);
    const float inv = 1.f / static_cast<float>(C);
    const bool has_dz = p.dz != nullptr;
    // this thread's granules: stage, then slot (dy, z, dz of each vector), then plane
    const int z_at = NV * kBranch, dz_at = z_at + NV * kStream;
    const int stage_granules = (dz_at + (has_dz ? NV * kStream : 0)) * threads;
    uint4* mine = reinterpret_cast<uint4*>(smem) + threadIdx.x;
    pdl_trigger();
    pdl_wait();
    DropState drop;
    drop.init(p.drop);

    auto fetch = [&](int stage, long long r) {
        if (r < p.rows) {
            const int room = static_cast<int>(min((p.rows - r) * C, 1LL << 30));   // elements to the tensor's end, at least
            uint4* to = mine + stage * stage_granules;
            const TB* dy = static_cast<const TB*>(p.dy) + r * p.ld_dy;
            const TS* z = static_cast<const TS*>(p.z) + r * p.ld_z;
            const TS* dz = static_cast<const TS*>(p.dz) + r * p.ld_dz;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int col = (k * width + lane) * 8 - shift;
                copy_slot<TB, GW>(to + k * kBranch * threads, threads, dy, sub, col, C, room);
                copy_slot<TS, GW>(to + (z_at + k * kStream) * threads, threads, z, sub, col, C, room);
                if (has_dz) copy_slot<TS, GW>(to + (dz_at + k * kStream) * threads, threads, dz, sub, col, C, room);
            }
        }
        copy_commit();
    };
#pragma unroll
    for (int i = 0; i < S; ++i) fetch(i, group + static_cast<long long>(i) * groups);

    float gam[8];
    ParamSource gsrc;
    if constexpr (NV == 1) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = lane * 8 + j - shift;
            gam[j] = static_cast<unsigned>(c) < static_cast<unsigned>(C) ? load_param(p.gamma, p.param_type, c, 1.f) : 0.f;
        }
    } else {
        gsrc.present = staged || p.gamma != nullptr;
        gsrc.p = static_cast<const float*>(p.gamma);
        if (staged) {
            const int span = width * NV * 8;
            float* g = smem + S * stage_granules * 4 + local * span;
            for (int i = lane; i < span; i += width) {
                const int c = i - shift;
                g[i] = static_cast<unsigned>(c) < static_cast<unsigned>(C) ? load_param(p.gamma, p.param_type, c, 1.f) : 0.f;
            }
            gsrc.p = g;
            if (kCta) group_barrier(1 + local, width); else __syncwarp();
        }
    }
    float sum_g[NV][8], sum_b[NV][8];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) sum_g[k][j] = sum_b[k][j] = 0.f;
    int parity = 0, stage = 0;
    float next_mean = 0.f, next_rstd = 0.f;
    if (group < p.rows) {
        next_mean = p.mean[group];
        next_rstd = p.rstd[group];
    }

    const int in_warp = kCta ? 0 : local % (32 / GW);
    for (long long r = group; r - in_warp < p.rows; r += groups) {
        const bool live = r < p.rows;
        const float mean = next_mean, rstd = next_rstd;
        if (r + groups < p.rows) {
            next_mean = p.mean[r + groups];
            next_rstd = p.rstd[r + groups];
        }
        copy_wait<S - 1>();
        __syncwarp();
        const uint4* from = mine + stage * stage_granules;
        float2 s = make_float2(0.f, 0.f);
        if (live) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int at = (k * width + lane) * 8, col = at - shift;
                if (col >= C) continue;
                if constexpr (NV > 1) gsrc.get(gam, at, 1.f);
                float f[8], x[8];
                read_slot<TB>(f, from + k * kBranch * threads, threads);
                read_slot<TS>(x, from + (z_at + k * kStream) * threads, threads);
                if (!inside(col, C)) {
                    mask8(f, col, C);
                    mask8(x, col, C);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float d = x[j] - mean;
                    const float a = f[j] * gam[j];
                    s.x += a;
                    s.y = fmaf(a, d, s.y);
                    sum_g[k][j] = fmaf(f[j], d * rstd, sum_g[k][j]);
                    sum_b[k][j] += f[j];
                }
            }
        }
        s.x = group_sum<GW>(s.x);
        s.y = group_sum<GW>(s.y);
        if (kCta) {
            if ((threadIdx.x & 31) == 0) merge[parity][threadIdx.x >> 5] = s;
            group_barrier(1 + local, width);
            s = make_float2(0.f, 0.f);
            for (int w = 0; w < (width >> 5); ++w) {
                s.x += merge[parity][first_warp + w].x;
                s.y += merge[parity][first_warp + w].y;
            }
            parity ^= 1;
        }
        // dx = rstd (a - c1 - xhat c2) = rstd a - k1 - (x - mean) k2
        const float k1 = rstd * s.x * inv, k2 = rstd * rstd * rstd * s.y * inv;
        if (live) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int at = (k * width + lane) * 8, col = at - shift;
                if (col >= C) continue;
                if constexpr (NV > 1) gsrc.get(gam, at, 1.f);
                float f[8], x[8], g[8];
                read_slot<TB>(f, from + k * kBranch * threads, threads);
                read_slot<TS>(x, from + (z_at + k * kStream) * threads, threads);
                if (has_dz) read_slot<TS>(g, from + (dz_at + k * kStream) * threads, threads);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float t = fmaf(-k2, x[j] - mean, fmaf(f[j] * gam[j], rstd, -k1));
                    g[j] = has_dz ? g[j] + t : t;
                }
                store_row8(static_cast<TS*>(p.d_stream) + r * C, g, col, C);
                if (p.d_branch != nullptr) {
                    if (drop.threshold != 0) drop8(drop, g, static_cast<uint64_t>(r * C + col) >> 3);
                    store_row8(static_cast<TB*>(p.d_branch) + r * C, g, col, C);
                }
            }
        }
        __syncwarp();   // all lanes have read the stage
        fetch(stage, r + static_cast<long long>(S) * groups);
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
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = col + j;
            if (static_cast<unsigned>(c) >= static_cast<unsigned>(C)) continue;
            float* to = combine ? smem + local * 2 * C : part;   // the groups' sums, [group][2][C]
            to[c] = sum_g[k][j];
            to[C + c] = sum_b[k][j];
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

template <typename TS, typename TB, bool kAdd, int G, int NV, int U>
cudaError_t fwd_launch(const NormFwd& p, int vectors) {
    auto kern = norm_fwd_rows_kernel<TS, TB, kAdd, G, NV, U>;
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

template <typename TS, typename TB, int G, int NV, int S>
cudaError_t bwd_launch(const NormBwd& p, int vectors) {
    auto kern = norm_bwd_rows_kernel<TS, TB, G, NV, S>;
    const int width = G > 0 ? G : (vectors + NV * 32 - 1) / (NV * 32) * 32;
    const int per_cta = G > 0 ? kWarpCta / G : static_cast<int>(std::min<long long>(kMaxCta / width, (p.rows + 7) / 8));
    const int threads = width * per_cta;
    const int staged = NV > 1 && !params_line_up(p.gamma, nullptr, p.param_type, p.C);
    const size_t per_thread = S * 8 * (sizeof(TB) + sizeof(TS) * (p.dz != nullptr ? 2 : 1)) + (staged ? 8 * sizeof(float) : 0);
    size_t bytes = per_thread * NV * threads;
    if (per_cta > 1 && p.partial != nullptr)
        bytes = std::max(bytes, static_cast<size_t>(per_cta) * 2 * p.C * sizeof(float));
    if (bytes > kDynamicSmem) return cudaErrorNotSupported;   // (fp32 rows near 16384 with all three tensors)
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

template <typename TS, typename TB, bool kAdd>
cudaError_t fwd_rows(const NormFwd& p) {
    const int v = row_vectors(p.C);
    if (v <= 8) return fwd_launch<TS, TB, kAdd, 8, 1, 4>(p, v);
    if (v <= 16) return fwd_launch<TS, TB, kAdd, 16, 1, 4>(p, v);
    if (v <= 32) return fwd_launch<TS, TB, kAdd, 32, 1, 4>(p, v);
    if (v <= 64) return fwd_launch<TS, TB, kAdd, 32, 2, 2>(p, v);
    if (v <= 128) return fwd_launch<TS, TB, kAdd, 32, 4, 1>(p, v);
    if (v <= kMaxCta * kCtaVecs) return fwd_launch<TS, TB, kAdd, 0, kCtaVecs, 1>(p, v);
    return cudaErrorNotSupported;
}

template <typename TS, typename TB>
cudaError_t bwd_rows(const NormBwd& p) {
    const int v = row_vectors(p.C);
    if (v <= 8) return bwd_launch<TS, TB, 8, 1, 2>(p, v);
    if (v <= 16) return bwd_launch<TS, TB, 16, 1, 2>(p, v);
    if (v <= 32) return bwd_launch<TS, TB, 32, 1, 2>(p, v);
    if (v <= 64) return bwd_launch<TS, TB, 32, 2, 2>(p, v);
    if (v <= 128) return bwd_launch<TS, TB, 32, 4, 1>(p, v);
    if (v <= kMaxCta * kCtaVecs) return bwd_launch<TS, TB, 0, kCtaVecs, 1>(p, v);
    return cudaErrorNotSupported;
}

}  // namespace norm
}  // namespace dwc

// dwc_norm_rows.cuh -- layer norm and its residual form, forward and backward, on rows of up to
// 65536 channels.
//
// Both passes are bound by memory: a row is read once, reduced in registers or shared memory and
// written once, 8 elements per access.  A group of threads serves one row:
//   rows of up to 8, 16 and 32 vectors: G = 8, 16, 32 lanes, one vector each; up to 64 vectors: a
//   warp with 2; up to 1280: several warps with 2 vectors a thread (up to 640 threads); beyond
//   that a cluster of 2, 4 or 8 CTAs, each with a share of the columns, which exchange their sums
//   through distributed shared memory.
//
// Alignment.  A dense row of C channels starts (row * C) mod 8 elements past a vector boundary, and
// so does every tensor of the call if its base is aligned and its row stride is congruent to C
// modulo 8.  The group works on the vectors of the address, shifted against the row by that
// amount; the first and last one may hang over and are masked (kAligned: C is a multiple of 8
// and nothing is).  Groups advance by a multiple of 8 rows, so a group's shift never changes:
// its columns (parameters, gradient sums) stay its own.  The dropout's blocks of 8 elements
// coincide with these vectors.
//
// Copies.  cp.async of 16 bytes per thread into the thread group's own slots of shared memory, one or two
// rows ahead: no registers wait for memory, and neither alignment of the row nor a barrier between
// producer and consumer is needed.  (Rows loaded straight into registers reached 64 % of the
// bandwidth with bf16, which leaves half the bytes in flight: 61 us forward for 16384 x 4096.)
//
// Measured (device time, GB300, of the bytes that must move at 6.79 TB/s): forward bf16 16384 x 4096
// 43 us (92 %), fp32 16384 x 4096 81 us (97 %), fp32 200704 x 128 35 us (88 %); residual form, fp32
// stream and bf16 branches with dropout, 16384 x 4096 forward 120 us (99 %), backward 174 us
// (91 %), bf16 stream 85 us (93 %) and 111 us (89 %); backward bf16 8192 x 4096 40 us (74 %, of which 6 us
// are the parameter gradients' second kernel), bf16 200704 x 128 29 us (79 %), fp32 x with bf16 dy
// 16384 x 4096 120 us (82 %).  Bound by memory from about 100 MB on; below that by the
// two launches' and the copies' latency, a few microseconds.
#pragma once

#include <algorithm>
#include <climits>

#include "dwc_norm_device.cuh"

namespace dwc {
namespace norm {

constexpr int kWarpCta = 256;            // threads of a CTA whose warps or lane groups serve rows
// Threads of a CTA otherwise: 512 of 128 registers where two rows go through together, 640 of 96
// where it is one (which serves rows of 4104 to 5120 channels with two groups instead of one).
constexpr int max_cta(int R) { return R == 2 ? 512 : 640; }
constexpr size_t kDynamicSmem = 220 * 1024;   // of 227 KB, beside the exchanges' static arrays

// Vectors that the longest-shifted row of C channels touches.
inline int row_vectors(int C) {
    int g = 8;                            // gcd(C, 8): the shifts are its multiples
    while (C % g != 0) g /= 2;
    return static_cast<int>((static_cast<long long>(C) + (8 - g) + 7) / 8);
}

__device__ __forceinline__ float shifted_param(const void* p, int type, int c, int C, float absent) {
    return in_row(c, C) ? load_param(p, type, c, absent) : 0.f;
}

// Where a thread's vectors lie: vector k of the thread begins at column first + 8 * (k * width +
// lane) and is the thread's if that is below `end`.  `first` is the CTA's first column (minus the
// row's shift), so a CTA of a cluster has the columns max(0, first) .. end - 1.
struct Columns {
    int first, end, width, lane;
    __device__ __forceinline__ int of(int k) const { return first + (k * width + lane) * 8; }
};

// What the warp's lanes have in common about their vectors k (a vote once, a uniform branch per use):
// `whole`: none of the row's vectors hangs over its ends; `full`: besides, none lies past the end.
template <int NV, bool kAligned>
struct Edges {
    bool whole[NV], full[NV];
    __device__ __forceinline__ Edges(const Columns& at, int C) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const bool some = at.of(k) < at.end, in = inside(at.of(k), C);
            whole[k] = kAligned || __all_sync(0xffffffffu, !some || in);
            full[k] = __all_sync(0xffffffffu, some && in);
        }
    }
};

// Elements of a row that warp `warp` of the group holds.
template <int NV>
__device__ __forceinline__ int warp_columns(const Columns& at, int warp) {
    int n = 0;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int lo = at.first + (k * at.width + warp * 32) * 8;
        n += max(0, min(at.end, lo + 32 * 8) - max(0, lo));
    }
    return n;
}

// Gamma or beta of a thread's vectors, in registers.
template <int NV>
__device__ __forceinline__ void load_params(float2 (&f)[NV][4], const void* p, int type, int C, const Columns& at, float absent) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = at.of(k) + 2 * j;
            f[k][j] = make_float2(shifted_param(p, type, c, C, absent), shifted_param(p, type, c + 1, C, absent));
        }
}

// ---- sums of several warps or CTAs ---------------------------------------------------------
constexpr int kWarps = 20;                   // places of one CTA in an exchange
constexpr int kMaxCluster = 8;

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// Barrier of all threads of the cluster; shared memory written before it, the other CTAs' too, is
// visible after it.
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// *p = v in the shared memory of CTA `rank` of the cluster (ordered by cluster_barrier()).
__device__ __forceinline__ void store_remote(float* p, float v, uint32_t rank) {
    asm volatile(
        "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\tst.shared::cluster.f32 [a], %2;\n\t}" ::"r"(smem_addr(p)),
        "r"(rank), "f"(v)
        : "memory");
}
// The same counted on that CTA's mbarrier: what a cluster exchanges per row.  (A cluster barrier in
// its place waits for the CTA's stores to global memory as well: 132 against 110 us for bf16
// 4096 x 16384 forward, before the number of clusters was set right, now 66.)
__device__ __forceinline__ void send_remote(float* p, float v, uint64_t* bar, uint32_t rank) {
    asm volatile(
        "{\n\t.reg .b32 a, b;\n\tmapa.shared::cluster.u32 a, %0, %2;\n\tmapa.shared::cluster.u32 b, %1, %2;\n\t"
        "st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [a], %3, [b];\n\t}" ::"r"(smem_addr(p)),
        "r"(smem_addr(bar)), "r"(rank), "r"(__float_as_uint(v))
        : "memory");
}
// Wait for a phase of the exchange, no longer than the limit; false if it ran out.
__device__ __forceinline__ bool await_exchange(uint64_t* bar, uint32_t phase, unsigned long long limit_ns, unsigned int* status) {
    const unsigned long long limit = limit_ns != 0 ? limit_ns : kWaitLimitNs, t0 = global_ns();
    for (;;) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(smem_addr(bar)), "r"(phase)
            : "memory");
        if (done) return true;
        if (global_ns() - t0 > limit) break;
    }
    record_status(status, DWC_DEVSTAT_TIMEOUT);
    return false;
}
// The end of a cluster's kernel.  A thread whose wait ran out (`lost`) has sent and awaited nothing since
// and goes on with wrong sums; its CTA stays until what was on its way to it must have come.
__device__ __forceinline__ void leave_cluster(bool lost) {
    cluster_barrier();
    if (!lost) return;
    const unsigned long long t0 = global_ns();
    while (global_ns() - t0 < 100000ull) {
    }
}
// A warp's value to the place in the exchange where its row's threads find it.
template <bool kCluster>
__device__ __forceinline__ void publish(float* p, float v, uint64_t* bar, int cluster) {
    if constexpr (!kCluster) {
        *p = v;
    } else {
        for (int q = 0; q < cluster; ++q) send_remote(p, v, bar, q);
    }
}

// Asynchronous copies of one row's tensors into the thread group's own part of shared memory.
// Each thread holds 8 elements of every vector slot: one 16-byte granule of a 16-bit type or two of
// fp32, of which the lanes of a warp copy consecutive ones (whole sectors; `lane` counts them).  A warp's granules stay
// in the tensor's order, so each copy fills 512 contiguous bytes; the fp32 reads then meet in
// banks two by two, which costs little: with the halves of the vectors parted into two planes
// (no conflicts) the copies themselves were the limit, 238 us instead of 185 for 16384 x 4096 with
// an fp32 stream.  Vectors past the row's end are filled with zeros (a copy of no bytes), so the
// arithmetic needs no branches (copy_column: what such a copy names).  Granules that hang over the row's ends are copied whole while
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
__device__ __forceinline__ void copy_granule(uint4* dst, const T* row, int col, int end, int C, int low, int room) {
    constexpr int n = 16 / sizeof(T);
    const bool some = col < end;
    if (kAligned || !some || (col >= low && col + n <= room)) {
        copy16(dst, row + (kAligned ? (some ? col : 0) : copy_column(col, end, n)), some);
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
__device__ __forceinline__ void copy_slot(uint4* slot, const T* row, int lane, int col, int end, int C, int low, int room) {
    if constexpr (sizeof(T) == 2) {
        copy_granule<kAligned>(slot, row, col, end, C, low, room);
    } else {
        const int first = col - 4 * lane;       // this lane's granule of the group's 2 * GW
        copy_granule<kAligned>(slot - lane, row, first, end, C, low, room);
        copy_granule<kAligned>(slot - lane + GW, row, first + 4 * GW, end, C, low, room);
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
template <typename TS, typename TB, bool kAdd, bool kAligned, bool kCluster, int G, int NV, int R, int S>
__global__ void __launch_bounds__(G > 0 ? kWarpCta : kCluster ? 512 : max_cta(R), fwd_min_ctas(G, NV))
norm_fwd_rows_kernel(NormFwd p, int group_threads, int cluster_ctas, int cta_vectors, int) {
    const int cluster = kCluster ? cluster_ctas : 1;
    extern __shared__ __align__(16) float smem[];
    __shared__ float exchange[2][R][2][kWarps * (kCluster ? kMaxCluster : 1)], counts[kWarps * (kCluster ? kMaxCluster : 1)];
    __shared__ uint64_t arrived[2];
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
    const int groups = gridDim.x / cluster * per_cta;
    const int group = blockIdx.x / cluster * per_cta + local;
    const int rank = kCluster ? cluster_rank() : 0;
    const int C = p.C;
    const int shift = kAligned ? 0 : static_cast<int>((static_cast<long long>(group) * C) & 7);
    const int first = rank * cta_vectors * 8 - shift;
    const Columns at{first, min(C, first + cta_vectors * 8), width, lane};
    const float inv = 1.f / static_cast<float>(C);
    // (an update in place overwrites the neighbouring rows: then only the row's own elements are read)
    const bool whole = !p.in_place;
    const int low = whole ? -8 : 0;
    // shared memory: stage, row, then slot (the stream's vectors, the branch's), then thread
    const int x_at = NV * kStream * threads;
    const int row_granules = x_at + (kAdd ? NV * kBranch * threads : 0);
    uint4* const slots = reinterpret_cast<uint4*>(smem);
    const int mine_b = threadIdx.x * kBranch, mine_s = threadIdx.x * kStream;   // this thread's granules of a slot
    pdl_trigger();
    if (kCluster) {
        if (threadIdx.x == 0) {
            mbar_init(&arrived[0], 1);
            mbar_init(&arrived[1], 1);
            fence_barrier_init();
        }
        cluster_barrier();   // every CTA of the cluster is ready before any writes to it
    }
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
                copy_slot<kAligned, TS, GW>(to + k * kStream * threads + mine_s, in, sub, at.of(k), at.end, C, low, room);
                if (kAdd)
                    copy_slot<kAligned, TB, GW>(to + x_at + k * kBranch * threads + mine_b, x, sub, at.of(k), at.end, C, low,
                                                room);
            }
        }
        copy_commit();
    };
#pragma unroll
    for (int i = 0; i < S; ++i) fetch(i, group + static_cast<long long>(i) * R * groups);

    const Edges<NV, kAligned> edges(at, C);
    float2 gamma[NV][4], beta[NV][4];
    load_params(gamma, p.gamma, p.param_type, C, at, 1.f);
    load_params(beta, p.beta, p.param_type, C, at, 0.f);
    // elements of this thread's warp (or group) in a row; its place in the exchange, and the places
    // that one row's sums come from
    const int warps = width >> 5;
    const int place = kCluster ? rank * kWarps + (lane >> 5) : threadIdx.x >> 5;
    const int from_place = local * warps, places = cluster * kWarps;
    int mine = C;
    float peer = 0.f;              // elements of the warp whose sums this lane merges (one CTA to a row)
    if constexpr (kCta) {
        mine = warp_columns<NV>(at, lane >> 5);
        const int w = sub % kPart;
        if (w < warps) peer = static_cast<float>(warp_columns<NV>(at, w));
        if (kCluster) {
            // (places of warps that do not exist count nothing)
            for (int i = threadIdx.x; i < cluster * kWarps; i += threads) counts[i] = 0.f;
            cluster_barrier();
            if (sub == 0)
                for (int q = 0; q < cluster; ++q) store_remote(&counts[place], static_cast<float>(mine), q);
            cluster_barrier();
        }
    }
    const float mine_inv = mine > 0 ? 1.f / static_cast<float>(mine) : 0.f;
    int parity = 0, stage = 0;
    uint32_t phase = 0;                 // of the exchange barrier that is next in use
    bool lost = kCluster && p.stall && rank == cluster - 1;   // a wait of this thread ran out (or is to)

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
                const int col = at.of(k);
                read_slot<TS>(v[u][k], row + k * kStream * threads + mine_s);
                if constexpr (kAdd) {
                    float2 b[4];
                    read_slot<TB>(b, row + x_at + k * kBranch * threads + mine_b);
                    if (drop.threshold != 0) drop8(drop, b, static_cast<uint64_t>(r * C + col) >> 3);
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[u][k][j] = __fadd2_rn(v[u][k][j], b[j]);
                    if (live && col < at.end) store_row8(static_cast<TS*>(p.z) + r * C, v[u][k], col, C, edges.whole[k]);
                }
                if (!edges.whole[k]) mask8(v[u][k], col, C);
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
                const int col = at.of(k);
                float2 d[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) d[j] = __fadd2_rn(v[u][k][j], both(-mean[u]));
                if (!edges.full[k]) mask8(d, col, col >= at.end ? 0 : C);
#pragma unroll
                for (int j = 0; j < 4; ++j) q2 = __ffma2_rn(d[j], d[j], q2);
            }
            s[u] = q2.x + q2.y;
        }
        t = parted_sum<GW, R>(s, sub);
        float m = mean[0];
        if constexpr (R == 2) m = sub < kPart ? mean[0] : mean[1];
        if constexpr (kCta) {
            // the part of a warp that holds row u's sums merges that row over the warps (and CTAs)
            float(&e)[2][kWarps * (kCluster ? kMaxCluster : 1)] = exchange[parity][sub / kPart];
            if (kCluster && threadIdx.x == 0 && !lost)
                mbar_arrive_expect_tx(&arrived[parity], R * 2 * sizeof(float) * warps * cluster);
            if (sub % kPart == 0 && !lost) {
                publish<kCluster>(&e[0][place], m, &arrived[parity], cluster);
                publish<kCluster>(&e[1][place], t, &arrived[parity], cluster);
            }
            if constexpr (!kCluster) {
                group_barrier(1 + local, width);
                const int w = sub % kPart;
                const float em = w < warps ? e[0][from_place + w] : 0.f, eq = w < warps ? e[1][from_place + w] : 0.f;
                m = peer * em;
#pragma unroll
                for (int x = kPart / 2; x > 0; x >>= 1) m += __shfl_xor_sync(0xffffffffu, m, x);
                m *= inv;
                const float d = em - m;
                t = peer > 0.f ? fmaf(peer * d, d, eq) : 0.f;
            } else {
                if (!lost) lost = !await_exchange(&arrived[parity], phase, p.wait_ns, p.status);
                m = 0.f;
                for (int w = sub % kPart; w < places; w += kPart)
                    if (counts[w] > 0.f) m = fmaf(counts[w], e[0][w], m);
#pragma unroll
                for (int x = kPart / 2; x > 0; x >>= 1) m += __shfl_xor_sync(0xffffffffu, m, x);
                m *= inv;
                t = 0.f;
                for (int w = sub % kPart; w < places; w += kPart)
                    if (counts[w] > 0.f) {
                        const float d = e[0][w] - m;
                        t += fmaf(counts[w] * d, d, e[1][w]);
                    }
            }
#pragma unroll
            for (int x = kPart / 2; x > 0; x >>= 1) t += __shfl_xor_sync(0xffffffffu, t, x);
            phase ^= parity;                // both barriers have been used once: their next phase
            parity ^= 1;
        }
        t = 1.f / sqrtf(t * inv + p.eps);
#pragma unroll
        for (int u = 0; u < R; ++u) {
            mean[u] = __shfl_sync(0xffffffffu, m, u * kPart, GW);
            rstd[u] = __shfl_sync(0xffffffffu, t, u * kPart, GW);
        }
#pragma unroll
        for (int u = 0; u < R; ++u) {
            const long long r = r0 + static_cast<long long>(u) * groups;
            if (r >= p.rows) continue;     // (no barrier and no shuffle below)
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                float2 y[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 xhat = __fmul2_rn(__fadd2_rn(v[u][k][j], both(-mean[u])), both(rstd[u]));
                    y[j] = __ffma2_rn(xhat, gamma[k][j], beta[k][j]);
                }
                if (at.of(k) < at.end) store_row8(static_cast<TB*>(p.y) + r * C, y, at.of(k), C, edges.whole[k]);
            }
            if (lane == 0 && rank == 0) {
                if (p.mean != nullptr) p.mean[r] = mean[u];
                if (p.rstd != nullptr) p.rstd[r] = rstd[u];
            }
        }
    }
    copy_wait<0>();
    if (kCluster) leave_cluster(lost);
}

// ------------------------------------------------------------------------------ backward

// CTAs per SM that the register budget allows: 80 registers a thread for one vector, 128 for 2, of
// which 16 a vector hold the gradient sums and 8 gamma.
constexpr int bwd_min_ctas(int G, int NV) { return G == 0 ? 1 : NV == 1 ? 3 : 2; }

// A thread's sums of its columns (null: not wanted).
template <bool kAligned, int NV>
__device__ __forceinline__ void store_sums(float* to, const float2 (&f)[NV][4], const Columns& at, int C) {
    if (to == nullptr) return;
    const bool vec = kAligned && reinterpret_cast<uintptr_t>(to) % 16 == 0;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int col = at.of(k);
        if (col >= at.end) continue;
        if (vec) {
            *reinterpret_cast<float4*>(to + col) = make_float4(f[k][0].x, f[k][0].y, f[k][1].x, f[k][1].y);
            *reinterpret_cast<float4*>(to + col + 4) = make_float4(f[k][2].x, f[k][2].y, f[k][3].x, f[k][3].y);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (in_row(col + j, C)) to[col + j] = j & 1 ? f[k][j / 2].y : f[k][j / 2].x;
        }
    }
}

// dgamma and dbeta of a call of few rows: each CTA adds up a share of the columns over all rows, whose dy
// and z are read once more (from L2).  No partial sums, so no second kernel: a launch of the host and
// some of the GPU's time less (bf16 64 x 4096: 6.1 us and 6.8 call to call, with partial sums 7.9 and
// 9.1).  32 columns are a chunk; `slots` warps share the rows of one, 8 rows at a time in flight, and a
// CTA's warps work on warps / slots chunks together.  `red` holds 32 pairs a warp.
template <typename TS, typename TB>
__device__ __forceinline__ void column_sums(const NormBwd& p, float2* red, int threads, int slots) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, together = (threads >> 5) / slots;
    const int chunks = (p.C + 31) / 32, share = (chunks + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
    const int first = min(chunks, static_cast<int>(blockIdx.x) * share), last = min(chunks, first + share);
    const int slot = warp % slots, mine = warp / slots;
    for (int k = first; k < last; k += together) {
        const int c = (k + mine) * 32 + lane;
        const bool in = mine < together && k + mine < last && c < p.C;
        float2 s = both(0.f);
        if (in) {
            for (long long r0 = slot; r0 < p.rows; r0 += 8 * slots) {
                float f[8], x[8], m[8], rs[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const long long r = r0 + i * slots;
                    const bool live = r < p.rows;
                    f[i] = live ? to_f32(static_cast<const TB*>(p.dy)[r * p.ld_dy + c]) : 0.f;
                    x[i] = live ? to_f32(static_cast<const TS*>(p.z)[r * p.ld_z + c]) : 0.f;
                    m[i] = live ? p.mean[r] : 0.f;
                    rs[i] = live ? p.rstd[r] : 0.f;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    s.x = fmaf(f[i], (x[i] - m[i]) * rs[i], s.x);
                    s.y += f[i];
                }
            }
        }
        __syncthreads();              // red is free: nothing reads the rows or an earlier result any more
        red[warp * 32 + lane] = s;
        __syncthreads();
        if (slot == 0 && in) {
            for (int w = 1; w < slots; ++w) {
                s.x += red[(warp + w) * 32 + lane].x;
                s.y += red[(warp + w) * 32 + lane].y;
            }
            if (p.dgamma != nullptr) p.dgamma[c] = s.x;
            if (p.dbeta != nullptr) p.dbeta[c] = s.y;
        }
    }
}

// Each thread keeps the sums of dy * xhat and dy of its columns in registers over all rows of its
// group; at the end the groups of a CTA are added in order and the CTA writes one row of partial
// sums.  The sums and gamma take the registers, so the rows wait in
// shared memory, S times R rows per group, and are read twice there (before and after a row's
// two means are known).  R rows go through together: one reduction and one barrier for both,
// and two independent chains of latencies.  G == 0: groups of `group_threads` threads, several
// to a CTA where they are short: one CTA per SM, so that there are few rows of partial sums.
// kAdd: the residual form (dz, a branch gradient, dropout).
template <typename TS, typename TB, bool kAdd, bool kAligned, bool kCluster, int G, int NV, int R, int S>
__global__ void __launch_bounds__(G > 0 ? kWarpCta : kCluster ? 512 : max_cta(R), bwd_min_ctas(G, NV))
norm_bwd_rows_kernel(NormBwd p, int group_threads, int cluster_ctas, int cta_vectors, int row_slots) {
    const int cluster = kCluster ? cluster_ctas : 1;
    extern __shared__ __align__(16) float smem[];
    __shared__ float exchange[2][2 * R][kWarps * (kCluster ? kMaxCluster : 1)];
    __shared__ uint64_t arrived[2];
    constexpr bool kCta = G == 0;                  // several warps serve a row
    constexpr int GW = kCta ? 32 : G;              // lanes whose vectors are adjacent
    constexpr int kBranch = sizeof(TB) / 2, kStream = sizeof(TS) / 2;  // granules of a slot
    const int threads = kCta ? blockDim.x : kWarpCta;
    const int width = kCta ? group_threads : G;
    const int local = threadIdx.x / width;         // group within the CTA
    const int lane = threadIdx.x - local * width;
    const int sub = threadIdx.x % GW;
    const int per_cta = threads / width;
    const int groups = gridDim.x / cluster * per_cta;
    const int group = blockIdx.x / cluster * per_cta + local;
    const int rank = kCluster ? cluster_rank() : 0;
    const int C = p.C;
    const int shift = kAligned ? 0 : static_cast<int>((static_cast<long long>(group) * C) & 7);
    const int first = rank * cta_vectors * 8 - shift;
    const Columns at{first, min(C, first + cta_vectors * 8), width, lane};
    const float inv = 1.f / static_cast<float>(C);
    const bool has_dz = kAdd && p.dz != nullptr;
    const bool has_branch = kAdd && p.d_branch != nullptr;
    const bool whole = !p.in_place;                // (as forward)
    const int low = whole ? -8 : 0;
    // shared memory: stage, row, then slot (dy, z, dz of each vector), then thread
    const int z_at = NV * kBranch * threads, dz_at = z_at + NV * kStream * threads;
    const int row_granules = dz_at + (has_dz ? NV * kStream * threads : 0);
    uint4* const slots = reinterpret_cast<uint4*>(smem);
    const int mine_b = threadIdx.x * kBranch, mine_s = threadIdx.x * kStream;   // this thread's granules of a slot
    pdl_trigger();
    if (kCluster) {
        if (threadIdx.x == 0) {
            mbar_init(&arrived[0], 1);
            mbar_init(&arrived[1], 1);
            fence_barrier_init();
        }
        cluster_barrier();   // every CTA of the cluster is ready before any writes to it
    }
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
            const TB* dy = static_cast<const TB*>(p.dy) + r * p.ld_dy;
            const TS* z = static_cast<const TS*>(p.z) + r * p.ld_z;
            const TS* dz = has_dz ? static_cast<const TS*>(p.dz) + r * p.ld_dz : nullptr;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                copy_slot<kAligned, TB, GW>(to + k * kBranch * threads + mine_b, dy, sub, at.of(k), at.end, C, low, room);
                copy_slot<kAligned, TS, GW>(to + z_at + k * kStream * threads + mine_s, z, sub, at.of(k), at.end, C, low, room);
            }
            if (has_dz) {
#pragma unroll
                for (int k = 0; k < NV; ++k)
                    copy_slot<kAligned, TS, GW>(to + dz_at + k * kStream * threads + mine_s, dz, sub, at.of(k), at.end, C, low,
                                                room);
            }
        }
        copy_commit();
    };
#pragma unroll
    for (int i = 0; i < S; ++i) fetch(i, group + static_cast<long long>(i) * R * groups);

    const Edges<NV, kAligned> edges(at, C);
    float2 gamma[NV][4];
    load_params(gamma, p.gamma, p.param_type, C, at, 1.f);
    float2 sum_g[NV][4], sum_b[NV][4];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) sum_g[k][j] = sum_b[k][j] = both(0.f);
    // the warp's place in the exchange, and the places that one row's sums come from
    const int warps = width >> 5;
    const int place = kCluster ? rank * kWarps + (lane >> 5) : threadIdx.x >> 5;
    const int from_place = local * warps;
    int parity = 0, stage = 0;
    uint32_t phase = 0;                 // of the exchange barrier that is next in use
    bool lost = kCluster && p.stall && rank == cluster - 1;   // a wait of this thread ran out (or is to)
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
                    if (!edges.whole[k]) {
                        mask8(f, at.of(k), C);
                        mask8(x, at.of(k), C);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 xhat = __fmul2_rn(__fadd2_rn(x[j], both(-mean[u])), both(rstd[u]));
                        const float2 a = __fmul2_rn(f[j], gamma[k][j]);
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
            // the part of a warp that holds sum q adds it up over the warps (and CTAs)
            float(&e)[kWarps * (kCluster ? kMaxCluster : 1)] = exchange[parity][sub / kPart];
            if (kCluster && threadIdx.x == 0 && !lost)
                mbar_arrive_expect_tx(&arrived[parity], 2 * R * sizeof(float) * warps * cluster);
            if (sub % kPart == 0 && !lost) publish<kCluster>(&e[place], t, &arrived[parity], cluster);
            t = 0.f;
            if constexpr (!kCluster) {
                group_barrier(1 + local, width);
                for (int w = sub % kPart; w < warps; w += kPart) t += e[from_place + w];
            } else {
                if (!lost) lost = !await_exchange(&arrived[parity], phase, p.wait_ns, p.status);
                for (int w = sub % kPart; w < cluster * kWarps; w += kPart)
                    if (w % kWarps < warps) t += e[w];
            }
#pragma unroll
            for (int m = kPart / 2; m > 0; m >>= 1) t += __shfl_xor_sync(0xffffffffu, t, m);
            phase ^= parity;                // both barriers have been used once: their next phase
            parity ^= 1;
        }
#pragma unroll
        for (int q = 0; q < 2 * R; ++q) s[q] = __shfl_sync(0xffffffffu, t, q * kPart, GW);
#pragma unroll
        for (int u = 0; u < R; ++u) {
            const long long r = r0 + static_cast<long long>(u) * groups;
            if (r >= p.rows) continue;        // (no barrier and no shuffle below)
            // dx = rstd (a - c1 - xhat c2) = rstd (a - c1 - (x - mean) k2), k2 = rstd c2.  rstd comes last: its square
            // would overflow for rows of very little spread (eps = 0) whose dx is finite, k2 only where dx does.
            const float c1 = s[2 * u] * inv, k2 = rstd[u] * (s[2 * u + 1] * inv);
            const uint4* row = from + u * row_granules;
            TS* ds = static_cast<TS*>(p.d_stream) + r * C;
            TB* db = has_branch ? static_cast<TB*>(p.d_branch) + r * C : nullptr;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int col = at.of(k);
                float2 f[4], x[4], g[4];
                read_slot<TB>(f, row + k * kBranch * threads + mine_b);
                read_slot<TS>(x, row + z_at + k * kStream * threads + mine_s);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 a = __ffma2_rn(f[j], gamma[k][j], both(-c1));
                    g[j] = __fmul2_rn(__ffma2_rn(__fadd2_rn(x[j], both(-mean[u])), both(-k2), a), both(rstd[u]));
                }
                if (has_dz) {
                    read_slot<TS>(x, row + dz_at + k * kStream * threads + mine_s);
#pragma unroll
                    for (int j = 0; j < 4; ++j) g[j] = __fadd2_rn(g[j], x[j]);
                }
                if (col < at.end) {
                    store_row8(ds, g, col, C, edges.whole[k]);
                    if (has_branch) {
                        if (drop.threshold != 0) drop8(drop, g, static_cast<uint64_t>(r * C + col) >> 3);
                        store_row8(db, g, col, C, edges.whole[k]);
                    }
                }
            }
        }
        __syncwarp();   // all lanes have read the stage
        fetch(stage, r0 + S * step);
        if (++stage == S) stage = 0;
    }
    copy_wait<0>();
    if (kCluster) leave_cluster(lost);
    if (p.dgamma == nullptr && p.dbeta == nullptr) return;
    // a lone CTA (or cluster) has the whole sums, others write a row of partial ones, or where a call of
    // few rows has no place for them each adds up a share of the columns
    const bool alone = gridDim.x == cluster;
    if (!alone && p.partial == nullptr) {
        column_sums<TS, TB>(p, reinterpret_cast<float2*>(smem), threads, row_slots);
        return;
    }
    float* part = alone ? nullptr : p.partial + static_cast<size_t>(blockIdx.x / cluster) * 2 * C;
    float *to_g = alone ? p.dgamma : part, *to_b = alone ? p.dbeta : part + C;
    if (per_cta == 1) {
        // (one group: its threads hold each column once)
        store_sums<kAligned, NV>(to_g, sum_g, at, C);
        store_sums<kAligned, NV>(to_b, sum_b, at, C);
        return;
    }
    __syncthreads();                 // no group reads its rows any more
    float* mine_sums = smem + local * 2 * C;   // the groups' sums, [group][2][C]
    store_sums<kAligned, NV>(mine_sums, sum_g, at, C);
    store_sums<kAligned, NV>(mine_sums + C, sum_b, at, C);
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * C; i += threads) {
        float t = 0.f;
        for (int g = 0; g < per_cta; ++g) t += smem[g * 2 * C + i];
        float* to = i < C ? to_g : to_b;
        if (to != nullptr) to[i < C ? i : i - C] = t;
    }
}

// ------------------------------------------------------------------------------- launches

// What a launch needs to know of its kernel, asked from the runtime once per kernel.
struct KernelFacts {
    DeviceOnce smem;
    std::atomic<int> regs{0};
    ClusterCounts clusters;
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

// How the rows of a call are laid over CTAs.
struct Layout {
    int width;          // threads of a group
    int per_cta;        // groups of a CTA
    int cluster;        // CTAs that share a row
    int cta_vectors;    // vectors of a row in one of them
    int threads;        // of a CTA
    int slots = 0;      // warps that share a column's rows (column_sums), 0: partial sums
};

// G > 0: a row to G lanes.  Else NV vectors a thread: one CTA to a row (several
// groups to a CTA once there are more rows than SMs), or a cluster of 2, 4 or 8 CTAs of up to 512
// threads.  (Twice as many CTAs of 256, two to an SM, wait longer for one another: bf16 4096 x 12288
// 78 against 58 us forward, 102 against 74 backward.)  No layout: threads = 0.
inline Layout layout(bool cluster, int G, int NV, int R, long long rows, int vectors) {
    if (G > 0) return {G, kWarpCta / G, 1, vectors, kWarpCta};
    const int most = cluster ? 512 : max_cta(R);
    Layout l{};
    l.cluster = cluster ? 2 : 1;
    while (cluster && l.cluster < kMaxCluster && vectors > l.cluster * NV * most) l.cluster *= 2;
    if (vectors > l.cluster * NV * most) return Layout{};
    l.cta_vectors = (vectors + l.cluster - 1) / l.cluster;
    l.width = (l.cta_vectors + NV * 32 - 1) / (NV * 32) * 32;
    // as many groups as serve an SM's share of the rows in the fewest rounds, and no more (fp32 3136 x
    // 1024, all tensors: 7 groups and two stages of shared memory 17 us, 10 groups and one 19)
    const long long share = (rows + device_info().sm_count - 1) / device_info().sm_count;
    const long long rounds = (share + most / l.width * R - 1) / (most / l.width * R);
    l.per_cta = cluster ? 1 : static_cast<int>((share + rounds * R - 1) / (rounds * R));
    l.threads = l.width * l.per_cta;
    return l;
}

// Rows that fill no CTA go to clusters.  (Those that do are faster in one: bf16 8192 x 8192 44 against
// 61 us forward, 70 against 80 backward.)
inline bool fits_cta(int vectors) { return vectors <= 2 * max_cta(1); }
// Whether rows of this many vectors go through two at a time: unless one at a time makes so much
// better use of the threads (bf16 8192 x 5003, groups of 320 threads: 50 us forward and 76 backward in
// pairs, one group to a CTA; 42 and 66 one at a time, two groups).
inline bool in_pairs(int vectors) {
    const int width = (vectors + 63) / 64 * 32;
    return max_cta(2) >= width && max_cta(2) / width * 3 > max_cta(1) / width * 2;
}
// Most shared memory of rows on their way, where one row goes through at a time: above it one stage
// serves, not two.  (Copies beyond that only crowd the memory system.  Forward, fp32 branch and
// stream: 8192 x 8192 186 us with two stages of 128 KB in all, 171 with one; fp32 stream with bf16
// branches, 96 KB: 120 against 127.  Backward, fp32 stream with bf16 branches: 65536 x 1024 188 us with
// 200 KB, 164 with 100; 16384 x 4096 174 us with 160 KB, 189 with 80.)
constexpr size_t kFwdFlight = 112 * 1024, kBwdFlight = 176 * 1024;

// Warps that share the rows of a column (column_sums) in a call of `ctas` CTAs of `threads` threads, or 0
// where that would take more than 4 rounds of loads (about 1 us each; partial sums cost as much and a launch).
inline int column_slots(long long rows, int C, int threads, long long ctas) {
    if (rows > 256) return 0;
    int slots = 1;
    while (slots * 2 <= threads / 32 && slots * 8 < rows) slots *= 2;
    const int together = threads / 32 / slots, chunks = (C + 31) / 32;
    const long long share = (chunks + ctas - 1) / ctas;
    return (share + together - 1) / together * ((rows + 8 * slots - 1) / (8 * slots)) <= 4 ? slots : 0;
}

// Rows of a lane group that go through the backward pass together, in two stages: two of a 16-bit
// stream, one of an fp32 stream or where edges are masked (80 registers hold no more; bf16
// 524288 x 128: 66 us, 76 with one stage of two rows).
template <typename TS, bool kAligned>
constexpr int kBwdLaneRows = sizeof(TS) == 2 && kAligned ? 2 : 1;

template <class P>
struct RowLaunch {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    RowLaunch(const P& p, const Layout& l, size_t smem) {
        cfg.blockDim = dim3(static_cast<unsigned>(l.threads));
        cfg.dynamicSmemBytes = smem;
        cfg.stream = p.stream;
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = static_cast<unsigned>(l.cluster);
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = l.cluster > 1 ? 2 : 1;
    }
};

// CTAs (or clusters) for `want` of them: at most what the GPU holds together, since each takes its
// share of the rows and a late one would double the time.  Where rows are shifted they come in
// eights (a group's rows are a multiple of 8 apart, see the head of this file).
template <class K, class P>
cudaError_t launch_rows(K kern, KernelFacts& facts, const P& p, const Layout& l, long long want, size_t smem, int* grid) {
    RowLaunch<P> launch(p, l, smem);
    long long all;
    if (l.cluster == 1) {
        all = static_cast<long long>(device_info().sm_count) * resident_ctas(smem, l.threads, facts.registers(kern));
    } else {
        // clusters need their CTAs on one GPC, whose SMs they do not always divide: 4 CTAs, two to an SM,
        // fit 74 times, not 76
        int device = 0;
        cudaError_t err = cudaGetDevice(&device);
        if (err != cudaSuccess) return err;
        all = facts.clusters.get(device, smem, l.threads, l.cluster, [&] {
            launch.cfg.gridDim = dim3(static_cast<unsigned>(l.cluster));
            int n = 0;
            err = cudaOccupancyMaxActiveClusters(&n, kern, &launch.cfg);
            return err == cudaSuccess ? n : 0;
        });
        if (err != cudaSuccess) return err;
        if (all < 1) return cudaErrorNotSupported;
    }
    if (p.C % 8 != 0) all = std::max(8LL, all / 8 * 8);
    *grid = static_cast<int>(std::min(want, all));
    // what the kernels' accesses rest on: a group's rows all have one shift
    const long long groups = static_cast<long long>(*grid) * l.per_cta;
    if (p.C % 8 != 0 && groups % 8 != 0 && groups < p.rows) return cudaErrorInvalidConfiguration;
    launch.cfg.gridDim = dim3(static_cast<unsigned>(*grid) * static_cast<unsigned>(l.cluster));
    P args = p;
    if (l.cluster > 1) args.stall = take_norm_stall();
    return cudaLaunchKernelEx(&launch.cfg, kern, args, l.width, l.cluster, l.cta_vectors, l.slots);
}

template <typename TS, typename TB, bool kAdd, bool kAligned, bool kCluster, int G, int NV, int R, int S>
cudaError_t fwd_launch(const NormFwd& p, int vectors) {
    auto kern = norm_fwd_rows_kernel<TS, TB, kAdd, kAligned, kCluster, G, NV, R, S>;
    const Layout l = layout(kCluster, G, NV, R, p.rows, vectors);
    const size_t bytes = static_cast<size_t>(S * R * NV * l.threads) * 8 * (sizeof(TS) + (kAdd ? sizeof(TB) : 0));
    if (l.threads == 0 || bytes > (G == 0 && R == 1 && S == 2 ? kFwdFlight : kDynamicSmem)) return cudaErrorNotSupported;
    static KernelFacts facts;
    const cudaError_t err = opt_in_smem(kern, facts.smem, kDynamicSmem);
    if (err != cudaSuccess) return err;
    int grid = 0;
    return launch_rows(kern, facts, p, l, (p.rows + l.per_cta - 1) / l.per_cta, bytes, &grid);
}

template <typename TS, typename TB, bool kAdd, bool kAligned, bool kCluster, int G, int NV, int R, int S>
cudaError_t bwd_launch(const NormBwd& call, int vectors) {
    NormBwd p = call;
    auto kern = norm_bwd_rows_kernel<TS, TB, kAdd, kAligned, kCluster, G, NV, R, S>;
    Layout l = layout(kCluster, G, NV, R, p.rows, vectors);
    if (l.threads == 0) return cudaErrorNotSupported;
    const size_t slot = 8 * (sizeof(TB) + sizeof(TS) * (p.dz != nullptr ? 2 : 1));
    // A few rows go through one CTA, up to three to a group: it writes the parameter gradients itself,
    // and the second kernel that sums partial ones (4 us, as long as three rows) is not needed.
    const int groups = G > 0 ? l.per_cta : kCluster ? 1 : max_cta(R) / l.width;
    // (Shifted rows of a group must be a multiple of 8 apart: lane groups are, others come in one go.)
    const bool one_cta = p.partial != nullptr && !kCluster && p.rows <= (kAligned || G > 0 ? 3LL : 1LL) * groups;
    if (p.partial != nullptr && !kCluster && !one_cta && !p.in_place) {
        // up to 256 rows: the columns' sums in the same kernel, with more groups to a CTA where that
        // takes fewer rounds (not in place: it reads dy and z again, which other CTAs may have overwritten by then)
        l.slots = column_slots(p.rows, p.C, l.threads, (p.rows + l.per_cta - 1) / l.per_cta);
        if (G == 0 && l.slots == 0 && p.rows <= 256) {
            const int most = static_cast<int>(std::min<long long>(groups, p.rows));
            l.slots = column_slots(p.rows, p.C, l.width * most, (p.rows + most - 1) / most);
            if (l.slots != 0) l.per_cta = most;
        }
        if (l.slots != 0) p.partial = nullptr;
    }
    if (G == 0 && one_cta) l.per_cta = static_cast<int>(std::min<long long>(groups, p.rows));
    if (G == 0) l.threads = l.width * l.per_cta;
    size_t bytes = static_cast<size_t>(S * R * NV * l.threads) * slot;
    if (l.per_cta > 1) bytes = std::max(bytes, static_cast<size_t>(l.per_cta) * 2 * p.C * sizeof(float));
    if (bytes > (G == 0 && R == 1 && S == 2 ? kBwdFlight : kDynamicSmem)) return cudaErrorNotSupported;
    static KernelFacts facts;
    cudaError_t err = opt_in_smem(kern, facts.smem, kDynamicSmem);
    if (err != cudaSuccess) return err;
    long long want = one_cta ? 1 : (p.rows + l.per_cta - 1) / l.per_cta;
    const int parts = p.partial != nullptr ? norm_bwd_partials(p.rows, p.C) : INT_MAX;
    if (parts < want) want = p.C % 8 != 0 ? std::max(8, parts / 8 * 8) : parts;   // (eights: see launch_rows)
    int grid = 0;
    err = launch_rows(kern, facts, p, l, want, bytes, &grid);
    if (err != cudaSuccess || p.partial == nullptr || grid == 1) return err;
    return launch_norm_param_sum(p.partial, grid, p.C, p.dgamma, p.dbeta, p.stream);
}

// Rows of several warps: pairs in two stages for 16-bit streams (the arithmetic and the generator need
// them: bf16 16384 x 4096 with dropout 85 us, 98 with one row at a time; they always fit), one row at a
// time in two stages or one for fp32 streams (twice the bytes, and copies in flight beyond them only
// get in the way of the stores: fp32 16384 x 4096 81 us, 93 in pairs).
template <typename TS, typename TB, bool kAdd, bool kAligned, bool kCluster>
cudaError_t fwd_rows_c(const NormFwd& p, int v) {
    if constexpr (sizeof(TS) == 2) {
        if constexpr (!kCluster)
            if (!in_pairs(v)) return fwd_launch<TS, TB, kAdd, kAligned, kCluster, 0, 2, 1, 2>(p, v);
        return fwd_launch<TS, TB, kAdd, kAligned, kCluster, 0, 2, 2, 2>(p, v);
    } else {
        // (a cluster's exchange is paid per pair of rows where pairs go through: fp32 4096 x 16384 102 us, 127
        // with one row at a time)
        if constexpr (kCluster) {
            const cudaError_t err = fwd_launch<TS, TB, kAdd, kAligned, kCluster, 0, 2, 2, 2>(p, v);
            if (err != cudaErrorNotSupported) return err;
        }
        const cudaError_t err = fwd_launch<TS, TB, kAdd, kAligned, kCluster, 0, 2, 1, 2>(p, v);
        return err != cudaErrorNotSupported ? err : fwd_launch<TS, TB, kAdd, kAligned, kCluster, 0, 2, 1, 1>(p, v);
    }
}

template <typename TS, typename TB, bool kAdd, bool kAligned>
cudaError_t fwd_rows_a(const NormFwd& p) {
    const int v = row_vectors(p.C);
    if (v <= 8) return fwd_launch<TS, TB, kAdd, kAligned, false, 8, 1, 2, 2>(p, v);
    if (v <= 16) return fwd_launch<TS, TB, kAdd, kAligned, false, 16, 1, 2, 2>(p, v);
    if (v <= 32) return fwd_launch<TS, TB, kAdd, kAligned, false, 32, 1, 2, 2>(p, v);
    if (v <= 64) return fwd_launch<TS, TB, kAdd, kAligned, false, 32, 2, 2, 1>(p, v);
    return fits_cta(v) ? fwd_rows_c<TS, TB, kAdd, kAligned, false>(p, v) : fwd_rows_c<TS, TB, kAdd, kAligned, true>(p, v);
}

template <typename TS, typename TB, bool kAdd>
cudaError_t fwd_rows(const NormFwd& p) {
    return p.C % 8 == 0 ? fwd_rows_a<TS, TB, kAdd, true>(p) : fwd_rows_a<TS, TB, kAdd, false>(p);
}

// As forward; fp32 rows go in pairs where those fit (bf16 16384 x 4096: 67 us, with one row at a time 76).
template <typename TS, typename TB, bool kAdd, bool kAligned, bool kCluster>
cudaError_t bwd_rows_c(const NormBwd& p, int v) {
    // the residual form on an fp32 stream, where one vector a thread fills most of a CTA: one group to an SM
    // with three rows on their way, instead of two groups with two each (fp32 stream, bf16 branches:
    // 16384 x 4096 174 against 180 us, 13107 x 5120 168 against 182; fp32 16384 x 4096 207 against 217)
    if constexpr (sizeof(TS) == 4 && kAdd && !kCluster)
        if (v > 480 && v <= max_cta(1)) return bwd_launch<TS, TB, kAdd, kAligned, kCluster, 0, 1, 1, 3>(p, v);
    cudaError_t err = cudaErrorNotSupported;
    if (kCluster || in_pairs(v)) err = bwd_launch<TS, TB, kAdd, kAligned, kCluster, 0, 2, 2, 2>(p, v);
    if constexpr (sizeof(TS) == 4 || !kCluster)
        if (err == cudaErrorNotSupported) err = bwd_launch<TS, TB, kAdd, kAligned, kCluster, 0, 2, 1, 2>(p, v);
    if constexpr (sizeof(TS) == 4)
        if (err == cudaErrorNotSupported) err = bwd_launch<TS, TB, kAdd, kAligned, kCluster, 0, 2, 1, 1>(p, v);
    return err;
}

template <typename TS, typename TB, bool kAdd, bool kAligned>
cudaError_t bwd_rows_a(const NormBwd& p) {
    const int v = row_vectors(p.C);
    if (v <= 8) return bwd_launch<TS, TB, kAdd, kAligned, false, 8, 1, kBwdLaneRows<TS, kAligned>, 2>(p, v);
    if (v <= 16) return bwd_launch<TS, TB, kAdd, kAligned, false, 16, 1, kBwdLaneRows<TS, kAligned>, 2>(p, v);
    if (v <= 32) return bwd_launch<TS, TB, kAdd, kAligned, false, 32, 1, kBwdLaneRows<TS, kAligned>, 2>(p, v);
    if (v <= 64) return bwd_launch<TS, TB, kAdd, kAligned, false, 32, 2, 1, 2>(p, v);
    return fits_cta(v) ? bwd_rows_c<TS, TB, kAdd, kAligned, false>(p, v) : bwd_rows_c<TS, TB, kAdd, kAligned, true>(p, v);
}

template <typename TS, typename TB, bool kAdd>
cudaError_t bwd_rows(const NormBwd& p) {
    return p.C % 8 == 0 ? bwd_rows_a<TS, TB, kAdd, true>(p) : bwd_rows_a<TS, TB, kAdd, false>(p);
}

}  // namespace norm
}  // namespace dwc

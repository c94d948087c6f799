// dwc_block_norm_rows.cuh -- the block norm on rows of up to 8192 channels whose tensors line up.
//
//     n = x rstd_post gamma_post,  z = alpha res + scale act(gate) n,  y = z rstd_pre gamma_pre
//
// Bound by memory: forward reads x, gate and res and writes z and y, backward reads dy, dz, x, gate
// and z and writes dx, dgate and dres.  Rows wait in shared memory as in the layer norm's kernels
// (dwc_norm_rows.cuh: asynchronous copies of each thread's own vectors, shifted against rows that do not
// start at a vector boundary), and every value is worked on in registers.  Two sums over a row follow one
// another, since z (backward: the stream's gradient) needs the first: two barriers a row.
//
// Measured (bf16 branches, fp32 stream, gate, 16384 x 4096): forward 139 us, 99 % of the copy bandwidth (one CTA a row that
// reads its row three times: 440), backward 213 us and 5.6 for the parameters (1958).  One bf16 row of 4096 channels
// 3.0 us call to call (17.4).  fp16 4190 x 1024 backward 17.7 us in a graph, 1000 channels 19.0, of 1001, rows that no vector
// divides, 24.2: first and last vectors of a row, which are stored value by value, and parameters cut out of two vectors.
#pragma once

#include "dwc_norm_rows.cuh"
#include "dwc_block_norm_device.cuh"

namespace dwc {
namespace block_norm {

using namespace norm;

// Threads of a CTA whose warps serve rows, one to an SM: with 128 registers each, or 96.
constexpr int kMost = 512, kWide = 640;
// (lane groups of a warp: 256 threads, two or three CTAs to an SM)
constexpr int block_threads(int G, int M) { return G > 0 ? kWarpCta : M; }

// The sum of one value over the threads of a group (G lanes, or several warps of a CTA of up to M threads).
template <int G, int M>
struct GroupSum {
    float (&e)[2][2][M / 32];
    int local, width, parity;
    // which: 0 or 1, the first or second sum of a row
    __device__ __forceinline__ float operator()(float v, int which) const {
        constexpr int GW = G > 0 ? G : 32;
#pragma unroll
        for (int m = GW / 2; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
        if constexpr (G > 0) return v;
        const int warp = threadIdx.x >> 5, warps = width >> 5, lane = threadIdx.x & 31;
        if (warps == 1) return v;
        if (lane == 0) e[parity][which][warp] = v;
        group_barrier(1 + local, width);
        if (warps <= 4) {           // (fewer steps than exchanges)
            v = 0.f;
            for (int w = 0; w < warps; ++w) v += e[parity][which][local * warps + w];
            return v;
        }
        v = lane < warps ? e[parity][which][local * warps + lane] : 0.f;
#pragma unroll
        for (int m = M > 512 ? 16 : 8; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);    // (of M / 32 lanes)
        return __shfl_sync(0xffffffffu, v, 0);
    }
};

// 8 parameters from column c on, zeros beside the row: cut out of the two vectors they lie in (`whole`: the parameters are
// aligned; single loads, 32 bytes apart from lane to lane, take 8 wavefronts each: fp16 4190 x 1001 forward 14.1 us,
// 13.3 so), or
// one by one, on their way together (with a choice of the type around each of them they were waited for in turn).
template <typename T>
__device__ __forceinline__ void params_at(float2 (&f)[4], const T* p, int c, int C, bool whole) {
    const int base = c & ~7, d = c - base;
    if (whole && base >= 0 && base + 16 <= C) {
        Vec8<T> raw[2];
        raw[0].load(p + base);
        raw[1].load(p + base + 8);
        float2 w[2][4];
        raw[0].widen(w[0]);
        raw[1].widen(w[1]);
        float v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = j & 1 ? w[j / 8][j % 8 / 2].y : w[j / 8][j % 8 / 2].x;
#pragma unroll
        for (int j = 0; j < 12; ++j) v[j] = d & 4 ? v[j + 4] : v[j];
#pragma unroll
        for (int j = 0; j < 10; ++j) v[j] = d & 2 ? v[j + 2] : v[j];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = d & 1 ? v[j + 1] : v[j];
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = make_float2(v[2 * j], v[2 * j + 1]);
        return;
    }
    T v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = p[min(max(c + j, 0), C - 1)];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        f[j] = make_float2(in_row(c + 2 * j, C) ? to_f32(v[2 * j]) : 0.f, in_row(c + 2 * j + 1, C) ? to_f32(v[2 * j + 1]) : 0.f);
}

// Parameters of a thread's vectors: one access each where the parameters are aligned and the vectors are not shifted.
template <bool kAligned, int NV>
__device__ __forceinline__ void params(float2 (&f)[NV][4], const void* p, int type, int C, const Columns& at) {
    const size_t align = type == kF32 ? 32 : 16;
    const bool lines_up = reinterpret_cast<uintptr_t>(p) % align == 0, single = !kAligned || !lines_up;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = at.of(k);
        if (p == nullptr) {
#pragma unroll
            for (int j = 0; j < 4; ++j) f[k][j] = make_float2(in_row(c + 2 * j, C) ? 1.f : 0.f, in_row(c + 2 * j + 1, C) ? 1.f : 0.f);
            continue;
        }
        if (single && c < at.end) {
            if (type == kF32) params_at(f[k], static_cast<const float*>(p), c, C, lines_up);
            else if (type == kBF16) params_at(f[k], static_cast<const __nv_bfloat16*>(p), c, C, lines_up);
            else params_at(f[k], static_cast<const __half*>(p), c, C, lines_up);
            continue;
        }
        if (c >= at.end) {
#pragma unroll
            for (int j = 0; j < 4; ++j) f[k][j] = both(0.f);
        } else if (type == kF32) {
            Vec8<float> v;
            v.load(static_cast<const float*>(p) + c);
            v.widen(f[k]);
        } else if (type == kBF16) {
            Vec8<__nv_bfloat16> v;
            v.load(static_cast<const __nv_bfloat16*>(p) + c);
            v.widen(f[k]);
        } else {
            Vec8<__half> v;
            v.load(static_cast<const __half*>(p) + c);
            v.widen(f[k]);
        }
    }
}

// Common to both passes: which columns and rows a thread has.
template <bool kAligned, int G, int NV>
struct Place {
    static constexpr int GW = G > 0 ? G : 32;
    int threads, width, local, lane, sub, groups, group, shift;
    Columns at;
    __device__ __forceinline__ Place(int C, int vectors, int group_threads) {
        threads = G > 0 ? kWarpCta : blockDim.x;
        width = G > 0 ? G : group_threads;
        local = threadIdx.x / width;
        lane = threadIdx.x - local * width;
        sub = threadIdx.x % GW;
        const int per_cta = threads / width;
        groups = gridDim.x * per_cta;
        group = blockIdx.x * per_cta + local;
        shift = kAligned ? 0 : static_cast<int>((static_cast<long long>(group) * C) & 7);
        at = Columns{-shift, min(C, vectors * 8 - shift), width, lane};
    }
};

template <typename TS, typename TB, bool kAligned, int G, int NV, int S, int M>
__global__ void __launch_bounds__(block_threads(G, M), G > 0 ? 2 : 1) block_norm_fwd_rows_kernel(BlockNorm p, int group_threads, int vectors) {
    extern __shared__ __align__(16) float smem[];
    __shared__ float exchange[2][2][M / 32];
    constexpr int kBranch = sizeof(TB) / 2, kStream = sizeof(TS) / 2;  // granules of a slot
    const int C = p.C;
    const Place<kAligned, G, NV> me(C, vectors, group_threads);
    constexpr int GW = Place<kAligned, G, NV>::GW;
    const Columns& at = me.at;
    const bool has_gate = p.gate != nullptr;
    // (an update in place overwrites the neighbouring rows: then only the row's own elements are read)
    const bool whole = !p.in_place;
    const int low = whole ? -8 : 0, threads = me.threads;
    const int x_at = NV * kStream * threads, gate_at = x_at + NV * kBranch * threads;
    const int row_granules = gate_at + (has_gate ? NV * kBranch * threads : 0);
    uint4* const slots = reinterpret_cast<uint4*>(smem);
    const int mine_b = threadIdx.x * kBranch, mine_s = threadIdx.x * kStream;
    const float inv = 1.f / static_cast<float>(C);
    pdl_trigger();
    pdl_wait();

    auto fetch = [&](int stage, long long r) {
        if (r < p.rows) {
            const int room = kAligned ? 0 : whole ? static_cast<int>(min((p.rows - r) * C, 1LL << 30)) : C;
            uint4* to = slots + stage * row_granules;
            const TS* res = static_cast<const TS*>(p.res) + r * p.ld_res;
            const TB* x = static_cast<const TB*>(p.x) + r * p.ld_x;
            const TB* gate = static_cast<const TB*>(p.gate) + r * p.ld_gate;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                copy_slot<kAligned, TB, GW>(to + x_at + k * kBranch * threads + mine_b, x, me.sub, at.of(k), at.end, C, low, room);
                copy_slot<kAligned, TS, GW>(to + k * kStream * threads + mine_s, res, me.sub, at.of(k), at.end, C, low, room);
                if (has_gate)
                    copy_slot<kAligned, TB, GW>(to + gate_at + k * kBranch * threads + mine_b, gate, me.sub, at.of(k), at.end, C, low, room);
            }
        }
        copy_commit();
    };
#pragma unroll
    for (int i = 0; i < S; ++i) fetch(i, me.group + static_cast<long long>(i) * me.groups);
    const Edges<NV, kAligned> edges(at, C);
    float2 w[NV][4], pre_w[NV][4];       // scale * gamma_post, gamma_pre
    params<kAligned>(w, p.gamma_post, p.param_type, C, at);
    params<kAligned>(pre_w, p.scale, p.param_type, C, at);
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) w[k][j] = __fmul2_rn(w[k][j], pre_w[k][j]);
    params<kAligned>(pre_w, p.gamma_pre, p.param_type, C, at);
    GroupSum<G, M> sum{exchange, me.local, me.width, 0};
    int stage = 0;
    const int in_warp = G > 0 ? me.local % (32 / GW) : 0;   // (the lane groups of a warp stay together)
    for (long long r = me.group; r - in_warp < p.rows; r += me.groups) {
        copy_wait<S - 1>();
        __syncwarp();
        const uint4* row = slots + stage * row_granules;
        const bool live = r < p.rows;
        float2 x[NV][4], z[NV][4], q = both(0.f);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            read_slot<TB>(x[k], row + x_at + k * kBranch * threads + mine_b);
            read_slot<TS>(z[k], row + k * kStream * threads + mine_s);
            if (!edges.full[k]) mask8(x[k], at.of(k), at.of(k) >= at.end ? 0 : C);
#pragma unroll
            for (int j = 0; j < 4; ++j) q = __ffma2_rn(x[k][j], x[k][j], q);
        }
        const float post = 1.f / sqrtf(fmaf(sum(q.x + q.y, 0), inv, p.eps));
        q = both(0.f);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float2 m[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) m[j] = __fmul2_rn(__fmul2_rn(x[k][j], both(post)), w[k][j]);
            if (has_gate) {
                float2 g[4];
                read_slot<TB>(g, row + gate_at + k * kBranch * threads + mine_b);
                gate8(g, p.act);
#pragma unroll
                for (int j = 0; j < 4; ++j) m[j] = __fmul2_rn(m[j], g[j]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) z[k][j] = __ffma2_rn(both(p.alpha), z[k][j], m[j]);
            if (!edges.full[k]) mask8(z[k], at.of(k), at.of(k) >= at.end ? 0 : C);
#pragma unroll
            for (int j = 0; j < 4; ++j) q = __ffma2_rn(z[k][j], z[k][j], q);
        }
        __syncwarp();
        fetch(stage, r + static_cast<long long>(S) * me.groups);   // (the stage is read)
        if (++stage == S) stage = 0;
        const float pre = 1.f / sqrtf(fmaf(sum(q.x + q.y, 1), inv, p.eps));
        sum.parity ^= 1;
        if (!live) continue;                // (no barrier and no shuffle below)
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (at.of(k) >= at.end) continue;
            store_row8(static_cast<TS*>(p.z) + r * C, z[k], at.of(k), C, edges.whole[k]);
#pragma unroll
            for (int j = 0; j < 4; ++j) z[k][j] = __fmul2_rn(__fmul2_rn(z[k][j], both(pre)), pre_w[k][j]);
            store_row8(static_cast<TB*>(p.y) + r * C, z[k], at.of(k), C, edges.whole[k]);
        }
        if (me.lane == 0) {
            if (p.rstd_post_out != nullptr) p.rstd_post_out[r] = post;
            if (p.rstd_pre_out != nullptr) p.rstd_pre_out[r] = pre;
        }
    }
    copy_wait<0>();
}

template <typename TB>
constexpr bool params_in_registers(int NV) { return NV == 1 || sizeof(TB) == 4; }

// With zhat = z rstd_pre, xhat = x rstd_post, a = dy gamma_pre, w = scale gamma_post:
//     g = dz + rstd_pre (a - zhat mean(a zhat)),  t = act g,  b = w t
//     dx = rstd_post (b - xhat mean(b xhat)),  dres = alpha g,  dgate = w g xhat act'
// and of the parameters only two sums over the rows, S = sum t xhat and sum dy zhat: dgamma_post is
// scale S, dscale is gamma_post S.  They stay in registers; the groups of a CTA are added at its end.
template <typename TS, typename TB, bool kAligned, int G, int NV, int S, int M>
__global__ void __launch_bounds__(block_threads(G, M), G > 0 ? 2 : 1) block_norm_bwd_rows_kernel(BlockNorm p, int group_threads, int vectors) {
    extern __shared__ __align__(16) float smem[];
    __shared__ float exchange[2][2][M / 32];
    constexpr int kBranch = sizeof(TB) / 2, kStream = sizeof(TS) / 2;
    const int C = p.C;
    const Place<kAligned, G, NV> me(C, vectors, group_threads);
    constexpr int GW = Place<kAligned, G, NV>::GW;
    const Columns& at = me.at;
    const bool has_gate = p.gate != nullptr, has_dz = p.dz != nullptr;
    const bool whole = !p.in_place;
    const int low = whole ? -8 : 0, threads = me.threads;
    const int b_slot = NV * kBranch * threads, s_slot = NV * kStream * threads;
    const int x_at = b_slot, z_at = 2 * b_slot, dz_at = z_at + s_slot, gate_at = dz_at + (has_dz ? s_slot : 0);
    const int row_granules = gate_at + (has_gate ? b_slot : 0);
    uint4* const slots = reinterpret_cast<uint4*>(smem);
    const int mine_b = threadIdx.x * kBranch, mine_s = threadIdx.x * kStream;
    const float inv = 1.f / static_cast<float>(C);
    pdl_trigger();
    pdl_wait();

    auto fetch = [&](int stage, long long r) {
        if (r < p.rows) {
            const int room = kAligned ? 0 : whole ? static_cast<int>(min((p.rows - r) * C, 1LL << 30)) : C;
            uint4* to = slots + stage * row_granules;
            const TB* dy = static_cast<const TB*>(p.dy) + r * p.ld_dy;
            const TB* x = static_cast<const TB*>(p.x) + r * p.ld_x;
            const TS* z = static_cast<const TS*>(p.z_in) + r * p.ld_z;
            const TS* dz = has_dz ? static_cast<const TS*>(p.dz) + r * p.ld_dz : nullptr;
            const TB* gate = has_gate ? static_cast<const TB*>(p.gate) + r * p.ld_gate : nullptr;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int col = at.of(k);
                copy_slot<kAligned, TB, GW>(to + k * kBranch * threads + mine_b, dy, me.sub, col, at.end, C, low, room);
                copy_slot<kAligned, TS, GW>(to + z_at + k * kStream * threads + mine_s, z, me.sub, col, at.end, C, low, room);
                copy_slot<kAligned, TB, GW>(to + x_at + k * kBranch * threads + mine_b, x, me.sub, col, at.end, C, low, room);
                if (has_dz) copy_slot<kAligned, TS, GW>(to + dz_at + k * kStream * threads + mine_s, dz, me.sub, col, at.end, C, low, room);
                if (has_gate) copy_slot<kAligned, TB, GW>(to + gate_at + k * kBranch * threads + mine_b, gate, me.sub, col, at.end, C, low, room);
            }
        }
        copy_commit();
    };
#pragma unroll
    for (int i = 0; i < S; ++i) fetch(i, me.group + static_cast<long long>(i) * me.groups);
    const Edges<NV, kAligned> edges(at, C);
    // scale * gamma_post and gamma_pre of a vector: in registers; where a thread has two vectors of 16-bit branches in its own
    // places in shared memory (registers would be spilled: bf16 4096 x 8192 151 us, 124 so; beside fp32 branches of 8192
    // channels there is no room)
    constexpr bool kKept = params_in_registers<TB>(NV);
    float2 held_w[NV][4], held_pre[NV][4], sum_t[NV][4], sum_pre[NV][4];
    float4* const places = reinterpret_cast<float4*>(slots + S * row_granules) + threadIdx.x;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const Columns one{at.of(k), at.end, 1, 0};
        float2 f[1][4], g[1][4];
        params<kAligned>(f, p.gamma_post, p.param_type, C, one);
        params<kAligned>(g, p.scale, p.param_type, C, one);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            held_w[k][j] = __fmul2_rn(f[0][j], g[0][j]);
            sum_t[k][j] = sum_pre[k][j] = both(0.f);
        }
        params<kAligned>(f, p.gamma_pre, p.param_type, C, one);
#pragma unroll
        for (int j = 0; j < 4; ++j) held_pre[k][j] = f[0][j];
        if constexpr (!kKept) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                places[(k * 4 + q) * threads] = make_float4(held_w[k][2 * q].x, held_w[k][2 * q].y, held_w[k][2 * q + 1].x, held_w[k][2 * q + 1].y);
                places[(k * 4 + 2 + q) * threads] = make_float4(held_pre[k][2 * q].x, held_pre[k][2 * q].y, held_pre[k][2 * q + 1].x, held_pre[k][2 * q + 1].y);
            }
        }
    }
    const auto params_of = [&](float2 (&f)[4], int k, int which) {
        if constexpr (kKept) {
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = which == 0 ? held_w[k][j] : held_pre[k][j];
        } else {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const float4 v = places[(k * 4 + 2 * which + q) * threads];
                f[2 * q] = make_float2(v.x, v.y), f[2 * q + 1] = make_float2(v.z, v.w);
            }
        }
    };
    GroupSum<G, M> sum{exchange, me.local, me.width, 0};
    int stage = 0;
    const int in_warp = G > 0 ? me.local % (32 / GW) : 0;
    float next_post = me.group < p.rows ? p.rstd_post[me.group] : 0.f, next_pre = me.group < p.rows ? p.rstd_pre[me.group] : 0.f;
    for (long long r = me.group; r - in_warp < p.rows; r += me.groups) {
        const float post = next_post, pre = next_pre;
        if (r + me.groups < p.rows) {
            next_post = p.rstd_post[r + me.groups];
            next_pre = p.rstd_pre[r + me.groups];
        }
        copy_wait<S - 1>();
        __syncwarp();
        const uint4* row = slots + stage * row_granules;
        const bool live = r < p.rows;
        float2 q = both(0.f), zhat[NV][4], t[NV][4];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            // (a row that does not exist left the slot as it was: nothing of it may count)
            const int limit = !live || at.of(k) >= at.end ? 0 : C;
            read_slot<TB>(t[k], row + k * kBranch * threads + mine_b);
            read_slot<TS>(zhat[k], row + z_at + k * kStream * threads + mine_s);
            float2 pre_w[4];
            params_of(pre_w, k, 1);
            if (!live || !edges.full[k]) {
                mask8(t[k], at.of(k), limit);
                mask8(zhat[k], at.of(k), limit);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                zhat[k][j] = __fmul2_rn(zhat[k][j], both(pre));
                sum_pre[k][j] = __ffma2_rn(t[k][j], zhat[k][j], sum_pre[k][j]);
                t[k][j] = __fmul2_rn(t[k][j], pre_w[j]);          // a
                q = __ffma2_rn(t[k][j], zhat[k][j], q);
            }
        }
        const float m_pre = sum(q.x + q.y, 0) * inv;
        q = both(0.f);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int limit = !live || at.of(k) >= at.end ? 0 : C;
            float2 x[4], v[4], w[4];
            params_of(w, k, 0);
            read_slot<TB>(x, row + x_at + k * kBranch * threads + mine_b);
            if (!live || !edges.full[k]) mask8(x, at.of(k), limit);
#pragma unroll
            for (int j = 0; j < 4; ++j) t[k][j] = __fmul2_rn(__ffma2_rn(zhat[k][j], both(-m_pre), t[k][j]), both(pre));
            if (has_dz) {
                read_slot<TS>(v, row + dz_at + k * kStream * threads + mine_s);
                if (!live || !edges.full[k]) mask8(v, at.of(k), limit);
#pragma unroll
                for (int j = 0; j < 4; ++j) t[k][j] = __fadd2_rn(t[k][j], v[j]);
            }
            if (live && at.of(k) < at.end) {
                float2 o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) o[j] = __fmul2_rn(both(p.alpha), t[k][j]);
                store_row8(static_cast<TS*>(p.dres) + r * C, o, at.of(k), C, edges.whole[k]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = __fmul2_rn(x[j], both(post));      // xhat
            if (has_gate) {
                read_slot<TB>(v, row + gate_at + k * kBranch * threads + mine_b);
                if (!live || !edges.full[k]) mask8(v, at.of(k), limit);
                float2 o[4];
                gate8(v, o, p.act);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    o[j] = __fmul2_rn(__fmul2_rn(__fmul2_rn(w[j], t[k][j]), x[j]), o[j]);
                    t[k][j] = __fmul2_rn(t[k][j], v[j]);
                }
                if (live && at.of(k) < at.end && p.dgate != nullptr)
                    store_row8(static_cast<TB*>(p.dgate) + r * C, o, at.of(k), C, edges.whole[k]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sum_t[k][j] = __ffma2_rn(t[k][j], x[j], sum_t[k][j]);
                t[k][j] = __fmul2_rn(t[k][j], w[j]);             // b
                q = __ffma2_rn(t[k][j], x[j], q);
                zhat[k][j] = x[j];
            }
        }
        __syncwarp();
        fetch(stage, r + static_cast<long long>(S) * me.groups);   // (the stage is read)
        if (++stage == S) stage = 0;
        const float m_post = sum(q.x + q.y, 1) * inv;
        sum.parity ^= 1;
        if (!live) continue;                // (no barrier and no shuffle below)
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (at.of(k) >= at.end) continue;
#pragma unroll
            for (int j = 0; j < 4; ++j) t[k][j] = __fmul2_rn(__ffma2_rn(zhat[k][j], both(-m_post), t[k][j]), both(post));
            store_row8(static_cast<TB*>(p.dx) + r * C, t[k], at.of(k), C, edges.whole[k]);
        }
    }
    copy_wait<0>();
    if (p.partial == nullptr) return;
    const int per_cta = threads / me.width;
    float* part = p.partial + static_cast<size_t>(blockIdx.x) * 2 * C;
    if (kAligned && per_cta == 1) {
        store_sums<kAligned, NV>(part, sum_t, at, C);
        store_sums<kAligned, NV>(part + C, sum_pre, at, C);
        return;
    }
    __syncthreads();                 // no group reads its rows any more
    // the groups' sums, [group][2][vectors], each vector in its own place (a group's columns are shifted by `shift`)
    const int room = vectors * 8;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        if (at.of(k) >= at.end) continue;
        float4* to = reinterpret_cast<float4*>(smem + me.local * 2 * room + at.of(k) + me.shift);
        to[0] = make_float4(sum_t[k][0].x, sum_t[k][0].y, sum_t[k][1].x, sum_t[k][1].y);
        to[1] = make_float4(sum_t[k][2].x, sum_t[k][2].y, sum_t[k][3].x, sum_t[k][3].y);
        to += room / 4;
        to[0] = make_float4(sum_pre[k][0].x, sum_pre[k][0].y, sum_pre[k][1].x, sum_pre[k][1].y);
        to[1] = make_float4(sum_pre[k][2].x, sum_pre[k][2].y, sum_pre[k][3].x, sum_pre[k][3].y);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * C; i += threads) {
        const int from = i < C ? i : i - C + room;
        float s = 0.f;
        for (int g = 0; g < per_cta; ++g) {
            const int shift = kAligned ? 0 : static_cast<int>((static_cast<long long>(blockIdx.x * per_cta + g) * C) & 7);
            s += smem[g * 2 * room + shift + from];
        }
        part[i] = s;
    }
}

// ------------------------------------------------------------------------------- launches

struct Plan {
    int width, per_cta, threads, grid;
    size_t smem;
};

// `slot`: bytes of a vector's tensors in a stage, `more`: besides the stages.
// One CTA to an SM (lane groups: as many as fit), groups of the fewest threads that hold a row; as many
// groups to a CTA as serve its share of the rows in the fewest rounds.  Where rows are shifted the
// number of groups is a multiple of 8, so that a group's rows all have one shift.
template <class K>
cudaError_t plan_rows(K kern, KernelFacts& facts, const BlockNorm& p, int G, int NV, int S, int M, size_t slot, size_t more, int vectors, int parts, Plan& l) {
    const int sms = device_info().sm_count;
    if (G > 0) {
        l.width = G;
        l.per_cta = kWarpCta / G;
    } else {
        l.width = (vectors + NV * 32 - 1) / (NV * 32) * 32;
        if (l.width > M) return cudaErrorNotSupported;
        const long long share = (p.rows + sms - 1) / sms, most = M / l.width;
        const long long rounds = (share + most - 1) / most;
        l.per_cta = static_cast<int>((share + rounds - 1) / rounds);
    }
    l.threads = l.width * l.per_cta;
    l.smem = static_cast<size_t>(l.threads) * NV * (S * slot + more);
    if (parts > 0) l.smem = std::max(l.smem, static_cast<size_t>(l.per_cta) * 2 * vectors * 8 * sizeof(float));
    if (l.smem > kDynamicSmem) return cudaErrorNotSupported;
    const cudaError_t err = opt_in_smem(kern, facts.smem, kDynamicSmem);
    if (err != cudaSuccess) return err;
    long long all = static_cast<long long>(sms) * resident_ctas(l.smem, l.threads, facts.registers(kern));
    long long want = (p.rows + l.per_cta - 1) / l.per_cta;
    if (parts > 0) all = std::min<long long>(all, parts);
    if (p.C % 8 != 0) all = std::max(8LL, all / 8 * 8);
    l.grid = static_cast<int>(std::min(want, all));
    const long long groups = static_cast<long long>(l.grid) * l.per_cta;
    if (p.C % 8 != 0 && groups % 8 != 0 && groups < p.rows) return cudaErrorInvalidConfiguration;
    if (parts > 0 && l.grid > parts) return cudaErrorNotSupported;      // (more eights than the workspace has rows)
    return cudaSuccess;
}

template <typename TS, typename TB, bool kAligned, int G, int NV, int S, int M = kMost>
cudaError_t fwd_launch(const BlockNorm& p, int vectors) {
    auto kern = block_norm_fwd_rows_kernel<TS, TB, kAligned, G, NV, S, M>;
    static KernelFacts facts;
    Plan l;
    const size_t slot = 8 * (sizeof(TS) + sizeof(TB) * (p.gate != nullptr ? 2 : 1));
    const cudaError_t err = plan_rows(kern, facts, p, G, NV, S, M, slot, 0, vectors, 0, l);
    if (err != cudaSuccess) return err;
    return launch_pdl(kern, dim3(static_cast<unsigned>(l.grid)), dim3(static_cast<unsigned>(l.threads)), l.smem, p.stream, p, l.width,
                      vectors);
}

template <typename TS, typename TB, bool kAligned, int G, int NV, int S, int M = kMost>
cudaError_t bwd_launch(const BlockNorm& p, int vectors) {
    auto kern = block_norm_bwd_rows_kernel<TS, TB, kAligned, G, NV, S, M>;
    static KernelFacts facts;
    Plan l;
    const size_t slot = 8 * (sizeof(TB) * (p.gate != nullptr ? 3 : 2) + sizeof(TS) * (p.dz != nullptr ? 2 : 1));
    cudaError_t err = plan_rows(kern, facts, p, G, NV, S, M, slot, params_in_registers<TB>(NV) ? 0 : 64, vectors,
                                p.partial != nullptr ? block_norm_partials(p.rows, p.C) : 0, l);
    if (err != cudaSuccess) return err;
    err = launch_pdl(kern, dim3(static_cast<unsigned>(l.grid)), dim3(static_cast<unsigned>(l.threads)), l.smem, p.stream, p, l.width,
                     vectors);
    return err != cudaSuccess || p.partial == nullptr ? err : launch_block_norm_params(p, l.grid);
}

// Whether CTAs of kWide threads hold so many more groups of a row than those of kMost (or one where there was none) that
// fewer registers pay: half as many again; twice as many where rows are shifted; with fp32 branches, whose kernels
// have room for two CTAs to an SM, only where there was none.  bf16, kWide and kMost threads: 6553 x 5120 forward 61 and 78 us,
// backward 106 and 154; 13107 x 2560 backward 104 and 134; 21845 x 1536 105 and 116, of 1501 channels 93 and 88; fp32
// 3276 x 5120 backward 108 and 130, 6553 x 2560 96 and 84.
template <typename TB, bool kAligned>
inline bool wide_cta(int vectors, int NV) {
    const int width = (vectors + NV * 32 - 1) / (NV * 32) * 32;
    if (width > kWide) return false;
    return sizeof(TB) == 4 ? width > kMost : 2 * (kWide / width) >= (kAligned ? 3 : 4) * (kMost / width);
}

template <typename TS, typename TB, bool kAligned>
cudaError_t fwd_rows(const BlockNorm& p) {
    const int v = row_vectors(p.C);
    if (v <= 8) return fwd_launch<TS, TB, kAligned, 8, 1, 2>(p, v);
    if (v <= 16) return fwd_launch<TS, TB, kAligned, 16, 1, 2>(p, v);
    if (v <= 32) return fwd_launch<TS, TB, kAligned, 32, 1, 2>(p, v);
    // (a row to an SM: the most threads it can take)
    if (v <= kMost && p.rows <= device_info().sm_count) return fwd_launch<TS, TB, kAligned, 0, 1, 1>(p, v);
    if (wide_cta<TB, kAligned>(v, 2)) {
        const cudaError_t err = fwd_launch<TS, TB, kAligned, 0, 2, 2, kWide>(p, v);
        if (err != cudaErrorNotSupported) return err;
    }
    const cudaError_t err = fwd_launch<TS, TB, kAligned, 0, 2, 2>(p, v);
    return err == cudaErrorNotSupported ? fwd_launch<TS, TB, kAligned, 0, 2, 1>(p, v) : err;
}

template <typename TS, typename TB, bool kAligned>
cudaError_t bwd_rows(const BlockNorm& p) {
    const int v = row_vectors(p.C);
    if (v <= 8) return bwd_launch<TS, TB, kAligned, 8, 1, 2>(p, v);
    if (v <= 16) return bwd_launch<TS, TB, kAligned, 16, 1, 2>(p, v);
    if (v <= 32) return bwd_launch<TS, TB, kAligned, 32, 1, 2>(p, v);
    cudaError_t err = wide_cta<TB, kAligned>(v, 1) ? bwd_launch<TS, TB, kAligned, 0, 1, 2, kWide>(p, v) : cudaErrorNotSupported;
    if (err == cudaErrorNotSupported && v <= kMost) err = bwd_launch<TS, TB, kAligned, 0, 1, 2>(p, v);
    // (two vectors a thread: one stage, whose kernel has registers enough; bf16 4681 x 7168 124 us, 157 with two)
    return err == cudaErrorNotSupported ? bwd_launch<TS, TB, kAligned, 0, 2, 1>(p, v) : err;
}

template <typename TS, typename TB>
cudaError_t fwd_rows(const BlockNorm& p) {
    return p.C % 8 == 0 ? fwd_rows<TS, TB, true>(p) : fwd_rows<TS, TB, false>(p);
}
template <typename TS, typename TB>
cudaError_t bwd_rows(const BlockNorm& p) {
    return p.C % 8 == 0 ? bwd_rows<TS, TB, true>(p) : bwd_rows<TS, TB, false>(p);
}

}  // namespace block_norm
}  // namespace dwc

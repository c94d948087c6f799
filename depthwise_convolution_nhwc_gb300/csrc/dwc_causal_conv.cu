// dwc_causal_conv.cu -- the short causal depthwise convolution along sequences, forward, backward and
// for single tokens.
//
//     pre[t, c] = bias[c] + sum_k w[k, c] x[t - K + 1 + k, c],  y = act(pre)
//     dpre = dy act'(pre),  dx[t] = sum_k w[k] dpre[t + K - 1 - k],  dw[k] = sum_t dpre[t] x[t - K + 1 + k]
//
// Bound by memory: x (and dy) are read once and y (dx) written once.  A thread owns V adjacent
// channels and walks along a run of positions with the last K inputs in registers; the run's K - 1
// rows in front (and, backward, behind) are read again from L1 or L2.
//
// Measured (bf16, 8 sequences of 2048 positions, 4096 channels, 4 taps, SiLU): forward 44 us (89 % of the copy bandwidth),
// with one load at a time 107; backward 85 us with 4 us for the sums of partial rows (its bytes take 59).  In fp32, whose
// bytes bind both, 82 (96 %) and 128 (92 %).  The bf16 backward pass waits on its instructions, 24 a value, of which 16 warps
// to an SM (128 registers a thread) issue one every other cycle.  fp32 packed rows of 1001 channels, one channel a thread:
// 22 us (9).
#include <algorithm>
#include <type_traits>

#include "dwc_seq_device.cuh"

namespace dwc {
namespace {

constexpr int kThreads = 128;

// fp32 values of V adjacent channels, in pairs for the packed arithmetic.
template <int V>
struct Lanes {
    float2 v[V / 2];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int j = 0; j < V / 2; ++j) v[j] = both(0.f);
    }
    __device__ __forceinline__ void fma(const Lanes& a, const Lanes& b) {        // += a b
#pragma unroll
        for (int j = 0; j < V / 2; ++j) v[j] = __ffma2_rn(a.v[j], b.v[j], v[j]);
    }
    __device__ __forceinline__ void add(const Lanes& a) {
#pragma unroll
        for (int j = 0; j < V / 2; ++j) v[j] = __fadd2_rn(v[j], a.v[j]);
    }
    __device__ __forceinline__ void to_silu() {
#pragma unroll
        for (int j = 0; j < V / 2; ++j) v[j] = silu2(v[j]);
    }
    __device__ __forceinline__ void by_slope(const Lanes& a) {                   // *= silu'(a)
#pragma unroll
        for (int j = 0; j < V / 2; ++j) v[j] = __fmul2_rn(v[j], silu_slope2(a.v[j]));
    }
    __device__ __forceinline__ float get(int j) const { return j & 1 ? v[j / 2].y : v[j / 2].x; }
    __device__ __forceinline__ void set(int j, float f) { (j & 1 ? v[j / 2].y : v[j / 2].x) = f; }
};
template <>
struct Lanes<1> {
    float v;
    __device__ __forceinline__ void clear() { v = 0.f; }
    __device__ __forceinline__ void fma(const Lanes& a, const Lanes& b) { v = fmaf(a.v, b.v, v); }
    __device__ __forceinline__ void add(const Lanes& a) { v += a.v; }
    __device__ __forceinline__ void to_silu() { v = silu(v); }
    __device__ __forceinline__ void by_slope(const Lanes& a) { v *= silu_slope(a.v, sigmoid(a.v)); }
    __device__ __forceinline__ float get(int) const { return v; }
    __device__ __forceinline__ void set(int, float f) { v = f; }
};

// The same as they lie in memory.
template <typename T, int V>
struct Raw {
    static constexpr int kBytes = V * sizeof(T);
    using Word = typename std::conditional<kBytes == 16, uint4, typename std::conditional<kBytes == 8, uint2, typename std::conditional<kBytes == 4, uint32_t, uint16_t>::type>::type>::type;
    Word w;
    __device__ __forceinline__ void zero() { w = Word{}; }
    __device__ __forceinline__ void load(const T* p) { w = *reinterpret_cast<const Word*>(p); }
    __device__ __forceinline__ void put(T* p) const { *reinterpret_cast<Word*>(p) = w; }
    __device__ __forceinline__ Lanes<V> widen() const {
        Lanes<V> f;
        if constexpr (V == 1) {
            f.v = to_f32(*reinterpret_cast<const T*>(&w));
        } else {
            using Pair = typename Elem<T>::pair_t;
#pragma unroll
            for (int j = 0; j < V / 2; ++j) f.v[j] = Elem<T>::load_pair(reinterpret_cast<const T*>(reinterpret_cast<const Pair*>(&w) + j));
        }
        return f;
    }
    __device__ static __forceinline__ void store(T* p, const Lanes<V>& f) {
        Raw r;
        if constexpr (V == 1) {
            store_out(reinterpret_cast<T*>(&r.w), f.v);
        } else {
            using Pair = typename Elem<T>::pair_t;
            Pair* v = reinterpret_cast<Pair*>(&r.w);
#pragma unroll
            for (int j = 0; j < V / 2; ++j) {
                if constexpr (std::is_same<T, float>::value) v[j] = f.v[j];
                else if constexpr (std::is_same<T, __half>::value) v[j] = __float22half2_rn(f.v[j]);
                else v[j] = __float22bfloat162_rn(f.v[j]);
            }
        }
        r.put(p);
    }
};

// Input at position t of a sequence (negative: from its state).
template <typename T, int V>
__device__ __forceinline__ Lanes<V> input(const T* x, long long row, const T* state, int C, int K, long long t) {
    Raw<T, V> r;
    r.zero();
    if (t >= 0) r.load(x + t * row);
    else if (state != nullptr) r.load(state + (t + K - 1) * C);
    return r.widen();
}

// Parameters of V channels: w[i] is the tap on the input i positions back.
template <int KM, int V>
__device__ __forceinline__ void load_taps(Lanes<V> (&w)[KM], Lanes<V>& bias, const CausalConv& p, int K, int c) {
#pragma unroll
    for (int i = 0; i < KM; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) w[i].set(j, i < K ? load_param(p.w, p.param_type, (K - 1 - i) * p.C + c + j, 0.f) : 0.f);
#pragma unroll
    for (int j = 0; j < V; ++j) bias.set(j, load_param(p.bias, p.param_type, c + j, 0.f));
}

template <int KM, int V>
__device__ __forceinline__ Lanes<V> convolve(const Lanes<V> (&w)[KM], const Lanes<V>& bias, const Lanes<V> (&win)[KM], int K) {
    Lanes<V> f = bias;
#pragma unroll
    for (int i = KM - 1; i >= 0; --i)
        if (i < K) f.fma(w[i], win[i]);
    return f;
}

template <int KM, int V>
__device__ __forceinline__ void shift(Lanes<V> (&win)[KM]) {
#pragma unroll
    for (int i = KM - 1; i > 0; --i) win[i] = win[i - 1];
}

// Rows that a thread brings in together, batches ahead of the one it works on: what is in flight is what counts
// (bf16 8 x 2048 x 4096, 4 taps, forward: 8 rows of 4 channels, two batches under way, five CTAs to an SM 44 us, one batch in registers
// 46, of 4 rows 54, of 4 rows of 8 channels 58; backward: 4 rows 90, 8 rows 103, 2 rows 96).
constexpr int kFwdBatch = 8, kBwdBatch = 4;

template <int kBytes>
__device__ __forceinline__ void copy_async(void* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_addr(dst)), "l"(src), "n"(kBytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Where batches wait: in shared memory, brought there by each thread for itself (no barrier), or in registers.
// Backward in registers only where a thread's values are less than the 4 bytes that a copy takes (8 x 2048 x 4096 as above: two
// batches under way in shared memory 90 us, one 94, one in registers 99; fp32 129 and 256).  Forward with several channels and
// taps (bf16 44 us, in registers 46, fp32 82 and 97; one channel 26 and 25, one tap of 2048 channels 26 and 20).
template <typename T, int V, bool kWanted>
struct Stage {
    using Word = typename Raw<T, V>::Word;
    static constexpr bool kOn = kWanted && sizeof(Word) >= 4;
    static constexpr int kBatches = !kOn || sizeof(Word) == 16 ? 2 : 3;      // one of them in work
};

// KM: taps held in registers; up to 4 it is the number of taps, 8 and 16 serve the numbers up to it.
template <typename T, int KM, int V>
__global__ void __launch_bounds__(kThreads, KM < 8 ? 5 : 1) causal_conv_fwd_kernel(CausalConv p, int columns, int run, int blocks) {
    using S = Stage<T, V, (V > 1 && KM > 1)>;
    __shared__ __align__(16) typename S::Word ring[S::kOn ? S::kBatches * kFwdBatch : 1][kThreads];
    pdl_trigger();
    pdl_wait();
    const int K = KM >= 8 ? p.K : KM, C = p.C;
    const long long slot = blockIdx.x / blocks;
    const int block = static_cast<int>(blockIdx.x - slot * blocks);
    const int column = threadIdx.x % columns, group = threadIdx.x / columns;
    const int c = (block * columns + column) * V;
    const Piece r = find_piece(p.seqs, slot, p.span);
    if (!r.some || c >= C) return;
    const T* x = view_at<T>(p.x, p.seqs, r) + c;
    const T* state = p.state == nullptr ? nullptr : static_cast<const T*>(p.state) + static_cast<long long>(r.s) * (K - 1) * C + c;
    const long long first = r.first + static_cast<long long>(group) * run;
    const int n = static_cast<int>((first + run < r.end ? first + run : r.end) - first);      // positions of this thread
    if (n > 0) {
        const T* from = x + first * p.x.row;
        T* to = static_cast<T*>(p.y) + (dense_row(p.seqs, r) + first) * C + c;
        Raw<T, V> next[kFwdBatch];               // (without copies)
        int place = 0;                           // of the next batch in the ring
        const auto fetch = [&](int t) {       // (positions t .. t + kFwdBatch - 1, in turn)
            typename S::Word* to = &ring[S::kOn ? place * kFwdBatch : 0][threadIdx.x];
#pragma unroll
            for (int q = 0; q < kFwdBatch; ++q) {
                if (t + q < n) {
                    if constexpr (S::kOn) copy_async<sizeof(typename S::Word)>(to + q * kThreads, from);
                    else next[q].load(from);
                }
                from += p.x.row;
            }
            if constexpr (S::kOn) {
                copy_commit();
                place = place == S::kBatches - 1 ? 0 : place + 1;
            }
        };
#pragma unroll
        for (int i = 0; i < S::kBatches - 1; ++i) fetch(i * kFwdBatch);
        Lanes<V> w[KM], bias, win[KM];        // win[i]: the input i positions back
        load_taps(w, bias, p, K, c);
#pragma unroll
        for (int i = 1; i < KM; ++i)
            if (i < K) win[i] = input<T, V>(x, p.x.row, state, C, K, first - i);
        for (int t0 = 0; t0 < n; t0 += kFwdBatch) {
            Raw<T, V> raw[kFwdBatch];
            // the oldest batch of the ring, whose copies came before the others'
            const typename S::Word* batch = &ring[S::kOn ? (place == S::kBatches - 1 ? 0 : place + 1) * kFwdBatch : 0][threadIdx.x];
            if constexpr (S::kOn) {
                copy_wait<S::kBatches - 2>();
            } else {
#pragma unroll
                for (int q = 0; q < kFwdBatch; ++q) raw[q] = next[q];
            }
            // (into the place of the batch before, whose values are used up)
            fetch(t0 + (S::kBatches - 1) * kFwdBatch);
#pragma unroll
            for (int q = 0; q < kFwdBatch; ++q) {
                if constexpr (S::kOn) raw[q].w = batch[q * kThreads];
                win[0] = raw[q].widen();
                Lanes<V> f = convolve(w, bias, win, K);
                if (p.silu) f.to_silu();
                if (t0 + q < n) Raw<T, V>::store(to, f);
                to += C;
                shift(win);
            }
        }
    }
    if (r.last && p.final_state != nullptr) {
        T* out = static_cast<T*>(p.final_state) + static_cast<long long>(r.s) * (K - 1) * C + c;
        for (int i = group; i < K - 1; i += kThreads / columns)
            Raw<T, V>::store(out + static_cast<long long>(i) * C, input<T, V>(x, p.x.row, state, C, K, r.length - (K - 1) + i));
    }
}

// A thread walks K - 1 positions past its run: position t gives dpre[t], and with it dx[t - K + 1] is
// complete.  Parameter gradients count the run's own positions; the CTA's groups are added in order.
template <typename T, int KM, int V>
__global__ void __launch_bounds__(kThreads, KM < 8 ? 4 : 1) causal_conv_bwd_kernel(CausalConv p, int columns, int run, int blocks) {
    using S = Stage<T, V, true>;
    __shared__ float sums[kThreads * V];
    __shared__ __align__(16) typename S::Word ring[S::kOn ? S::kBatches * 2 * kBwdBatch : 1][kThreads];
    pdl_trigger();
    pdl_wait();
    const int K = KM >= 8 ? p.K : KM, C = p.C;
    const long long slot = blockIdx.x / blocks;
    const int block = static_cast<int>(blockIdx.x - slot * blocks);
    const int column = threadIdx.x % columns, group = threadIdx.x / columns, groups = kThreads / columns;
    const int c = (block * columns + column) * V;
    const Piece r = find_piece(p.seqs, slot, p.span);
    const bool here = r.some && c < C;
    Lanes<V> dw[KM], db;             // dw[i]: of the tap on the input i positions back
    db.clear();
#pragma unroll
    for (int i = 0; i < KM; ++i) dw[i].clear();
    const long long first = r.first + static_cast<long long>(group) * run;
    const int n = first < r.end ? static_cast<int>((first + run < r.end ? first + run : r.end) - first) : 0;
    if (here && (n > 0 || first == 0)) {
        const T* x = view_at<T>(p.x, p.seqs, r) + c;
        const long long kept = static_cast<long long>(r.s) * (K - 1) * C + c, rest = r.length - first;
        const T* state = p.state == nullptr ? nullptr : static_cast<const T*>(p.state) + kept;
        const T* dfinal = p.dfinal == nullptr ? nullptr : static_cast<const T*>(p.dfinal) + kept;
        T* dstate = p.dstate == nullptr ? nullptr : static_cast<T*>(p.dstate) + kept;
        // the first run's walk gives the state's positions as well
        const int low = first == 0 ? -(K - 1) : 0, stop = n + K - 1, known = stop < rest ? stop : static_cast<int>(rest);
        // (positions that the last inputs kept have a gradient through them: from this one on)
        const int kept_from = dfinal != nullptr && rest - (K - 1) < stop ? static_cast<int>(rest) - (K - 1) : stop;
        const T* from_x = x + first * p.x.row;
        const T* from_dy = view_at<T>(p.dy, p.seqs, r) + c + first * p.dy.row;
        T* to = static_cast<T*>(p.dx) + (dense_row(p.seqs, r) + first - (K - 1)) * C + c;
        Raw<T, V> next_x[kBwdBatch], next_dy[kBwdBatch];        // (without copies)
        int place = 0;                                           // of the next batch in the ring
        const auto fetch = [&](int t) {       // (positions t .. t + kBwdBatch - 1, in turn)
            typename S::Word* to = &ring[S::kOn ? place * 2 * kBwdBatch : 0][threadIdx.x];
#pragma unroll
            for (int q = 0; q < kBwdBatch; ++q) {
                if (t + q < known) {
                    if constexpr (S::kOn) {
                        copy_async<sizeof(typename S::Word)>(to + 2 * q * kThreads, from_x);
                        copy_async<sizeof(typename S::Word)>(to + (2 * q + 1) * kThreads, from_dy);
                    } else {
                        next_x[q].load(from_x);
                        next_dy[q].load(from_dy);
                    }
                }
                from_x += p.x.row;
                from_dy += p.dy.row;
            }
            if constexpr (S::kOn) {
                copy_commit();
                place = place == S::kBatches - 1 ? 0 : place + 1;
            }
        };
#pragma unroll
        for (int i = 0; i < S::kBatches - 1; ++i) fetch(i * kBwdBatch);
        Lanes<V> w[KM], bias, win[KM], dpre[KM];
        load_taps(w, bias, p, K, c);
        // (the number of taps is not known: the same in the other order, since registers have no variable index)
        Lanes<V> ahead[KM < 8 ? 1 : KM];
        if constexpr (KM >= 8) {
#pragma unroll
            for (int i = 0; i < KM; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) ahead[i].set(j, i < K ? load_param(p.w, p.param_type, i * C + c + j, 0.f) : 0.f);
        }
#pragma unroll
        for (int i = 0; i < KM; ++i) dpre[i].clear();
#pragma unroll
        for (int i = 1; i < KM; ++i)
            if (i < K) win[i] = input<T, V>(x, p.x.row, state, C, K, first - i);
        for (int t0 = 0; t0 < stop; t0 += kBwdBatch) {
            Raw<T, V> raw_x[kBwdBatch], raw_dy[kBwdBatch];
            // the oldest batch of the ring, whose copies came before the others'
            const typename S::Word* batch = &ring[S::kOn ? (place == S::kBatches - 1 ? 0 : place + 1) * 2 * kBwdBatch : 0][threadIdx.x];
            if constexpr (S::kOn) {
                copy_wait<S::kBatches - 2>();
            } else {
#pragma unroll
                for (int q = 0; q < kBwdBatch; ++q) raw_x[q] = next_x[q], raw_dy[q] = next_dy[q];
            }
            // (into the place of the batch before, whose values are used up)
            fetch(t0 + (S::kBatches - 1) * kBwdBatch);
            // (nearly every batch lies within the run and needs no test of its rows)
            const auto work = [&](auto whole) {
                constexpr bool kWhole = decltype(whole)::value;
#pragma unroll
                for (int q = 0; q < kBwdBatch; ++q) {
                    const int t = t0 + q, at = t - (K - 1);
                    if (kWhole || t < known) {
                        if constexpr (S::kOn) raw_x[q].w = batch[2 * q * kThreads], raw_dy[q].w = batch[(2 * q + 1) * kThreads];
                        win[0] = raw_x[q].widen();
                        dpre[0] = raw_dy[q].widen();
                        if (p.silu) dpre[0].by_slope(convolve(w, bias, win, K));
                    } else {
                        dpre[0].clear();
                    }
                    if (kWhole || t < n) {
#pragma unroll
                        for (int i = 0; i < KM; ++i)
                            if (i < K) dw[i].fma(dpre[0], win[i]);
                        db.add(dpre[0]);
                    }
                    if (kWhole || (at >= low && t < stop)) {
                        // dx[at] = sum_k w_k dpre[at + K - 1 - k]: the tap i back goes with dpre of i positions on
                        Lanes<V> f;
                        f.clear();
#pragma unroll
                        for (int i = 0; i < KM; ++i) {
                            if (i >= K) continue;
                            if constexpr (KM < 8) f.fma(w[KM - 1 - i], dpre[i]);
                            else f.fma(ahead[i], dpre[i]);
                        }
                        if (!kWhole && at >= kept_from) {
                            Raw<T, V> g;
                            g.load(dfinal + (first + at - (r.length - (K - 1))) * C);
                            f.add(g.widen());
                        }
                        if (kWhole || at >= 0) Raw<T, V>::store(to, f);
                        else if (dstate != nullptr) Raw<T, V>::store(dstate + (at + K - 1) * C, f);
                    }
                    to += C;
                    shift(win);
                    shift(dpre);
                }
            };
            if (t0 >= K - 1 && t0 + kBwdBatch <= n && t0 + kBwdBatch - (K - 1) <= kept_from) work(std::true_type{});
            else work(std::false_type{});
        }
    }
    if (p.partial == nullptr) return;
    float* part = p.partial + slot * (K + 1) * C;
#pragma unroll
    for (int i = 0; i <= KM; ++i) {
        if (i > K) break;
        const Lanes<V>& mine = i < KM && i < K ? dw[i < KM ? i : 0] : db;
#pragma unroll
        for (int j = 0; j < V; ++j) sums[j * kThreads + threadIdx.x] = mine.get(j);
        __syncthreads();
        if (group == 0 && c < C) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float s = 0.f;
                for (int g = 0; g < groups; ++g) s += sums[j * kThreads + g * columns + column];
                part[static_cast<long long>(i < K ? K - 1 - i : K) * C + c + j] = s;
            }
        }
        __syncthreads();
    }
}

// One position a sequence, V channels to a thread; the state's rows move up by one in place.  KM as above.
template <typename T, int KM, int V>
__global__ void __launch_bounds__(kThreads) causal_conv_step_kernel(CausalConv p, T* states, long long state_stride) {
    pdl_trigger();
    pdl_wait();
    const int K = KM >= 8 ? p.K : KM, C = p.C, vectors = C / V;
    const long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
    if (i >= static_cast<long long>(p.seqs.count) * vectors) return;
    const int s = static_cast<int>(i / vectors), c = static_cast<int>(i - static_cast<long long>(s) * vectors) * V;
    T* state = states + s * state_stride + c;
    Raw<T, V> rows[KM];          // rows[j]: the input j positions back
#pragma unroll
    for (int j = 1; j < KM; ++j)
        if (j < K) rows[j].load(state + static_cast<long long>(K - 1 - j) * C);
    rows[0].load(static_cast<const T*>(p.x.p) + s * p.x.seq + c);
    Lanes<V> f;
#pragma unroll
    for (int j = 0; j < V; ++j) f.set(j, load_param(p.bias, p.param_type, c + j, 0.f));
#pragma unroll
    for (int j = KM - 1; j >= 0; --j) {
        if (j >= K) continue;
        Lanes<V> w;
#pragma unroll
        for (int q = 0; q < V; ++q) w.set(q, load_param(p.w, p.param_type, (K - 1 - j) * C + c + q, 0.f));
        f.fma(w, rows[j].widen());
    }
    if (p.silu) f.to_silu();
    Raw<T, V>::store(static_cast<T*>(p.y) + static_cast<long long>(s) * C + c, f);
#pragma unroll
    for (int j = 0; j < KM - 1; ++j)
        if (j < K - 1) rows[j].put(state + static_cast<long long>(K - 2 - j) * C);
}

// Column sums of the rows: a CTA takes 32 columns, each of its kSlots warps every kSlots-th row, 8 loads in flight.  (Few
// rows leave most of 32 warps idle: 8 rows of 73728 columns 24 us with 32 warps.)
template <int kSlots>
__global__ void __launch_bounds__(32 * kSlots) row_sum_kernel(RowSum p) {
    __shared__ float sums[kSlots][33];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long j = static_cast<long long>(blockIdx.x) * 32 + lane, width = p.widths[0] + p.widths[1] + p.widths[2];
    float s = 0.f;
    if (j < width)
        for (long long k = warp; k < p.count; k += 8 * kSlots) {
            float t[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) t[i] = k + kSlots * i < p.count ? p.rows[(k + kSlots * i) * p.stride + j] : 0.f;
            s += ((t[0] + t[1]) + (t[2] + t[3])) + ((t[4] + t[5]) + (t[6] + t[7]));
        }
    sums[warp][lane] = s;
    __syncthreads();
    if (warp != 0) return;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < kSlots; ++i) s += sums[i][lane];
    long long o = j;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        if (o >= 0 && o < p.widths[i] && p.out[i] != nullptr) p.out[i][o] = s;
        o -= p.widths[i];
    }
}

// (nearly always there is nothing to do: the CTAs read two offsets and leave)
__global__ void __launch_bounds__(256) zero_beside_kernel(ZeroBeside p) {
    pdl_trigger();
    pdl_wait();
    const long long first = seq_offset(p.seqs, 0), last = seq_offset(p.seqs, p.seqs.count);
    const long long at = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x, step = static_cast<long long>(gridDim.x) * 256;
    for (int i = 0; i < p.count; ++i) {
        uint16_t* to = static_cast<uint16_t*>(p.p[i]);
        for (long long j = at; j < first * p.halves[i]; j += step) to[j] = 0;
        for (long long j = max(first, last) * p.halves[i] + at; j < p.seqs.length * p.halves[i]; j += step) to[j] = 0;
    }
}

// Vectors of a row that lie side by side in a CTA; the rest of its threads have other runs of positions.
int columns_for(int vectors) {
    int n = 1;
    while (n < vectors && n < 32) n *= 2;
    return n;
}

// Positions to a thread: 64, fewer where that leaves SMs without their eight CTAs.
constexpr int kRun = 64;

template <typename T, int KM, int V>
cudaError_t fwd_t(CausalConv p) {
    const int vectors = (p.C + V - 1) / V, columns = columns_for(vectors), blocks = (vectors + columns - 1) / columns;
    int run = kRun;
    while (run > kFwdBatch && seq_rows(p.seqs) / (kThreads / columns * run) * blocks < 8LL * device_info().sm_count) run /= 2;
    p.span = static_cast<long long>(kThreads / columns) * run;
    const long long grid = seq_slots(p.seqs, p.span) * blocks;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    return launch_pdl(causal_conv_fwd_kernel<T, KM, V>, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, p.stream, p, columns,
                      run, blocks);
}

// Positions to a slot of the backward pass, for V channels a thread: runs of 128, fewer where that leaves SMs without
// the CTAs that they hold together, 4 of several channels a thread, 8 of one (8 x 2048 x 4096 as above: runs of 128 85 us,
// 64 90, 256 94; fp32 packed 5005 x 1001: runs of 32 23 us, 64 25).
long long bwd_span(const Seqs& s, int C, int V) {
    const int vectors = (C + V - 1) / V, columns = columns_for(vectors), groups = kThreads / columns;
    const long long blocks = (vectors + columns - 1) / columns, enough = (V > 1 ? 4LL : 8LL) * device_info().sm_count;
    long long span = static_cast<long long>(groups) * 128;
    while (span > groups * 8 && seq_rows(s) / span * blocks < enough) span /= 2;
    return span;
}

template <typename T, int KM, int V>
cudaError_t bwd_t(CausalConv p) {
    p.span = bwd_span(p.seqs, p.C, V);
    const int vectors = (p.C + V - 1) / V, columns = columns_for(vectors), blocks = (vectors + columns - 1) / columns;
    const int groups = kThreads / columns;
    const long long slots = seq_slots(p.seqs, p.span), grid = slots * blocks;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const cudaError_t err = launch_pdl(causal_conv_bwd_kernel<T, KM, V>, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0,
                                       p.stream, p, columns, static_cast<int>((p.span + groups - 1) / groups), blocks);
    if (err != cudaSuccess || p.partial == nullptr) return err;
    const long long taps = static_cast<long long>(p.K) * p.C;
    return launch_row_sum(p.partial, slots, taps + p.C, {p.dw, p.dbias}, {taps, p.C}, p.stream);
}

// Several channels a thread where every tensor allows it, else one.
// (bf16 8 x 2048 x 2048, two channels a thread and one: 12 taps forward 66 and 88 us, backward 174 and 243, 8 taps backward
// 97 and 138; four: 12 taps forward 87, 8 taps backward 116.)
bool vectors_of(const CausalConv& p, bool backward) {
    const size_t a = 8 * static_cast<size_t>(elem_bytes(p.type));
    const auto off = [&](const void* t) { return reinterpret_cast<uintptr_t>(t) % a != 0; };
    return p.C % 8 == 0 && p.x.vec && !off(p.state) &&
           (backward ? p.dy.vec && !off(p.dx) && !off(p.dstate) && !off(p.dfinal) : !off(p.y) && !off(p.final_state));
}

template <typename T>
cudaError_t fwd_k(const CausalConv& p) {
    const bool vec = vectors_of(p, false);
    switch (p.K) {
        case 1: return vec ? fwd_t<T, 1, 4>(p) : fwd_t<T, 1, 1>(p);
        case 2: return vec ? fwd_t<T, 2, 4>(p) : fwd_t<T, 2, 1>(p);
        case 3: return vec ? fwd_t<T, 3, 4>(p) : fwd_t<T, 3, 1>(p);
        case 4: return vec ? fwd_t<T, 4, 4>(p) : fwd_t<T, 4, 1>(p);
    }
    if (p.K > 8) return vec ? fwd_t<T, 16, 2>(p) : fwd_t<T, 16, 1>(p);
    return vec ? fwd_t<T, 8, 4>(p) : fwd_t<T, 8, 1>(p);
}

template <typename T>
cudaError_t bwd_k(const CausalConv& p) {
    const bool vec = vectors_of(p, true);
    switch (p.K) {
        case 1: return vec ? bwd_t<T, 1, 4>(p) : bwd_t<T, 1, 1>(p);
        case 2: return vec ? bwd_t<T, 2, 4>(p) : bwd_t<T, 2, 1>(p);
        case 3: return vec ? bwd_t<T, 3, 4>(p) : bwd_t<T, 3, 1>(p);
        case 4: return vec ? bwd_t<T, 4, 4>(p) : bwd_t<T, 4, 1>(p);
    }
    if (p.K > 8) return vec ? bwd_t<T, 16, 2>(p) : bwd_t<T, 16, 1>(p);
    return vec ? bwd_t<T, 8, 2>(p) : bwd_t<T, 8, 1>(p);
}

template <typename T, int KM, int V>
cudaError_t step_t(const CausalConv& p, void* state, long long state_stride) {
    const long long grid = (static_cast<long long>(p.seqs.count) * (p.C / V) + kThreads - 1) / kThreads;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    return launch_pdl(causal_conv_step_kernel<T, KM, V>, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, p.stream, p,
                      static_cast<T*>(state), state_stride);
}

template <typename T>
cudaError_t step_k(const CausalConv& p, void* state, long long state_stride) {
    const auto off = [](const void* t) { return reinterpret_cast<uintptr_t>(t) % (2 * sizeof(T)) != 0; };
    const bool one = p.seqs.count <= 1;
    const bool vec = p.C % 2 == 0 && !off(p.x.p) && !off(state) && !off(p.y) && (one || (p.x.seq % 2 == 0 && state_stride % 2 == 0));
    // Numbers of taps as in the other passes: rows that a kernel has registers for and the call does not have cost as if they were
    // there (bf16, 64 sequences of 4096 channels, in a graph, this kernel and that of 16 taps: 1 tap 1.4 and 3.7 us, 2 taps 2.0
    // and 3.8, 4 taps 2.2 and 4.0, 8 taps 4.0 and 4.4; 256 of 8192: 2 taps 8.6 and 19.1, 8 taps 12.5 and 20.5).
    switch (p.K) {
        case 1: return vec ? step_t<T, 1, 2>(p, state, state_stride) : step_t<T, 1, 1>(p, state, state_stride);
        case 2: return vec ? step_t<T, 2, 2>(p, state, state_stride) : step_t<T, 2, 1>(p, state, state_stride);
        case 3: return vec ? step_t<T, 3, 2>(p, state, state_stride) : step_t<T, 3, 1>(p, state, state_stride);
        case 4: return vec ? step_t<T, 4, 2>(p, state, state_stride) : step_t<T, 4, 1>(p, state, state_stride);
    }
    if (p.K > 8) return vec ? step_t<T, 16, 2>(p, state, state_stride) : step_t<T, 16, 1>(p, state, state_stride);
    return vec ? step_t<T, 8, 2>(p, state, state_stride) : step_t<T, 8, 1>(p, state, state_stride);
}

}  // namespace

// (Whatever the alignment: of the kernels' vectors the one with the most slots.)
long long causal_conv_bwd_slots(const Seqs& s, int C) {
    long long most = 0;
    for (int V : {1, 2, 4}) most = std::max(most, seq_slots(s, bwd_span(s, C, V)));
    return most;
}

cudaError_t launch_causal_conv_fwd(const CausalConv& p) {
    switch (p.type) {
        case kF32: return fwd_k<float>(p);
        case kBF16: return fwd_k<__nv_bfloat16>(p);
        default: return fwd_k<__half>(p);
    }
}

cudaError_t launch_causal_conv_bwd(const CausalConv& p) {
    switch (p.type) {
        case kF32: return bwd_k<float>(p);
        case kBF16: return bwd_k<__nv_bfloat16>(p);
        default: return bwd_k<__half>(p);
    }
}

cudaError_t launch_causal_conv_step(const CausalConv& p, void* state, long long state_stride) {
    switch (p.type) {
        case kF32: return step_k<float>(p, state, state_stride);
        case kBF16: return step_k<__nv_bfloat16>(p, state, state_stride);
        default: return step_k<__half>(p, state, state_stride);
    }
}

cudaError_t launch_zero_beside(const ZeroBeside& p) {
    return launch_pdl(zero_beside_kernel, dim3(static_cast<unsigned>(device_info().sm_count)), dim3(256), 0, p.stream, p);
}

cudaError_t launch_row_sum(const float* rows, long long count, long long stride, std::initializer_list<float*> out,
                           std::initializer_list<long long> widths, cudaStream_t stream) {
    RowSum p{rows, count, stride, {}, {}};
    std::copy(out.begin(), out.end(), p.out);
    std::copy(widths.begin(), widths.end(), p.widths);
    const long long grid = (p.widths[0] + p.widths[1] + p.widths[2] + 31) / 32;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const dim3 ctas(static_cast<unsigned>(grid));
    if (count <= 16) return launch_pdl(row_sum_kernel<2>, ctas, dim3(64), 0, stream, p);
    if (count <= 128) return launch_pdl(row_sum_kernel<8>, ctas, dim3(256), 0, stream, p);
    return launch_pdl(row_sum_kernel<32>, ctas, dim3(1024), 0, stream, p);
}

}  // namespace dwc

// dwc_seq_device.cuh -- device-side parts shared by the kernels along sequences.
#pragma once

#include "dwc_norm_device.cuh"
#include "dwc_seq_host.h"

namespace dwc {

// A piece of a sequence: positions first .. end - 1 of sequence `s`, whose position t lies at row
// base + t (packed) or in batch entry s (base 0).
struct Piece {
    int s;
    long long base, length;     // of the sequence
    long long first, end;
    long long index;            // of the piece in its sequence
    bool last;                  // the sequence's last piece (an empty sequence has one, empty)
    bool some;                  // false: the slot has no piece
};

__device__ __forceinline__ long long seq_offset(const Seqs& q, int s) {
    const long long o = q.offsets[s];
    return o < 0 ? 0 : o > q.length ? q.length : o;
}

__device__ __forceinline__ Piece find_piece(const Seqs& q, long long slot, long long span) {
    Piece r;
    if (q.offsets == nullptr) {
        const long long n = q.length == 0 ? 1 : (q.length + span - 1) / span;
        r.s = static_cast<int>(slot / n);
        r.index = slot - r.s * n;
        r.base = 0;
        r.length = q.length;
        r.some = true;
    } else {
        // the last sequence whose first slot is not behind this one
        int lo = 0, hi = q.count - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (seq_offset(q, mid) / span + mid <= slot) lo = mid;
            else hi = mid - 1;
        }
        r.s = lo;
        r.base = seq_offset(q, lo);
        const long long end = seq_offset(q, lo + 1);
        r.length = end > r.base ? end - r.base : 0;
        r.index = slot - (r.base / span + lo);
        r.some = r.index >= 0 && (r.index == 0 || r.index * span < r.length);
    }
    r.first = r.index * span;
    r.end = r.first + span < r.length ? r.first + span : r.length;
    r.last = r.first + span >= r.length;
    return r;
}

// Row of an input view at position 0 of the piece's sequence, and of a dense tensor of `width` values.
template <typename T>
__device__ __forceinline__ const T* view_at(const RowsView& v, const Seqs& q, const Piece& r) {
    return static_cast<const T*>(v.p) + (q.offsets != nullptr ? r.base * v.row : r.s * v.seq);
}
__device__ __forceinline__ long long seq_rows_device(const Seqs& q) {
    return q.offsets != nullptr ? q.length : q.count * q.length;
}
__device__ __forceinline__ long long dense_row(const Seqs& q, const Piece& r) {
    return q.offsets != nullptr ? r.base : r.s * q.length;
}

// 8 values, of which `left` exist (the others: zeros, not stored).  vec: one access for all 8.
template <typename T>
__device__ __forceinline__ void load8(Vec8<T>& v, const T* p, int left, bool vec) {
    if (vec) {
        v.load(p);
    } else {
        v.zero();
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < left) v.set(j, p[j]);
    }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float2 (&f)[4], int left, bool vec) {
    if (vec) {
        Vec8<T>::store(p, f);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (2 * j < left) store_out(p + 2 * j, f[j].x);
            if (2 * j + 1 < left) store_out(p + 2 * j + 1, f[j].y);
        }
    }
}
// Brings a line that a later load reads from DRAM to L2.
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

}  // namespace dwc

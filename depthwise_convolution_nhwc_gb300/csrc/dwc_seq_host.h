// dwc_seq_host.h -- host-side interface between the C ABI of the sequence operators and their kernel
// launchers.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

#include "dwc_host.h"

namespace dwc {

// A view of positions x values; `vec`: 8 values at a time can be read from any multiple of 8.
struct RowsView {
    const void* p;
    long long seq, row;
    bool vec;
};

// Sequences of a batch (offsets null) or packed.
struct Seqs {
    const int* offsets;
    int count;
    long long length;       // of each sequence; packed: rows in all
};

// Sequences cut into pieces of `span` positions, one slot each (at least one per sequence, an empty
// one too).  Packed: piece k of sequence s has slot offsets[s] / span + s + k; a sequence of n rows
// has at most (offsets[s] + n) / span - offsets[s] / span + 1 pieces, so slots never meet, and some
// stay empty.
inline long long seq_slots(const Seqs& s, long long span) {
    if (s.count == 0) return 0;
    if (s.offsets != nullptr) return s.length / span + s.count;
    const long long n = (s.length + span - 1) / span;
    return s.count * (n < 1 ? 1 : n);
}
inline long long seq_rows(const Seqs& s) { return s.offsets != nullptr ? s.length : s.count * s.length; }

struct CausalConv {
    Seqs seqs;
    int C, K;
    bool silu;
    int type, param_type;
    RowsView x;
    const void* w;
    const void* bias;       // may be null
    const void* state;      // may be null
    // forward
    void* y;
    void* final_state;      // may be null
    // backward
    RowsView dy;
    const void* dfinal;     // may be null
    void* dx;
    void* dstate;           // may be null
    float* dw;              // may be null
    float* dbias;           // may be null
    float* partial;         // slots x (K + 1) x C (with a parameter gradient only)
    long long span;         // positions to a slot
    cudaStream_t stream;
};

// Slots that the backward pass may take.
long long causal_conv_bwd_slots(const Seqs& s, int C);
cudaError_t launch_causal_conv_fwd(const CausalConv& p);
cudaError_t launch_causal_conv_bwd(const CausalConv& p);
cudaError_t launch_causal_conv_step(const CausalConv& p, void* state, long long state_stride);

// Positions between the states that the forward pass keeps for the backward pass.
constexpr int kScanTile = 16;
constexpr int kScanMaxStates = 128;

struct Scan {
    Seqs seqs;
    int C, N, G;
    bool softplus;
    int type;
    RowsView u, dt, z, b, c;
    const float* A;
    const float* D;
    const float* dt_bias;
    // forward
    const float* state;     // may be null
    void* y;
    float* final_state;     // may be null
    float* saved;           // may be null in the forward pass
    // backward
    RowsView dy;
    const float* dfinal;    // may be null
    void* du;
    void* ddt;
    void* dz;
    void* db;
    void* dc;
    float* dA;
    float* dD;
    float* ddt_bias;
    float* dstate;          // may be null
    float* workspace;
    long long span;         // positions to a chunk
    cudaStream_t stream;
};

// Positions to a chunk (a multiple of 16; a sequence's length or more: no chunks) and, with them, the workspaces.
long long scan_fwd_span(const Scan& p);
long long scan_bwd_span(const Scan& p);
size_t scan_fwd_workspace_floats(const Scan& p);
size_t scan_bwd_workspace_floats(const Scan& p);
#define DWC_SCAN_TYPE(name)                            \
    cudaError_t launch_scan_fwd_##name(const Scan& p); \
    cudaError_t launch_scan_bwd_##name(const Scan& p);
DWC_SCAN_TYPE(f32)
DWC_SCAN_TYPE(bf16)
DWC_SCAN_TYPE(f16)
#undef DWC_SCAN_TYPE
cudaError_t launch_scan_step(const Scan& p, float* state, long long state_stride);

struct ZeroBeside {
    Seqs seqs;
    void* p[8];
    long long halves[8];    // 16-bit words to a row
    int count;
    cudaStream_t stream;
};
cudaError_t launch_zero_beside(const ZeroBeside& p);

// Sums of `count` rows that lie `stride` floats apart, in a fixed order: of the first widths[0] columns to out[0]
// (may be null), of the next widths[1] to out[1] and so on.
struct RowSum {
    const float* rows;
    long long count, stride;
    float* out[3];
    long long widths[3];
};
cudaError_t launch_row_sum(const float* rows, long long count, long long stride, std::initializer_list<float*> out,
                           std::initializer_list<long long> widths, cudaStream_t stream);

}  // namespace dwc

// dwc_norm_host.h -- host-side interface between the C ABI of the norm and dropout operators
// and their kernel launchers.
//
// All three operators are written over a stream tensor (layer norm's x, the residual sum z) and
// a branch tensor (layer norm's y, the residual form's x and y); the pairs of types are equal,
// or an fp32 stream with a 16-bit branch.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <mutex>

#include "dwc_host.h"

namespace dwc {

// Counter-based dropout: 16-bit draws below `threshold` are dropped (0: no dropout, 65536: all).
struct Dropout {
    uint32_t threshold = 0;
    float scale = 1.f;              // 65536 / (65536 - threshold)
    uint32_t k0 = 0, k1 = 0;        // the seed's words
    uint64_t offset = 0;
    const unsigned long long* step = nullptr;
};

// z = stream (+ dropout(branch)), y = layer_norm(z).
struct NormFwd {
    const void* in;                 // rows x C of the stream type, row stride ld_in
    const void* x;                  // the branch (row stride ld_x), or null: plain layer norm
    void* z;                        // sum, stream type (with a branch only)
    void* y;                        // branch type
    float* mean;                    // may be null
    float* rstd;                    // may be null
    const void* gamma;              // may be null
    const void* beta;               // may be null
    int param_type;
    float eps;
    long long rows, ld_in, ld_x;
    int C;
    int stream_type, branch_type;
    Dropout drop;
    cudaStream_t stream;
    bool in_place = false;            // an output is one of the inputs
    bool stall = false;               // test of the wait limit: each cluster's last CTA sends its sums to nobody
    unsigned int* status = nullptr;   // of the kernels whose waits have a limit
    unsigned long long wait_ns = 0;   // that limit (0: the default)
};

// g = dz + layer_norm_bwd(dy; z): d_stream = g, d_branch = dropout map of g.
struct NormBwd {
    const void* dy;                 // branch type, row stride ld_dy
    const void* dz;                 // stream type, row stride ld_dz, or null
    const void* z;                  // stream type, row stride ld_z
    const float* mean;
    const float* rstd;
    const void* gamma;              // may be null
    int param_type;
    void* d_stream;                 // stream type
    void* d_branch;                 // branch type, or null
    float* dgamma;                  // may be null
    float* dbeta;                   // may be null
    float* partial;                 // workspace (with a parameter gradient only)
    long long rows, ld_dy, ld_dz, ld_z;
    int C;
    int stream_type, branch_type;
    Dropout drop;
    cudaStream_t stream;
    bool in_place = false;            // an output is one of the inputs
    bool stall = false;               // test of the wait limit: each cluster's last CTA sends its sums to nobody
    unsigned int* status = nullptr;
    unsigned long long wait_ns = 0;
};

struct DropoutCall {
    const void* x;
    void* y;
    long long rows, ld_x;
    int C;
    int type;
    Dropout drop;
    cudaStream_t stream;
};

// First element, counted from a row's start, that a 16-byte copy of the granule of `n` elements at column `col` names
// in global memory.  A granule past the row's `end` is a copy of no bytes (zeros), but the copy's address has to
// be aligned all the same, and the start of a shifted row is not: it names the boundary at or before that start
// (col is minus the row's shift modulo n, and the tensor's base lies on a boundary).
constexpr int copy_column(int col, int end, int n) { return col < end ? col : -(-col & (n - 1)); }

// How many clusters of a kernel a device holds together, by device and launch shape, each asked for once
// (a runtime call of its own).  `ask()` gives the number; none (below 1) is not kept.  No allocation: a kernel
// has at most 96 shapes (threads in steps of 32 up to 512, clusters of 2, 4 and 8, with and without
// dz), and what finds no place any more, with many devices, is asked for at every call.
class ClusterCounts {
public:
    template <class Ask>
    int get(int device, size_t smem, int threads, int cluster, Ask ask) {
        std::lock_guard<std::mutex> lock(mu_);
        for (int i = 0; i < count_; ++i) {
            const Place& k = known_[i];
            if (k.device == device && k.smem == smem && k.threads == threads && k.cluster == cluster) return k.n;
        }
        const int n = ask();
        if (n >= 1 && count_ < kPlaces) known_[count_++] = {smem, device, threads, cluster, n};
        return n;
    }

private:
    static constexpr int kPlaces = 192;
    struct Place {
        size_t smem;
        int device, threads, cluster, n;
    };
    std::mutex mu_;
    Place known_[kPlaces];
    int count_ = 0;
};

// General kernels: any row stride, alignment and channel count.
cudaError_t launch_norm_fwd_general(const NormFwd& p);
cudaError_t launch_norm_bwd_general(const NormBwd& p);
cudaError_t launch_dropout_general(const DropoutCall& p);

// Dropout from bases aligned to 8 elements: dense rows, or rows of a multiple of 8 channels whose stride is
// one too; cudaErrorNotSupported for others.
cudaError_t launch_dropout_vec(const DropoutCall& p);

// Rows in registers (aligned tensors, up to 65536 channels), one file per
// pair of types; cudaErrorNotSupported beyond that.
#define DWC_NORM_PAIR(name)                           \
    cudaError_t launch_norm_fwd_##name(const NormFwd& p); \
    cudaError_t launch_norm_bwd_##name(const NormBwd& p);
DWC_NORM_PAIR(f32)
DWC_NORM_PAIR(bf16)
DWC_NORM_PAIR(f16)
DWC_NORM_PAIR(f32_bf16)
DWC_NORM_PAIR(f32_f16)
#undef DWC_NORM_PAIR

// Rows of partial parameter gradients (2 x C floats each) that a backward pass may write.
int norm_bwd_partials(long long rows, int C);
// dgamma / dbeta = the sum of `count` partial rows [dgamma | dbeta], in a fixed order.
cudaError_t launch_norm_param_sum(const float* partial, int count, int C, float* dgamma,
                                  float* dbeta, cudaStream_t stream);

}  // namespace dwc

/*
 * dwc_seq.h -- operators along the positions of sequences, per channel (libdwc_gb300.so): the short
 * causal depthwise convolution and the selective scan of state space layers, forward, backward and
 * for single tokens.  The conventions of dwc.h hold: device pointers owned by the caller,
 * asynchronous calls on `stream`, host-side validation, status codes, no call aborts or throws,
 * programmatic dependent launches.
 *
 * Sequences lie as a batch (offsets NULL): `count` sequences of `length` positions each; or packed
 * one behind the other: `length` rows in all, sequence s the rows offsets[s] .. offsets[s+1]-1
 * (count + 1 ascending 32-bit values on the device, within 0 .. length; a sequence may be empty, but
 * with a count of 0 length is 0 too: packed rows of no sequence are DWC_ERR_INVALID_ARG).  Rows in
 * front of the first and behind the last sequence are neither read nor written (outputs keep there
 * what they held).  The offsets are read on the device; values outside 0 .. length are clamped, and
 * descending ones give undefined results but no access outside the tensors.
 *
 * Views: position t of sequence s of an input lies at data + s * seq_stride + t * row_stride (a
 * batch) or data + (offsets[s] + t) * row_stride (packed), strides in elements, 0 or more (0
 * repeats a row); its values are adjacent.  Outputs are dense.  Outputs must not overlap inputs or
 * one another, except where a call says that it works in place.
 *
 * Arithmetic is fp32: 16-bit inputs are widened exactly; sums, states and gradients of parameters
 * are fp32; 16-bit outputs are rounded to nearest even once, at the store.  Exponentials (decays, SiLU,
 * softplus) and quotients are the hardware's approximations, off by up to 2 ulp, with results below
 * 2^-126 zero.  The order of every sum is fixed by the sizes, the types and the number of SMs, so
 * results are bit-identical from run to run (no atomics).  No call allocates device memory.
 */
#ifndef DWC_SEQ_GB300_H
#define DWC_SEQ_GB300_H

#include "dwc.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    const void* data;
    long long seq_stride; /* a batch's sequences; not used for packed ones */
    long long row_stride;
} dwc_rows_t;

typedef struct {
    int count;
    long long length;
    const int* offsets;
} dwc_seqs_t;

/* Zeros in the packed rows that lie in front of the first and behind the last sequence, of up to 8
 * dense tensors of `length` rows of row_bytes[i] bytes (aligned to 2): what an output that is new
 * memory wants there.  Nothing for a batch. */
dwc_status_t dwc_zero_beside_sequences(const dwc_seqs_t* seqs, void* const* tensors, const long long* row_bytes,
                                       int count, dwc_stream_t stream);

/* ---- short causal depthwise convolution ---------------------------------------------------
 *     pre[t, c] = bias[c] + sum_{k < K} w[k, c] * x[t - K + 1 + k, c],   y = act(pre)
 * (a cross-correlation, the last tap on the position itself).  Positions before a sequence's first
 * come from its state: state[s, j] is position j - (K - 1); zeros without one. */
typedef struct {
    dwc_seqs_t seqs;
    int C, K;                /* K from 1 to 16 */
    dwc_gate_t act;          /* DWC_GATE_NONE or DWC_GATE_SILU */
    dwc_dtype_t dtype;       /* of x, y, the states and dx */
    dwc_dtype_t param_dtype; /* of w and bias */
    dwc_rows_t x;
    const void* w;           /* K x C */
    const void* bias;        /* C values, or NULL (0) */
    const void* state;       /* count x (K - 1) x C, dense, or NULL (0) */
} dwc_causal_conv_t;

/* y: dense like x.  final_state: count x (K - 1) x C, the last K - 1 inputs of each sequence (with
 * its state in front), the state of a later call; or NULL.
 * DWC_ERR_INVALID_ARG: null x, w or y with positions to work on, negative sizes or strides, C < 1,
 * K < 1, unknown types or activation.  DWC_ERR_UNSUPPORTED: K above 16, C above 2^20, more than
 * 2^31 - 64 positions, more than 2^40 elements.  DWC_ERR_ALIGNMENT: a pointer not aligned to its
 * element.  No sequences or no positions: DWC_OK (the final states are written). */
dwc_status_t dwc_causal_conv_fwd(const dwc_causal_conv_t* conv, void* y, void* final_state, dwc_stream_t stream);

/* Bytes of workspace dwc_causal_conv_bwd needs on the CURRENT device when dw or dbias is wanted
 * (0 for invalid sizes). */
size_t dwc_causal_conv_bwd_workspace_size(const dwc_causal_conv_t* conv);

/* With dpre = dy * act'(pre):
 *     dx[t] = sum_k w[k] * dpre[t + K - 1 - k],  dw[k] = sum_t dpre[t] * x[t - K + 1 + k],
 *     dbias = sum_t dpre
 *   dy: a view like x     dfinal: the gradient of final_state (dense, dtype), or NULL
 *   dx: dense     dstate: count x (K - 1) x C (out, dtype), or NULL
 *   dw: K x C, dbias: C fp32 values (out), or NULL each
 *   workspace: 16-byte aligned, contents ignored and clobbered (not needed without dw and dbias)
 * Errors as the forward pass, and DWC_ERR_WORKSPACE. */
dwc_status_t dwc_causal_conv_bwd(const dwc_causal_conv_t* conv, const dwc_rows_t* dy, const void* dfinal, void* dx,
                                 void* dstate, float* dw, float* dbias, void* workspace, size_t workspace_bytes,
                                 dwc_stream_t stream);

/* One position for each of `count` sequences (length 1, no offsets): y as in the forward pass, and
 * `state` moves on by one row in place; its sequences lie state_stride elements apart (at least
 * (K - 1) * C), conv->state is not used. */
dwc_status_t dwc_causal_conv_step(const dwc_causal_conv_t* conv, void* state, long long state_stride, void* y,
                                  dwc_stream_t stream);

/* ---- selective scan -------------------------------------------------------------------------
 * Per channel c, with N states and the group g = c / (C / G) of B and C:
 *     delta[t] = dt[t] + dt_bias, or log(1 + exp(dt[t] + dt_bias)) with softplus
 *     h[t, n]  = exp(delta[t] * A[n]) * h[t-1, n] + delta[t] * u[t] * B[t, g, n]
 *     y[t]     = (sum_n C[t, g, n] * h[t, n] + D * u[t]) * silu(z[t])
 * h before a sequence's first position is its state (zero without one).  A counts as at most 2.35e38
 * either way: a state of A = minus infinity keeps nothing wherever delta is above 1e-36, and delta = 0
 * leaves it alone, as it does every state; the gradient that reaches delta through such a state is 0. */
typedef struct {
    dwc_seqs_t seqs;
    int C, N, G;             /* N from 1 to 128; G divides C */
    int softplus;
    dwc_dtype_t dtype;       /* of u, dt, z, B, C, y and their gradients */
    dwc_rows_t u, dt;        /* C values a position */
    dwc_rows_t z;            /* the same; data NULL: no gate */
    dwc_rows_t b, c;         /* G x N values a position */
    const float* A;          /* C x N */
    const float* D;          /* C values, or NULL (0) */
    const float* dt_bias;    /* C values, or NULL (0) */
} dwc_scan_t;

/* Floats of `saved`: the states in front of every 16th position of each sequence, what the
 * backward pass starts from (0 for invalid sizes). */
size_t dwc_selective_scan_saved_floats(const dwc_scan_t* scan);
/* Bytes of workspace of the two passes on the CURRENT device (0: none, or invalid sizes).  Forward:
 * none, or 4 C (N + 1) a chunk where sequences are few.  Backward:
 *     8 N a position and block of channels (of one group: up to 64 of them with up to 8 states, 32 with
 *     up to 16, 16 with up to 32, else 8) for partial rows of dB and dC, but not more than 8 GB or
 *     what `saved` takes, the larger: past it the positions are worked on in parts of 64 and more;
 *     and 4 C (N + 2) a sequence, 4 C (2 N + 3) a chunk where sequences are few or worked on in parts. */
size_t dwc_selective_scan_fwd_workspace_size(const dwc_scan_t* scan);
size_t dwc_selective_scan_bwd_workspace_size(const dwc_scan_t* scan);

/*   state: count x C x N, or NULL     y: dense like u
 *   final_state: count x C x N (out), or NULL (state and final_state may be the same)
 *   saved: dwc_selective_scan_saved_floats values (out), or NULL: no backward pass follows
 *   workspace: 16-byte aligned, contents ignored and clobbered
 * Errors as dwc_causal_conv_fwd (the views, A and y in place of x, w and y), DWC_ERR_INVALID_ARG
 * also for G that does not divide C, DWC_ERR_UNSUPPORTED for N above 128, DWC_ERR_WORKSPACE. */
dwc_status_t dwc_selective_scan_fwd(const dwc_scan_t* scan, const float* state, void* y, float* final_state,
                                    float* saved, void* workspace, size_t workspace_bytes, dwc_stream_t stream);

/* Gradients from dy (a view like u), the forward pass's inputs and its `saved`; dfinal: the
 * gradient of final_state (count x C x N), or NULL.
 *   du, ddt, dz: dense like u (dz only, and always, with z)
 *   db, dc: dense, G x N values a position
 *   dA: C x N, dD: C, ddt_bias: C fp32 values (out)
 *   dstate: count x C x N (out), or NULL */
dwc_status_t dwc_selective_scan_bwd(const dwc_scan_t* scan, const dwc_rows_t* dy, const float* saved,
                                    const float* dfinal, void* du, void* ddt, void* dz, void* db, void* dc, float* dA,
                                    float* dD, float* ddt_bias, float* dstate, void* workspace,
                                    size_t workspace_bytes, dwc_stream_t stream);

/* One position for each of `count` sequences (length 1, no offsets), `state` updated in place; its
 * sequences lie state_stride floats apart (at least C * N). */
dwc_status_t dwc_selective_scan_step(const dwc_scan_t* scan, float* state, long long state_stride, void* y,
                                     dwc_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DWC_SEQ_GB300_H */

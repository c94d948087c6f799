/*
 * dwc_norm.h -- layer norm, dropout, their residual form and the block norm over channels-last rows
 * (libdwc_gb300.so; the conventions of dwc.h hold: device pointers owned by the caller,
 * asynchronous calls on `stream`, host-side validation, status codes, no call aborts or throws,
 * programmatic dependent launches).
 *
 * Rows: a tensor of `rows` x C values, C the channels of one position (the last axis of an
 * N x H x W x C tensor, rows = N*H*W, or of tokens x C).  Inputs have a row stride `ld*` in
 * elements (at least C; channels are adjacent); outputs are dense (row stride C).
 *
 * Arithmetic is fp32: 16-bit inputs are widened exactly, sums, means, variances and their
 * merges are fp32, 16-bit outputs are rounded to nearest even once, at the store.  The order of
 * every sum is fixed by the shape, the types, the alignment, whether the call works in place and
 * the number of SMs (beyond 10240 channels: of clusters that the GPU holds), so results are
 * bit-identical from run to run (no atomics).
 *
 * In place: an output of rows x C values may be one of the call's inputs of rows x C values, from the same
 * address, of the same type and with dense rows (z over res, y over x, dx over dy or x, ...); the same
 * address with another type or row stride is DWC_ERR_INVALID_ARG.  Outputs must not overlap inputs or one
 * another in any other way.
 *
 * No call allocates device memory; the backward passes take a caller workspace for the partial
 * sums of the parameter gradients.
 *
 * Kernels: rows of up to 65536 channels whose tensors are aligned to 8 elements and whose row strides
 * are congruent to C modulo 8 (dense tensors from aligned bases are, for any C) run on kernels that
 * read every input once; other views and wider rows run on general kernels (same results within
 * the rounding of another order of sums, slower).  Rows beyond 10240 channels use clusters of CTAs
 * whose waits have the limit of dwc_set_wait_limit_ns and report to dwc_device_status.
 *
 * Dropout: p in [0, 1] is held as q = floor(p * 65536 + 0.5) / 65536 and kept values are scaled
 * by 1 / (1 - q), so the expected value is exact.  Element i of the tensor (i = row * C + channel,
 * whatever the row stride) is kept where h(i) >= q * 65536; h(i) is the 16-bit value i % 8 (of
 * each 32-bit word the low half first) of the Philox4x32-10 block (Salmon, Moraes, Dror and Shaw,
 * "Parallel random numbers: as easy as 1, 2, 3", 2011) with the key `seed` (low word first) and
 * the 128-bit counter (i / 8 as 64 bits, offset + *step as 64 bits, low words first).  The mask is
 * never stored: the backward pass draws it again from the same (seed, offset, *step).  `step` may
 * be NULL (0); it is read on the device, so a captured graph draws new masks when the caller
 * advances it.  A dropped value gives +0 whatever it was (infinities and NaN included); q = 0 is
 * the identity, q = 1 gives zeros.
 */
#ifndef DWC_NORM_GB300_H
#define DWC_NORM_GB300_H

#include "dwc.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Layer norm over the channels of each row:
 *     mean = sum_c x / C,  rstd = 1 / sqrt(sum_c (x - mean)^2 / C + eps),
 *     y = (x - mean) * rstd * gamma + beta
 *   x : rows x C, dtype, row stride ldx       y : rows x C, out_dtype (out)
 *   gamma, beta : C values of param_dtype each, or NULL (1 and 0)
 *   mean, rstd : rows fp32 values each (out), or NULL
 *   out_dtype : dtype, or a 16-bit type for fp32 x (the next product's operand)
 *   eps >= 0; a row of equal values gives y = beta (with eps = 0: NaN, 0 * infinity).
 * DWC_ERR_INVALID_ARG: null x or y with rows > 0, rows < 0, C < 1, ldx < C, unknown or
 * unsupported types, negative or non-finite eps.  DWC_ERR_UNSUPPORTED: C above 2^24, rows * C or
 * rows * ld above 2^40.  DWC_ERR_ALIGNMENT: a pointer not aligned to its element.  rows = 0 is
 * DWC_OK without a launch. */
dwc_status_t dwc_layer_norm_fwd(const void* x, long long ldx, const void* gamma, const void* beta,
                                dwc_dtype_t param_dtype, float eps, void* y, float* mean,
                                float* rstd, long long rows, int C, dwc_dtype_t dtype,
                                dwc_dtype_t out_dtype, dwc_stream_t stream);

/* Bytes of workspace the backward passes need for rows x C on the CURRENT device (0 for invalid
 * sizes; the pass then reports the error). */
size_t dwc_layer_norm_bwd_workspace_size(long long rows, int C);

/* Backward of dwc_layer_norm_fwd; with xhat = (x - mean) * rstd and a = dy * gamma:
 *     dx = rstd * (a - mean_c(a) - xhat * mean_c(a * xhat))
 *     dgamma = sum over rows of dy * xhat,   dbeta = sum over rows of dy
 *   dy : rows x C, dy_dtype (the forward's out_dtype), row stride lddy
 *   x, mean, rstd, gamma : as in the forward pass     dx : rows x C, dtype (out)
 *   dgamma, dbeta : C fp32 values each (out), or NULL; rows = 0 writes zeros
 *   workspace : at least dwc_layer_norm_bwd_workspace_size(rows, C) bytes, 16-byte aligned,
 *               contents ignored and clobbered (not needed when dgamma and dbeta are NULL).
 * Errors as the forward pass; also DWC_ERR_INVALID_ARG for a null mean or rstd with rows > 0 and
 * DWC_ERR_WORKSPACE. */
dwc_status_t dwc_layer_norm_bwd(const void* dy, long long lddy, const void* x, long long ldx,
                                const float* mean, const float* rstd, const void* gamma,
                                dwc_dtype_t param_dtype, void* dx, float* dgamma, float* dbeta,
                                long long rows, int C, dwc_dtype_t dtype, dwc_dtype_t dy_dtype,
                                void* workspace, size_t workspace_bytes, dwc_stream_t stream);

/* Dropout of rows x C values (see above), and its backward pass dx = the same map of dy.
 *   x, dy : rows x C, dtype, row stride ldx / lddy      y, dx : rows x C, dtype (out)
 * DWC_ERR_INVALID_ARG also for p outside [0, 1] or NaN; DWC_ERR_ALIGNMENT for a step pointer not
 * 8-byte aligned. */
dwc_status_t dwc_dropout_fwd(const void* x, long long ldx, void* y, long long rows, int C, double p,
                             unsigned long long seed, unsigned long long offset,
                             const unsigned long long* step, dwc_dtype_t dtype, dwc_stream_t stream);
dwc_status_t dwc_dropout_bwd(const void* dy, long long lddy, void* dx, long long rows, int C,
                             double p, unsigned long long seed, unsigned long long offset,
                             const unsigned long long* step, dwc_dtype_t dtype, dwc_stream_t stream);

/* The end of a residual branch and the norm in front of the next one, in one pass:
 *     z = res + dropout(x),   y = layer_norm(z)
 * (statistics and y from the fp32 sum, z rounded once where it is stored).
 *   x : rows x C, dtype, row stride ldx (the branch)   y : rows x C, dtype (out)
 *   res : rows x C, res_dtype, row stride ldres (the residual stream)
 *   z : rows x C, res_dtype (out); may be res itself (see "In place" above)
 *   res_dtype : dtype, or DWC_F32 (an fp32 stream with 16-bit branches)
 *   p = 0 : no dropout (serving); seed, offset and step are then not used
 * The rest and the errors as dwc_layer_norm_fwd and dwc_dropout_fwd. */
dwc_status_t dwc_add_layer_norm_fwd(const void* x, long long ldx, const void* res, long long ldres,
                                    double p, unsigned long long seed, unsigned long long offset,
                                    const unsigned long long* step, const void* gamma,
                                    const void* beta, dwc_dtype_t param_dtype, float eps, void* z,
                                    void* y, float* mean, float* rstd, long long rows, int C,
                                    dwc_dtype_t dtype, dwc_dtype_t res_dtype, dwc_stream_t stream);

/* Backward of dwc_add_layer_norm_fwd:
 *     g = dz + layer_norm_bwd(dy),   dres = g,   dx = dropout map of g
 *   dy : rows x C, dtype     dz : rows x C, res_dtype: the gradient that reaches z from the rest of
 *   the residual stream, or NULL (zero)     z : the forward's sum, res_dtype
 *   dx : rows x C, dtype (out), or NULL when p = 0 and dtype == res_dtype (dres is the same then)
 *   dres : rows x C, res_dtype (out)
 * The rest and the errors as dwc_layer_norm_bwd and dwc_dropout_bwd. */
dwc_status_t dwc_add_layer_norm_bwd(const void* dy, long long lddy, const void* dz, long long lddz,
                                    const void* z, long long ldz, const float* mean,
                                    const float* rstd, const void* gamma, dwc_dtype_t param_dtype,
                                    double p, unsigned long long seed, unsigned long long offset,
                                    const unsigned long long* step, void* dx, void* dres,
                                    float* dgamma, float* dbeta, long long rows, int C,
                                    dwc_dtype_t dtype, dwc_dtype_t res_dtype, void* workspace,
                                    size_t workspace_bytes, dwc_stream_t stream);

/* The norms on either side of a residual connection, with a gate and residual scales, in one pass:
 *     rstd_post = 1 / sqrt(sum_c x^2 / C + eps),   n = x * rstd_post * gamma_post
 *     z = alpha * res + scale * act(gate) * n
 *     rstd_pre = 1 / sqrt(sum_c z^2 / C + eps),    y = z * rstd_pre * gamma_pre
 * (the norm after a block, its gate and scale, the residual sum, the norm in front of the next
 * block; statistics and y from the fp32 sum, z rounded once where it is stored).
 *   x : rows x C, dtype, row stride ldx (the block's output)
 *   res : rows x C, res_dtype, row stride ldres (the residual stream)
 *   gate : rows x C, dtype, row stride ldgate, or NULL (act is then not used)
 *   gamma_post, gamma_pre, scale : C values of param_dtype each, or NULL (1)
 *   z : rows x C, res_dtype (out)   y : rows x C, dtype (out); in place as above
 *   rstd_post, rstd_pre : rows fp32 values each (out), or NULL
 *   res_dtype : dtype, or DWC_F32
 * The rest and the errors as dwc_layer_norm_fwd; DWC_ERR_INVALID_ARG also for an unknown act and a
 * non-finite alpha.  A row of zeros gives zeros (with eps = 0: NaN, 0 * infinity). */
dwc_status_t dwc_block_norm_fwd(const void* x, long long ldx, const void* res, long long ldres, const void* gate,
                                long long ldgate, dwc_gate_t act, const void* gamma_post, const void* gamma_pre,
                                const void* scale, dwc_dtype_t param_dtype, float alpha, float eps, void* z, void* y,
                                float* rstd_post, float* rstd_pre, long long rows, int C, dwc_dtype_t dtype,
                                dwc_dtype_t res_dtype, dwc_stream_t stream);

/* Bytes of workspace dwc_block_norm_bwd needs for rows x C on the CURRENT device (0 for invalid
 * sizes). */
size_t dwc_block_norm_bwd_workspace_size(long long rows, int C);

/* Backward of dwc_block_norm_fwd; with zhat = z * rstd_pre, xhat = x * rstd_post, a = dy * gamma_pre:
 *     g = dz + rstd_pre * (a - zhat * mean_c(a * zhat)),   dres = alpha * g
 *     dn = scale * act(gate) * g,   b = dn * gamma_post
 *     dx = rstd_post * (b - xhat * mean_c(b * xhat)),   dgate = scale * g * n * act'(gate)
 *     dgamma_pre = sum of dy * zhat, dgamma_post = sum of dn * xhat, dscale = sum of g * act(gate) * n
 *   dy : rows x C, dtype     dz : rows x C, res_dtype: the gradient that reaches z from the rest of the
 *   residual stream, or NULL (zero)     x, gate, z, rstd_post, rstd_pre : as in the forward pass
 *   dx : rows x C, dtype (out)     dres : rows x C, res_dtype (out)
 *   dgate : rows x C, dtype (out), or NULL
 *   dgamma_post, dgamma_pre, dscale : C fp32 values each (out), or NULL; rows = 0 writes zeros
 *   workspace : 16-byte aligned, contents ignored and clobbered (not needed without parameter gradients)
 * Errors as dwc_layer_norm_bwd and dwc_block_norm_fwd; DWC_ERR_INVALID_ARG also for a dgate without a gate. */
dwc_status_t dwc_block_norm_bwd(const void* dy, long long lddy, const void* dz, long long lddz, const void* x,
                                long long ldx, const void* z, long long ldz, const void* gate, long long ldgate,
                                dwc_gate_t act, const float* rstd_post, const float* rstd_pre, const void* gamma_post,
                                const void* gamma_pre, const void* scale, dwc_dtype_t param_dtype, float alpha,
                                void* dx, void* dres, void* dgate, float* dgamma_post, float* dgamma_pre,
                                float* dscale, long long rows, int C, dwc_dtype_t dtype, dwc_dtype_t res_dtype,
                                void* workspace, size_t workspace_bytes, dwc_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DWC_NORM_GB300_H */

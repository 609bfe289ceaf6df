/*
 * C ABI of the backward pass of the causal depthwise convolution front-end
 * (mamba_conv1d_fwd of mamba_conv.h), in the same library (libmamba_scan.so).
 *
 * With v_t = bias[d] + sum_j weight[d,j] xin[t - (width-1) + j] recomputed from
 * the inputs (those before t = 0 from state_in, or zero) and
 * dv_t = dout_t silu'(v_t):
 *
 *   dxin_t       = sum_j weight[d,j] dv_{t + (width-1) - j}   (dv = 0 past the end)
 *   dweight[d,j] = sum_{b,t} dv_t xin[t - (width-1) + j]
 *   dbias[d]     = sum_{b,t} dv_t
 *
 * and the same sum at the steps before 0 for dstate_in. dstate_out, the
 * gradient of the forward's state_out, joins the gradients of the last
 * width - 1 inputs (state_in's, where the sequence is shorter).
 *
 * Conventions as in mamba_conv.h. xin, state_in, dout and dxin are in the io
 * dtype; every other gradient (the states' too) is float32. Deterministic.
 */
#ifndef MAMBA_CONV_BWD_H
#define MAMBA_CONV_BWD_H

#include <stddef.h>
#include <stdint.h>

#include "../mamba_conv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of device workspace mamba_conv1d_bwd needs (0 when none, or for an
 * invalid descriptor). The amount depends on the sizes and on the compute-unit
 * count of the current device: call it with the device current that the
 * backward will run on. */
size_t mamba_conv1d_bwd_workspace_size(const mamba_conv_desc *desc);

/*
 *   xin, weight, bias, state_in : as given to mamba_conv1d_fwd (bias and
 *                state_in may be NULL; weight is read for empty sequences too).
 *   dout       : (batch, seqlen, dim) io dtype.
 *   dstate_out : (batch, dim, width-1) float32 or NULL (zero).
 *   dxin       : (batch, seqlen, dim) io dtype, written.
 *   dweight    : (dim, width) float32, written (zeros for no tokens).
 *   dbias      : (dim) float32 or NULL (skip), written.
 *   dstate_in  : (batch, dim, width-1) float32 or NULL (skip), written.
 *   workspace  : at least mamba_conv1d_bwd_workspace_size(desc) bytes, 256-byte
 *                aligned, not shared by calls that run concurrently.
 * Outputs must not overlap any input, the workspace or each other. Alignment:
 * io tensors to their element size, float32 tensors to 4 bytes.
 */
mamba_status mamba_conv1d_bwd(const mamba_conv_desc *desc, const void *xin,
                              const float *weight, const float *bias,
                              const void *state_in, const void *dout,
                              const float *dstate_out, void *dxin,
                              float *dweight, float *dbias, float *dstate_in,
                              void *workspace, size_t workspace_bytes,
                              void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MAMBA_CONV_BWD_H */

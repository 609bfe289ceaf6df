/*
 * C ABI of the gated linear recurrence (gfx950), in the same library as
 * mamba_scan.h (libmamba_scan.so): full sequences, their backward pass, and
 * one decode token.
 *
 * The operation, per batch row b and channel d (one state per channel: the
 * recurrence of mamba_scan.h at N = 1 with the decay and the input's weight
 * given by two gates):
 *
 *   a_t = exp(A[d] sigmoid(r[b,t,d]))
 *   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(g[b,t,d]) x[b,t,d]
 *   out[b,t,d] = h_t,    h_{-1} = h0[b,d] (zero without one)
 *
 * With reset[b,t] nonzero, step t starts a new sequence: a_t = 0, so that
 * h_t = sigmoid(g) x and nothing of the state before it remains (not even a
 * non-finite one); r gets no gradient there. last_state is the state after the
 * last step, so of several sequences in one row the last one's. (The
 * convolution of mamba_conv.h in front of the recurrence has no resets: it sees
 * the width - 1 inputs before a step whatever sequence they belong to.)
 *
 * A must be finite and <= 0 (A = -c softplus(lambda), or c log of the decay of
 * an open gate); A = 0 holds the state (a = 1, weight 0). A > 0 makes the
 * square root NaN, and the gradients with it. r = -inf holds the state too;
 * r = +inf, g = +-inf are the gates' limits. The weight's derivative with
 * respect to a gate that holds the state exactly (1 - a^2 = 0) is taken as 0.
 * Where sigmoid(r) is below float32's normal range (2^-126) it counts as 0; in
 * the forward and the decode token a weight below 2^-63 does too, in the
 * gradients it keeps its value.
 *
 * Conventions as in mamba_scan.h: device pointers of the current device owned
 * by the caller, asynchronous on `stream`, validation before any HIP call,
 * mamba_last_error(), calls on different streams independent as long as their
 * outputs and workspaces are. io tensors (x, r, g, out and their gradients)
 * are float32 or bfloat16 (mamba_dtype); A, states, checkpoints, dA and dh0
 * are float32, and so is all arithmetic. Results are deterministic: whatever
 * the order in which workgroups run, each is computed by the same sums.
 */
#ifndef MAMBA_GATED_H
#define MAMBA_GATED_H

#include <stddef.h>
#include <stdint.h>

#include "../mamba_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Sizes. flags must be 0. */
typedef struct mamba_gated_desc {
  int64_t batch;    /* >= 0                                       */
  int64_t seqlen;   /* L >= 0 (must be 1 for mamba_gated_update)  */
  int64_t dim;      /* channels, 0 .. 2^26                        */
  int32_t io_dtype; /* mamba_dtype of the io tensors              */
  uint32_t flags;   /* 0                                          */
} mamba_gated_desc;

/*
 * Elements between consecutive token rows (steps; batch row b starts
 * b * seqlen rows in), per tensor, so that r and g can be halves of one
 * projection's rows and dr and dg halves of its gradient's; 0 = contiguous
 * (dim). Elements within a row stay contiguous. `out` is out's, or dout's in
 * the backward. A stride below dim is MAMBA_ERR_INVALID_ARG, one above 2^26
 * MAMBA_ERR_UNSUPPORTED. A NULL struct means all contiguous.
 * dr and dg may interleave in one buffer, and so may any two inputs.
 */
typedef struct mamba_gated_strides {
  int64_t x, r, g, out, dx, dr, dg;
} mamba_gated_strides;

/* Steps between two checkpoints: checkpoint k is the state before step
 * k * MAMBA_GATED_CHECKPOINT. */
#define MAMBA_GATED_CHECKPOINT 64

/* Bytes of device workspace mamba_gated_scan_fwd / _bwd need (0 when none, or
 * for an invalid descriptor). */
size_t mamba_gated_scan_workspace_size(const mamba_gated_desc *desc);
size_t mamba_gated_scan_bwd_workspace_size(const mamba_gated_desc *desc);

/*
 * Full sequences.
 *   x, r, g     : (batch, seqlen, dim) io dtype.
 *   A           : (dim) float32.
 *   h0          : (batch, dim) float32 or NULL (zeros).
 *   reset       : (batch, seqlen) bytes, nonzero where a sequence starts, or NULL.
 *   out         : (batch, seqlen, dim) io dtype, written.
 *   last_state  : (batch, dim) float32 or NULL; receives h_{L-1} (h0 or zeros
 *                 when seqlen == 0).
 *   checkpoints : (batch, ceil(seqlen / MAMBA_GATED_CHECKPOINT), dim) float32
 *                 or NULL; receives the states that the backward starts from.
 *   workspace   : at least mamba_gated_scan_workspace_size(desc) bytes,
 *                 256-byte aligned; contents on entry ignored; not shared by
 *                 calls that run concurrently.
 * Outputs must not overlap any input, the workspace or each other. Alignment:
 * io tensors to their element size, float32 tensors to 4 bytes.
 */
mamba_status mamba_gated_scan_fwd(const mamba_gated_desc *desc,
                                  const mamba_gated_strides *strides,
                                  const void *x, const void *r, const void *g,
                                  const float *A, const float *h0,
                                  const uint8_t *reset, void *out,
                                  float *last_state, float *checkpoints,
                                  void *workspace, size_t workspace_bytes,
                                  void *stream);

/*
 * Gradients of mamba_gated_scan_fwd for dout = dLoss/dout and dlast =
 * dLoss/d(last_state). The states are recomputed from the forward's
 * checkpoints, in float32. With lam_t = dout_t + a_{t+1} lam_{t+1} (lam_{L-1} =
 * dout_{L-1} + dlast), sr = sigmoid(r_t), sg = sigmoid(g_t), w = sqrt(1 - a_t^2):
 *   dx_t = lam_t w sg              dg_t = lam_t w x_t sg (1 - sg)
 *   dv_t = lam_t (a_t h_{t-1} - a_t^2 / w sg x_t)    (0 where reset is set)
 *   dr_t = dv_t A sr (1 - sr)      dA = sum_{b,t} dv_t sr     dh0 = a_0 lam_0
 *   x, r, g, A, reset : as given to the forward.
 *   checkpoints : as the forward wrote them.
 *   dout        : (batch, seqlen, dim) io dtype.
 *   dlast       : (batch, dim) float32 or NULL (zero).
 *   dx, dr, dg  : (batch, seqlen, dim) io dtype, written.
 *   dA          : (dim) float32, written.
 *   dh0         : (batch, dim) float32 or NULL (skip), written.
 * With seqlen == 0 (or batch == 0) dA is zero and dh0 = dlast (zero without
 * it). Overlap and alignment as the forward, except that dr and dg may
 * interleave.
 */
mamba_status mamba_gated_scan_bwd(const mamba_gated_desc *desc,
                                  const mamba_gated_strides *strides,
                                  const void *x, const void *r, const void *g,
                                  const float *A, const uint8_t *reset,
                                  const float *checkpoints, const void *dout,
                                  const float *dlast, void *dx, void *dr,
                                  void *dg, float *dA, float *dh0,
                                  void *workspace, size_t workspace_bytes,
                                  void *stream);

/*
 * One decode token for every sequence (desc->seqlen must be 1).
 *   state       : (batch, dim) float32, read and overwritten in place.
 *   x, r, g     : (batch, dim) io dtype; out : (batch, dim) io dtype, written.
 * out must not overlap any input or the state. Row strides as above (dx, dr,
 * dg unused).
 */
mamba_status mamba_gated_update(const mamba_gated_desc *desc,
                                const mamba_gated_strides *strides,
                                float *state, const void *x, const void *r,
                                const void *g, const float *A, void *out,
                                void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MAMBA_GATED_H */

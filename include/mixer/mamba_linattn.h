/*
 * C ABI of linear attention with a decay for each head (gfx950), in the same
 * library as mamba_scan.h (libmamba_scan.so): whole sequences, their backward
 * pass, and one decode token.
 *
 * The operation, per sequence and head h (queries and keys of group
 * h / (nheads / ngroups)); the state S is a K x V matrix, as that of
 * mamba_ssd.h with the decay given as it is:
 *
 *   S_t = exp(g_t) S_{t-1} + k_t v_t^T,     S_{-1} = h0 (zeros without one)
 *   o_t = scale S_t^T q_t
 *
 * g is the log of the decay, per token and head or one per head
 * (MAMBA_LINATTN_HEAD_DECAY). g <= -104, -inf included, is a decay that float32
 * holds as 0: the state before such a token is dropped, whatever it is, so that
 * the token starts anew. g > 0 makes the state grow, until it overflows; where a sum
 * of them passes 88 the factor is infinite, also for a state of zeros, which is
 * NaN then.
 *
 * A token's values reach the outputs of its own and later tokens of its
 * sequence and no other's, non-finite ones too; within one sequence they reach
 * later tokens until a decay of 0 (one g <= -104: decays that underflow together
 * leave what is not finite as it is).
 *
 * Sequences are `batch` runs of seqlen tokens, or with MAMBA_LINATTN_PACKED lie
 * one after another in seqlen token rows: sequence i is rows offsets[i] ..
 * offsets[i + 1] - 1 (none when they are equal), offsets being batch + 1 values
 * on the device that do not decrease, in 0 .. seqlen. They are read when the
 * kernels run; a value outside 0 .. seqlen counts as the nearer end. With values
 * that decrease the outputs hold unspecified numbers, but nothing outside them
 * is written. Rows of no sequence are left as they were, unless
 * MAMBA_LINATTN_ZERO_REST asks for zeros in those before the first and behind
 * the last sequence.
 *
 * Conventions as in mamba_scan.h: device pointers of the current device owned
 * by the caller, asynchronous on `stream`, validation before any HIP call,
 * mamba_last_error(), calls on different streams independent as long as their
 * outputs and workspaces are. io tensors (q, k, v, out and their gradients) are
 * float32 or bfloat16; g, states, dg and dh0 are float32. States, products and
 * sums are held in float32; with bfloat16 io the products are taken on the
 * matrix cores from bfloat16 operands, and what is float32 goes in as a sum of
 * bfloat16 parts: three, whose sum is the value, where it makes the state, and
 * two, off by 2^-17 of each term, where it makes an output. The outputs are
 * rounded once. (Parts of an infinity, or of a value that rounds to one in
 * bfloat16, add up to NaN: such a state or score reaches the outputs as NaN.)
 * Results are deterministic.
 */
#ifndef MAMBA_LINATTN_H
#define MAMBA_LINATTN_H

#include <stddef.h>
#include <stdint.h>

#include "../mamba_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MAMBA_LINATTN_HEAD_DECAY (1u << 0) /* g is (nheads), the same for every token        */
#define MAMBA_LINATTN_PACKED (1u << 1)     /* offsets given; seqlen counts all token rows    */
#define MAMBA_LINATTN_ZERO_REST (1u << 2)  /* zeros in rows before / behind packed sequences */

/* Sizes and options. K and V are multiples of 8 in 8 .. 256 (others:
 * MAMBA_ERR_UNSUPPORTED). */
typedef struct mamba_linattn_desc {
  int64_t batch;    /* sequences >= 0                                       */
  int64_t seqlen;   /* tokens of each, or all token rows with PACKED, >= 0
                       (must be 1 for mamba_linattn_update)                 */
  int64_t nheads;   /* H >= 0                                               */
  int64_t ngroups;  /* G >= 1 dividing H: head h reads q, k of h / (H / G)  */
  int64_t dkey;     /* K                                                    */
  int64_t dvalue;   /* V                                                    */
  int32_t io_dtype; /* mamba_dtype of the io tensors                        */
  uint32_t flags;   /* MAMBA_LINATTN_*                                      */
  float scale;      /* finite                                               */
} mamba_linattn_desc;

/*
 * Elements between consecutive token rows, per tensor, so that q, k and v can
 * be column slices of one projection's rows and their gradients of one
 * gradient's; 0 = contiguous (heads * head size). Elements within a row stay
 * contiguous. `out` is out's, or dout's in the backward. Below a row's length:
 * MAMBA_ERR_INVALID_ARG; above 2^23, also of contiguous rows:
 * MAMBA_ERR_UNSUPPORTED. A NULL struct means all contiguous. Any two inputs may
 * interleave, and so may dq, dk and dv.
 */
typedef struct mamba_linattn_strides {
  int64_t q, k, v, out, dq, dk, dv;
} mamba_linattn_strides;

/* Bytes of device workspace the calls need (0 when none, or for an invalid
 * descriptor). The amount depends on the sizes and on the compute-unit count of
 * the current device: call it with the device current that the call will run
 * on. */
size_t mamba_linattn_workspace_size(const mamba_linattn_desc *desc);
size_t mamba_linattn_bwd_workspace_size(const mamba_linattn_desc *desc);

/*
 * Whole sequences. `rows` below is batch * seqlen, or seqlen with PACKED.
 *   q, k       : (rows, G, K) io dtype.
 *   v          : (rows, H, V) io dtype.
 *   g          : (rows, H) float32, or (H) with HEAD_DECAY.
 *   h0         : (batch, H, K, V) float32 or NULL (zeros).
 *   offsets    : (batch + 1) int64 with PACKED, else NULL.
 *   out        : (rows, H, V) io dtype, written.
 *   last_state : (batch, H, K, V) float32 or NULL; receives the state after each
 *                sequence's last token (h0 or zeros for one of no tokens).
 *   workspace  : at least mamba_linattn_workspace_size(desc) bytes, 256-byte
 *                aligned; contents on entry ignored; not shared by calls that
 *                run concurrently.
 * Outputs must not overlap any input, the workspace or each other. Alignment: io
 * tensors to their element size, float32 tensors to 4 bytes, offsets to 8.
 */
mamba_status mamba_linattn_fwd(const mamba_linattn_desc *desc,
                               const mamba_linattn_strides *strides,
                               const void *q, const void *k, const void *v,
                               const float *g, const float *h0,
                               const int64_t *offsets, void *out,
                               float *last_state, void *workspace,
                               size_t workspace_bytes, void *stream);

/*
 * Gradients of mamba_linattn_fwd for dout = dLoss/dout and dlast =
 * dLoss/d(last_state), from the forward's inputs alone. With dS_t =
 * exp(g_{t+1}) dS_{t+1} + scale q_t dout_t^T (the last token's with dlast in
 * the place of the first term):
 *   dq_t = scale S_t dout_t     dk_t = dS_t v_t     dv_t = dS_t^T k_t
 *   dg_t = exp(g_t) <dS_t, S_{t-1}>                 dh0 = exp(g_0) dS_0
 * dq and dk are sums over the heads of a group, rounded once; dg is a sum over
 * all tokens with HEAD_DECAY. A decay of 0 gets a zero gradient. dg_t is added up
 * from terms of its own, in float32 states and products and float64 sums: its error
 * goes by the magnitudes of what crosses token t, not by other tokens' gradients,
 * however large these are. For it the workspace takes the states at every 64 tokens
 * (bfloat16) or 32 (float32), twice, of all heads or, past 8 GiB, of some at a
 * time. With bfloat16 io dq, dk and dv are other roundings of the same sums where
 * dg is NULL.
 *   q, k, v, g, h0, offsets : as given to the forward.
 *   dout       : (rows, H, V) io dtype.
 *   dlast      : (batch, H, K, V) float32 or NULL (zero).
 *   dq, dk     : (rows, G, K) io dtype, written.
 *   dv         : (rows, H, V) io dtype, written.
 *   dg         : as g, float32, written, or NULL (skip, which takes less time).
 *   dh0        : (batch, H, K, V) float32 or NULL (skip), written.
 * Overlap and alignment as the forward, except that dq, dk and dv may
 * interleave.
 */
mamba_status mamba_linattn_bwd(const mamba_linattn_desc *desc,
                               const mamba_linattn_strides *strides,
                               const void *q, const void *k, const void *v,
                               const float *g, const float *h0,
                               const int64_t *offsets, const void *dout,
                               const float *dlast, void *dq, void *dk, void *dv,
                               float *dg, float *dh0, void *workspace,
                               size_t workspace_bytes, void *stream);

/*
 * One decode token for every sequence (desc->seqlen must be 1, no PACKED).
 *   state   : (batch, H, K, V) float32, read and overwritten in place.
 *   q, k    : (batch, G, K) io dtype; v : (batch, H, V) io dtype.
 *   g       : (batch, H) float32, or (H) with HEAD_DECAY.
 *   out     : (batch, H, V) io dtype, written.
 * out must not overlap any input or the state. Row strides as above (dq, dk, dv
 * unused). All arithmetic is float32.
 */
mamba_status mamba_linattn_update(const mamba_linattn_desc *desc,
                                  const mamba_linattn_strides *strides,
                                  float *state, const void *q, const void *k,
                                  const void *v, const float *g, void *out,
                                  void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MAMBA_LINATTN_H */

/*
 * C ABI of the norm of queries and keys for each head with the rotation by the
 * token's position in the same pass (gfx950), in the same library as
 * mamba_scan.h (libmamba_scan.so), and its backward pass.
 *
 * Per token and head, over its D channels x (a query head with q_weight, a key
 * head with k_weight; a weight that is NULL counts as ones):
 *
 *   n_d = x_d rstd weight[d],     rstd = 1 / sqrt(mean_d x_d^2 + eps)
 *   y   = n with the pairs (a, b) of its first `rotary` channels turned:
 *         a' = a cos - b sin,  b' = b cos + a sin,
 *         angle = positions[axis(i)][token] * freqs[i]  for pair i
 *
 * Pair i is channels i and i + rotary / 2, or 2 i and 2 i + 1 with
 * MAMBA_QKNORM_INTERLEAVED; channels from `rotary` on are not turned. With several
 * axes (1 to 4; such as time, height, width) the pairs are split into
 * consecutive sections, sections[a] pairs turning by axis a's positions. The
 * angle is the product of the position and the float32 frequency in 64 bits,
 * exact for positions below 2^28 in magnitude, and so are sine and cosine to
 * float32's precision; farther off they lose a bit each time the position doubles.
 *
 * Conventions as in mamba_scan.h and block/mamba_norm.h: io tensors are float32 or
 * bfloat16, weights, freqs and the weights' gradients float32, arithmetic
 * float32; non-finite values propagate within their head's row (in the backward
 * the row is NaN). Sums of squares are float32 ones: a head whose sum is above their
 * range (values of 1e19 and more) has rstd 0 as an infinite one has. With eps 0 a
 * head of zeros has no norm and is NaN, and one whose squares are all below the range
 * (values of 1e-23 and less) has an infinite rstd. Results are deterministic.
 */
#ifndef MAMBA_QKNORM_H
#define MAMBA_QKNORM_H

#include <stddef.h>
#include <stdint.h>

#include "../mamba_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MAMBA_QKNORM_INTERLEAVED (1u << 0) /* pairs of neighbouring channels */
#define MAMBA_QKNORM_AXES 4

/* Sizes and options. headdim is a multiple of 8 in 8 .. 256 (others:
 * MAMBA_ERR_UNSUPPORTED). */
typedef struct mamba_qknorm_desc {
  int64_t tokens;   /* >= 0                                            */
  int64_t qheads;   /* >= 0                                            */
  int64_t kheads;   /* >= 0 (0: queries only, the keys' pointers NULL) */
  int64_t headdim;  /* D                                               */
  int64_t rotary;   /* a multiple of 8, 0 .. D                         */
  int64_t sections[MAMBA_QKNORM_AXES]; /* pairs of each axis; their sum is
                       rotary / 2; those from naxes on are 0           */
  int32_t naxes;    /* 1 .. 4                                          */
  int32_t io_dtype; /* mamba_dtype                                     */
  float eps;        /* >= 0, finite                                    */
  uint32_t flags;   /* 0 or MAMBA_QKNORM_INTERLEAVED                   */
} mamba_qknorm_desc;

/* Elements between consecutive token rows, per tensor, so that q and k can be
 * column slices of one projection's rows; 0 (or a NULL struct) = contiguous.
 * Below a row's length: MAMBA_ERR_INVALID_ARG; above 2^26:
 * MAMBA_ERR_UNSUPPORTED. qo, ko are the outputs', or the gradients' of the
 * outputs in the backward. */
typedef struct mamba_qknorm_strides {
  int64_t q, k, qo, ko, dq, dk;
} mamba_qknorm_strides;

/*
 *   q, k      : (tokens, qheads, D), (tokens, kheads, D) io dtype.
 *   positions : (naxes, tokens) int64.
 *   freqs     : (rotary / 2) float32, radians for each position.
 *   q_weight, k_weight : (D) float32 or NULL.
 *   qo, ko    : as q and k, written. Each may be its input (same pointer and
 *               stride: normed and turned in place).
 * Otherwise outputs must not overlap any input or each other; outputs may
 * interleave. Alignment: to the element size.
 */
mamba_status mamba_qknorm_fwd(const mamba_qknorm_desc *desc,
                              const mamba_qknorm_strides *strides,
                              const void *q, const void *k,
                              const int64_t *positions, const float *freqs,
                              const float *q_weight, const float *k_weight,
                              void *qo, void *ko, void *stream);

/* Bytes of device workspace mamba_qknorm_bwd needs (0 when none, or for an
 * invalid descriptor). The amount depends on the sizes and on the compute-unit
 * count of the current device. */
size_t mamba_qknorm_bwd_workspace_size(const mamba_qknorm_desc *desc);

/*
 * Gradients of mamba_qknorm_fwd for dqo and dko, from the forward's inputs (as
 * they were before it). With u the output's gradient turned back and n_d = x_d
 * rstd:
 *   dx_d = rstd (weight[d] u_d - n_d mean_d(weight[d] u_d n_d))
 *   dweight[d] = sum over tokens and heads of u_d n_d
 *   dq, dk    : as q and k, written. Each may be its output's gradient (same
 *               pointer and stride).
 *   dq_weight, dk_weight : (D) float32 or NULL (skip), written.
 *   workspace : at least mamba_qknorm_bwd_workspace_size(desc) bytes, 256-byte
 *               aligned, not shared by calls that run concurrently.
 */
mamba_status mamba_qknorm_bwd(const mamba_qknorm_desc *desc,
                              const mamba_qknorm_strides *strides,
                              const void *q, const void *k,
                              const int64_t *positions, const float *freqs,
                              const float *q_weight, const float *k_weight,
                              const void *dqo, const void *dko, void *dq,
                              void *dk, float *dq_weight, float *dk_weight,
                              void *workspace, size_t workspace_bytes,
                              void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MAMBA_QKNORM_H */

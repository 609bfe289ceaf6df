/*
 * C ABI of the root-mean-square norm at a block's entry (gfx950), in the same
 * library as mamba_scan.h (libmamba_scan.so): with the residual stream's
 * addition, with an 8-bit output and its scales, and its backward pass.
 *
 * Per token (row) over its dim channels:
 *
 *   s_d   = x_d + residual_d       (rounded to the residual's dtype: the
 *                                   stream as it is stored is what is normed;
 *                                   s = x without a residual)
 *   y_d   = s_d rstd weight[d],    rstd = 1 / sqrt(mean_d s_d^2 + eps)
 *
 * The 8-bit form gives q = e4m3(y / scale), rounded to nearest even, with one
 * float32 scale per row (group 0) or per run of `group` channels (the last
 * run may be shorter): scale = max(max |y|, 2^-100) / 448, 448 being e4m3's
 * largest finite value. y is a float32 value, not rounded to the io dtype in
 * between, and y / scale its float32 quotient by the scale as it is stored.
 * Rows of zeros give q = 0.
 *
 * Non-finite inputs propagate within their row: a NaN makes the row NaN; an
 * infinity makes rstd 0, so its own outputs NaN and the row's others 0. NaN
 * values do not take part in a scale's maximum. With eps 0 a row of zeros has
 * no norm and is NaN. Squares and their sum are float32 numbers: a row whose sum
 * of squares is above their range (values of 1e19 and more) has rstd 0 as an
 * infinite one has, and with eps 0 one whose squares are all below it (values
 * of 1e-23 and less) an infinite rstd. In the backward a row of the stream with a
 * non-finite value has a NaN ds.
 *
 * Conventions as in mamba_scan.h. x, out, dout and dx have the io dtype;
 * residual, sum, dsum and dresidual the residual dtype, which is the io dtype
 * or float32; weight and dweight are float32. Arithmetic is float32. Results
 * are deterministic.
 */
#ifndef MAMBA_NORM_H
#define MAMBA_NORM_H

#include <stddef.h>
#include <stdint.h>

#include "../mamba_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Sizes and options. dim is 0 .. 65536. */
typedef struct mamba_norm_desc {
  int64_t rows;           /* tokens >= 0                                   */
  int64_t dim;            /* channels                                      */
  int64_t group;          /* mamba_rmsnorm_quant_fwd: 0 or 128; else 0     */
  int32_t io_dtype;       /* mamba_dtype                                   */
  int32_t residual_dtype; /* io_dtype or MAMBA_F32                         */
  float eps;              /* >= 0, finite                                  */
  uint32_t flags;         /* 0                                             */
} mamba_norm_desc;

/* Elements between consecutive rows, per tensor; 0 (or a NULL struct) =
 * contiguous. Below dim: MAMBA_ERR_INVALID_ARG; above 2^26:
 * MAMBA_ERR_UNSUPPORTED. `out` is out's, q's or dout's; `dsum` and `dresidual`,
 * `dx` are the backward's. */
typedef struct mamba_norm_strides {
  int64_t x, residual, sum, out, dsum, dresidual, dx;
} mamba_norm_strides;

/*
 *   x        : (rows, dim) io dtype.
 *   residual : (rows, dim) residual dtype, or NULL (then residual_dtype must be
 *              io_dtype and sum NULL: x itself is the stream).
 *   weight   : (dim) float32.
 *   out      : (rows, dim) io dtype, written.
 *   sum      : (rows, dim) residual dtype, receives s; required with a
 *              residual. It may be the residual itself (same pointer and
 *              stride: the stream is updated in place).
 * Otherwise outputs must not overlap any input or each other. Alignment: to
 * the element size.
 */
mamba_status mamba_rmsnorm_fwd(const mamba_norm_desc *desc,
                               const mamba_norm_strides *strides, const void *x,
                               const void *residual, const float *weight,
                               void *out, void *sum, void *stream);

/*
 * The same with an 8-bit output.
 *   q     : (rows, dim) e4m3 bytes (the OCP format: no infinities, largest
 *           value 448), written.
 *   scale : (rows, group ? ceil(dim / group) : 1) float32, contiguous, written.
 */
mamba_status mamba_rmsnorm_quant_fwd(const mamba_norm_desc *desc,
                                     const mamba_norm_strides *strides,
                                     const void *x, const void *residual,
                                     const float *weight, void *q, float *scale,
                                     void *sum, void *stream);

/* Bytes of device workspace mamba_rmsnorm_bwd needs (0 when none, or for an
 * invalid descriptor). The amount depends on the sizes and on the compute-unit
 * count of the current device: call it with the device current that the
 * backward will run on. */
size_t mamba_rmsnorm_bwd_workspace_size(const mamba_norm_desc *desc);

/*
 * Gradients of mamba_rmsnorm_fwd for dout = dLoss/dout and dsum = dLoss/d(sum)
 * (what the stream's later readers send back). With n_d = s_d rstd and
 * u_d = weight[d] dout_d:
 *   ds_d = dsum_d + rstd (u_d - n_d mean_d(u_d n_d)),  dweight[d] = sum_rows dout_d n_d
 * ds is the gradient of both x and the residual.
 *   sum       : (rows, dim) residual dtype, as the forward wrote it (x without
 *               a residual).
 *   dout      : (rows, dim) io dtype.
 *   dsum      : (rows, dim) residual dtype or NULL (zero).
 *   dresidual : (rows, dim) residual dtype, ds, written. It may be dsum itself
 *               (same pointer and stride).
 *   dx        : (rows, dim) io dtype, ds, written; NULL to skip, and must be
 *               NULL when both dtypes are the same (dresidual is dx then).
 *   dweight   : (dim) float32, written (zeros for no rows).
 *   workspace : at least mamba_rmsnorm_bwd_workspace_size(desc) bytes, 256-byte
 *               aligned, not shared by calls that run concurrently.
 */
mamba_status mamba_rmsnorm_bwd(const mamba_norm_desc *desc,
                               const mamba_norm_strides *strides,
                               const void *sum, const float *weight,
                               const void *dout, const void *dsum,
                               void *dresidual, void *dx, float *dweight,
                               void *workspace, size_t workspace_bytes,
                               void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MAMBA_NORM_H */

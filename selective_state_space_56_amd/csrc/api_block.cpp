// C ABI of the block operators around the scan: argument validation and
// dispatch to the HIP kernels. See include/block/ for the contracts.
#include "block/mamba_conv_bwd.h"
#include "block/mamba_gated.h"
#include "block/mamba_norm.h"

#include <hip/hip_runtime_api.h>

#include <cmath>
#include <initializer_list>

#include "api_rows.h"
#include "block.h"

using mscan::check_align;
using mscan::check_conv_desc;
using mscan::check_io;
using mscan::check_outputs;
using mscan::check_present;
using mscan::check_row_align;
using mscan::check_workspace;
using mscan::collide;
using mscan::fail;
using mscan::flat;
using mscan::io_bytes;
using mscan::kMaxElems;
using mscan::kMaxStride;
using mscan::launched;
using mscan::ok;
using mscan::resolve;
using mscan::Rows;

namespace {

static_assert(MAMBA_GATED_CHECKPOINT == mscan::kGatedCheckpoint, "the header states the spacing");

mamba_status check_gated(const char* who, const mamba_gated_desc* d) {
  if (!d) return fail(MAMBA_ERR_INVALID_ARG, "%s: desc is NULL", who);
  if (d->batch < 0 || d->seqlen < 0 || d->dim < 0)
    return fail(MAMBA_ERR_INVALID_ARG, "%s: negative size (batch=%lld seqlen=%lld dim=%lld)", who,
                (long long)d->batch, (long long)d->seqlen, (long long)d->dim);
  mamba_status st = check_io(who, "io_dtype", d->io_dtype);
  if (st != MAMBA_OK) return st;
  if (d->flags != 0) return fail(MAMBA_ERR_INVALID_ARG, "%s: flags must be 0", who);
  if (d->dim > kMaxStride)
    return fail(MAMBA_ERR_UNSUPPORTED, "%s: dim %lld too large", who, (long long)d->dim);
  // states and tokens are counted in 31 bits, elements in 40
  const int64_t count = (int64_t(1) << 31) - 1;
  if (d->batch > count || d->seqlen > count || (d->dim > 0 && d->batch > count / d->dim) ||
      (d->batch > 0 && d->seqlen > count / d->batch) ||
      (d->batch * d->dim > 0 && d->seqlen > kMaxElems / (d->batch * d->dim)) ||
      mscan::gated_tiles(d->batch, d->seqlen, d->dim) > mscan::kGatedMaxTiles)
    return fail(MAMBA_ERR_UNSUPPORTED, "%s: problem too large", who);
  return MAMBA_OK;
}

struct GatedRows {
  int64_t x, r, g, out, dx, dr, dg;
};

mamba_status resolve_gated(const char* who, const mamba_gated_desc* d, const mamba_gated_strides* s,
                           GatedRows* to) {
  const mamba_gated_strides none = {0, 0, 0, 0, 0, 0, 0};
  const mamba_gated_strides& v = s ? *s : none;
  const struct {
    const char* name;
    int64_t given;
    int64_t* to;
  } f[] = {{"x", v.x, &to->x},    {"r", v.r, &to->r},    {"g", v.g, &to->g},   {"out", v.out, &to->out},
           {"dx", v.dx, &to->dx}, {"dr", v.dr, &to->dr}, {"dg", v.dg, &to->dg}};
  const int64_t tokens = d->batch * d->seqlen;
  for (const auto& e : f) {
    const mamba_status st = resolve(who, e.name, e.given, d->dim, e.to);
    if (st != MAMBA_OK) return st;
    if (tokens > 0 && *e.to > kMaxElems / tokens)
      return fail(MAMBA_ERR_UNSUPPORTED, "%s: problem too large", who);
  }
  return MAMBA_OK;
}

int64_t checkpoints_of(const mamba_gated_desc* d) {
  return (d->seqlen + MAMBA_GATED_CHECKPOINT - 1) / MAMBA_GATED_CHECKPOINT;
}

}  // namespace

extern "C" {

size_t mamba_gated_scan_workspace_size(const mamba_gated_desc* d) {
  if (check_gated("mamba_gated_scan_workspace_size", d) != MAMBA_OK) return 0;
  return mscan::gated_fwd_workspace_bytes(d->batch, d->seqlen, d->dim);
}

size_t mamba_gated_scan_bwd_workspace_size(const mamba_gated_desc* d) {
  if (check_gated("mamba_gated_scan_bwd_workspace_size", d) != MAMBA_OK) return 0;
  return mscan::gated_bwd_workspace_bytes(d->batch, d->seqlen, d->dim);
}

mamba_status mamba_gated_scan_fwd(const mamba_gated_desc* d, const mamba_gated_strides* strides,
                                  const void* x, const void* r, const void* g, const float* A,
                                  const float* h0, const uint8_t* reset, void* out,
                                  float* last_state, float* checkpoints, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  const char* who = "mamba_gated_scan_fwd";
  GatedRows s;
  mamba_status st = check_gated(who, d);
  if (st != MAMBA_OK || (st = resolve_gated(who, d, strides, &s)) != MAMBA_OK) return st;
  const int64_t rows = d->batch * d->dim, tokens = d->batch * d->seqlen;
  const bool work = rows > 0 && tokens > 0;
  if (rows == 0 || (!work && !last_state)) return ok();
  if (work && (st = check_present(who, {{"x", x, 0}, {"r", r, 0}, {"g", g, 0}, {"A", A, 0}, {"out", out, 0}})) !=
                  MAMBA_OK)
    return st;
  const size_t need = mamba_gated_scan_workspace_size(d);
  if ((st = check_workspace(who, workspace, workspace_bytes, need)) != MAMBA_OK) return st;
  const size_t eb = io_bytes(d->io_dtype);
  const int64_t n = work ? tokens : 0;
  const Rows ix{"x", x, n, s.x, d->dim, eb}, ir{"r", r, n, s.r, d->dim, eb}, ig{"g", g, n, s.g, d->dim, eb};
  const Rows ia = flat("A", A, d->dim, 4), ih = flat("h0", h0, rows, 4), im = flat("reset", reset, n, 1);
  const Rows oo{"out", out, n, s.out, d->dim, eb}, ol = flat("last_state", last_state, rows, 4);
  const Rows oc = flat("checkpoints", checkpoints, work ? d->batch * checkpoints_of(d) * d->dim : 0, 4);
  const Rows ow = flat("workspace", need ? workspace : nullptr, static_cast<int64_t>(need), 1);
  if ((st = check_outputs(who, {ix, ir, ig, ia, ih, im}, {oo, ol, oc, ow})) != MAMBA_OK) return st;
  if ((st = check_row_align(who, {ix, ir, ig, ia, ih, oo, ol, oc})) != MAMBA_OK) return st;
  mscan::GatedProblem p;
  p.x = x;
  p.r = r;
  p.g = g;
  p.A = A;
  p.h0 = h0;
  p.reset = reset;
  p.out = out;
  p.last_state = last_state;
  p.checkpoints = checkpoints;
  p.batch = d->batch;
  p.seqlen = d->seqlen;
  p.dim = d->dim;
  p.io = d->io_dtype;
  p.sx = s.x;
  p.sr = s.r;
  p.sg = s.g;
  p.so = s.out;
  return launched(who, mscan::launch_gated_fwd(p, workspace, static_cast<hipStream_t>(stream)));
}

mamba_status mamba_gated_scan_bwd(const mamba_gated_desc* d, const mamba_gated_strides* strides,
                                  const void* x, const void* r, const void* g, const float* A,
                                  const uint8_t* reset, const float* checkpoints, const void* dout,
                                  const float* dlast, void* dx, void* dr, void* dg, float* dA,
                                  float* dh0, void* workspace, size_t workspace_bytes, void* stream) {
  const char* who = "mamba_gated_scan_bwd";
  GatedRows s;
  mamba_status st = check_gated(who, d);
  if (st != MAMBA_OK || (st = resolve_gated(who, d, strides, &s)) != MAMBA_OK) return st;
  const int64_t rows = d->batch * d->dim, tokens = d->batch * d->seqlen;
  const bool work = rows > 0 && tokens > 0;
  if (d->dim == 0) return ok();
  if ((st = check_present(who, {{"dA", dA, 0}})) != MAMBA_OK) return st;
  if (work &&
      (st = check_present(who, {{"x", x, 0}, {"r", r, 0}, {"g", g, 0}, {"A", A, 0}, {"checkpoints", checkpoints, 0},
                                {"dout", dout, 0}, {"dx", dx, 0}, {"dr", dr, 0}, {"dg", dg, 0}})) != MAMBA_OK)
    return st;
  const size_t need = mamba_gated_scan_bwd_workspace_size(d);
  if ((st = check_workspace(who, workspace, workspace_bytes, need)) != MAMBA_OK) return st;
  const size_t eb = io_bytes(d->io_dtype);
  const int64_t n = work ? tokens : 0;
  const Rows ix{"x", x, n, s.x, d->dim, eb}, ir{"r", r, n, s.r, d->dim, eb}, ig{"g", g, n, s.g, d->dim, eb};
  const Rows io{"dout", dout, n, s.out, d->dim, eb};
  const Rows ia = flat("A", A, d->dim, 4), im = flat("reset", reset, n, 1), il = flat("dlast", dlast, rows, 4);
  const Rows ic = flat("checkpoints", checkpoints, work ? d->batch * checkpoints_of(d) * d->dim : 0, 4);
  const Rows ox{"dx", dx, n, s.dx, d->dim, eb}, orr{"dr", dr, n, s.dr, d->dim, eb};
  const Rows og{"dg", dg, n, s.dg, d->dim, eb};
  const Rows oa = flat("dA", dA, d->dim, 4), oh = flat("dh0", dh0, rows, 4);
  const Rows ow = flat("workspace", need ? workspace : nullptr, static_cast<int64_t>(need), 1);
  if ((st = check_outputs(who, {ix, ir, ig, io, ia, im, il, ic}, {ox, orr, og, oa, oh, ow})) != MAMBA_OK) return st;
  if ((st = check_row_align(who, {ix, ir, ig, io, ia, il, ic, ox, orr, og, oa, oh})) != MAMBA_OK) return st;
  mscan::GatedBwdProblem p;
  p.x = x;
  p.r = r;
  p.g = g;
  p.A = A;
  p.reset = reset;
  p.checkpoints = checkpoints;
  p.dout = dout;
  p.dlast = dlast;
  p.dx = dx;
  p.dr = dr;
  p.dg = dg;
  p.dA = dA;
  p.dh0 = dh0;
  p.batch = d->batch;
  p.seqlen = d->seqlen;
  p.dim = d->dim;
  p.io = d->io_dtype;
  p.sx = s.x;
  p.sr = s.r;
  p.sg = s.g;
  p.so = s.out;
  p.sdx = s.dx;
  p.sdr = s.dr;
  p.sdg = s.dg;
  return launched(who, mscan::launch_gated_bwd(p, workspace, static_cast<hipStream_t>(stream)));
}

mamba_status mamba_gated_update(const mamba_gated_desc* d, const mamba_gated_strides* strides,
                                float* state, const void* x, const void* r, const void* g,
                                const float* A, void* out, void* stream) {
  const char* who = "mamba_gated_update";
  GatedRows s;
  mamba_status st = check_gated(who, d);
  if (st != MAMBA_OK) return st;
  if (d->seqlen != 1)
    return fail(MAMBA_ERR_INVALID_ARG, "%s: seqlen %lld must be 1", who, (long long)d->seqlen);
  if ((st = resolve_gated(who, d, strides, &s)) != MAMBA_OK) return st;
  const int64_t n = d->batch, rows = d->batch * d->dim;
  if (rows == 0) return ok();
  if ((st = check_present(who, {{"state", state, 0}, {"x", x, 0}, {"r", r, 0}, {"g", g, 0}, {"A", A, 0},
                                {"out", out, 0}})) != MAMBA_OK)
    return st;
  const size_t eb = io_bytes(d->io_dtype);
  const Rows ix{"x", x, n, s.x, d->dim, eb}, ir{"r", r, n, s.r, d->dim, eb}, ig{"g", g, n, s.g, d->dim, eb};
  const Rows ia = flat("A", A, d->dim, 4), oh = flat("state", state, rows, 4);
  const Rows oo{"out", out, n, s.out, d->dim, eb};
  if ((st = check_outputs(who, {ix, ir, ig, ia}, {oo, oh})) != MAMBA_OK) return st;
  if ((st = check_row_align(who, {ix, ir, ig, ia, oh, oo})) != MAMBA_OK) return st;
  mscan::GatedUpdateProblem p;
  p.state = state;
  p.x = x;
  p.r = r;
  p.g = g;
  p.A = A;
  p.out = out;
  p.batch = d->batch;
  p.dim = d->dim;
  p.io = d->io_dtype;
  p.sx = s.x;
  p.sr = s.r;
  p.sg = s.g;
  p.so = s.out;
  return launched(who, mscan::launch_gated_update(p, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

mamba_status check_norm(const char* who, const mamba_norm_desc* d, bool quant) {
  if (!d) return fail(MAMBA_ERR_INVALID_ARG, "%s: desc is NULL", who);
  if (d->rows < 0 || d->dim < 0)
    return fail(MAMBA_ERR_INVALID_ARG, "%s: negative size (rows=%lld dim=%lld)", who, (long long)d->rows,
                (long long)d->dim);
  mamba_status st = check_io(who, "io_dtype", d->io_dtype);
  if (st != MAMBA_OK || (st = check_io(who, "residual_dtype", d->residual_dtype)) != MAMBA_OK) return st;
  if (d->residual_dtype != d->io_dtype && d->residual_dtype != MAMBA_F32)
    return fail(MAMBA_ERR_UNSUPPORTED, "%s: a bfloat16 residual needs bfloat16 io", who);
  if (d->flags != 0) return fail(MAMBA_ERR_INVALID_ARG, "%s: flags must be 0", who);
  if (!(d->eps >= 0.0f) || !std::isfinite(d->eps))
    return fail(MAMBA_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", who);
  if (d->group != 0 && !(quant && d->group == 128))
    return fail(quant && d->group > 0 ? MAMBA_ERR_UNSUPPORTED : MAMBA_ERR_INVALID_ARG, "%s: group %lld is not %s",
                who, (long long)d->group, quant ? "0 or 128" : "0");
  if (d->dim > mscan::kNormMaxDim)
    return fail(MAMBA_ERR_UNSUPPORTED, "%s: dim %lld too large (at most %lld)", who, (long long)d->dim,
                (long long)mscan::kNormMaxDim);
  if (d->rows > (int64_t(1) << 31) - 1 || (d->dim > 0 && d->rows > kMaxElems / d->dim))
    return fail(MAMBA_ERR_UNSUPPORTED, "%s: problem too large", who);
  return MAMBA_OK;
}

struct NormRows {
  int64_t x, residual, sum, out, dsum, dresidual, dx;
};

mamba_status resolve_norm(const char* who, const mamba_norm_desc* d, const mamba_norm_strides* s,
                          NormRows* to) {
  const mamba_norm_strides none = {0, 0, 0, 0, 0, 0, 0};
  const mamba_norm_strides& v = s ? *s : none;
  const struct {
    const char* name;
    int64_t given;
    int64_t* to;
  } f[] = {{"x", v.x, &to->x},          {"residual", v.residual, &to->residual},
           {"sum", v.sum, &to->sum},    {"out", v.out, &to->out},
           {"dsum", v.dsum, &to->dsum}, {"dresidual", v.dresidual, &to->dresidual},
           {"dx", v.dx, &to->dx}};
  for (const auto& e : f) {
    const mamba_status st = resolve(who, e.name, e.given, d->dim, e.to);
    if (st != MAMBA_OK) return st;
    if (d->rows > 0 && *e.to > kMaxElems / d->rows)
      return fail(MAMBA_ERR_UNSUPPORTED, "%s: problem too large", who);
  }
  return MAMBA_OK;
}

bool same_rows(const Rows& a, const Rows& b) { return a.p == b.p && a.stride == b.stride && a.eb == b.eb; }

mamba_status norm_fwd_impl(const char* who, const mamba_norm_desc* d, const mamba_norm_strides* strides,
                           const void* x, const void* residual, const float* weight, void* out,
                           float* scale, void* sum, void* stream, bool quant) {
  NormRows s;
  mamba_status st = check_norm(who, d, quant);
  if (st != MAMBA_OK || (st = resolve_norm(who, d, strides, &s)) != MAMBA_OK) return st;
  if (!residual && (sum || d->residual_dtype != d->io_dtype))
    return fail(MAMBA_ERR_INVALID_ARG, "%s: without a residual sum must be NULL and both dtypes the same", who);
  if (d->rows == 0 || d->dim == 0) {
    // no channels: a row's only output is its scale, of an empty maximum
    if (d->rows == 0 || !quant || d->group != 0) return ok();
    return fail(MAMBA_ERR_UNSUPPORTED, "%s: dim 0 has no values to scale", who);
  }
  if ((st = check_present(who, {{"x", x, 0}, {"weight", weight, 0}, {quant ? "q" : "out", out, 0}})) != MAMBA_OK)
    return st;
  if (quant && (st = check_present(who, {{"scale", scale, 0}})) != MAMBA_OK) return st;
  if (residual && (st = check_present(who, {{"sum", sum, 0}})) != MAMBA_OK) return st;
  const size_t eb = io_bytes(d->io_dtype), rb = io_bytes(d->residual_dtype);
  const Rows ix{"x", x, d->rows, s.x, d->dim, eb}, ir{"residual", residual, d->rows, s.residual, d->dim, rb};
  const Rows iw = flat("weight", weight, d->dim, 4);
  const Rows oo{quant ? "q" : "out", out, d->rows, s.out, d->dim, quant ? 1 : eb};
  const Rows os{"sum", sum, d->rows, s.sum, d->dim, rb};
  const int64_t groups = d->group ? (d->dim + d->group - 1) / d->group : 1;
  const Rows oc = flat("scale", scale, d->rows * groups, 4);
  if (sum && same_rows(ir, os))  // in place: every element is read before it is written
    st = check_outputs(who, {ix, iw}, {oo, oc, os});
  else
    st = check_outputs(who, {ix, ir, iw}, {oo, oc, os});
  if (st != MAMBA_OK || (st = check_row_align(who, {ix, ir, iw, oo, os, oc})) != MAMBA_OK) return st;
  mscan::NormProblem p;
  p.x = x;
  p.residual = residual;
  p.weight = weight;
  p.out = out;
  p.scale = scale;
  p.sum = sum;
  p.rows = d->rows;
  p.dim = d->dim;
  p.group = d->group;
  p.io = d->io_dtype;
  p.res = d->residual_dtype;
  p.eps = d->eps;
  p.sx = s.x;
  p.sres = s.residual;
  p.ssum = s.sum;
  p.so = s.out;
  return launched(who, mscan::launch_norm(p, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

mamba_status mamba_rmsnorm_fwd(const mamba_norm_desc* d, const mamba_norm_strides* strides, const void* x,
                               const void* residual, const float* weight, void* out, void* sum,
                               void* stream) {
  return norm_fwd_impl("mamba_rmsnorm_fwd", d, strides, x, residual, weight, out, nullptr, sum, stream,
                       false);
}

mamba_status mamba_rmsnorm_quant_fwd(const mamba_norm_desc* d, const mamba_norm_strides* strides,
                                     const void* x, const void* residual, const float* weight, void* q,
                                     float* scale, void* sum, void* stream) {
  return norm_fwd_impl("mamba_rmsnorm_quant_fwd", d, strides, x, residual, weight, q, scale, sum, stream,
                       true);
}

size_t mamba_rmsnorm_bwd_workspace_size(const mamba_norm_desc* d) {
  if (check_norm("mamba_rmsnorm_bwd_workspace_size", d, false) != MAMBA_OK) return 0;
  return mscan::norm_bwd_workspace_bytes(d->rows, d->dim);
}

mamba_status mamba_rmsnorm_bwd(const mamba_norm_desc* d, const mamba_norm_strides* strides,
                               const void* sum, const float* weight, const void* dout, const void* dsum,
                               void* dresidual, void* dx, float* dweight, void* workspace,
                               size_t workspace_bytes, void* stream) {
  const char* who = "mamba_rmsnorm_bwd";
  NormRows s;
  mamba_status st = check_norm(who, d, false);
  if (st != MAMBA_OK || (st = resolve_norm(who, d, strides, &s)) != MAMBA_OK) return st;
  if (dx && d->io_dtype == d->residual_dtype)
    return fail(MAMBA_ERR_INVALID_ARG, "%s: dx must be NULL when both dtypes are the same", who);
  if (d->dim == 0) return ok();
  if ((st = check_present(who, {{"dweight", dweight, 0}})) != MAMBA_OK) return st;
  if (d->rows > 0 && (st = check_present(who, {{"sum", sum, 0}, {"weight", weight, 0}, {"dout", dout, 0},
                                               {"dresidual", dresidual, 0}})) != MAMBA_OK)
    return st;
  const size_t need = mamba_rmsnorm_bwd_workspace_size(d);
  if ((st = check_workspace(who, workspace, workspace_bytes, need)) != MAMBA_OK) return st;
  const size_t eb = io_bytes(d->io_dtype), rb = io_bytes(d->residual_dtype);
  const Rows is{"sum", sum, d->rows, s.sum, d->dim, rb}, io{"dout", dout, d->rows, s.out, d->dim, eb};
  const Rows id{"dsum", dsum, d->rows, s.dsum, d->dim, rb}, iw = flat("weight", weight, d->dim, 4);
  const Rows od{"dresidual", dresidual, d->rows, s.dresidual, d->dim, rb};
  const Rows ox{"dx", dx, d->rows, s.dx, d->dim, eb}, ow = flat("dweight", dweight, d->dim, 4);
  const Rows wk = flat("workspace", need ? workspace : nullptr, static_cast<int64_t>(need), 1);
  if (dsum && same_rows(id, od))
    st = check_outputs(who, {is, io, iw}, {od, ox, ow, wk});
  else
    st = check_outputs(who, {is, io, id, iw}, {od, ox, ow, wk});
  if (st != MAMBA_OK || (st = check_row_align(who, {is, io, id, iw, od, ox, ow})) != MAMBA_OK) return st;
  mscan::NormBwdProblem p;
  p.sum = sum;
  p.weight = weight;
  p.dout = dout;
  p.dsum = dsum;
  p.dresidual = dresidual;
  p.dx = dx;
  p.dweight = dweight;
  p.rows = d->rows;
  p.dim = d->dim;
  p.io = d->io_dtype;
  p.res = d->residual_dtype;
  p.eps = d->eps;
  p.ssum = s.sum;
  p.so = s.out;
  p.sdsum = s.dsum;
  p.sdres = s.dresidual;
  p.sdx = s.dx;
  return launched(who, mscan::launch_norm_bwd(p, workspace, static_cast<hipStream_t>(stream)));
}

size_t mamba_conv1d_bwd_workspace_size(const mamba_conv_desc* d) {
  if (check_conv_desc(d, "mamba_conv1d_bwd_workspace_size") != MAMBA_OK) return 0;
  return mscan::conv_bwd_workspace_bytes(d->batch, d->seqlen, d->dim, static_cast<int>(d->width));
}

mamba_status mamba_conv1d_bwd(const mamba_conv_desc* d, const void* xin, const float* weight,
                              const float* bias, const void* state_in, const void* dout,
                              const float* dstate_out, void* dxin, float* dweight, float* dbias,
                              float* dstate_in, void* workspace, size_t workspace_bytes, void* stream) {
  const char* who = "mamba_conv1d_bwd";
  mamba_status st = check_conv_desc(d, who);
  if (st != MAMBA_OK) return st;
  const int64_t rows = d->batch * d->dim, elems = rows * d->seqlen, W = d->width;
  if (d->dim == 0) return ok();
  if ((st = check_present(who, {{"dweight", dweight, 0}})) != MAMBA_OK) return st;
  if (rows > 0 && (st = check_present(who, {{"weight", weight, 0}})) != MAMBA_OK) return st;  // also of no tokens
  if (elems > 0 && (st = check_present(who, {{"xin", xin, 0}, {"dout", dout, 0}, {"dxin", dxin, 0}})) != MAMBA_OK)
    return st;
  const size_t need = mamba_conv1d_bwd_workspace_size(d);
  if ((st = check_workspace(who, workspace, workspace_bytes, need)) != MAMBA_OK) return st;
  const size_t eb = io_bytes(d->io_dtype);
  const int64_t states = rows * (W - 1);
  const Rows ix = flat("xin", xin, elems, eb), iw = flat("weight", weight, d->dim * W, 4);
  const Rows ib = flat("bias", bias, d->dim, 4), is = flat("state_in", state_in, states, eb);
  const Rows io = flat("dout", dout, elems, eb), il = flat("dstate_out", dstate_out, states, 4);
  const Rows ox = flat("dxin", dxin, elems, eb), ow = flat("dweight", dweight, d->dim * W, 4);
  const Rows ob = flat("dbias", dbias, d->dim, 4), os = flat("dstate_in", dstate_in, states, 4);
  const Rows wk = flat("workspace", need ? workspace : nullptr, static_cast<int64_t>(need), 1);
  if ((st = check_outputs(who, {ix, iw, ib, is, io, il}, {ox, ow, ob, os, wk})) != MAMBA_OK) return st;
  if ((st = check_row_align(who, {ix, iw, ib, is, io, il, ox, ow, ob, os})) != MAMBA_OK) return st;
  mscan::ConvBwdProblem p;
  p.xin = xin;
  p.weight = weight;
  p.bias = bias;
  p.state_in = W > 1 ? state_in : nullptr;
  p.dout = dout;
  p.dstate_out = W > 1 ? dstate_out : nullptr;
  p.dxin = dxin;
  p.dweight = dweight;
  p.dbias = dbias;
  p.dstate_in = W > 1 ? dstate_in : nullptr;
  p.batch = d->batch;
  p.seqlen = d->seqlen;
  p.dim = d->dim;
  p.width = static_cast<int>(W);
  p.io = d->io_dtype;
  return launched(who, mscan::launch_conv_bwd(p, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

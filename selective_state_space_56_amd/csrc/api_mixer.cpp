// C ABI of the matrix-state mixer's operators: argument validation and dispatch
// to the HIP kernels. See include/mixer/ for the contracts.
#include "mixer/mamba_linattn.h"
#include "mixer/mamba_qknorm.h"

#include <hip/hip_runtime_api.h>

#include <cmath>

#include "api_rows.h"
#include "mixer.h"

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
using mscan::launched;
using mscan::ok;
using mscan::resolve;
using mscan::Rows;

namespace {

constexpr uint32_t kLinattnFlags = MAMBA_LINATTN_HEAD_DECAY | MAMBA_LINATTN_PACKED | MAMBA_LINATTN_ZERO_REST;

static_assert(MAMBA_QKNORM_AXES == mscan::kQkNormAxes, "the header states the axes");

mamba_status check_head_size(const char* who, const char* name, int64_t size) {
  if (size <= 0) return fail(MAMBA_ERR_INVALID_ARG, "%s: %s %lld < 1", who, name, (long long)size);
  if (size % 8 || size > 256)
    return fail(MAMBA_ERR_UNSUPPORTED, "%s: %s %lld is not a multiple of 8 in 8 .. 256", who, name, (long long)size);
  return MAMBA_OK;
}

// Sizes of a valid descriptor.
mamba_status check_linattn(const char* who, const mamba_linattn_desc* d, mscan::LinattnSizes* to) {
  if (!d) return fail(MAMBA_ERR_INVALID_ARG, "%s: desc is NULL", who);
  if (d->batch < 0 || d->seqlen < 0 || d->nheads < 0)
    return fail(MAMBA_ERR_INVALID_ARG, "%s: negative size (batch=%lld seqlen=%lld nheads=%lld)", who,
                (long long)d->batch, (long long)d->seqlen, (long long)d->nheads);
  if (d->ngroups < 1 || d->nheads % d->ngroups)
    return fail(MAMBA_ERR_INVALID_ARG, "%s: ngroups %lld must be >= 1 and divide nheads %lld", who,
                (long long)d->ngroups, (long long)d->nheads);
  mamba_status st = check_io(who, "io_dtype", d->io_dtype);
  if (st != MAMBA_OK) return st;
  if (d->flags & ~kLinattnFlags) return fail(MAMBA_ERR_INVALID_ARG, "%s: unknown flags 0x%x", who, (unsigned)d->flags);
  const bool packed = d->flags & MAMBA_LINATTN_PACKED;
  if ((d->flags & MAMBA_LINATTN_ZERO_REST) && !packed)
    return fail(MAMBA_ERR_INVALID_ARG, "%s: ZERO_REST is for packed sequences", who);
  if (!std::isfinite(d->scale)) return fail(MAMBA_ERR_INVALID_ARG, "%s: scale is not finite", who);
  if ((st = check_head_size(who, "dkey", d->dkey)) != MAMBA_OK) return st;
  if ((st = check_head_size(who, "dvalue", d->dvalue)) != MAMBA_OK) return st;
  const int64_t most = mscan::kLinattnMaxRowHeads, states = mscan::kLinattnMaxStates;
  // rows times heads are counted in 31 bits, and so are the rows alone
  if (d->batch > states || d->nheads > states || d->batch * d->nheads > states || d->seqlen > most ||
      (!packed && d->batch > 0 && d->seqlen > most / d->batch))
    return fail(MAMBA_ERR_UNSUPPORTED, "%s: problem too large", who);
  const int64_t rows = packed ? d->seqlen : d->batch * d->seqlen;
  if (d->nheads > 0 && rows > most / d->nheads) return fail(MAMBA_ERR_UNSUPPORTED, "%s: problem too large", who);
  *to = mscan::LinattnSizes{d->batch, d->seqlen, rows, d->nheads, d->ngroups, d->dkey, d->dvalue, d->io_dtype, packed};
  return MAMBA_OK;
}

struct Stride {
  const char* name;
  int64_t given, row;
  int64_t* to;
};

mamba_status resolve_all(const char* who, int64_t rows, std::initializer_list<Stride> strides) {
  for (const Stride& s : strides) {
    const mamba_status st = resolve(who, s.name, s.given, s.row, s.to);
    if (st != MAMBA_OK) return st;
    if (rows > 0 && *s.to > kMaxElems / rows) return fail(MAMBA_ERR_UNSUPPORTED, "%s: problem too large", who);
  }
  return MAMBA_OK;
}

struct LinattnRows {
  int64_t q, k, v, out, dq, dk, dv;
};

mamba_status resolve_linattn(const char* who, const mscan::LinattnSizes& n, const mamba_linattn_strides* s,
                             LinattnRows* to) {
  const mamba_linattn_strides none = {0, 0, 0, 0, 0, 0, 0};
  const mamba_linattn_strides& v = s ? *s : none;
  const int64_t qk = n.groups * n.K, hv = n.heads * n.V;
  for (int64_t given : {qk, hv, v.q, v.k, v.v, v.out, v.dq, v.dk, v.dv})
    if (given > mscan::kMixMaxStride)
      return fail(MAMBA_ERR_UNSUPPORTED, "%s: rows of %lld elements are too far apart", who, (long long)given);
  return resolve_all(who, n.rows,
                     {{"q", v.q, qk, &to->q}, {"k", v.k, qk, &to->k}, {"v", v.v, hv, &to->v}, {"out", v.out, hv, &to->out},
                      {"dq", v.dq, qk, &to->dq}, {"dk", v.dk, qk, &to->dk}, {"dv", v.dv, hv, &to->dv}});
}

mamba_status check_offsets(const char* who, const mscan::LinattnSizes& n, const int64_t* offsets) {
  if (n.packed && !offsets) return fail(MAMBA_ERR_INVALID_ARG, "%s: offsets is NULL", who);
  if (!n.packed && offsets) return fail(MAMBA_ERR_INVALID_ARG, "%s: offsets without MAMBA_LINATTN_PACKED", who);
  return MAMBA_OK;
}

int64_t gates_of(const mamba_linattn_desc* d, int64_t rows) {
  return d->flags & MAMBA_LINATTN_HEAD_DECAY ? d->nheads : rows * d->nheads;
}

mscan::LinattnProblem problem(const mamba_linattn_desc* d, const mscan::LinattnSizes& n, const LinattnRows& s,
                              const void* q, const void* k, const void* v, const float* g, const float* h0,
                              const int64_t* offsets) {
  mscan::LinattnProblem p{};
  p.n = n;
  p.q = q;
  p.k = k;
  p.v = v;
  p.g = g;
  p.h0 = h0;
  p.offsets = offsets;
  p.scale = d->scale;
  p.head_decay = d->flags & MAMBA_LINATTN_HEAD_DECAY;
  p.zero_rest = d->flags & MAMBA_LINATTN_ZERO_REST;
  p.sq = s.q;
  p.sk = s.k;
  p.sv = s.v;
  p.so = s.out;
  return p;
}

struct QkNormRows {
  int64_t q, k, qo, ko, dq, dk;
};

mamba_status check_qknorm(const char* who, const mamba_qknorm_desc* d, const mamba_qknorm_strides* strides,
                          QkNormRows* to) {
  if (!d) return fail(MAMBA_ERR_INVALID_ARG, "%s: desc is NULL", who);
  if (d->tokens < 0 || d->qheads < 0 || d->kheads < 0)
    return fail(MAMBA_ERR_INVALID_ARG, "%s: negative size (tokens=%lld qheads=%lld kheads=%lld)", who,
                (long long)d->tokens, (long long)d->qheads, (long long)d->kheads);
  mamba_status st = check_io(who, "io_dtype", d->io_dtype);
  if (st != MAMBA_OK) return st;
  if (d->flags & ~MAMBA_QKNORM_INTERLEAVED)
    return fail(MAMBA_ERR_INVALID_ARG, "%s: unknown flags 0x%x", who, (unsigned)d->flags);
  if (!(d->eps >= 0.0f) || !std::isfinite(d->eps))
    return fail(MAMBA_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", who);
  if ((st = check_head_size(who, "headdim", d->headdim)) != MAMBA_OK) return st;
  if (d->rotary < 0 || d->rotary > d->headdim)
    return fail(MAMBA_ERR_INVALID_ARG, "%s: rotary %lld is not in 0 .. headdim", who, (long long)d->rotary);
  if (d->rotary % 8)
    return fail(MAMBA_ERR_UNSUPPORTED, "%s: rotary %lld is not a multiple of 8", who, (long long)d->rotary);
  if (d->naxes < 1 || d->naxes > MAMBA_QKNORM_AXES)
    return fail(MAMBA_ERR_INVALID_ARG, "%s: naxes %d is not in 1 .. %d", who, (int)d->naxes, MAMBA_QKNORM_AXES);
  int64_t pairs = 0;
  for (int a = 0; a < MAMBA_QKNORM_AXES; ++a) {
    if (d->sections[a] < 0 || d->sections[a] > 128 || (a >= d->naxes && d->sections[a] != 0))
      return fail(MAMBA_ERR_INVALID_ARG, "%s: sections[%d] is %lld", who, a, (long long)d->sections[a]);
    pairs += d->sections[a];
  }
  if (pairs != d->rotary / 2)
    return fail(MAMBA_ERR_INVALID_ARG, "%s: the sections hold %lld pairs, rotary / 2 is %lld", who, (long long)pairs,
                (long long)(d->rotary / 2));
  const int64_t most = (int64_t(1) << 31) - 1, heads = int64_t(1) << 20;
  if (d->tokens > most || d->qheads > heads || d->kheads > heads ||
      (d->qheads + d->kheads > 0 && d->tokens > most / (d->qheads + d->kheads)))
    return fail(MAMBA_ERR_UNSUPPORTED, "%s: problem too large", who);
  const mamba_qknorm_strides none = {0, 0, 0, 0, 0, 0};
  const mamba_qknorm_strides& v = strides ? *strides : none;
  const int64_t qw = d->qheads * d->headdim, kw = d->kheads * d->headdim;
  return resolve_all(who, d->tokens,
                     {{"q", v.q, qw, &to->q}, {"k", v.k, kw, &to->k}, {"qo", v.qo, qw, &to->qo}, {"ko", v.ko, kw, &to->ko},
                      {"dq", v.dq, qw, &to->dq}, {"dk", v.dk, kw, &to->dk}});
}

// Outputs against inputs, except that an output may be just `own`'s place.
mamba_status check_in_place(const char* who, const Rows& o, const Rows& own, std::initializer_list<Rows> others) {
  if (!(o.p == own.p && o.stride == own.stride) && collide(o, own))
    return fail(MAMBA_ERR_INVALID_ARG, "%s: %s overlaps %s", who, o.name, own.name);
  return check_outputs(who, others, {o});
}

mscan::QkNormProblem qk_problem(const mamba_qknorm_desc* d, const QkNormRows& s, const void* q, const void* k,
                                const int64_t* positions, const float* freqs, const float* q_weight,
                                const float* k_weight) {
  mscan::QkNormProblem p{};
  p.q = q;
  p.k = k;
  p.positions = positions;
  p.freqs = freqs;
  p.q_weight = q_weight;
  p.k_weight = k_weight;
  p.tokens = d->tokens;
  p.qheads = d->qheads;
  p.kheads = d->kheads;
  p.dim = d->headdim;
  p.rotary = d->rotary;
  int64_t end = 0;
  for (int a = 0; a < MAMBA_QKNORM_AXES; ++a) p.ends[a] = end += d->sections[a];
  p.io = d->io_dtype;
  p.interleaved = d->flags & MAMBA_QKNORM_INTERLEAVED;
  p.eps = d->eps;
  p.sq = s.q;
  p.sk = s.k;
  return p;
}

}  // namespace

extern "C" {

size_t mamba_linattn_workspace_size(const mamba_linattn_desc* d) {
  mscan::LinattnSizes n;
  if (check_linattn("mamba_linattn_workspace_size", d, &n) != MAMBA_OK) return 0;
  return mscan::linattn_fwd_workspace_bytes(n);
}

size_t mamba_linattn_bwd_workspace_size(const mamba_linattn_desc* d) {
  mscan::LinattnSizes n;
  if (check_linattn("mamba_linattn_bwd_workspace_size", d, &n) != MAMBA_OK) return 0;
  return mscan::linattn_bwd_workspace_bytes(n, d->flags & MAMBA_LINATTN_HEAD_DECAY);
}

mamba_status mamba_linattn_fwd(const mamba_linattn_desc* d, const mamba_linattn_strides* strides, const void* q,
                               const void* k, const void* v, const float* g, const float* h0, const int64_t* offsets,
                               void* out, float* last_state, void* workspace, size_t workspace_bytes, void* stream) {
  const char* who = "mamba_linattn_fwd";
  mscan::LinattnSizes n;
  LinattnRows s;
  mamba_status st = check_linattn(who, d, &n);
  if (st != MAMBA_OK || (st = resolve_linattn(who, n, strides, &s)) != MAMBA_OK) return st;
  const int64_t states = n.batch * n.heads * n.K * n.V;
  if (n.heads == 0 || (n.rows == 0 && (!last_state || states == 0))) return ok();
  if ((st = check_offsets(who, n, offsets)) != MAMBA_OK) return st;
  if (n.rows > 0 && (st = check_present(who, {{"q", q, 0}, {"k", k, 0}, {"v", v, 0}, {"g", g, 0}, {"out", out, 0}})) !=
                        MAMBA_OK)
    return st;
  const size_t need = mscan::linattn_fwd_workspace_bytes(n);
  if ((st = check_workspace(who, workspace, workspace_bytes, need)) != MAMBA_OK) return st;
  const size_t eb = io_bytes(d->io_dtype);
  const int64_t qk = n.groups * n.K, hv = n.heads * n.V;
  const Rows iq{"q", q, n.rows, s.q, qk, eb}, ik{"k", k, n.rows, s.k, qk, eb}, iv{"v", v, n.rows, s.v, hv, eb};
  const Rows ig = flat("g", g, n.rows > 0 ? gates_of(d, n.rows) : 0, 4), ih = flat("h0", h0, states, 4);
  const Rows ioff = flat("offsets", offsets, n.packed ? n.batch + 1 : 0, 8);
  const Rows oo{"out", out, n.rows, s.out, hv, eb}, ol = flat("last_state", last_state, states, 4);
  const Rows ow = flat("workspace", need ? workspace : nullptr, static_cast<int64_t>(need), 1);
  if ((st = check_outputs(who, {iq, ik, iv, ig, ih, ioff}, {oo, ol, ow})) != MAMBA_OK) return st;
  if ((st = check_row_align(who, {iq, ik, iv, ig, ih, ioff, oo, ol})) != MAMBA_OK) return st;
  mscan::LinattnProblem p = problem(d, n, s, q, k, v, g, h0, offsets);
  p.out = out;
  p.last_state = last_state;
  return launched(who, mscan::launch_linattn_fwd(p, workspace, static_cast<hipStream_t>(stream)));
}

mamba_status mamba_linattn_bwd(const mamba_linattn_desc* d, const mamba_linattn_strides* strides, const void* q,
                               const void* k, const void* v, const float* g, const float* h0, const int64_t* offsets,
                               const void* dout, const float* dlast, void* dq, void* dk, void* dv, float* dg, float* dh0,
                               void* workspace, size_t workspace_bytes, void* stream) {
  const char* who = "mamba_linattn_bwd";
  mscan::LinattnSizes n;
  LinattnRows s;
  mamba_status st = check_linattn(who, d, &n);
  if (st != MAMBA_OK || (st = resolve_linattn(who, n, strides, &s)) != MAMBA_OK) return st;
  const int64_t states = n.batch * n.heads * n.K * n.V;
  const bool shared = d->flags & MAMBA_LINATTN_HEAD_DECAY;
  if (n.heads == 0 || (n.rows == 0 && (!dh0 || states == 0) && !(dg && shared))) return ok();
  if ((st = check_offsets(who, n, offsets)) != MAMBA_OK) return st;
  if (n.rows > 0 &&
      (st = check_present(who, {{"q", q, 0}, {"k", k, 0}, {"v", v, 0}, {"g", g, 0}, {"dout", dout, 0}, {"dq", dq, 0},
                                {"dk", dk, 0}, {"dv", dv, 0}})) != MAMBA_OK)
    return st;
  const size_t need = mscan::linattn_bwd_workspace_bytes(n, shared);
  if ((st = check_workspace(who, workspace, workspace_bytes, need)) != MAMBA_OK) return st;
  const size_t eb = io_bytes(d->io_dtype);
  const int64_t qk = n.groups * n.K, hv = n.heads * n.V, gates = shared ? n.heads : n.rows * n.heads;
  const Rows iq{"q", q, n.rows, s.q, qk, eb}, ik{"k", k, n.rows, s.k, qk, eb}, iv{"v", v, n.rows, s.v, hv, eb};
  const Rows id{"dout", dout, n.rows, s.out, hv, eb};
  const Rows ig = flat("g", g, n.rows > 0 ? gates : 0, 4), ih = flat("h0", h0, states, 4);
  const Rows il = flat("dlast", dlast, states, 4), ioff = flat("offsets", offsets, n.packed ? n.batch + 1 : 0, 8);
  const Rows oq{"dq", dq, n.rows, s.dq, qk, eb}, ok_{"dk", dk, n.rows, s.dk, qk, eb};
  const Rows ov{"dv", dv, n.rows, s.dv, hv, eb};
  const Rows og = flat("dg", dg, gates, 4), oh = flat("dh0", dh0, states, 4);
  const Rows ow = flat("workspace", need ? workspace : nullptr, static_cast<int64_t>(need), 1);
  if ((st = check_outputs(who, {iq, ik, iv, ig, ih, id, il, ioff}, {oq, ok_, ov, og, oh, ow})) != MAMBA_OK) return st;
  if ((st = check_row_align(who, {iq, ik, iv, ig, ih, id, il, ioff, oq, ok_, ov, og, oh})) != MAMBA_OK) return st;
  mscan::LinattnBwdProblem p{};
  p.f = problem(d, n, s, q, k, v, g, h0, offsets);
  p.dout = dout;
  p.dlast = dlast;
  p.dq = dq;
  p.dk = dk;
  p.dv = dv;
  p.dg = dg;
  p.dh0 = dh0;
  p.sdq = s.dq;
  p.sdk = s.dk;
  p.sdv = s.dv;
  return launched(who, mscan::launch_linattn_bwd(p, workspace, static_cast<hipStream_t>(stream)));
}

mamba_status mamba_linattn_update(const mamba_linattn_desc* d, const mamba_linattn_strides* strides, float* state,
                                  const void* q, const void* k, const void* v, const float* g, void* out,
                                  void* stream) {
  const char* who = "mamba_linattn_update";
  mscan::LinattnSizes n;
  LinattnRows s;
  mamba_status st = check_linattn(who, d, &n);
  if (st != MAMBA_OK) return st;
  if (n.packed) return fail(MAMBA_ERR_INVALID_ARG, "%s: PACKED is for whole sequences", who);
  if (n.seqlen != 1) return fail(MAMBA_ERR_INVALID_ARG, "%s: seqlen %lld must be 1", who, (long long)n.seqlen);
  if ((st = resolve_linattn(who, n, strides, &s)) != MAMBA_OK) return st;
  const int64_t states = n.batch * n.heads * n.K * n.V;
  if (states == 0) return ok();
  if ((st = check_present(who, {{"state", state, 0}, {"q", q, 0}, {"k", k, 0}, {"v", v, 0}, {"g", g, 0},
                                {"out", out, 0}})) != MAMBA_OK)
    return st;
  const size_t eb = io_bytes(d->io_dtype);
  const int64_t qk = n.groups * n.K, hv = n.heads * n.V;
  const Rows iq{"q", q, n.rows, s.q, qk, eb}, ik{"k", k, n.rows, s.k, qk, eb}, iv{"v", v, n.rows, s.v, hv, eb};
  const Rows ig = flat("g", g, gates_of(d, n.rows), 4), os = flat("state", state, states, 4);
  const Rows oo{"out", out, n.rows, s.out, hv, eb};
  if ((st = check_outputs(who, {iq, ik, iv, ig}, {oo, os})) != MAMBA_OK) return st;
  if ((st = check_row_align(who, {iq, ik, iv, ig, os, oo})) != MAMBA_OK) return st;
  mscan::LinattnUpdateProblem p{};
  p.state = state;
  p.q = q;
  p.k = k;
  p.v = v;
  p.g = g;
  p.out = out;
  p.batch = n.batch;
  p.heads = n.heads;
  p.groups = n.groups;
  p.K = n.K;
  p.V = n.V;
  p.io = n.io;
  p.head_decay = d->flags & MAMBA_LINATTN_HEAD_DECAY;
  p.scale = d->scale;
  p.sq = s.q;
  p.sk = s.k;
  p.sv = s.v;
  p.so = s.out;
  return launched(who, mscan::launch_linattn_update(p, static_cast<hipStream_t>(stream)));
}

mamba_status mamba_qknorm_fwd(const mamba_qknorm_desc* d, const mamba_qknorm_strides* strides, const void* q,
                              const void* k, const int64_t* positions, const float* freqs, const float* q_weight,
                              const float* k_weight, void* qo, void* ko, void* stream) {
  const char* who = "mamba_qknorm_fwd";
  QkNormRows s;
  mamba_status st = check_qknorm(who, d, strides, &s);
  if (st != MAMBA_OK) return st;
  if (d->tokens == 0 || d->qheads + d->kheads == 0) return ok();
  if (d->qheads > 0 && (st = check_present(who, {{"q", q, 0}, {"qo", qo, 0}})) != MAMBA_OK) return st;
  if (d->kheads > 0 && (st = check_present(who, {{"k", k, 0}, {"ko", ko, 0}})) != MAMBA_OK) return st;
  if (d->rotary > 0 && (st = check_present(who, {{"positions", positions, 0}, {"freqs", freqs, 0}})) != MAMBA_OK)
    return st;
  const size_t eb = io_bytes(d->io_dtype);
  const int64_t qw = d->qheads * d->headdim, kw = d->kheads * d->headdim, n = d->tokens;
  const Rows iq{"q", q, n, s.q, qw, eb}, ik{"k", k, n, s.k, kw, eb};
  const Rows ip = flat("positions", positions, d->rotary ? n * d->naxes : 0, 8);
  const Rows fr = flat("freqs", freqs, d->rotary / 2, 4);
  const Rows wq = flat("q_weight", q_weight, d->headdim, 4), wk = flat("k_weight", k_weight, d->headdim, 4);
  const Rows oq{"qo", qo, n, s.qo, qw, eb}, ok_{"ko", ko, n, s.ko, kw, eb};
  if ((st = check_in_place(who, oq, iq, {ik, ip, fr, wq, wk})) != MAMBA_OK) return st;
  if ((st = check_in_place(who, ok_, ik, {iq, ip, fr, wq, wk})) != MAMBA_OK) return st;
  if ((st = check_outputs(who, {}, {oq, ok_})) != MAMBA_OK) return st;
  if ((st = check_row_align(who, {iq, ik, ip, fr, wq, wk, oq, ok_})) != MAMBA_OK) return st;
  mscan::QkNormProblem p = qk_problem(d, s, q, k, positions, freqs, q_weight, k_weight);
  p.qo = qo;
  p.ko = ko;
  p.sqo = s.qo;
  p.sko = s.ko;
  return launched(who, mscan::launch_qknorm_fwd(p, static_cast<hipStream_t>(stream)));
}

size_t mamba_qknorm_bwd_workspace_size(const mamba_qknorm_desc* d) {
  QkNormRows s;
  if (check_qknorm("mamba_qknorm_bwd_workspace_size", d, nullptr, &s) != MAMBA_OK) return 0;
  return mscan::qknorm_bwd_workspace_bytes(d->tokens, d->qheads, d->kheads, d->headdim);
}

mamba_status mamba_qknorm_bwd(const mamba_qknorm_desc* d, const mamba_qknorm_strides* strides, const void* q,
                              const void* k, const int64_t* positions, const float* freqs, const float* q_weight,
                              const float* k_weight, const void* dqo, const void* dko, void* dq, void* dk,
                              float* dq_weight, float* dk_weight, void* workspace, size_t workspace_bytes,
                              void* stream) {
  const char* who = "mamba_qknorm_bwd";
  QkNormRows s;
  mamba_status st = check_qknorm(who, d, strides, &s);
  if (st != MAMBA_OK) return st;
  const bool work = d->tokens > 0 && d->qheads + d->kheads > 0;
  if (!work && !dq_weight && !dk_weight) return ok();
  const int64_t n = work ? d->tokens : 0;
  if (n > 0 && d->qheads > 0 && (st = check_present(who, {{"q", q, 0}, {"dqo", dqo, 0}, {"dq", dq, 0}})) != MAMBA_OK)
    return st;
  if (n > 0 && d->kheads > 0 && (st = check_present(who, {{"k", k, 0}, {"dko", dko, 0}, {"dk", dk, 0}})) != MAMBA_OK)
    return st;
  if (n > 0 && d->rotary > 0 &&
      (st = check_present(who, {{"positions", positions, 0}, {"freqs", freqs, 0}})) != MAMBA_OK)
    return st;
  const size_t need = mscan::qknorm_bwd_workspace_bytes(d->tokens, d->qheads, d->kheads, d->headdim);
  if ((st = check_workspace(who, workspace, workspace_bytes, need)) != MAMBA_OK) return st;
  const size_t eb = io_bytes(d->io_dtype);
  const int64_t qw = d->qheads * d->headdim, kw = d->kheads * d->headdim;
  const Rows iq{"q", q, n, s.q, qw, eb}, ik{"k", k, n, s.k, kw, eb};
  const Rows ip = flat("positions", positions, d->rotary ? n * d->naxes : 0, 8);
  const Rows fr = flat("freqs", freqs, d->rotary / 2, 4);
  const Rows wq = flat("q_weight", q_weight, d->headdim, 4), wk = flat("k_weight", k_weight, d->headdim, 4);
  const Rows iy{"dqo", dqo, n, s.qo, qw, eb}, iz{"dko", dko, n, s.ko, kw, eb};
  const Rows oq{"dq", dq, n, s.dq, qw, eb}, ok_{"dk", dk, n, s.dk, kw, eb};
  const Rows gq = flat("dq_weight", dq_weight, d->headdim, 4), gk = flat("dk_weight", dk_weight, d->headdim, 4);
  const Rows ow = flat("workspace", need ? workspace : nullptr, static_cast<int64_t>(need), 1);
  if ((st = check_in_place(who, oq, iy, {iq, ik, ip, fr, wq, wk, iz})) != MAMBA_OK) return st;
  if ((st = check_in_place(who, ok_, iz, {iq, ik, ip, fr, wq, wk, iy})) != MAMBA_OK) return st;
  if ((st = check_outputs(who, {iq, ik, ip, fr, wq, wk, iy, iz}, {gq, gk, ow})) != MAMBA_OK) return st;
  if ((st = check_outputs(who, {}, {oq, ok_, gq, gk, ow})) != MAMBA_OK) return st;
  if ((st = check_row_align(who, {iq, ik, ip, fr, wq, wk, iy, iz, oq, ok_, gq, gk})) != MAMBA_OK) return st;
  mscan::QkNormProblem p = qk_problem(d, s, q, k, positions, freqs, q_weight, k_weight);
  p.dqo = dqo;
  p.dko = dko;
  p.qo = dq;
  p.ko = dk;
  p.dq_weight = dq_weight;
  p.dk_weight = dk_weight;
  p.sdqo = s.qo;
  p.sdko = s.ko;
  p.sqo = s.dq;
  p.sko = s.dk;
  return launched(who, mscan::launch_qknorm_bwd(p, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

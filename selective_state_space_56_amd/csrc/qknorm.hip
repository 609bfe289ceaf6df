// RMS norm of each query and key head with the rotation by the token's position,
// and its backward.
//
// Bound by HBM: every element is read once and written once (16384 tokens of 48 heads of
// 128 bf16: 86 us, 4.7 TB/s; the gradients of 40 heads 118 us, 4.3 TB/s). A head's row is D / 8
// lanes of 8 channels each, chosen so that a lane holds whole pairs: four
// channels i and the four rotary / 2 further on, or eight neighbours (interleaved
// pairs, and channels that are not turned). The row's sums go over those lanes, the
// rows of a wave are heads of one token, so that its angles are formed once for all
// of them.
//
// Angles: a = position x freq is exact in float64 for positions below 2^28 (24 bits
// of a float32 frequency); the nearest multiple of pi / 2 is taken off in two
// pieces, and sine and cosine of what is left, at most pi / 4, are their Taylor
// series to x^9 and x^10 (the next terms are 2e-9 and 1e-10).
#include "block_math.h"
#include "colsum.h"
#include "mamba_scan.h"
#include "mixer.h"

namespace mscan {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

struct Turn {
  float c[4], s[4];
};

__device__ __forceinline__ void turn_of(double a, float& c, float& s) {
  const double n = rint(a * 0.63661977236758134308);       // 2 / pi
  double y = fma(n, -1.57079632679489655800, a);           // pi / 2 in two pieces
  y = fma(n, -6.12323399573676603587e-17, y);
  const int quarter = static_cast<int>(static_cast<long long>(n) & 3);
  const float x = static_cast<float>(y), x2 = x * x;
  float ps = fmaf(x2, 1.0f / 362880.0f, -1.0f / 5040.0f);
  ps = fmaf(x2, ps, 1.0f / 120.0f);
  ps = fmaf(x2, ps, -1.0f / 6.0f);
  const float sn = fmaf(x * x2, ps, x);
  float pc = fmaf(x2, -1.0f / 3628800.0f, 1.0f / 40320.0f);
  pc = fmaf(x2, pc, -1.0f / 720.0f);
  pc = fmaf(x2, pc, 1.0f / 24.0f);
  pc = fmaf(x2, pc, -0.5f);
  const float cs = fmaf(x2, pc, 1.0f);
  const bool swap = quarter & 1;
  c = swap ? sn : cs;
  s = swap ? cs : sn;
  if (quarter == 1 || quarter == 2) c = -c;
  if (quarter >= 2) s = -s;
}

// A lane's place in a row: LP lanes (a power of two) per row, D / 8 of them with channels.
struct Place {
  int lane, at;            // at: the lane's first channel
  int gap;                 // channels from its first four to its last four
  bool has, turns;
};

__device__ __forceinline__ Place place_of(const QkNormProblem& p, int LP) {
  Place s;
  s.lane = threadIdx.x & (LP - 1);
  s.has = 8 * s.lane < p.dim;
  s.turns = 8 * s.lane < p.rotary;
  const bool apart = s.turns && !p.interleaved;
  s.at = apart ? 4 * s.lane : 8 * s.lane;
  s.gap = apart ? static_cast<int>(p.rotary / 2) : 4;
  return s;
}

__device__ __forceinline__ void angles_of(const QkNormProblem& p, const Place& s, int64_t token, Turn& t) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    t.c[e] = 1.0f;
    t.s[e] = 0.0f;
    if (!s.turns) continue;
    const int pair = 4 * s.lane + e;
    int axis = 0;
    while (axis < kQkNormAxes - 1 && pair >= p.ends[axis]) ++axis;
    turn_of(static_cast<double>(p.positions[axis * p.tokens + token]) * static_cast<double>(p.freqs[pair]), t.c[e], t.s[e]);
  }
}

template <class IO>
__device__ __forceinline__ void load_row(float (&x)[8], const typename IO::raw* row, const Place& s) {
  Piece<IO, 4> a, b;
  a.load(row + s.at);
  b.load(row + s.at + s.gap);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[e] = a.get(e);
    x[4 + e] = b.get(e);
  }
}

template <class IO>
__device__ __forceinline__ void store_row(const float (&x)[8], typename IO::raw* row, const Place& s) {
  Piece<IO, 4> a, b;
  const float lo[4] = {x[0], x[1], x[2], x[3]}, hi[4] = {x[4], x[5], x[6], x[7]};
  a.set(lo);
  b.set(hi);
  a.store(row + s.at);
  b.store(row + s.at + s.gap);
}

// The lane's pairs turned; BACK: by the angles' negatives.
template <bool BACK, bool INTER>
__device__ __forceinline__ void turn_row(float (&x)[8], const Turn& t, const Place& s) {
  if (!s.turns) return;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float sn = BACK ? -t.s[e] : t.s[e];
    const int i = INTER ? 2 * e : e, j = INTER ? 2 * e + 1 : 4 + e;
    const float a = x[i], b = x[j];
    x[i] = fmaf(a, t.c[e], -b * sn);
    x[j] = fmaf(b, t.c[e], a * sn);
  }
}

__device__ __forceinline__ float over_row(float v, int LP) {
  for (int off = LP >> 1; off > 0; off >>= 1) v += __shfl_xor(v, off);
  return v;
}

__device__ __forceinline__ void load_weight(float (&w)[8], const float* from, const Place& s) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
    w[e] = from && s.has ? from[s.at + (e < 4 ? e : s.gap + e - 4)] : 1.0f;
}

// 1 / sqrt, to float32
__device__ __forceinline__ float rstd_of(float ms, float eps) { return 1.0f / sqrtf(ms + eps); }

// A wave takes `each` heads of one token at a time, 64 / LP of them side by side, one row per
// lane in flight. (Rows loaded two, three and four ahead cost registers and with them waves:
// 89 us became 94, 94 and 98, and 194 for a training step 266, 277 and 285. INTER as a
// run-time choice took 97 and 213. Queries and keys in workgroups of their own need fewer
// registers, one weight's, but took 91 and 207: a token's rows are no longer read together.)
template <class IO, bool INTER>
__global__ __launch_bounds__(kThreads) void qknorm_fwd_kernel(QkNormProblem p, int LP, int each, int64_t units, int parts) {
  using raw = typename IO::raw;
  const Place s = place_of(p, LP);
  const int sub = (threadIdx.x & 63) / LP, rows = 64 / LP;
  const int64_t heads = p.qheads + p.kheads;
  float wq[8], wk[8];
  load_weight(wq, p.q_weight, s);
  load_weight(wk, p.k_weight, s);
  const float scale = 1.0f / static_cast<float>(p.dim);
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWaves + (threadIdx.x >> 6); u < units;
       u += static_cast<int64_t>(gridDim.x) * kWaves) {
    const int64_t token = u / parts, h0 = u % parts * each;
    const int64_t h1 = h0 + each < heads ? h0 + each : heads;
    Turn t;
    angles_of(p, s, token, t);
    for (int64_t h = h0 + sub; h - sub < h1; h += rows) {
      const bool on = h < h1 && s.has, key = h >= p.qheads;
      const int64_t at = (key ? h - p.qheads : h) * p.dim;
      float x[8] = {};
      if (on)
        load_row<IO>(x, key ? static_cast<const raw*>(p.k) + token * p.sk + at : static_cast<const raw*>(p.q) + token * p.sq + at, s);
      float sq = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) sq = fmaf(x[e], x[e], sq);
      const float r = rstd_of(over_row(sq, LP) * scale, p.eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = x[e] * r * (key ? wk[e] : wq[e]);
      turn_row<false, INTER>(x, t, s);
      if (on)
        store_row<IO>(x, key ? static_cast<raw*>(p.ko) + token * p.sko + at : static_cast<raw*>(p.qo) + token * p.sqo + at, s);
    }
  }
}

template <class IO, bool INTER>
__global__ __launch_bounds__(kThreads) void qknorm_bwd_kernel(QkNormProblem p, int LP, int each, int64_t units, int parts,
                                                              float* sums) {
  using raw = typename IO::raw;
  __shared__ float s_sum[kThreads][17];
  const Place s = place_of(p, LP);
  const int sub = (threadIdx.x & 63) / LP, rows = 64 / LP;
  const int64_t heads = p.qheads + p.kheads;
  float wq[8], wk[8], dwq[8] = {}, dwk[8] = {};
  load_weight(wq, p.q_weight, s);
  load_weight(wk, p.k_weight, s);
  const float scale = 1.0f / static_cast<float>(p.dim);
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWaves + (threadIdx.x >> 6); u < units;
       u += static_cast<int64_t>(gridDim.x) * kWaves) {
    const int64_t token = u / parts, h0 = u % parts * each;
    const int64_t h1 = h0 + each < heads ? h0 + each : heads;
    Turn t;
    angles_of(p, s, token, t);
    for (int64_t h = h0 + sub; h - sub < h1; h += rows) {
      const bool on = h < h1 && s.has, key = h >= p.qheads;
      const int64_t at = (key ? h - p.qheads : h) * p.dim;
      float x[8] = {}, dy[8] = {};
      if (on) {
        load_row<IO>(x, key ? static_cast<const raw*>(p.k) + token * p.sk + at : static_cast<const raw*>(p.q) + token * p.sq + at, s);
        load_row<IO>(dy, key ? static_cast<const raw*>(p.dko) + token * p.sdko + at
                             : static_cast<const raw*>(p.dqo) + token * p.sdqo + at, s);
      }
      turn_row<true, INTER>(dy, t, s);
      float sq = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) sq = fmaf(x[e], x[e], sq);
      const float r = rstd_of(over_row(sq, LP) * scale, p.eps);
      float dot = 0.0f, wu[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] *= r;
        wu[e] = dy[e] * (key ? wk[e] : wq[e]);
        dot = fmaf(wu[e], x[e], dot);
        const float d = on ? dy[e] * x[e] : 0.0f;  // (no row: r may be infinite)
        dwq[e] += key ? 0.0f : d;
        dwk[e] += key ? d : 0.0f;
      }
      dot = over_row(dot, LP) * scale;
#pragma unroll
      for (int e = 0; e < 8; ++e) wu[e] = r * fmaf(-x[e], dot, wu[e]);
      if (on)
        store_row<IO>(wu, key ? static_cast<raw*>(p.ko) + token * p.sko + at : static_cast<raw*>(p.qo) + token * p.sqo + at, s);
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    s_sum[threadIdx.x][e] = dwq[e];
    s_sum[threadIdx.x][8 + e] = dwk[e];
  }
  __syncthreads();
  // thread l < LP adds lane l's sums of every row and wave, in order
  if (threadIdx.x < LP && s.has) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float a = 0.0f, b = 0.0f;
      for (int i = threadIdx.x; i < kThreads; i += LP) {
        a += s_sum[i][e];
        b += s_sum[i][8 + e];
      }
      const int c = s.at + (e < 4 ? e : s.gap + e - 4);
      sums[blockIdx.x * 2 * p.dim + c] = a;
      sums[blockIdx.x * 2 * p.dim + p.dim + c] = b;
    }
  }
}

struct StoreWeights {
  float* q;
  float* k;
  int64_t dim;
  __device__ __forceinline__ void operator()(int64_t c, float v) const {
    if (c < dim) {
      if (q) q[c] = v;
    } else if (k) {
      k[c - dim] = v;
    }
  }
};

int64_t compute_units() {
  int dev = 0, n = 0;
  if (hipGetDevice(&dev) != hipSuccess ||
      hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0)
    n = 256;
  return n;
}

struct Plan {
  int LP, each, parts;
  int64_t units, groups;
};

// A token's heads are shared by several waves where there are few tokens.
Plan plan_of(int64_t tokens, int64_t heads, int64_t dim, int64_t waves) {
  Plan s;
  s.LP = 1;
  while (8 * s.LP < dim) s.LP *= 2;
  const int64_t rows = 64 / s.LP, rounds = (heads + rows - 1) / rows;
  int64_t parts = (waves + tokens - 1) / tokens;
  if (parts > rounds) parts = rounds;
  const int64_t per = (rounds + parts - 1) / parts;
  s.each = static_cast<int>(per * rows);
  s.parts = static_cast<int>((rounds + per - 1) / per);
  s.units = tokens * s.parts;
  s.groups = (s.units + kWaves - 1) / kWaves;
  return s;
}

constexpr int kFwdWavesPerCu = 32, kBwdGroupsPerCu = 4;

Plan bwd_plan(int64_t tokens, int64_t heads, int64_t dim) {
  const int64_t most = compute_units() * kBwdGroupsPerCu;
  Plan s = plan_of(tokens, heads, dim, most * kWaves);
  if (s.groups > most) s.groups = most;
  return s;
}

}  // namespace

hipError_t launch_qknorm_fwd(const QkNormProblem& p, hipStream_t stream) {
  const Plan s = plan_of(p.tokens, p.qheads + p.kheads, p.dim, compute_units() * kFwdWavesPerCu);
  const dim3 grid(static_cast<unsigned>(s.groups < (1 << 22) ? s.groups : 1 << 22));
  const auto kernel = p.io == MAMBA_BF16 ? p.interleaved ? qknorm_fwd_kernel<Bf16Io, true> : qknorm_fwd_kernel<Bf16Io, false>
                      : p.interleaved    ? qknorm_fwd_kernel<F32Io, true>
                                         : qknorm_fwd_kernel<F32Io, false>;
  hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, stream, p, s.LP, s.each, s.units, s.parts);
  return hipGetLastError();
}

size_t qknorm_bwd_workspace_bytes(int64_t tokens, int64_t qheads, int64_t kheads, int64_t dim) {
  if (tokens == 0 || qheads + kheads == 0) return 0;
  return static_cast<size_t>(bwd_plan(tokens, qheads + kheads, dim).groups) * 2 * dim * 4;
}

hipError_t launch_qknorm_bwd(const QkNormProblem& p, void* workspace, hipStream_t stream) {
  int64_t groups = 0;
  float* sums = static_cast<float*>(workspace);
  if (p.tokens > 0 && p.qheads + p.kheads > 0) {
    const Plan s = bwd_plan(p.tokens, p.qheads + p.kheads, p.dim);
    const dim3 grid(static_cast<unsigned>(s.groups));
    groups = s.groups;
    const auto kernel = p.io == MAMBA_BF16 ? p.interleaved ? qknorm_bwd_kernel<Bf16Io, true> : qknorm_bwd_kernel<Bf16Io, false>
                        : p.interleaved    ? qknorm_bwd_kernel<F32Io, true>
                                           : qknorm_bwd_kernel<F32Io, false>;
    hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, stream, p, s.LP, s.each, s.units, s.parts, sums);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!p.dq_weight && !p.dk_weight) return hipSuccess;
  return launch_colsum(sums, groups, 2 * p.dim, StoreWeights{p.dq_weight, p.dk_weight, p.dim}, stream);
}

}  // namespace mscan

// RMS norm of a block's entry: y = s rstd w with s = x + residual and
// rstd = 1 / sqrt(mean s^2 + eps), as an io output or as e4m3 with scales, and
// its backward.
#include "block.h"
#include "block_math.h"
#include "colsum.h"

namespace mscan {

namespace {

constexpr int kThreads = 256;
constexpr float kE4m3Max = 448.0f;
constexpr float kTiny = 0x1p-100f;

__device__ __forceinline__ float load_any(const void* p, int io, int64_t i) {
  return io == kIoBf16 ? Bf16Io::load(static_cast<const uint16_t*>(p) + i) : static_cast<const float*>(p)[i];
}

__device__ __forceinline__ void store_any(void* p, int io, int64_t i, float v) {
  if (io == kIoBf16)
    static_cast<uint16_t*>(p)[i] = Bf16Io::from_f32(v);
  else
    static_cast<float*>(p)[i] = v;
}

__device__ __forceinline__ float rounded(int io, float v) {
  return io == kIoBf16 ? Bf16Io::to_f32(Bf16Io::from_f32(v)) : v;
}

// Sum (or maximum) over the workgroup, the same in every thread.
template <bool MAX>
__device__ float over_block(float v, float* scratch) {
  const int t = threadIdx.x;
  __syncthreads();
  scratch[t] = v;
  __syncthreads();
  for (int k = kThreads / 2; k > 0; k /= 2) {
    if (t < k) scratch[t] = MAX ? fmaxf(scratch[t], scratch[t + k]) : scratch[t] + scratch[t + k];
    __syncthreads();
  }
  return scratch[0];
}

__device__ __forceinline__ uint8_t e4m3(float v) {
  v = v > kE4m3Max ? kE4m3Max : v < -kE4m3Max ? -kE4m3Max : v;  // keeps NaN
  return static_cast<uint8_t>(__builtin_amdgcn_cvt_pk_fp8_f32(v, v, 0, false) & 0xff);
}

// One workgroup per row, the row read again for each of its uses.
__device__ void norm_row(const NormProblem& p, int64_t row, float* scratch) {
  const auto s_at = [&](int64_t d) {
    if (p.sum) return load_any(p.sum, p.res, row * p.ssum + d);
    return load_any(p.x, p.io, row * p.sx + d);
  };
  float ss = 0.0f;
  for (int64_t d = threadIdx.x; d < p.dim; d += kThreads) {
    float s = load_any(p.x, p.io, row * p.sx + d);
    if (p.residual) {
      s = rounded(p.res, s + load_any(p.residual, p.res, row * p.sres + d));
      store_any(p.sum, p.res, row * p.ssum + d, s);
    }
    ss = fmaf(s, s, ss);
  }
  const float rstd = 1.0f / sqrtf(over_block<false>(ss, scratch) / static_cast<float>(p.dim) + p.eps);
  if (!p.scale) {
    for (int64_t d = threadIdx.x; d < p.dim; d += kThreads)
      store_any(p.out, p.io, row * p.so + d, s_at(d) * rstd * p.weight[d]);
    return;
  }
  const int64_t group = p.group ? p.group : p.dim, groups = (p.dim + group - 1) / group;
  for (int64_t k = 0; k < groups; ++k) {
    const int64_t end = (k + 1) * group < p.dim ? (k + 1) * group : p.dim;
    float top = kTiny;
    for (int64_t d = k * group + threadIdx.x; d < end; d += kThreads)
      top = fmaxf(top, fabsf(s_at(d) * rstd * p.weight[d]));
    const float scale = over_block<true>(top, scratch) / kE4m3Max;
    for (int64_t d = k * group + threadIdx.x; d < end; d += kThreads)
      static_cast<uint8_t*>(p.out)[row * p.so + d] = e4m3(s_at(d) * rstd * p.weight[d] / scale);
    if (threadIdx.x == 0) p.scale[row * groups + k] = scale;
  }
}

constexpr int64_t kMaxGrid = 65536;

__global__ __launch_bounds__(kThreads) void norm_kernel(NormProblem p) {
  __shared__ float scratch[kThreads];
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) norm_row(p, row, scratch);
}

constexpr int64_t kParts = 256;  // workgroups of the backward, each with a part of dweight

__global__ __launch_bounds__(kThreads) void norm_bwd_kernel(NormBwdProblem p, float* parts) {
  __shared__ float scratch[kThreads];
  float* part = parts + blockIdx.x * p.dim;
  for (int64_t d = threadIdx.x; d < p.dim; d += kThreads) part[d] = 0.0f;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    float ss = 0.0f, su = 0.0f;
    for (int64_t d = threadIdx.x; d < p.dim; d += kThreads) {
      const float s = load_any(p.sum, p.res, row * p.ssum + d);
      ss = fmaf(s, s, ss);
      su = fmaf(s, p.weight[d] * load_any(p.dout, p.io, row * p.so + d), su);
    }
    const float n = static_cast<float>(p.dim);
    const float rstd = 1.0f / sqrtf(over_block<false>(ss, scratch) / n + p.eps);
    const float mean = over_block<false>(su, scratch) * rstd / n;
    for (int64_t d = threadIdx.x; d < p.dim; d += kThreads) {
      const float norm = load_any(p.sum, p.res, row * p.ssum + d) * rstd;
      const float dy = load_any(p.dout, p.io, row * p.so + d);
      float ds = rstd * (p.weight[d] * dy - norm * mean);
      if (p.dsum) ds += load_any(p.dsum, p.res, row * p.sdsum + d);
      store_any(p.dresidual, p.res, row * p.sdres + d, ds);
      if (p.dx) store_any(p.dx, p.io, row * p.sdx + d, ds);
      part[d] = fmaf(dy, norm, part[d]);
    }
  }
}

}  // namespace

hipError_t launch_norm(const NormProblem& p, hipStream_t stream) {
  hipLaunchKernelGGL(norm_kernel, dim3(static_cast<unsigned>(p.rows < kMaxGrid ? p.rows : kMaxGrid)), dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

size_t norm_bwd_workspace_bytes(int64_t rows, int64_t dim) {
  const int64_t parts = rows < kParts ? rows : kParts;
  return (static_cast<size_t>(parts * dim) * 4 + 255) / 256 * 256;
}

hipError_t launch_norm_bwd(const NormBwdProblem& p, void* workspace, hipStream_t stream) {
  const int64_t n = p.rows < kParts ? p.rows : kParts;
  float* parts = static_cast<float*>(workspace);
  if (n > 0) {
    hipLaunchKernelGGL(norm_bwd_kernel, dim3(static_cast<unsigned>(n)), dim3(kThreads), 0, stream, p, parts);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return launch_colsum(parts, n, p.dim, StoreFlat{p.dweight}, stream);
}

}  // namespace mscan

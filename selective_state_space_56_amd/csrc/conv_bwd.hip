// Backward of the causal depthwise convolution + SiLU:
//   v_t = bias + sum_j w_j x_{t-(W-1)+j},  dv_t = dout_t silu'(v_t),
//   dx_t = sum_j w_j dv_{t+(W-1)-j},  dw_j = sum_t dv_t x_{t-(W-1)+j},  dbias = sum_t dv_t.
#include "block.h"
#include "block_math.h"
#include "colsum.h"

namespace mscan {

namespace {

constexpr int kThreads = 64;
constexpr int kSpan = 64;  // time steps per thread

// One channel of one batch row per thread, kSpan steps: v and dv are formed in
// time order and kept for W steps; a step's dx is ready W - 1 steps later, so a
// span reads W - 1 steps past its end (and those add nothing to its dw).
template <class IO, int W>
__global__ __launch_bounds__(kThreads) void conv_bwd_kernel(ConvBwdProblem p, float* parts) {
  using raw = typename IO::raw;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (c >= p.dim) return;
  const int64_t b = blockIdx.z;
  const int64_t t0 = static_cast<int64_t>(blockIdx.y) * kSpan;
  const int64_t t1 = t0 + kSpan < p.seqlen ? t0 + kSpan : p.seqlen;
  const raw* xin = static_cast<const raw*>(p.xin);
  const raw* sin = static_cast<const raw*>(p.state_in);
  float w[W], dw[W], x[W], dv[W];  // x[j] = input t - (W-1) + j, dv[j] = dv at t - j
  const float bias = p.bias ? p.bias[c] : 0.0f;
#pragma unroll
  for (int j = 0; j < W; ++j) {
    w[j] = p.weight[c * W + j];
    dw[j] = 0.0f;
    x[j] = 0.0f;
    dv[j] = 0.0f;
  }
  const auto input = [&](int64_t t) {
    if (t >= 0) return IO::load(xin + (b * p.seqlen + t) * p.dim + c);
    return sin ? IO::load(sin + (b * p.dim + c) * (W - 1) + (W - 1) + t) : 0.0f;
  };
  float db = 0.0f;
#pragma unroll
  for (int j = 0; j < W - 1; ++j) x[j + 1] = input(t0 - (W - 1) + j);
  // steps t0 .. t1 + W - 2: the inputs at t - (W-1) get their gradient at step t.
  // The first span also covers the state's inputs, the last those up to the end.
  for (int64_t t = t0; t < t1 + W - 1; ++t) {
#pragma unroll
    for (int j = 0; j + 1 < W; ++j) x[j] = x[j + 1];
#pragma unroll
    for (int j = W - 1; j > 0; --j) dv[j] = dv[j - 1];
    dv[0] = 0.0f;
    if (t < p.seqlen) {
      x[W - 1] = input(t);
      float v = bias;
#pragma unroll
      for (int j = 0; j < W; ++j) v = fmaf(w[j], x[j], v);
      const float sig = sigmoid_f(v);
      dv[0] = IO::load(static_cast<const raw*>(p.dout) + (b * p.seqlen + t) * p.dim + c) * sig *
              fmaf(v, 1.0f - sig, 1.0f);
      if (t < t1) {
        db += dv[0];
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j] = fmaf(dv[0], x[j], dw[j]);
      }
    }
    const int64_t at = t - (W - 1);  // this span's own inputs only; the first span's state inputs too
    if (at < t0 && blockIdx.y > 0) continue;
    float d = 0.0f;
#pragma unroll
    for (int j = 0; j < W; ++j) d = fmaf(w[j], dv[j], d);
    // the forward's last W - 1 inputs are its state_out
    const int64_t slot = at - (p.seqlen - (W - 1));
    if (W > 1 && slot >= 0 && p.dstate_out) d += p.dstate_out[(b * p.dim + c) * (W - 1) + slot];
    if (at >= 0)
      static_cast<raw*>(p.dxin)[(b * p.seqlen + at) * p.dim + c] = IO::from_f32(d);
    else if (p.dstate_in)
      p.dstate_in[(b * p.dim + c) * (W - 1) + (W - 1) + at] = d;
  }
  float* part = parts + (b * gridDim.y + blockIdx.y) * (W + 1) * p.dim;
#pragma unroll
  for (int j = 0; j < W; ++j) part[j * p.dim + c] = dw[j];
  part[W * p.dim + c] = db;
}

// column j * dim + c of the parts: tap j's sum, or the bias's for j = width
struct StoreTaps {
  float* dweight;
  float* dbias;
  int64_t dim;
  int width;
  __device__ __forceinline__ void operator()(int64_t i, float v) const {
    const int64_t j = i / dim, c = i % dim;
    if (j < width)
      dweight[c * width + j] = v;
    else if (dbias)
      dbias[c] = v;
  }
};

int64_t spans_of(int64_t seqlen) { return seqlen > 0 ? (seqlen + kSpan - 1) / kSpan : 1; }

template <class IO>
hipError_t launch_io(const ConvBwdProblem& p, float* parts, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>((p.dim + kThreads - 1) / kThreads),
                  static_cast<unsigned>(spans_of(p.seqlen)), static_cast<unsigned>(p.batch));
  switch (p.width) {
    case 1: hipLaunchKernelGGL((conv_bwd_kernel<IO, 1>), grid, dim3(kThreads), 0, stream, p, parts); break;
    case 2: hipLaunchKernelGGL((conv_bwd_kernel<IO, 2>), grid, dim3(kThreads), 0, stream, p, parts); break;
    case 3: hipLaunchKernelGGL((conv_bwd_kernel<IO, 3>), grid, dim3(kThreads), 0, stream, p, parts); break;
    case 4: hipLaunchKernelGGL((conv_bwd_kernel<IO, 4>), grid, dim3(kThreads), 0, stream, p, parts); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace

size_t conv_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim, int width) {
  return (static_cast<size_t>(batch * spans_of(seqlen) * (width + 1) * dim) * 4 + 255) / 256 * 256;
}

hipError_t launch_conv_bwd(const ConvBwdProblem& p, void* workspace, hipStream_t stream) {
  float* parts = static_cast<float*>(workspace);
  if (p.batch > 0) {
    const hipError_t e = p.io == kIoBf16 ? launch_io<Bf16Io>(p, parts, stream) : launch_io<F32Io>(p, parts, stream);
    if (e != hipSuccess) return e;
  }
  return launch_colsum(parts, p.batch * spans_of(p.seqlen), (p.width + 1) * p.dim,
                       StoreTaps{p.dweight, p.dbias, p.dim, p.width}, stream);
}

}  // namespace mscan

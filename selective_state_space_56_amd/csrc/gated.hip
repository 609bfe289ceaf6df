// Gated linear recurrence, one state per channel:
//   a_t = exp(A sigmoid(r_t)),  h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(g_t) x_t,
// over full sequences, its backward, and one decode token.
#include "block.h"
#include "block_math.h"
#include "colsum.h"

namespace mscan {

namespace {

constexpr int kLanes = 64;

// One lane per channel of one batch row, step by step.
template <class IO>
__global__ __launch_bounds__(kLanes) void gated_fwd_kernel(GatedProblem p) {
  using raw = typename IO::raw;
  const unsigned tiles = static_cast<unsigned>((p.dim + kLanes - 1) / kLanes);
  const int64_t c = static_cast<int64_t>(blockIdx.x % tiles) * kLanes + threadIdx.x, b = blockIdx.x / tiles;
  if (c >= p.dim) return;
  const float A = p.A ? p.A[c] : 0.0f;
  float h = p.h0 ? p.h0[b * p.dim + c] : 0.0f;
  const int64_t marks = (p.seqlen + kGatedCheckpoint - 1) / kGatedCheckpoint;
  for (int64_t t = 0; t < p.seqlen; ++t) {
    const int64_t row = b * p.seqlen + t;
    if (p.checkpoints && t % kGatedCheckpoint == 0)
      p.checkpoints[(b * marks + t / kGatedCheckpoint) * p.dim + c] = h;
    const float x = IO::load(static_cast<const raw*>(p.x) + row * p.sx + c);
    const float sr = sigmoid_f(IO::load(static_cast<const raw*>(p.r) + row * p.sr + c));
    const float sg = sigmoid_f(IO::load(static_cast<const raw*>(p.g) + row * p.sg + c));
    float a, w;
    decay_gain(A * sr, a, w);
    h = p.reset && p.reset[row] ? sg * x : fmaf(a, h, w * (sg * x));
    static_cast<raw*>(p.out)[row * p.so + c] = IO::from_f32(h);
  }
  if (p.last_state) p.last_state[b * p.dim + c] = h;
}

// Checkpoint to checkpoint, from the last: the states of the span are
// recomputed into LDS, then the adjoint runs back through it. One part of dA
// per batch row.
template <class IO>
__global__ __launch_bounds__(kLanes) void gated_bwd_kernel(GatedBwdProblem p, float* parts) {
  using raw = typename IO::raw;
  __shared__ float before[kGatedCheckpoint][kLanes];
  const unsigned tiles = static_cast<unsigned>((p.dim + kLanes - 1) / kLanes);
  const int64_t c = static_cast<int64_t>(blockIdx.x % tiles) * kLanes + threadIdx.x, b = blockIdx.x / tiles;
  if (c >= p.dim) return;
  const float A = p.A ? p.A[c] : 0.0f;
  float carry = p.dlast ? p.dlast[b * p.dim + c] : 0.0f, dA = 0.0f;
  const int64_t marks = (p.seqlen + kGatedCheckpoint - 1) / kGatedCheckpoint;
  for (int64_t k = marks - 1; k >= 0; --k) {
    const int64_t t0 = k * kGatedCheckpoint;
    const int64_t t1 = t0 + kGatedCheckpoint < p.seqlen ? t0 + kGatedCheckpoint : p.seqlen;
    float h = p.checkpoints[(b * marks + k) * p.dim + c];
    for (int pass = 0; pass < 2; ++pass) {
      for (int64_t i = 0; i < t1 - t0; ++i) {
        const int64_t t = pass ? t1 - 1 - i : t0 + i;
        const int64_t row = b * p.seqlen + t;
        const float x = IO::load(static_cast<const raw*>(p.x) + row * p.sx + c);
        const float sr = sigmoid_f(IO::load(static_cast<const raw*>(p.r) + row * p.sr + c));
        const float sg = sigmoid_f(IO::load(static_cast<const raw*>(p.g) + row * p.sg + c));
        const bool start = p.reset && p.reset[row];
        float a, w;
        decay_gain(A * sr, a, w);
        if (start) w = 1.0f;
        if (pass == 0) {
          before[t - t0][threadIdx.x] = h;
          h = start ? sg * x : fmaf(a, h, w * (sg * x));
          continue;
        }
        const float lam = IO::load(static_cast<const raw*>(p.dout) + row * p.so + c) + carry;
        const float slope = w > 0.0f ? a * a * hw_rcp(w) : 0.0f;
        const float dv = start ? 0.0f : lam * fmaf(a, before[t - t0][threadIdx.x], -slope * sg * x);
        carry = start ? 0.0f : a * lam;
        dA = fmaf(dv, sr, dA);
        static_cast<raw*>(p.dx)[row * p.sdx + c] = IO::from_f32(lam * w * sg);
        static_cast<raw*>(p.dg)[row * p.sdg + c] = IO::from_f32(lam * w * x * sg * (1.0f - sg));
        static_cast<raw*>(p.dr)[row * p.sdr + c] = IO::from_f32(dv * A * sr * (1.0f - sr));
      }
    }
  }
  if (p.dh0) p.dh0[b * p.dim + c] = carry;
  parts[b * p.dim + c] = dA;
}

// One decode token per (batch row, channel).
template <class IO>
__global__ __launch_bounds__(256) void gated_update_kernel(GatedUpdateProblem p) {
  using raw = typename IO::raw;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= p.batch * p.dim) return;
  const int64_t b = i / p.dim, c = i % p.dim;
  const float x = IO::load(static_cast<const raw*>(p.x) + b * p.sx + c);
  const float sr = sigmoid_f(IO::load(static_cast<const raw*>(p.r) + b * p.sr + c));
  const float sg = sigmoid_f(IO::load(static_cast<const raw*>(p.g) + b * p.sg + c));
  float a, w;
  decay_gain(p.A[c] * sr, a, w);
  const float h = fmaf(a, p.state[i], w * (sg * x));
  p.state[i] = h;
  static_cast<raw*>(p.out)[b * p.so + c] = IO::from_f32(h);
}

dim3 channel_grid(int64_t batch, int64_t dim) {
  return dim3(static_cast<unsigned>((dim + kLanes - 1) / kLanes * batch));
}

}  // namespace

size_t gated_fwd_workspace_bytes(int64_t, int64_t, int64_t, int) { return 0; }

size_t gated_bwd_workspace_bytes(int64_t batch, int64_t, int64_t dim, int) {
  return (static_cast<size_t>(batch * dim) * 4 + 255) / 256 * 256;
}

hipError_t launch_gated_fwd(const GatedProblem& p, void*, hipStream_t stream) {
  if (p.io == kIoBf16)
    hipLaunchKernelGGL((gated_fwd_kernel<Bf16Io>), channel_grid(p.batch, p.dim), dim3(kLanes), 0, stream, p);
  else
    hipLaunchKernelGGL((gated_fwd_kernel<F32Io>), channel_grid(p.batch, p.dim), dim3(kLanes), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_gated_bwd(const GatedBwdProblem& p, void* workspace, hipStream_t stream) {
  float* parts = static_cast<float*>(workspace);
  if (p.batch > 0) {
    if (p.io == kIoBf16)
      hipLaunchKernelGGL((gated_bwd_kernel<Bf16Io>), channel_grid(p.batch, p.dim), dim3(kLanes), 0, stream, p, parts);
    else
      hipLaunchKernelGGL((gated_bwd_kernel<F32Io>), channel_grid(p.batch, p.dim), dim3(kLanes), 0, stream, p, parts);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return launch_colsum(parts, p.batch, p.dim, StoreFlat{p.dA}, stream);
}

hipError_t launch_gated_update(const GatedUpdateProblem& p, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>((p.batch * p.dim + 255) / 256));
  if (p.io == kIoBf16)
    hipLaunchKernelGGL((gated_update_kernel<Bf16Io>), grid, dim3(256), 0, stream, p);
  else
    hipLaunchKernelGGL((gated_update_kernel<F32Io>), grid, dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace mscan

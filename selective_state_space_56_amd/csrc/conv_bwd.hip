// Backward of the causal depthwise convolution + SiLU:
//   v_t = bias + sum_j w_j x_{t-(W-1)+j},  dv_t = dout_t silu'(v_t),
//   dx_t = sum_j w_j dv_{t+(W-1)-j},  dw_j = sum_t dv_t x_{t-(W-1)+j},  dbias = sum_t dv_t.
//
// Streaming and bound by HBM: x and dout in, dx out (503 MB for 8 x 2048 x 5120
// bf16), and 9 % on top for the W - 1 steps that neighbouring spans both read
// and for the parts of dw. That takes 108 us and 6 for the sums of dw on an
// MI355X, 5.1 TB/s of what is moved; a plain copy reaches 5.3.
#include "block.h"
#include "block_math.h"
#include "colsum.h"

namespace mscan {

namespace {

constexpr int kThreads = 64;
// Channels per thread (1 where there is one), steps whose loads are in flight
// together. 8 x 2048 x 5120 bf16, with the sums and plain loads: two channels and 4
// steps 115 us, 2 steps 119, 6 steps 128, 8 steps 121; four channels and 4 steps 142.
constexpr int kVec = 2;
constexpr int kGroup = 4;

// V channels of one batch row per thread, `span` steps: v and dv are formed in
// time order and kept for W steps; a step's dx is ready W - 1 steps later, so a
// span reads W - 1 steps past its end (and those add nothing to its dw). The
// next group's loads are in flight while the current group is computed.
// Threads past the last channel take the last V channels: they compute what
// their owner does, and what both write is the same.
template <class IO, int W, int V, bool LAST>
__global__ __launch_bounds__(kThreads) void conv_bwd_kernel(ConvBwdProblem p, int span, float* parts) {
  using raw = typename IO::raw;
  const int64_t own = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) * V;
  const int64_t c = own < p.dim - V ? own : p.dim - V;
  const int64_t b = blockIdx.z;
  const int64_t t0 = static_cast<int64_t>(blockIdx.y) * span;
  const int64_t t1 = t0 + span < p.seqlen ? t0 + span : p.seqlen;
  const raw* xin = static_cast<const raw*>(p.xin) + b * p.seqlen * p.dim + c;
  const raw* dout = static_cast<const raw*>(p.dout) + b * p.seqlen * p.dim + c;
  raw* dxin = static_cast<raw*>(p.dxin) + b * p.seqlen * p.dim + c;
  const int64_t state = (b * p.dim + c) * (W - 1);
  float w[W][V], dw[W][V], bias[V], db[V];
  float x[W][V], dv[W][V];  // x[j] = input t - (W-1) + j, dv[j] = dv at t - j
#pragma unroll
  for (int k = 0; k < V; ++k) {
    bias[k] = p.bias ? p.bias[c + k] : 0.0f;
    db[k] = 0.0f;
#pragma unroll
    for (int j = 0; j < W; ++j) {
      w[j][k] = p.weight[(c + k) * W + j];
      dw[j][k] = dv[j][k] = x[j][k] = 0.0f;
    }
  }
  // the W - 1 inputs before the span
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    const int64_t t = t0 - (W - 1) + j;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      if (t >= 0)
        x[j + 1][k] = IO::load(xin + t * p.dim + k);
      else if (p.state_in)
        x[j + 1][k] = IO::load(static_cast<const raw*>(p.state_in) + state + k * (W - 1) + (W - 1) + t);
    }
  }
  // steps t0 .. end - 1: the inputs at t - (W-1) get their gradient at step t.
  // The first span also covers the state's inputs, the last those up to the end.
  const int64_t end = t1 + W - 1;
  Piece<IO, V> xr[kGroup], yr[kGroup];
  const auto load = [&](int64_t t) {
#pragma unroll
    for (int i = 0; i < kGroup; ++i) {
      const int64_t at = (t + i < p.seqlen ? t + i : p.seqlen - 1) * p.dim;  // past the end: not used
      xr[i].template load_if<LAST>(xin + at);
      yr[i].template load_if<LAST>(dout + at);
    }
  };
  // the windows move on by a step
  const auto shift = [&] {
#pragma unroll
    for (int k = 0; k < V; ++k) {
#pragma unroll
      for (int j = 0; j + 1 < W; ++j) x[j][k] = x[j + 1][k];
#pragma unroll
      for (int j = W - 1; j > 0; --j) dv[j][k] = dv[j - 1][k];
      dv[0][k] = 0.0f;
    }
  };
  const auto output = [&](const Piece<IO, V>& in, const Piece<IO, V>& dy) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      x[W - 1][k] = in.get(k);
      float v = bias[k];
#pragma unroll
      for (int j = 0; j < W; ++j) v = fmaf(w[j][k], x[j][k], v);
      const float sig = sigmoid_f(v);
      dv[0][k] = dy.get(k) * sig * fmaf(v, 1.0f - sig, 1.0f);
    }
  };
  const auto sums = [&] {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      db[k] += dv[0][k];
#pragma unroll
      for (int j = 0; j < W; ++j) dw[j][k] = fmaf(dv[0][k], x[j][k], dw[j][k]);
    }
  };
  const auto input_grad = [&](float (&d)[V]) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      d[k] = 0.0f;
#pragma unroll
      for (int j = 0; j < W; ++j) d[k] = fmaf(w[j][k], dv[j][k], d[k]);
    }
  };
  if (p.seqlen > 0) load(t0);
  for (int64_t t = t0; t < end; t += kGroup) {
    Piece<IO, V> x0[kGroup], y0[kGroup];
#pragma unroll
    for (int i = 0; i < kGroup; ++i) {
      x0[i] = xr[i];
      y0[i] = yr[i];
    }
    if (t + kGroup < end && p.seqlen > 0) load(t + kGroup);
    // inside the span every step is an output's and its oldest input is the span's
    if (t >= t0 + W - 1 && t + kGroup <= t1) {
#pragma unroll
      for (int i = 0; i < kGroup; ++i) {
        float d[V];
        shift();
        output(x0[i], y0[i]);
        sums();
        input_grad(d);
        Piece<IO, V> dx;
        dx.set(d);
        dx.template store_if<LAST>(dxin + (t + i - (W - 1)) * p.dim);
      }
      continue;
    }
#pragma unroll
    for (int i = 0; i < kGroup; ++i) {
      const int64_t now = t + i, at = now - (W - 1);
      if (now >= end) break;
      shift();
      if (now < p.seqlen) {
        output(x0[i], y0[i]);
        if (now < t1) sums();
      }
      if (at < t0 && blockIdx.y > 0) continue;  // the span before writes it
      float d[V];
      input_grad(d);
      // the forward's last W - 1 inputs are its state_out
      const int64_t slot = at - (p.seqlen - (W - 1));
      if (W > 1 && slot >= 0 && p.dstate_out)
#pragma unroll
        for (int k = 0; k < V; ++k) d[k] += p.dstate_out[state + k * (W - 1) + slot];
      if (at >= 0) {
        Piece<IO, V> dx;
        dx.set(d);
        dx.store(dxin + at * p.dim);
      } else if (p.dstate_in) {
#pragma unroll
        for (int k = 0; k < V; ++k) p.dstate_in[state + k * (W - 1) + (W - 1) + at] = d[k];
      }
    }
  }
  float* part = parts + (b * gridDim.y + blockIdx.y) * (W + 1) * p.dim + c;
#pragma unroll
  for (int k = 0; k < V; ++k) {
#pragma unroll
    for (int j = 0; j < W; ++j) part[j * p.dim + k] = dw[j][k];
    part[W * p.dim + k] = db[k];
  }
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

// Steps per thread: 64, and fewer, down to 16, while that gives fewer than four
// waves per compute unit. (8 x 2048 x 5120 bf16: 115 us at 64 steps, 114 at 128,
// 125 at 32; 3 x 301 x 771 fp32, 105 waves at 64 steps: 23 us then, 18 with 16.)
int span_of(int64_t batch, int64_t seqlen, int64_t dim) {
  const int64_t groups = batch * ((dim + kThreads * kVec - 1) / (kThreads * kVec));
  int span = 64;
  while (span > 16 && groups * ((seqlen + span - 1) / span) < 4 * device_cu_count()) span /= 2;
  return span;
}

int64_t spans_of(int64_t batch, int64_t seqlen, int64_t dim) {
  const int span = span_of(batch, seqlen, dim);
  return seqlen > 0 ? (seqlen + span - 1) / span : 1;
}

template <class IO, int V, bool LAST>
hipError_t launch_width(const ConvBwdProblem& p, float* parts, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>((p.dim + kThreads * V - 1) / (kThreads * V)),
                  static_cast<unsigned>(spans_of(p.batch, p.seqlen, p.dim)), static_cast<unsigned>(p.batch));
  const int span = span_of(p.batch, p.seqlen, p.dim);
  const auto kernel = p.width == 1   ? conv_bwd_kernel<IO, 1, V, LAST>
                      : p.width == 2 ? conv_bwd_kernel<IO, 2, V, LAST>
                      : p.width == 3 ? conv_bwd_kernel<IO, 3, V, LAST>
                                     : conv_bwd_kernel<IO, 4, V, LAST>;
  hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, stream, p, span, parts);
  return hipGetLastError();
}

template <class IO>
hipError_t launch_dim(const ConvBwdProblem& p, float* parts, hipStream_t stream) {
  if (p.dim < kVec) return launch_width<IO, 1, false>(p, parts, stream);
  if (streams(3 * p.batch * p.seqlen * p.dim * static_cast<int64_t>(sizeof(typename IO::raw))))
    return launch_width<IO, kVec, true>(p, parts, stream);
  return launch_width<IO, kVec, false>(p, parts, stream);
}

}  // namespace

size_t conv_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim, int width) {
  return (static_cast<size_t>(batch * spans_of(batch, seqlen, dim) * (width + 1) * dim) * 4 + 255) / 256 * 256;
}

hipError_t launch_conv_bwd(const ConvBwdProblem& p, void* workspace, hipStream_t stream) {
  float* parts = static_cast<float*>(workspace);
  if (p.batch > 0) {
    const hipError_t e = p.io == kIoBf16 ? launch_dim<Bf16Io>(p, parts, stream) : launch_dim<F32Io>(p, parts, stream);
    if (e != hipSuccess) return e;
  }
  return launch_colsum(parts, p.batch * spans_of(p.batch, p.seqlen, p.dim), (p.width + 1) * p.dim,
                       StoreTaps{p.dweight, p.dbias, p.dim, p.width}, stream);
}

}  // namespace mscan

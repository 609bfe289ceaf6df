// One decode token of linear attention: S <- e^g S + k v^T, o = scale S^T q, the
// state in place.
//
// Bound by HBM: every state is read and written once (8 K V bytes), the token's rows
// are nothing beside it (256 sequences of 40 heads, 128 x 128: 259 us, 5.2 TB/s; one
// sequence: 4.4 us, of which its 5 MB are one). A workgroup takes `cols` value channels of one (sequence,
// head); a thread four of them and every R-th row, several rows' loads in flight; the
// threads' sums meet in LDS, in a fixed order.
#include "block_math.h"
#include "mamba_scan.h"
#include "mixer.h"

namespace mscan {

namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 8;          // rows in flight per thread
constexpr int kMaxDim = 256;
constexpr float kNoDecay = -104.0f;

template <class IO>
__global__ __launch_bounds__(kThreads) void linattn_update_kernel(LinattnUpdateProblem p, int cols, int blocks) {
  using raw = typename IO::raw;
  __shared__ float s_q[kMaxDim], s_k[kMaxDim];
  __shared__ float s_sum[kThreads * 4];
  const int tid = threadIdx.x, K = static_cast<int>(p.K), V = static_cast<int>(p.V);
  const int64_t bh = blockIdx.x / blocks;
  const int c0 = static_cast<int>(blockIdx.x % blocks) * cols;
  const int64_t b = bh / p.heads;
  const int h = static_cast<int>(bh % p.heads);
  const int have = V - c0 < cols ? V - c0 : cols;
  const int quads = have / 4, R = kThreads / quads, r0 = tid / quads, x = 4 * (tid % quads);
  const int64_t qk = (h / (p.heads / p.groups)) * p.K;
  if (tid < K) {
    s_q[tid] = IO::to_f32(static_cast<const raw*>(p.q)[b * p.sq + qk + tid]) * p.scale;
    s_k[tid] = IO::to_f32(static_cast<const raw*>(p.k)[b * p.sk + qk + tid]);
  }
  const float g = p.g[p.head_decay ? h : bh];
  const float decay = hw_exp2(g * kLog2e);
  const bool drop = g <= kNoDecay;
  float v[4] = {}, sum[4] = {};
  if (r0 < R) {
    Piece<IO, 4> pv;
    pv.load(static_cast<const raw*>(p.v) + b * p.sv + static_cast<int64_t>(h) * V + c0 + x);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = pv.get(e);
  }
  __syncthreads();
  if (r0 < R) {
    float* state = p.state + bh * K * V + c0 + x;
    for (int k0 = r0; k0 < K; k0 += kAhead * R) {
      Piece<F32Io, 4> s[kAhead];
#pragma unroll
      for (int a = 0; a < kAhead; ++a)
        if (k0 + a * R < K) s[a].load(state + static_cast<int64_t>(k0 + a * R) * V);
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const int row = k0 + a * R;
        if (row >= K) break;
        float f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          f[e] = fmaf(s_k[row], v[e], drop ? 0.0f : decay * s[a].get(e));
          sum[e] = fmaf(s_q[row], f[e], sum[e]);
        }
        s[a].set(f);
        s[a].store(state + static_cast<int64_t>(row) * V);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) s_sum[r0 * have + x + e] = sum[e];
  }
  __syncthreads();
  if (tid < have) {
    float o = 0.0f;
    for (int r = 0; r < R; ++r) o += s_sum[r * have + tid];
    static_cast<raw*>(p.out)[b * p.so + static_cast<int64_t>(h) * V + c0 + tid] = IO::from_f32(o);
  }
}

}  // namespace

hipError_t launch_linattn_update(const LinattnUpdateProblem& p, hipStream_t stream) {
  const int64_t units = p.batch * p.heads;
  // few states are spread over more workgroups, 32 channels (128-byte pieces of rows) each: 40 and 160 states of
  // 128 x 128 take 4.7 and 6.9 us, with one workgroup each 5.7 and 7.2, 40 of 256 x 256 7.2 against 13.0. From
  // some 600 on neither is better throughout: 20.5 against 20.9 for 640 of 128 x 128 and 101.6 against
  // 103.9 for 3840, but 79 against 73 and 447 against 396 of 256 x 256, 7.1 against 6.7 and 28.6 against 27.3 of
  // 64 x 64.
  const int cols = units < 1024 && p.V > 32 ? 32 : static_cast<int>(p.V);
  const int blocks = static_cast<int>((p.V + cols - 1) / cols);
  const dim3 grid(static_cast<unsigned>(units * blocks));
  if (p.io == MAMBA_BF16)
    hipLaunchKernelGGL((linattn_update_kernel<Bf16Io>), grid, dim3(kThreads), 0, stream, p, cols, blocks);
  else
    hipLaunchKernelGGL((linattn_update_kernel<F32Io>), grid, dim3(kThreads), 0, stream, p, cols, blocks);
  return hipGetLastError();
}

}  // namespace mscan

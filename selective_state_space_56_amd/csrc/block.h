// Internal launch interface of the block operators around the scan: the gated
// linear recurrence, the RMS norm and the convolution's backward
// (api_block.cpp -> gated.hip, norm.hip, conv_bwd.hip).
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include "kernels.h"

namespace mscan {

// Gated linear recurrence. Strides count elements between consecutive steps
// (token rows); batch row b starts b * seqlen rows in.
struct GatedProblem {
  const void* x;
  const void* r;
  const void* g;
  const float* A;         // (dim)
  const float* h0;        // (batch, dim) or null
  const uint8_t* reset;   // (batch, seqlen) or null
  void* out;
  float* last_state;      // (batch, dim) or null
  float* checkpoints;     // (batch, ceil(seqlen / kGatedCheckpoint), dim) or null
  int64_t batch, seqlen, dim;
  int io;
  int64_t sx, sr, sg, so;
};

struct GatedBwdProblem {
  const void* x;
  const void* r;
  const void* g;
  const float* A;
  const uint8_t* reset;   // or null
  const float* checkpoints;
  const void* dout;
  const float* dlast;     // or null
  void* dx;
  void* dr;
  void* dg;
  float* dA;
  float* dh0;             // or null
  int64_t batch, seqlen, dim;
  int io;
  int64_t sx, sr, sg, so, sdx, sdr, sdg;
};

struct GatedUpdateProblem {
  float* state;
  const void* x;
  const void* r;
  const void* g;
  const float* A;
  void* out;
  int64_t batch, dim;
  int io;
  int64_t sx, sr, sg, so;
};

constexpr int64_t kGatedCheckpoint = 64;

// At least half the workgroups of a sequence call, counted as tiles of
// kGatedCheckpoint steps and 128 channels. The forward's tiles have twice the
// steps and 512 threads (64 channels only where there is one), the backward's 256
// threads and in fp32 64 channels, twice as many tiles: at most 2^24 - 2 of them.
inline int64_t gated_tiles(int64_t batch, int64_t seqlen, int64_t dim) {
  return batch * ((dim + 127) / 128) * ((seqlen + kGatedCheckpoint - 1) / kGatedCheckpoint);
}
constexpr int64_t kGatedMaxTiles = (int64_t(1) << 23) - 1;  // a launch holds fewer than 2^32 threads

size_t gated_fwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim);
size_t gated_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim);
hipError_t launch_gated_fwd(const GatedProblem& p, void* workspace, hipStream_t stream);
hipError_t launch_gated_bwd(const GatedBwdProblem& p, void* workspace, hipStream_t stream);
hipError_t launch_gated_update(const GatedUpdateProblem& p, hipStream_t stream);

// Whether a call that moves `bytes` streams past the caches: more than the 256 MB
// that the last-level cache holds, so that nothing of it would be found there
// by the next call. Such calls carry the non-temporal hint on their large
// tensors. With it the recurrence's training step of 8 x 2048 x 5120 bf16 (671 MB
// and more per call) takes 386 us instead of 404 and the convolution's backward
// 114.6 instead of 119.5; 3 x 1021 x 771 fp32 (38 MB), whose backward finds the
// forward's inputs in the cache, would take 51 us instead of 48.
inline bool streams(int64_t bytes) { return bytes > (int64_t(256) << 20); }

// RMS norm over rows, with the residual's addition and either an io output or
// an 8-bit one with scales.
struct NormProblem {
  const void* x;
  const void* residual;   // or null
  const float* weight;
  void* out;              // io, or e4m3 bytes when scale is set
  float* scale;           // (rows, ceil(dim / group)) or null: io output
  void* sum;              // null without a residual
  int64_t rows, dim, group;
  int io, res;
  float eps;
  int64_t sx, sres, ssum, so;
};

struct NormBwdProblem {
  const void* sum;
  const float* weight;
  const void* dout;
  const void* dsum;       // or null
  void* dresidual;
  void* dx;               // or null
  float* dweight;
  int64_t rows, dim;
  int io, res;
  float eps;
  int64_t ssum, so, sdsum, sdres, sdx;
};

constexpr int64_t kNormMaxDim = 65536;

hipError_t launch_norm(const NormProblem& p, hipStream_t stream);
size_t norm_bwd_workspace_bytes(int64_t rows, int64_t dim);
hipError_t launch_norm_bwd(const NormBwdProblem& p, void* workspace, hipStream_t stream);

// Backward of the causal convolution.
struct ConvBwdProblem {
  const void* xin;
  const float* weight;
  const float* bias;       // or null
  const void* state_in;    // or null
  const void* dout;
  const float* dstate_out; // or null
  void* dxin;
  float* dweight;
  float* dbias;            // or null
  float* dstate_in;        // or null
  int64_t batch, seqlen, dim;
  int width;
  int io;
};

size_t conv_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim, int width);
hipError_t launch_conv_bwd(const ConvBwdProblem& p, void* workspace, hipStream_t stream);

}  // namespace mscan

// Internal launch interface of the matrix-state mixer's operators: linear
// attention with a decay for each head, and the norm and rotation of its queries
// and keys (api_mixer.cpp -> linattn.hip, linattn_update.hip, qknorm.hip).
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include "kernels.h"

namespace mscan {

// Sizes of a linear attention call; `rows` token rows in all.
struct LinattnSizes {
  int64_t batch, seqlen, rows, heads, groups, K, V;
  int io;
  bool packed;
};

struct LinattnProblem {
  LinattnSizes n;
  const void* q;
  const void* k;
  const void* v;
  const float* g;
  const float* h0;           // or null
  const int64_t* offsets;    // packed only
  void* out;
  float* last_state;         // or null
  float scale;
  bool head_decay, zero_rest;
  int64_t sq, sk, sv, so;
};

struct LinattnBwdProblem {
  LinattnProblem f;          // out, last_state: null; so: dout's
  const void* dout;
  const float* dlast;        // or null
  void* dq;
  void* dk;
  void* dv;
  float* dg;                 // or null
  float* dh0;                // or null
  int64_t sdq, sdk, sdv;
};

struct LinattnUpdateProblem {
  float* state;
  const void* q;
  const void* k;
  const void* v;
  const float* g;
  void* out;
  int64_t batch, heads, groups, K, V;
  int io;
  bool head_decay;
  float scale;
  int64_t sq, sk, sv, so;
};

// Elements between two token rows at most: 64 rows are addressed in 31 bits.
constexpr int64_t kMixMaxStride = int64_t(1) << 23;

// Token rows times heads, and states, of one call at most: what the kernels
// count in 31 bits.
constexpr int64_t kLinattnMaxRowHeads = (int64_t(1) << 31) - 1;
constexpr int64_t kLinattnMaxStates = int64_t(1) << 21;

size_t linattn_fwd_workspace_bytes(const LinattnSizes& n);
size_t linattn_bwd_workspace_bytes(const LinattnSizes& n, bool head_decay);
hipError_t launch_linattn_fwd(const LinattnProblem& p, void* workspace, hipStream_t stream);
hipError_t launch_linattn_bwd(const LinattnBwdProblem& p, void* workspace, hipStream_t stream);
hipError_t launch_linattn_update(const LinattnUpdateProblem& p, hipStream_t stream);

constexpr int kQkNormAxes = 4;

struct QkNormProblem {
  const void* q;
  const void* k;
  const int64_t* positions;
  const float* freqs;
  const float* q_weight;     // or null
  const float* k_weight;     // or null
  void* qo;                  // the outputs, or (backward) the gradients of q and k
  void* ko;
  const void* dqo;           // backward: the outputs' gradients
  const void* dko;
  float* dq_weight;          // backward: or null
  float* dk_weight;
  int64_t tokens, qheads, kheads, dim, rotary;
  int64_t ends[kQkNormAxes]; // pairs of axis a: ends[a - 1] .. ends[a] - 1
  int io;
  bool interleaved;
  float eps;
  int64_t sq, sk, sqo, sko, sdqo, sdko;
};

hipError_t launch_qknorm_fwd(const QkNormProblem& p, hipStream_t stream);
size_t qknorm_bwd_workspace_bytes(int64_t tokens, int64_t qheads, int64_t kheads, int64_t dim);
hipError_t launch_qknorm_bwd(const QkNormProblem& p, void* workspace, hipStream_t stream);

}  // namespace mscan

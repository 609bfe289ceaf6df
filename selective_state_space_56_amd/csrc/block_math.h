// Device helpers of the block operators: wide accesses to rows of any
// alignment, the gates of the gated linear recurrence, column sums.
#pragma once

#include "device_math.h"

namespace mscan {

// V consecutive io values, as one access of V * sizeof(raw) bytes. gfx950's
// global loads and stores take any alignment of the element's size, so rows of
// odd lengths and odd first columns use the same path as aligned ones.
template <class IO, int V>
struct Piece {
  using raw = typename IO::raw;
  raw v[V];
  __device__ __forceinline__ void load(const raw* p) { __builtin_memcpy(v, p, sizeof(v)); }
  __device__ __forceinline__ void store(raw* p) const { __builtin_memcpy(p, v, sizeof(v)); }
  // the first n < V values only; the others are 0
  __device__ __forceinline__ void load_some(const raw* p, int n) {
#pragma unroll
    for (int k = 0; k < V; ++k) v[k] = k < n ? p[k] : IO::from_f32(0.0f);
  }
  __device__ __forceinline__ void store_some(raw* p, int n) const {
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (k < n) p[k] = v[k];
  }
  __device__ __forceinline__ float get(int k) const { return IO::to_f32(v[k]); }
  __device__ __forceinline__ void set(int k, float f) { v[k] = IO::from_f32(f); }
};

// 1 / (1 + e^-v): 0 and 1 at the infinities
__device__ __forceinline__ float sigmoid_f(float v) { return hw_rcp(1.0f + hw_exp2(-v * kLog2e)); }

// Decay a = e^v and input weight w = sqrt(1 - a^2) of one step, v = A sigmoid(r) <= 0.
// 1 - a^2 = 1 - e^-u with u = -2v: for u < 1/4, where 1 - a^2 would cancel, six
// terms of its series (the next is u^6 / 5040 < 5e-8 of the sum); above, a's
// rounding of 2^-24 is at most 3e-7 of 1 - a^2 >= 0.22.
__device__ __forceinline__ void decay_gain(float v, float& a, float& w) {
  a = hw_exp2(v * kLog2e);
  const float u = -2.0f * v;
  float p = fmaf(u, -1.0f / 720.0f, 1.0f / 120.0f);
  p = fmaf(u, p, -1.0f / 24.0f);
  p = fmaf(u, p, 1.0f / 6.0f);
  p = fmaf(u, p, -0.5f);
  p = fmaf(u, p, 1.0f);
  const float w2 = u < 0.25f ? u * p : fmaf(-a, a, 1.0f);
  w = __builtin_amdgcn_sqrtf(w2);
}

}  // namespace mscan

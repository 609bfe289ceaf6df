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

// Decay a = e^v and 1 - a^2 of one step, v = A sigmoid(r) <= 0, from v2 = v log2(e).
// 1 - a^2 = 1 - e^-u with u = -2v: for u < 1/4, where 1 - a^2 would cancel, six
// terms of its series u - u^2/2 + u^3/6 - ... (the next is u^6 / 5040 < 5e-8 of
// the sum), as a polynomial in v2; above, a's rounding of 2^-24 is at most 3e-7
// of 1 - a^2 >= 0.22.
__device__ __forceinline__ float decay_gap(float v2, float& a) {
  constexpr float k = 2.0f * kLn2;  // u = -k v2
  constexpr float c1 = -k, c2 = c1 * k / 2.0f, c3 = c2 * k / 3.0f, c4 = c3 * k / 4.0f, c5 = c4 * k / 5.0f,
                  c6 = c5 * k / 6.0f;
  a = hw_exp2(v2);
  float p = fmaf(v2, c6, c5);
  p = fmaf(v2, p, c4);
  p = fmaf(v2, p, c3);
  p = fmaf(v2, p, c2);
  p = fmaf(v2, p, c1);
  return v2 > -0.25f / k ? v2 * p : fmaf(-a, a, 1.0f);
}

}  // namespace mscan

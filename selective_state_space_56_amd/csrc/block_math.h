// Device helpers of the block operators: wide accesses to rows of any
// alignment, the gates of the gated linear recurrence, column sums.
#pragma once

#include "device_math.h"

namespace mscan {

// V consecutive io values, as one access of their size. gfx950's global loads
// and stores take any alignment of the element's size, so rows of odd lengths
// and odd first columns use the same path as aligned ones.
// load_last and store_last carry the non-temporal hint: for data that is not read
// again soon, so that it does not push out what is.
template <class T, int N, int ALIGN>
using Words = T __attribute__((ext_vector_type(N), aligned(ALIGN)));

template <class T, int N, int ALIGN>
__device__ __forceinline__ void load_streamed(const void* p, T (&to)[N]) {
  using W = Words<T, N, ALIGN>;
  const W w = __builtin_nontemporal_load(static_cast<const W*>(p));
#pragma unroll
  for (int k = 0; k < N; ++k) to[k] = w[k];
}

template <class T, int N, int ALIGN>
__device__ __forceinline__ void store_streamed(void* p, const T (&from)[N]) {
  using W = Words<T, N, ALIGN>;
  W w;
#pragma unroll
  for (int k = 0; k < N; ++k) w[k] = from[k];
  __builtin_nontemporal_store(w, static_cast<W*>(p));
}

template <class IO, int V>
struct Piece {
  using raw = typename IO::raw;
  raw v[V];
  __device__ __forceinline__ void load_last(const raw* p) { load_streamed<raw, V, sizeof(raw)>(p, v); }
  __device__ __forceinline__ void store_last(raw* p) const { store_streamed<raw, V, sizeof(raw)>(p, v); }
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
  template <bool LAST>
  __device__ __forceinline__ void load_if(const raw* p) {
    if constexpr (LAST)
      load_last(p);
    else
      load(p);
  }
  template <bool LAST>
  __device__ __forceinline__ void store_if(raw* p) const {
    if constexpr (LAST)
      store_last(p);
    else
      store(p);
  }
  __device__ __forceinline__ float get(int k) const { return IO::to_f32(v[k]); }
  __device__ __forceinline__ void set(const float (&f)[V]) {
#pragma unroll
    for (int k = 0; k < V; ++k) v[k] = IO::from_f32(f[k]);
  }
};

// bf16 in pairs: kept as the words that the access moves. (Held as single
// values, a piece that lives on past a branch or a loop's end is taken apart as
// soon as it arrives, so that every load is waited for where it was started.)
template <int V>
struct BfPiece {
  static_assert(V % 2 == 0, "whole words");
  using raw = uint16_t;
  uint32_t w[V / 2];
  __device__ __forceinline__ void load_last(const raw* p) { load_streamed<uint32_t, V / 2, 2>(p, w); }
  __device__ __forceinline__ void store_last(raw* p) const { store_streamed<uint32_t, V / 2, 2>(p, w); }
  __device__ __forceinline__ void load(const raw* p) { __builtin_memcpy(w, p, sizeof(w)); }
  __device__ __forceinline__ void store(raw* p) const { __builtin_memcpy(p, w, sizeof(w)); }
  __device__ __forceinline__ void load_some(const raw* p, int n) {
#pragma unroll
    for (int k = 0; k < V / 2; ++k) {
      const uint32_t low = 2 * k < n ? p[2 * k] : 0u, high = 2 * k + 1 < n ? p[2 * k + 1] : 0u;
      w[k] = low | (high << 16);
    }
  }
  __device__ __forceinline__ void store_some(raw* p, int n) const {
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (k < n) p[k] = static_cast<uint16_t>(w[k / 2] >> (16 * (k % 2)));
  }
  template <bool LAST>
  __device__ __forceinline__ void load_if(const raw* p) {
    if constexpr (LAST)
      load_last(p);
    else
      load(p);
  }
  template <bool LAST>
  __device__ __forceinline__ void store_if(raw* p) const {
    if constexpr (LAST)
      store_last(p);
    else
      store(p);
  }
  __device__ __forceinline__ float get(int k) const {
    return __uint_as_float(k % 2 ? w[k / 2] & 0xffff0000u : w[k / 2] << 16);
  }
  __device__ __forceinline__ void set(const float (&f)[V]) {
#pragma unroll
    for (int k = 0; k < V / 2; ++k)
      w[k] = static_cast<uint32_t>(Bf16Io::from_f32(f[2 * k])) |
             (static_cast<uint32_t>(Bf16Io::from_f32(f[2 * k + 1])) << 16);
  }
};
template <>
struct Piece<Bf16Io, 2> : BfPiece<2> {};
template <>
struct Piece<Bf16Io, 8> : BfPiece<8> {};

// 1 / (1 + e^-v): 0 and 1 at the infinities
__device__ __forceinline__ float sigmoid_f(float v) { return hw_rcp(1.0f + hw_exp2(-v * kLog2e)); }

// Decay a = e^v of one step, v = A s with the gate's sigmoid s, and 1 - a^2, from
// rate = A log2(e). With u = -2v and v2 = v log2(e): for u < 1/4 (`near`), where
// 1 - a^2 = 1 - e^-u would cancel, six terms of its series u - u^2/2 + u^3/6 - ...
// (the next is u^6 / 5040 < 5e-8 of the sum), as v2 times a polynomial in v2;
// above, a's rounding of 2^-24 is at most 3e-7 of 1 - a^2 >= 0.22. With SPLIT the
// series leaves out the factor |A|: s times a polynomial, which stays in float32's
// range where |A| s does not.
template <bool SPLIT>
__device__ __forceinline__ float decay_gap(float rate, float s, float& a, bool& near) {
  constexpr float k = 2.0f * kLn2;  // u = -k v2 = 2 |A| s
  constexpr float c1 = SPLIT ? 2.0f : -k, c2 = c1 * k / 2.0f, c3 = c2 * k / 3.0f, c4 = c3 * k / 4.0f,
                  c5 = c4 * k / 5.0f, c6 = c5 * k / 6.0f;
  const float v2 = rate * s;
  a = hw_exp2(v2);
  float p = fmaf(v2, c6, c5);
  p = fmaf(v2, p, c4);
  p = fmaf(v2, p, c3);
  p = fmaf(v2, p, c2);
  p = fmaf(v2, p, c1);
  near = v2 > -0.25f / k;
  return near ? (SPLIT ? s : v2) * p : fmaf(-a, a, 1.0f);
}

// a and w = sqrt(1 - a^2). The hardware's root takes numbers below its normal
// range as 0, so a weight below 2^-63 is 0. (Kept in range as the backward keeps it
// costs the forward 1.6 to 2 %: 129 -> 131.5 us for 8 x 2048 x 5120 bf16.)
__device__ __forceinline__ float decay_weight(float rate, float s, float& a) {
  bool near;
  return __builtin_amdgcn_sqrtf(decay_gap<false>(rate, s, a, near));
}

// What the weight's slope needs of a channel's A: sqrt(-A) and its reciprocal,
// NaN for A > 0; 0 both for A = 0, which holds the state.
struct RateRoot {
  float root, inv;
  __device__ __forceinline__ explicit RateRoot(float A) {
    const bool low = -A < 0x1p-100f;  // lifted: the hardware's roots take subnormal numbers as 0
    const float m = low ? -A * 0x1p64f : -A;
    root = __builtin_amdgcn_sqrtf(m) * (low ? 0x1p-32f : 1.0f);
    inv = A == 0.0f ? 0.0f : __builtin_amdgcn_rsqf(m) * (low ? 0x1p32f : 1.0f);
  }
};

}  // namespace mscan

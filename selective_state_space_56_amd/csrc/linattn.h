// What the kernels of linear attention share: a call's parts ("roles"), where
// sequences and their pieces lie, and the decays inside one chunk of steps.
//
// One map does all the work: per sequence and head, with a state S of K x V,
//   S_t = e^{g_t} S_{t-1} + k_t v_t^T,   o_t = S_t^T q_t
// over chunks of C steps. With ell_t the running sum of g inside the chunk,
//   o_t   = e^{ell_t} S_in^T q_t + sum_{s <= t} e^{ell_t - ell_s} (k_s . q_t) v_s
//   S_out = e^{ell_C} S_in + sum_s e^{ell_C - ell_s} k_s v_s^T
// so a chunk is four matrix products, and S stays in registers from the first
// chunk of a segment to its last. The gradients are the same map with other
// operands (dq: queries dout, keys v, values k, state S^T) and, for dk and dv,
// with time reversed; a reversed step's decay lies behind it, so there ell is
// the running sum before the step.
#pragma once

#include <stddef.h>

#include "block_math.h"
#include "mamba_scan.h"
#include "mixer.h"

namespace mscan {

constexpr float kNoDecay = -104.0f;  // e^g is 0 in float32 from here on: what was before is dropped

// One run of the map. Operands are rows of `heads / div` heads; e is what the
// sums for the decays' gradients take beside them.
struct MixRole {
  const void* q;
  const void* k;
  const void* v;
  const void* e;         // or null: no sums
  void* o;               // io rows, or null
  float* part;           // float32 rows (contiguous) in the place of o, or null
  int64_t sq, sk, sv, se, so;
  int qdiv, kdiv, vdiv, ediv;  // heads that share the operand's head
  int K, V;
  const float* s0;       // the state that enters a sequence, (batch, heads, K, V), or null
  const float* enter;    // the states that enter later segments, (slots, some, K, V), or null
  float* last;           // (batch, heads, K, V) or null
  float* entering;       // the state that enters each chunk, (chunk or inner slots, some, entering_size), or null
  float* sums;           // (value tiles, heads, rows) or null: for each step t, e_t . what S_in gives of o_t
  float* pairs;          // with it, the same shape, or null: for each step t, what crosses it of the chunk's
                         // own pairs, sum_{s < t <= u} of score (s, u) times e_u . v_s
  float* local;          // a segment's own state, (slots, some, K, V), instead of outputs; or null
  float* gone;           // with it: the segment's whole decay, (slots, some); -1 with a cut
  bool s0_turned;        // s0 is (.., V, K)
  bool reverse;
  float score, from, to; // factors of the chunk's scores, of what S_in gives, of what a step adds to S
};

struct MixCall {
  MixRole role[3];
  const int64_t* offsets;  // or null: sequences of seqlen steps
  const float* g;
  int64_t g_step;          // between steps: heads, or 0 with one decay per head
  int64_t seqlen, rows;
  int64_t slots;           // segments at most, over all sequences
  int batch, heads, roles, tiles;
  int head0, some;         // the heads of this call: `some` from head0 on; slots' arrays hold these
  int per;                 // chunks of a segment
  uint32_t together;       // consecutive workgroups that read the same rows
};

// Elements of a state as the runs leave it for each chunk: whole tiles of 32 x 32.
inline int64_t entering_size(int64_t K, int64_t V) { return (K + 31) / 32 * ((V + 31) / 32) * 1024; }

// Where a sequence lies. Offsets are read as they are found on the device, held
// to 0 .. rows.
struct Sequence {
  int64_t begin, len;
};
__device__ __forceinline__ int64_t offset_of(const int64_t* offsets, int64_t i, int64_t seqlen, int64_t rows) {
  if (!offsets) return i * seqlen;
  const int64_t v = offsets[i];
  return v < 0 ? 0 : v > rows ? rows : v;
}
__device__ __forceinline__ Sequence sequence_of(const int64_t* offsets, int64_t i, int64_t seqlen, int64_t rows) {
  const int64_t a = offset_of(offsets, i, seqlen, rows), b = offset_of(offsets, i + 1, seqlen, rows);
  return {a, b > a ? b - a : 0};
}

// Pieces of `steps` steps are counted through all sequences: piece p of sequence
// i has slot offset_i / steps + i + p, which leaves room for each sequence's last
// piece. The sequence of a slot is the last one that starts at or before it.
// (Rows are counted in 31 bits, and a segment has at most a chunk or two more.)
__device__ __forceinline__ int64_t first_slot(int64_t begin, int64_t i, uint32_t steps) {
  return static_cast<uint32_t>(begin) / steps + i;
}
inline int64_t slots_of(int64_t rows, int64_t batch, int64_t steps) { return rows / steps + batch; }

__device__ __forceinline__ int sequence_at(const int64_t* offsets, int batch, int64_t seqlen, int64_t rows, uint32_t steps,
                                           int64_t slot) {
  int lo = 0, hi = batch;  // lo: starts at or before the slot; hi: does not
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first_slot(offset_of(offsets, mid, seqlen, rows), mid, steps) <= slot)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Slots of chunks of C steps, and of the ends of those that another one of their sequence follows: chunk c's
// lies (c + 1) C steps into its sequence and before its end, so that counted through all rows its number is
// below the next sequence's first.
__device__ __forceinline__ int64_t chunk_slot(const int64_t* offsets, int64_t seqlen, int64_t begin, int64_t seq, int64_t c,
                                              int C) {
  return c + (offsets ? first_slot(begin, seq, C) : seq * ((seqlen + C - 1) / C));
}
__device__ __forceinline__ int64_t inner_slot(const int64_t* offsets, int64_t seqlen, int64_t begin, int64_t seq, int64_t c,
                                              int C) {
  return c + (offsets ? first_slot(begin, 1, C) : seq * ((seqlen + C - 1) / C - 1));
}
inline int64_t chunk_slots_of(const LinattnSizes& n, int64_t C) {
  return n.packed ? slots_of(n.rows, n.batch, C) : n.batch * ((n.seqlen + C - 1) / C);
}
inline int64_t inner_slots_of(const LinattnSizes& n, int64_t C) {
  return n.packed ? slots_of(n.rows, 1, C) : n.seqlen > 0 ? n.batch * ((n.seqlen + C - 1) / C - 1) : 0;
}

// The decays of one chunk of C <= 64 steps, by one wave, a step per lane. Sums
// are float64: among large decays the differences of float32 sums would lose the
// small ones (at 6400, half a step is 2^-12). A decay of 0 is no summand but cuts:
// step t sees steps s >= from[t] only. Steps past the chunk's end add nothing.
// (Aligned for the 16-byte reads of `down` and `end`, also where two of them follow each
// other in LDS.)
template <int C>
struct alignas(16) Decays {
  double ell[C];
  float in[C];     // of S_in in o_t, times `from`; 0 where a cut lies between (from[t] >= 0) or where it underflows
  float end[C];    // of a step in S_out, times `to`; 0 where a cut lies between (s < kept) or where it underflows
  int from[C];     // -1 without a cut before
  // Scores' factors e^{ell_t - ell_s} as up[t] down[s] (times `score`), where that is safe:
  // `flat` without a cut, with no g above 0 and 100 of decay at most.
  float up[C], down[C];
  int flat;
  float all;       // of S_in in S_out; 0 with a cut
  int cut;         // whether there is one
  int kept;        // the first step that S_out has
  double total;    // the sum of the others
};
static_assert(sizeof(Decays<32>) % 16 == 0 && offsetof(Decays<32>, down) % 16 == 0 && offsetof(Decays<32>, end) % 16 == 0 &&
                  sizeof(Decays<64>) % 16 == 0 && offsetof(Decays<64>, down) % 16 == 0 && offsetof(Decays<64>, end) % 16 == 0,
              "read 16 bytes at a time");

// e^v for the difference of two sums; the float32 argument is off by 2^-24 of |v|
__device__ __forceinline__ float exp_of(double v) { return hw_exp2(static_cast<float>(v) * kLog2e); }
// e^v to float32 whatever |v|: the whole part of log2 of it taken apart
__device__ __forceinline__ float exp_exactly(double v) {
  const double v2 = v * 1.44269504088896340736;
  const double whole = rint(v2 < -400.0 ? -400.0 : v2 > 400.0 ? 400.0 : v2);
  return ldexpf(hw_exp2(static_cast<float>(v2 - whole)), static_cast<int>(whole));
}

// Whether the product of the states that a chunk's steps lie between has a part in the gradients of its
// decays: not across a cut, nor where the decays between leave nothing in float32. `slack` (> 0) lets
// what stores the states reach further than what reads them, whose sums are not the same bits.
__device__ __forceinline__ bool passes(bool cut, double total, double slack = 0.0) { return !cut && !(total < -110.0 - slack); }

// Returns `all`.
template <int C>
__device__ __forceinline__ float chunk_decays(Decays<C>& d, float g, int n, bool reverse, float from, float to, float score) {
  const int i = threadIdx.x & 63;
  const bool live = i < n, cut = live && g <= kNoDecay;
  const double own = live && !cut ? static_cast<double>(g) : 0.0;
  double sum = own;
  int last = cut ? i : -1;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const double u = __shfl_up(sum, off);
    const int w = __shfl_up(last, off);
    if (i >= off) {
      sum += u;
      last = last > w ? last : w;
    }
  }
  const double total = __shfl(sum, 63);
  const int cuts = __shfl(last, 63);
  const float all = cuts < 0 ? exp_exactly(total) : 0.0f;
  const bool flat = cuts < 0 && total > -100.0 && !__any(live && !(g <= 0.0f));
  double ell = sum;
  int seen = last;
  if (reverse) {
    // not sum - own: the sums in the order in which they are made
    ell = __shfl_up(sum, 1);
    seen = __shfl_up(last, 1);
    if (i == 0) {
      ell = 0.0;
      seen = -1;
    }
  }
  if (i < C) {
    d.ell[i] = ell;
    d.in[i] = seen < 0 ? exp_exactly(ell) * from : 0.0f;
    d.up[i] = exp_exactly(ell - 0.5 * total) * score;
    d.down[i] = exp_exactly(0.5 * total - ell);
    d.from[i] = seen < 0 ? -1 : reverse ? seen + 1 : seen;
    d.end[i] = live && (reverse ? i > cuts : i >= cuts) ? exp_exactly(total - ell) * to : 0.0f;
    if (i == 0) {
      d.all = all;
      d.flat = flat;
      d.cut = cuts >= 0;
      d.kept = cuts < 0 ? 0 : reverse ? cuts + 1 : cuts;
      d.total = total;
    }
  }
  return all;
}

}  // namespace mscan

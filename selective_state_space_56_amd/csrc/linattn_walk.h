// A workgroup's way through one segment of one sequence: which chunks, which
// state it enters with and where it leaves it.
#pragma once

#include "linattn.h"

namespace mscan {

// 32-row tiles of a workgroup's state, and its waves, each with 32 value channels. (With
// 8 tiles, 128 registers of state, four waves' kernel would need more than there are.)
inline int key_tiles(int64_t K) { return K <= 64 ? 2 : K <= 128 ? 4 : 8; }
inline int value_waves(int64_t K, int64_t V) { return V <= 64 || key_tiles(K) == 8 ? 2 : 4; }
inline int value_tiles(int64_t K, int64_t V) {
  const int width = 32 * value_waves(K, V);
  return static_cast<int>((V + width - 1) / width);
}
inline int64_t walk_units(const MixCall& w) { return w.slots * w.heads * w.tiles * w.roles; }

// Sum over the 32 lanes of a half wave, in each of them.
__device__ __forceinline__ float over_32(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor(v, off);
  return v;
}

// A segment's whole decay.
struct Gone {
  double sum = 0.0;
  int cut = 0;
  __device__ __forceinline__ void add(int c, double s) {
    cut |= c;
    sum += s;
  }
};

struct Walk {
  int role, tile, head, seq;
  int64_t slot, begin, len, chunks;
  int first, stop, step;      // chunks: first, first + step, ... before stop
  bool entry, exit, reverse;  // whether the segment is its sequence's first or last on the way

  // False for a workgroup that has nothing to do.
  __device__ __forceinline__ bool find(const MixCall& w, int C) {
    int64_t u = blockIdx.x;
    role = static_cast<int>(u % w.roles);
    u /= w.roles;
    tile = static_cast<int>(u % w.tiles);
    u /= w.tiles;
    head = static_cast<int>(u % w.heads);
    slot = u / w.heads;
    const int64_t steps = static_cast<int64_t>(w.per) * C;
    seq = sequence_at(w.offsets, w.batch, w.seqlen, w.rows, steps, slot);
    const Sequence s = sequence_of(w.offsets, seq, w.seqlen, w.rows);
    begin = s.begin;
    len = s.len;
    chunks = (len + C - 1) / C;
    const int64_t segs = chunks > w.per ? (chunks + w.per - 1) / w.per : 1;
    const int64_t seg = slot - first_slot(begin, seq, steps);
    if (seg < 0 || seg >= segs) return false;
    reverse = w.role[role].reverse;
    entry = seg == (reverse ? segs - 1 : 0);
    exit = seg == (reverse ? 0 : segs - 1);
    if (w.role[role].local && exit) return false;  // nobody enters with what it leaves
    const int64_t a = seg * w.per, b = a + w.per < chunks ? a + w.per : chunks;
    first = static_cast<int>(reverse ? b - 1 : a);
    stop = static_cast<int>(reverse ? a - 1 : b);
    step = reverse ? -1 : 1;
    return true;
  }

  // The token of a chunk's row: the chunk starts c0 tokens into the sequence and has n.
  __device__ __forceinline__ int64_t token(int row, int64_t c0, int n) const {
    return c0 + (reverse ? n - 1 - row : row);
  }

  // Register i of tile kt holds S[32 kt + 8 (i / 4) + 4 hi + i % 4][col].
  static __device__ __forceinline__ int row_of(int kt, int i, int hi) { return 32 * kt + 8 * (i >> 2) + 4 * hi + (i & 3); }

  template <int KT, class Tile>
  __device__ __forceinline__ void write(const MixRole& r, float* to, const Tile (&S)[KT], int col, int hi) const {
    if (col >= r.V) return;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int row = row_of(kt, i, hi);
        if (row < r.K) to[static_cast<int64_t>(row) * r.V + col] = S[kt][i];
      }
  }

  template <int KT, class Tile>
  __device__ __forceinline__ void enter_state(const MixCall& w, const MixRole& r, Tile (&S)[KT], int col, int hi) const {
    const int64_t size = static_cast<int64_t>(r.K) * r.V;
    const float* from = entry ? r.s0 : r.enter;
    if (r.local) from = nullptr;
    if (from) from += ((entry ? seq : slot) * w.heads + head) * size;
    const bool turned = entry && r.s0_turned;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int row = row_of(kt, i, hi);
        S[kt][i] = from && row < r.K && col < r.V ? from[turned ? static_cast<int64_t>(col) * r.K + row
                                                                : static_cast<int64_t>(row) * r.V + col]
                                                  : 0.0f;
      }
  }

  // The state between chunks, for the gradients of the decays: with time running
  // forward what enters chunk c, in reverse what enters it from behind.
  template <int KT, class Tile>
  __device__ __forceinline__ void leave_mark(const MixCall& w, const MixRole& r, const Tile (&S)[KT], int64_t c, int64_t C,
                                             int col, int hi) const {
    if (!r.marks) return;
    const int64_t between = reverse ? c + 1 : c;
    if (between == 0 || between >= chunks || between % w.mark) return;
    const int64_t at = first_slot(begin, seq, w.mark * C) + between / w.mark;
    write<KT>(r, r.marks + (at * w.heads + head) * r.K * r.V, S, col, hi);
  }

  template <int KT, class Tile>
  __device__ __forceinline__ void leave_state(const MixCall& w, const MixRole& r, const Tile (&S)[KT], const Gone& gone,
                                              int col, int hi) const {
    const int64_t size = static_cast<int64_t>(r.K) * r.V;
    if (r.local) {
      write<KT>(r, r.local + (slot * w.heads + head) * size, S, col, hi);
      if (threadIdx.x == 0 && tile == 0) r.gone[slot * w.heads + head] = gone.cut ? 0.0f : exp_of(gone.sum);
    } else if (r.last && exit) {
      write<KT>(r, r.last + (static_cast<int64_t>(seq) * w.heads + head) * size, S, col, hi);
    }
  }

  // Outputs of the chunk's rows t0 + (as row_of), as far as there are tokens.
  template <class IO, class Tile>
  __device__ __forceinline__ void store(const MixCall& w, const MixRole& r, const Tile& o, int t0, int64_t c0, int n,
                                        int col, int hi) const {
    if (col >= r.V) return;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int t = t0 + row_of(0, i, hi);
      if (t >= n) continue;
      const int64_t row = begin + token(t, c0, n), at = static_cast<int64_t>(head) * r.V + col;
      if (r.part)
        r.part[row * w.heads * r.V + at] = o[i];
      else
        static_cast<typename IO::raw*>(r.o)[row * r.so + at] = IO::from_f32(o[i]);
    }
  }
};

hipError_t launch_walk_f32(const MixCall& w, int io, int chunk, hipStream_t stream);

}  // namespace mscan

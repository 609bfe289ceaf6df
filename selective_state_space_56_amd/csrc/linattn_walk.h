// A workgroup's way through one segment of one sequence: which chunks, which
// state it enters with and where it leaves it.
#pragma once

#include "linattn.h"

namespace mscan {

// 32-row tiles of a workgroup's state, and its value channels.
inline int key_tiles(int64_t K) { return K <= 64 ? 2 : K <= 128 ? 4 : 8; }
inline int value_width(int64_t V) { return V <= 64 ? 64 : 128; }
inline int value_tiles(int64_t V) { return static_cast<int>((V + value_width(V) - 1) / value_width(V)); }
inline int64_t walk_units(const MixCall& w) { return w.slots * w.some * w.tiles * w.roles; }

// Sum over the 32 lanes of a half wave, in each of them.
__device__ __forceinline__ float over_32(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor(v, off);
  return v;
}

__device__ __forceinline__ int segments_of(int chunks, int per) { return chunks > per ? (chunks + per - 1) / per : 1; }

__device__ __forceinline__ int64_t uniform(int64_t v) {
  const uint32_t a = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
  const uint32_t b = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
  return static_cast<int64_t>(static_cast<uint64_t>(b) << 32 | a);
}

// v where `on`, else 0. The value is formed either way: written as a condition around
// its expression, the compiler branches around each one.
__device__ __forceinline__ float where(bool on, float v) { return on ? v : 0.0f; }

// A value from another lane of its row of 16, as a DPP control says; 0 from outside the row.
template <int CTRL>
__device__ __forceinline__ float from_row(float v) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), CTRL, 0xf, 0xf, true));
}
constexpr int kMirror16 = 0x140, kMirror8 = 0x141, kSwapPairs = 0x4e, kSwapLanes = 0xb1;  // lane i: of 15 - i, 7 - i, i ^ 2, i ^ 1
constexpr int kFirst = 0x150, kNext = 0x100;                                              // of lane 0; of i + n

// Pairs of steps as a tile of D's registers: register i of a lane is step s = 8 (i / 4) + 4 hi + i % 4 with
// step u, the lane's column. prefix_of: each becomes the sum over s up to its own; returns a column's sum. All
// sums here are made in a fixed order, without LDS.
template <class Tile>
__device__ __forceinline__ float prefix_of(Tile& v, int hi) {
  float before = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
#pragma unroll
    for (int e = 1; e < 4; ++e) v[4 * j + e] += v[4 * j + e - 1];
    const uint32_t own = __float_as_uint(v[4 * j + 3]);
    const auto both = __builtin_amdgcn_permlane32_swap(own, own, false, false);
    const float low = __uint_as_float(both[0]), high = __uint_as_float(both[1]);
    const float base = hi ? before + low : before;
    before += low + high;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[4 * j + e] += base;
  }
  return before;
}

// The sums of each register over the 32 columns of a half wave, register i's in lanes 2 i and 2 i + 1: at each
// step a lane keeps half of its registers and adds the other lane's.
template <class Tile>
__device__ __forceinline__ float over_columns(const Tile& v, int lo) {
  float a[8], b[4], c[2];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const auto w = __builtin_amdgcn_permlane16_swap(__float_as_uint(v[i]), __float_as_uint(v[8 + i]), false, false);
    a[i] = __uint_as_float(w[0]) + __uint_as_float(w[1]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) b[i] = (lo & 8 ? a[4 + i] : a[i]) + from_row<kMirror16>(lo & 8 ? a[i] : a[4 + i]);
#pragma unroll
  for (int i = 0; i < 2; ++i) c[i] = (lo & 4 ? b[2 + i] : b[i]) + from_row<kMirror8>(lo & 4 ? b[i] : b[2 + i]);
  const float one = (lo & 2 ? c[1] : c[0]) + from_row<kSwapPairs>(lo & 2 ? c[0] : c[1]);
  return one + from_row<kSwapLanes>(one);
}

// The step s of a tile that over_columns' result of this lane is for.
__device__ __forceinline__ int column_step(int lo, int hi) { return 8 * (lo >> 3) + 4 * hi + ((lo >> 1) & 3); }

// The sum over the columns from the lane's own to the half wave's last.
__device__ __forceinline__ float over_later(float v, int lo) {
  v += from_row<kNext + 1>(v);
  v += from_row<kNext + 2>(v);
  v += from_row<kNext + 4>(v);
  v += from_row<kNext + 8>(v);
  const auto w = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  const float upper = from_row<kFirst>(__uint_as_float(w[1]));
  return lo < 16 ? v + upper : v;
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
  int role, tile, head, own, seq;  // own: the head among the call's
  int64_t slot, begin, len;
  int chunks;
  int first, stop, step;      // chunks: first, first + step, ... before stop
  bool entry, exit, reverse;  // whether the segment is its sequence's first or last on the way

  // False for a workgroup that has nothing to do.
  __device__ __forceinline__ bool find(const MixCall& w, int C) {
    uint32_t u = blockIdx.x;
    // Consecutive workgroups go to the eight dies in turn; those that read the same rows
    // (a head's runs and value tiles, heads that share their keys) are kept on one.
    const uint32_t run = w.together, whole = gridDim.x / (8 * run) * (8 * run);
    if (u < whole) u = (u / (8 * run) * 8 + u % 8) * run + u / 8 % run;
    role = u % w.roles;
    u /= w.roles;
    tile = u % w.tiles;
    u /= w.tiles;
    own = u % w.some;
    head = w.head0 + own;
    slot = u / w.some;
    const uint32_t steps = static_cast<uint32_t>(w.per) * C;
    // (the same in every lane, which the compiler cannot see of values read from memory)
    seq = __builtin_amdgcn_readfirstlane(sequence_at(w.offsets, w.batch, w.seqlen, w.rows, steps, slot));
    const Sequence s = sequence_of(w.offsets, seq, w.seqlen, w.rows);
    begin = uniform(s.begin);
    len = uniform(s.len);
    chunks = static_cast<int>((len + C - 1) / C);
    const int segs = segments_of(chunks, w.per);
    const int seg = static_cast<int>(slot - first_slot(begin, seq, steps));
    if (seg < 0 || seg >= segs) return false;
    reverse = w.role[role].reverse;
    entry = seg == (reverse ? segs - 1 : 0);
    exit = seg == (reverse ? 0 : segs - 1);
    if (w.role[role].local && exit) return false;  // nobody enters with what it leaves
    const int a = seg * w.per, b = a + w.per < chunks ? a + w.per : chunks;
    first = reverse ? b - 1 : a;
    stop = reverse ? a - 1 : b;
    step = reverse ? -1 : 1;
    return true;
  }

  // The token of a chunk's row: the chunk starts c0 tokens into the sequence and has n.
  __device__ __forceinline__ int64_t token(int row, int64_t c0, int n) const {
    return c0 + (reverse ? n - 1 - row : row);
  }

  // States are held as N tiles whose register i holds row L::row(tile, i) + L::kLane x
  // part of the state (and row0 rows on), part being the lane's group; the lane's column is col. They are
  // reached through a buffer resource, so that a register's address is a scalar beside
  // the lane's own; what lies past the state is out of its range.
  template <class L, class Tile, int N>
  __device__ __forceinline__ void write(const MixRole& r, float* to, const Tile (&S)[N], int col, int part,
                                        int row0 = 0) const {
    const auto rs = make_rsrc(to, static_cast<uint32_t>(r.K * r.V * 4));
    const int first = row0 + L::kLane * part;  // the lane's first row
    const uint32_t lane = col < r.V ? static_cast<uint32_t>((first * r.V + col) * 4) : kOffNone;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      int row_step = r.V * 4;
      asm volatile("" : "+s"(row_step));  // formed here, not kept for every register from the kernel's start on
#pragma unroll
      for (int i = 0; i < L::kRows; ++i)
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(S[k][i]), rs, first + L::row(k, i) < r.K ? lane : kOffNone,
                                              L::row(k, i) * row_step, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  template <class L, class Tile, int N>
  __device__ __forceinline__ void enter_state(const MixCall& w, const MixRole& r, Tile (&S)[N], int col, int part,
                                              int row0 = 0) const {
    const float* from = r.local ? nullptr : entry ? r.s0 : r.enter;
    if (!from) {
#pragma unroll
      for (int k = 0; k < N; ++k) S[k] = Tile{};
      return;
    }
    from += (entry ? static_cast<int64_t>(seq) * w.heads + head : slot * w.some + own) * r.K * r.V;
    const auto rs = make_rsrc(from, static_cast<uint32_t>(r.K * r.V * 4));
    const bool turned = entry && r.s0_turned;
    const int first = row0 + L::kLane * part;
    const uint32_t lane = static_cast<uint32_t>((turned ? col * r.K + first : first * r.V + col) * 4);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      int row_step = turned ? 4 : r.V * 4;
      asm volatile("" : "+s"(row_step));
#pragma unroll
      for (int i = 0; i < L::kRows; ++i) {
        const uint32_t at = col < r.V && first + L::row(k, i) < r.K ? lane : kOffNone;
        S[k][i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, at, L::row(k, i) * row_step, 0));
      }
      __builtin_amdgcn_sched_barrier(0);  // (a tile's addresses at a time)
    }
  }

  // The state that enters chunk c (in reverse, from behind, where another one follows), for the gradients
  // of the decays: as it stands in registers, 32 x 32 tiles of 16 bytes of each lane, since only its product
  // with another run's is asked for. (A training step of 8 x 2048 steps of 20 heads of 128 x 128, bf16: 755 us with rows of the
  // state written 4 bytes at a time, and 708 with 16, which is 685 with the non-temporal hint.)
  template <class Tile, int N, int C>
  __device__ __forceinline__ void leave_entering(const MixCall& w, const MixRole& r, const Tile (&S)[N], int c,
                                                 const Decays<C>& dec, int col_tile, int row_tile, int lane) const {
    typedef float Quad __attribute__((ext_vector_type(4)));
    if (!r.entering || (reverse ? c == chunks - 1 : c == 0 && !r.s0)) return;
    if (!__builtin_amdgcn_readfirstlane(passes(dec.cut, dec.total, 1.0))) return;
    const int rows = (r.K + 31) / 32, cols = (r.V + 31) / 32;
    if (col_tile >= cols) return;
    const int64_t at = (reverse ? inner_slot(w.offsets, w.seqlen, begin, seq, c, C)
                                : chunk_slot(w.offsets, w.seqlen, begin, seq, c, C)) * w.some + own;
    Quad* to = reinterpret_cast<Quad*>(r.entering) + ((at * cols + col_tile) * rows + row_tile) * 256 + lane;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      if (row_tile + k >= rows) break;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        __builtin_nontemporal_store(Quad{S[k][4 * j], S[k][4 * j + 1], S[k][4 * j + 2], S[k][4 * j + 3]}, to + 256 * k + 64 * j);
    }
  }

  template <class L, class Tile, int N>
  __device__ __forceinline__ void leave_state(const MixCall& w, const MixRole& r, const Tile (&S)[N], const Gone& gone,
                                              int col, int part, int row0 = 0) const {
    const int64_t size = static_cast<int64_t>(r.K) * r.V;
    if (r.local) {
      write<L>(r, r.local + (slot * w.some + own) * size, S, col, part, row0);
      if (threadIdx.x == 0 && tile == 0) r.gone[slot * w.some + own] = gone.cut ? -1.0f : exp_of(gone.sum);
    } else if (r.last && exit) {
      write<L>(r, r.last + (static_cast<int64_t>(seq) * w.heads + head) * size, S, col, part, row0);
    }
  }

  // Outputs as D's registers: rows t0 + L::row(0, i) + L::kLane x part of the chunk, as
  // far as there are tokens.
  template <class IO, class L, class Tile>
  __device__ __forceinline__ void store(const MixCall& w, const MixRole& r, const Tile& o, int t0, int64_t c0, int n,
                                        int col, int part) const {
    using raw = typename IO::raw;
    const int first = t0 + L::kLane * part;
    const int64_t stride = r.part ? static_cast<int64_t>(w.heads) * r.V : r.so, step = reverse ? -stride : stride;
    const int64_t at = (begin + token(0, c0, n)) * stride + static_cast<int64_t>(head) * r.V + col + first * step;
    if (col >= r.V) return;
#pragma unroll
    for (int i = 0; i < L::kRows; ++i) {
      if (first + L::row(0, i) >= n) continue;
      if (r.part)
        r.part[at + L::row(0, i) * step] = o[i];
      else
        static_cast<raw*>(r.o)[at + L::row(0, i) * step] = IO::from_f32(o[i]);
    }
  }
};

hipError_t launch_walk_f32(const MixCall& w, hipStream_t stream);
hipError_t launch_walk_bf16(const MixCall& w, hipStream_t stream);

}  // namespace mscan

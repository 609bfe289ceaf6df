// Gated linear recurrence, one state per channel:
//   a_t = exp(A sigmoid(r_t)),  h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(g_t) x_t,
// over full sequences, its backward, and one decode token.
#include "block.h"
#include "block_math.h"
#include "colsum.h"

namespace mscan {

namespace {

constexpr int kLanes = 64;
constexpr int kSteps = 8;   // steps of a tile per wave
constexpr int kWaves = 8;   // waves per workgroup
constexpr int kSpan = kSteps * kWaves;  // steps of a tile
static_assert(kSpan == kGatedCheckpoint, "a tile starts at a checkpoint");
constexpr int kThreads = kLanes * kWaves;
constexpr int kBack = 8;    // earlier tiles looked at together

using u64 = unsigned long long;

// How a step acts on a state, h -> A h + B, and how a run of steps does: the
// maps join as (A2 A1, A2 B1 + B2). A is a product of decays, so never below
// 0; exactly 0 says that the run has a reset, behind which nothing of the
// state before it is kept, not even a NaN. Products that underflow stop at the
// smallest float instead, so that a non-finite state is not lost in them.
__device__ __forceinline__ float through(float A, float B, float h) { return A == 0.0f ? B : fmaf(A, h, B); }
__device__ __forceinline__ float joined(float A1, float a) { return fmaxf(A1 * a, 0x1p-149f); }

// What a tile tells the later ones of its channels, one 64-bit word per
// channel (value in the low half), so that a relaxed access carries value and
// kind together. 0: nothing yet. Sign bit of the high half set: the tile's map,
// the high half being -A, the low half B. High half 1: the state that leaves the tile.
__device__ __forceinline__ u64 word_of_map(float A, float B) {
  return (static_cast<u64>(__float_as_uint(A) | 0x80000000u) << 32) | __float_as_uint(B);
}
__device__ __forceinline__ u64 word_of_state(float h) { return (u64(1) << 32) | __float_as_uint(h); }
__device__ __forceinline__ bool is_state(u64 w) { return (w >> 32) == 1; }
__device__ __forceinline__ float low_of(u64 w) { return __uint_as_float(static_cast<uint32_t>(w)); }
__device__ __forceinline__ float map_of(u64 w) { return __uint_as_float(static_cast<uint32_t>(w >> 32) & 0x7fffffffu); }

__device__ __forceinline__ void tell(u64* p, u64 w) {
  __hip_atomic_store(p, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ u64 heard(const u64* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The state that enters a tile whose predecessors' words are at from[0],
// from[-step], ... (`before` of them): the nearest state told among the last
// kBack tiles, carried forward through the maps of the tiles after it. The
// same products and sums in the same order as if each of those tiles had told
// its state already, so that the result does not depend on who was first.
// Waits until the words are there; the tiles waited for all started earlier.
__device__ __forceinline__ float state_before(const u64* from, int64_t step, int before) {
  const int n = before < kBack ? before : kBack;
  u64 w[kBack];
  for (;;) {
#pragma unroll
    for (int k = 0; k < kBack; ++k)
      if (k < n) w[k] = heard(from - k * step);
    int at = -1;  // the nearest state with every map after it known
    bool known = true;
#pragma unroll
    for (int k = 0; k < kBack; ++k)
      if (k < n) {
        if (at < 0 && known && is_state(w[k])) at = k;
        known = known && w[k] != 0;
      }
    if (at >= 0) {
      float h = 0.0f;
#pragma unroll
      for (int k = kBack - 1; k >= 0; --k) {
        if (k == at) h = low_of(w[k]);
        if (k < at) h = through(map_of(w[k]), low_of(w[k]), h);
      }
      return h;
    }
    __builtin_amdgcn_s_sleep(1);
  }
}

// The tiles' words and the counter that hands tiles out, cleared before each
// call by a kernel of its own.
__global__ __launch_bounds__(256) void clear_kernel(uint4* p, int64_t n) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * 256)
    p[i] = make_uint4(0, 0, 0, 0);
}

constexpr size_t kHeader = 256;  // bytes before the words: the counter

// Tiles are handed out in the order of a counter, all channels of all batch
// rows before the next span of time, so that a tile waits only for tiles that
// were handed out, to workgroups that were running, before it.
struct Order {
  int per_span;   // tiles of one span of time
  int tiles;      // channel tiles of one batch row
  int spans;
};

__device__ __forceinline__ int next_tile(unsigned* counter, int* shared) {
  if (threadIdx.x == 0) *shared = counter ? static_cast<int>(atomicAdd(counter, 1u)) : static_cast<int>(blockIdx.x);
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(*shared);
}

// First of a lane's V channels in a tile. Lanes past the last channel (and the
// last lane, when dim is not a multiple of V) take the last V channels: they
// compute what their owner does, and what both write is the same.
template <int V>
__device__ __forceinline__ int lane_channel(int tile, int64_t dim) {
  const int c = (tile * kLanes + static_cast<int>(threadIdx.x % kLanes)) * V;
  const int last = static_cast<int>(dim) - V;
  return c < last ? c : last;
}
// Whether channel c is this lane's own (only the owner tells words: a later
// map of another tile's lane must not take the place of a state).
template <int V>
__device__ __forceinline__ bool owns(int tile, int c, int64_t dim) {
  return c >= (tile * kLanes + static_cast<int>(threadIdx.x % kLanes)) * V && c < dim;
}

// The resets of a wave's steps, as bits.
__device__ __forceinline__ uint32_t reset_bits(const uint8_t* reset, int64_t row, int steps) {
  if (!reset) return 0;
  const int lane = threadIdx.x % kLanes;
  const bool on = lane < steps && reset[row + lane] != 0;
  return static_cast<uint32_t>(__ballot(on));
}

// One tile: kSpan steps of 64 V channels, kSteps of them per wave. Each wave
// turns its steps into maps, kept in registers, and joins them; the waves'
// maps meet in LDS, the last wave tells the tile's map, finds the state that
// enters the tile and tells the one that leaves it; then every wave runs its
// steps from its own entering state. Inputs are read once.
template <class IO, int V>
__global__ __launch_bounds__(kThreads) void gated_fwd_kernel(GatedProblem p, Order o, unsigned* counter, u64* words) {
  using raw = typename IO::raw;
  __shared__ float mapA[kWaves][kLanes * V], mapB[kWaves][kLanes * V], enter[kLanes * V];
  __shared__ int shared_tile;
  const int tile = next_tile(counter, &shared_tile);
  const int lane = threadIdx.x % kLanes, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kLanes);
  const int span = tile / o.per_span, of_span = tile % o.per_span;
  const int64_t b = of_span / o.tiles;
  const int c = lane_channel<V>(of_span % o.tiles, p.dim);
  const int64_t t0 = static_cast<int64_t>(span) * kSpan + wave * kSteps;
  const int64_t left = p.seqlen - t0;
  const int steps = left < 0 ? 0 : left < kSteps ? static_cast<int>(left) : kSteps;
  const int64_t row = b * p.seqlen + t0;
  float a[kSteps][V], u[kSteps][V];
  float A1[V], B1[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    A1[v] = 1.0f;
    B1[v] = 0.0f;
  }
  const uint32_t resets = reset_bits(p.reset, row, steps);
  const bool plain = steps == kSteps && resets == 0;
  if (steps > 0) {
    Piece<IO, V> x[kSteps], r[kSteps], g[kSteps];
    float rate[V];
#pragma unroll
    for (int v = 0; v < V; ++v) rate[v] = p.A[c + v];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int64_t at = row + (i < steps ? i : steps - 1);  // past the end: the last step again, not used
      r[i].load(static_cast<const raw*>(p.r) + at * p.sr + c);
      g[i].load(static_cast<const raw*>(p.g) + at * p.sg + c);
      x[i].load(static_cast<const raw*>(p.x) + at * p.sx + c);
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float w;
        decay_gain(rate[v] * sigmoid_f(r[i].get(v)), a[i][v], w);
        u[i][v] = sigmoid_f(g[i].get(v)) * x[i].get(v);
        if (!plain) {
          if (resets >> i & 1) {
            w = 1.0f;
            a[i][v] = 0.0f;
          }
          if (i >= steps) {
            a[i][v] = 1.0f;
            u[i][v] = 0.0f;
          }
        }
        u[i][v] *= w;
      }
    if (plain) {
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          B1[v] = fmaf(a[i][v], B1[v], u[i][v]);
          A1[v] *= a[i][v];
        }
    } else {
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const bool on = resets >> i & 1;
          B1[v] = on ? u[i][v] : fmaf(a[i][v], B1[v], u[i][v]);
          A1[v] = on ? 0.0f : A1[v] == 0.0f ? 0.0f : joined(A1[v], a[i][v]);
        }
    }
    if (plain)
#pragma unroll
      for (int v = 0; v < V; ++v) A1[v] = fmaxf(A1[v], 0x1p-149f);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    mapA[wave][lane * V + v] = A1[v];
    mapB[wave][lane * V + v] = B1[v];
  }
  __syncthreads();
  // the maps of the waves before this one, joined
  float A0[V], B0[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    A0[v] = 1.0f;
    B0[v] = 0.0f;
  }
  for (int k = 0; k < wave; ++k)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float Ak = mapA[k][lane * V + v], Bk = mapB[k][lane * V + v];
      B0[v] = through(Ak, Bk, B0[v]);
      A0[v] = Ak == 0.0f || A0[v] == 0.0f ? 0.0f : joined(A0[v], Ak);
    }
  if (wave == kWaves - 1) {
    float At[V], Bt[V];
    const bool tells = span + 1 < o.spans;
    u64* word = words + (static_cast<int64_t>(span) * p.batch + b) * p.dim + c;
    const int64_t step = p.batch * p.dim;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      At[v] = A1[v] == 0.0f || A0[v] == 0.0f ? 0.0f : joined(A0[v], A1[v]);
      Bt[v] = through(A1[v], B1[v], B0[v]);
      if (tells && span > 0 && owns<V>(of_span % o.tiles, c + v, p.dim)) tell(word + v, word_of_map(At[v], Bt[v]));
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float h;
      if (span > 0)
        h = state_before(word + v - step, step, span);
      else
        h = p.h0 ? p.h0[b * p.dim + c + v] : 0.0f;
      enter[lane * V + v] = h;
      if (p.checkpoints) p.checkpoints[(b * o.spans + span) * p.dim + c + v] = h;
      const float out = through(At[v], Bt[v], h);
      if (tells) {
        if (owns<V>(of_span % o.tiles, c + v, p.dim)) tell(word + v, word_of_state(out));
      } else if (p.last_state)
        p.last_state[b * p.dim + c + v] = out;
    }
  }
  __syncthreads();
  if (steps == 0) return;
  float h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = through(A0[v], B0[v], enter[lane * V + v]);
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    Piece<IO, V> y;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      h[v] = !plain && (resets >> i & 1) ? u[i][v] : fmaf(a[i][v], h[v], u[i][v]);
      y.set(v, h[v]);
    }
    if (i < steps) y.store(static_cast<raw*>(p.out) + (row + i) * p.so + c);
  }
}

// The state after no steps.
__global__ __launch_bounds__(256) void gated_no_steps_kernel(const float* from, float* to, int64_t n) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i < n) to[i] = from ? from[i] : 0.0f;
}

// One tile of the backward, handed out from the last span to the first. The
// steps' maps give the states before them (from the checkpoint) and, run from
// the end, the adjoint: m -> a (dout + m) from step t to the one before, where
// m enters step t from the one after it, so that lam_t = dout_t + m. Each wave
// keeps its steps' gates in registers, finds its entering state and adjoint as
// the forward does, and writes its steps' gradients. parts: one row of dA per tile.
template <class IO, int V>
__global__ __launch_bounds__(kThreads) void gated_bwd_kernel(GatedBwdProblem p, Order o, unsigned* counter, u64* words,
                                                             float* parts) {
  using raw = typename IO::raw;
  __shared__ float mapA[kWaves][kLanes * V], mapB[kWaves][kLanes * V], mapM[kWaves][kLanes * V], enter[kLanes * V];
  __shared__ int shared_tile;
  const int tile = next_tile(counter, &shared_tile);
  const int lane = threadIdx.x % kLanes, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kLanes);
  const int turn = tile / o.per_span, of_span = tile % o.per_span, span = o.spans - 1 - turn;
  const int64_t b = of_span / o.tiles;
  const int c = lane_channel<V>(of_span % o.tiles, p.dim);
  const int64_t t0 = static_cast<int64_t>(span) * kSpan + wave * kSteps;
  const int64_t left = p.seqlen - t0;
  const int steps = left < 0 ? 0 : left < kSteps ? static_cast<int>(left) : kSteps;
  const int64_t row = b * p.seqlen + t0;
  float a[kSteps][V], w[kSteps][V], sr[kSteps][V], sg[kSteps][V], rate[V];
  Piece<IO, V> x[kSteps], dy[kSteps];
  float A1[V], B1[V], M1[V], mark[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    A1[v] = 1.0f;
    B1[v] = M1[v] = 0.0f;
    rate[v] = p.A[c + v];
    mark[v] = p.checkpoints[(b * o.spans + span) * p.dim + c + v];
  }
  const uint32_t resets = reset_bits(p.reset, row, steps);
  if (steps > 0) {
    Piece<IO, V> r[kSteps], g[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int64_t at = row + (i < steps ? i : steps - 1);
      r[i].load(static_cast<const raw*>(p.r) + at * p.sr + c);
      g[i].load(static_cast<const raw*>(p.g) + at * p.sg + c);
      x[i].load(static_cast<const raw*>(p.x) + at * p.sx + c);
      dy[i].load(static_cast<const raw*>(p.dout) + at * p.so + c);
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        sr[i][v] = sigmoid_f(r[i].get(v));
        sg[i][v] = sigmoid_f(g[i].get(v));
        decay_gain(rate[v] * sr[i][v], a[i][v], w[i][v]);
        const bool on = resets >> i & 1;
        if (on) w[i][v] = 1.0f;
        if (i >= steps) a[i][v] = 1.0f;
        const float u = i < steps ? w[i][v] * (sg[i][v] * x[i].get(v)) : 0.0f;
        B1[v] = on ? u : fmaf(a[i][v], B1[v], u);
        A1[v] = on || A1[v] == 0.0f ? 0.0f : joined(A1[v], a[i][v]);
      }
#pragma unroll
    for (int i = kSteps - 1; i >= 0; --i)
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (i < steps) M1[v] = resets >> i & 1 ? 0.0f : a[i][v] * (dy[i].get(v) + M1[v]);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    mapA[wave][lane * V + v] = A1[v];
    mapB[wave][lane * V + v] = B1[v];
    mapM[wave][lane * V + v] = M1[v];
  }
  __syncthreads();
  if (wave == 0) {
    float At[V], Mt[V];
    const bool tells = span > 0;
    const int64_t step = p.batch * p.dim;
    u64* word = words + (static_cast<int64_t>(turn) * p.batch + b) * p.dim + c;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      At[v] = 1.0f;
      Mt[v] = 0.0f;
    }
    for (int k = kWaves - 1; k >= 0; --k)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float Ak = mapA[k][lane * V + v];
        Mt[v] = through(Ak, mapM[k][lane * V + v], Mt[v]);
        At[v] = Ak == 0.0f || At[v] == 0.0f ? 0.0f : joined(At[v], Ak);
      }
    if (tells && turn > 0)
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (owns<V>(of_span % o.tiles, c + v, p.dim)) tell(word + v, word_of_map(At[v], Mt[v]));
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float m;
      if (turn > 0)
        m = state_before(word + v - step, step, turn);
      else
        m = p.dlast ? p.dlast[b * p.dim + c + v] : 0.0f;
      enter[lane * V + v] = m;
      const float out = through(At[v], Mt[v], m);
      if (tells) {
        if (owns<V>(of_span % o.tiles, c + v, p.dim)) tell(word + v, word_of_state(out));
      } else if (p.dh0)
        p.dh0[b * p.dim + c + v] = out;
    }
  }
  // the states before this wave's steps
  float before[kSteps][V];
  {
    float h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = mark[v];
    for (int k = 0; k < wave; ++k)
#pragma unroll
      for (int v = 0; v < V; ++v) h[v] = through(mapA[k][lane * V + v], mapB[k][lane * V + v], h[v]);
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        before[i][v] = h[v];
        const float u = w[i][v] * (sg[i][v] * x[i].get(v));
        h[v] = resets >> i & 1 ? u : fmaf(a[i][v], h[v], u);
      }
  }
  __syncthreads();
  float dA[V];
#pragma unroll
  for (int v = 0; v < V; ++v) dA[v] = 0.0f;
  if (steps > 0) {
    float m[V];
#pragma unroll
    for (int v = 0; v < V; ++v) m[v] = enter[lane * V + v];
    for (int k = kWaves - 1; k > wave; --k)
#pragma unroll
      for (int v = 0; v < V; ++v) m[v] = through(mapA[k][lane * V + v], mapM[k][lane * V + v], m[v]);
#pragma unroll
    for (int i = kSteps - 1; i >= 0; --i) {
      if (i >= steps) continue;
      Piece<IO, V> dx, dr, dg;
      const bool on = resets >> i & 1;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float xv = x[i].get(v), lam = dy[i].get(v) + m[v], lw = lam * w[i][v] * sg[i][v];
        const float slope = w[i][v] > 0.0f ? a[i][v] * a[i][v] * hw_rcp(w[i][v]) : 0.0f;
        const float dv = on ? 0.0f : lam * fmaf(a[i][v], before[i][v], -slope * sg[i][v] * xv);
        m[v] = on ? 0.0f : a[i][v] * lam;
        dA[v] = fmaf(dv, sr[i][v], dA[v]);
        dx.set(v, lw);
        dg.set(v, lw * xv * (1.0f - sg[i][v]));
        dr.set(v, dv * rate[v] * sr[i][v] * (1.0f - sr[i][v]));
      }
      dx.store(static_cast<raw*>(p.dx) + (row + i) * p.sdx + c);
      dr.store(static_cast<raw*>(p.dr) + (row + i) * p.sdr + c);
      dg.store(static_cast<raw*>(p.dg) + (row + i) * p.sdg + c);
    }
  }
  // the waves' parts of dA, added in their order (mapB is read no more)
#pragma unroll
  for (int v = 0; v < V; ++v) mapB[wave][lane * V + v] = dA[v];
  __syncthreads();
  if (wave == 0)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float s = 0.0f;
      for (int k = 0; k < kWaves; ++k) s += mapB[k][lane * V + v];
      parts[(static_cast<int64_t>(turn) * p.batch + b) * p.dim + c + v] = s;
    }
}

// One decode token per (batch row, channel).
template <class IO>
__global__ __launch_bounds__(256) void gated_update_kernel(GatedUpdateProblem p) {
  using raw = typename IO::raw;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= p.batch * p.dim) return;
  const int64_t b = i / p.dim, c = i % p.dim;
  const float x = IO::load(static_cast<const raw*>(p.x) + b * p.sx + c);
  const float sr = sigmoid_f(IO::load(static_cast<const raw*>(p.r) + b * p.sr + c));
  const float sg = sigmoid_f(IO::load(static_cast<const raw*>(p.g) + b * p.sg + c));
  float a, w;
  decay_gain(p.A[c] * sr, a, w);
  const float h = fmaf(a, p.state[i], w * (sg * x));
  p.state[i] = h;
  static_cast<raw*>(p.out)[b * p.so + c] = IO::from_f32(h);
}

Order order_of(int64_t batch, int64_t seqlen, int64_t dim, int V) {
  Order o;
  o.tiles = static_cast<int>((dim + kLanes * V - 1) / (kLanes * V));
  o.per_span = static_cast<int>(batch * o.tiles);
  o.spans = static_cast<int>((seqlen + kSpan - 1) / kSpan);
  return o;
}

size_t rounded_up(size_t bytes) { return (bytes + 255) / 256 * 256; }

// The counter and one word per channel of every span but the last; nothing for
// sequences of one span, whose tiles wait for nobody.
size_t words_bytes(int64_t batch, int64_t seqlen, int64_t dim) {
  const int64_t spans = (seqlen + kSpan - 1) / kSpan;
  return spans > 1 && batch * dim > 0 ? kHeader + rounded_up(static_cast<size_t>((spans - 1) * batch * dim) * 8) : 0;
}

hipError_t clear_words(void* workspace, size_t bytes, hipStream_t stream) {
  const int64_t n = static_cast<int64_t>(bytes / 16), groups = (n + 1023) / 1024;
  hipLaunchKernelGGL(clear_kernel, dim3(static_cast<unsigned>(groups < 2048 ? groups : 2048)), dim3(256), 0, stream,
                     static_cast<uint4*>(workspace), n);
  return hipGetLastError();
}

template <class IO, int V>
hipError_t launch_fwd(const GatedProblem& p, void* workspace, hipStream_t stream) {
  const Order o = order_of(p.batch, p.seqlen, p.dim, V);
  const size_t bytes = words_bytes(p.batch, p.seqlen, p.dim);
  if (bytes) {
    const hipError_t e = clear_words(workspace, bytes, stream);
    if (e != hipSuccess) return e;
  }
  unsigned* counter = bytes ? static_cast<unsigned*>(workspace) : nullptr;
  u64* words = bytes ? reinterpret_cast<u64*>(static_cast<char*>(workspace) + kHeader) : nullptr;
  hipLaunchKernelGGL((gated_fwd_kernel<IO, V>), dim3(static_cast<unsigned>(o.per_span) * o.spans), dim3(kThreads), 0,
                     stream, p, o, counter, words);
  return hipGetLastError();
}

template <class IO, int V>
hipError_t launch_bwd(const GatedBwdProblem& p, void* workspace, hipStream_t stream) {
  const Order o = order_of(p.batch, p.seqlen, p.dim, V);
  const size_t bytes = words_bytes(p.batch, p.seqlen, p.dim);
  if (bytes) {
    const hipError_t e = clear_words(workspace, bytes, stream);
    if (e != hipSuccess) return e;
  }
  char* ws = static_cast<char*>(workspace);
  unsigned* counter = bytes ? reinterpret_cast<unsigned*>(ws) : nullptr;
  u64* words = bytes ? reinterpret_cast<u64*>(ws + kHeader) : nullptr;
  float* parts = reinterpret_cast<float*>(ws + bytes);
  hipLaunchKernelGGL((gated_bwd_kernel<IO, V>), dim3(static_cast<unsigned>(o.per_span) * o.spans), dim3(kThreads), 0,
                     stream, p, o, counter, words, parts);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return launch_colsum(parts, p.batch * o.spans, p.dim, StoreFlat{p.dA}, stream);
}

}  // namespace

size_t gated_fwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim, int) {
  return words_bytes(batch, seqlen, dim);
}

size_t gated_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim, int) {
  const int64_t spans = (seqlen + kSpan - 1) / kSpan;
  return words_bytes(batch, seqlen, dim) + rounded_up(static_cast<size_t>(spans * batch * dim) * 4);
}

hipError_t launch_gated_fwd(const GatedProblem& p, void* workspace, hipStream_t stream) {
  if (p.seqlen == 0) {
    const int64_t n = p.batch * p.dim;
    hipLaunchKernelGGL(gated_no_steps_kernel, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0, stream, p.h0,
                       p.last_state, n);
    return hipGetLastError();
  }
  if (p.io == kIoBf16) return p.dim > 1 ? launch_fwd<Bf16Io, 2>(p, workspace, stream) : launch_fwd<Bf16Io, 1>(p, workspace, stream);
  return p.dim > 1 ? launch_fwd<F32Io, 2>(p, workspace, stream) : launch_fwd<F32Io, 1>(p, workspace, stream);
}

hipError_t launch_gated_bwd(const GatedBwdProblem& p, void* workspace, hipStream_t stream) {
  if (p.batch == 0 || p.seqlen == 0) {
    const int64_t n = p.batch * p.dim;
    if (p.dh0 && n > 0)
      hipLaunchKernelGGL(gated_no_steps_kernel, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0, stream,
                         p.dlast, p.dh0, n);
    hipLaunchKernelGGL(gated_no_steps_kernel, dim3(static_cast<unsigned>((p.dim + 255) / 256)), dim3(256), 0, stream,
                       static_cast<const float*>(nullptr), p.dA, p.dim);
    return hipGetLastError();
  }
  if (p.io == kIoBf16) return p.dim > 1 ? launch_bwd<Bf16Io, 2>(p, workspace, stream) : launch_bwd<Bf16Io, 1>(p, workspace, stream);
  return p.dim > 1 ? launch_bwd<F32Io, 2>(p, workspace, stream) : launch_bwd<F32Io, 1>(p, workspace, stream);
}

hipError_t launch_gated_update(const GatedUpdateProblem& p, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>((p.batch * p.dim + 255) / 256));
  if (p.io == kIoBf16)
    hipLaunchKernelGGL((gated_update_kernel<Bf16Io>), grid, dim3(256), 0, stream, p);
  else
    hipLaunchKernelGGL((gated_update_kernel<F32Io>), grid, dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace mscan

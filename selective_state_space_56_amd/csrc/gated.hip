// Gated linear recurrence, one state per channel:
//   a_t = exp(A sigmoid(r_t)),  h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(g_t) x_t,
// over full sequences, its backward, and one decode token.
//
// A step is the affine map h -> a h + b, and maps join, so time is cut into
// tiles that work at once: a tile reads its inputs, keeps its steps' maps in
// registers, joins them, and needs from the tiles before it only the state that
// enters it, which it gets from a word per channel in global memory (below).
// One pass: every input is read once and every output written once.
//
// Measured on an MI355X, where a plain copy moves 5.3 TB/s: the forward of
// 8 x 2048 x 5120 bf16 takes 132 us (671 MB, 5.1 TB/s), of 1 x 131072 x 5120
// 990 us (5.37 GB, 5.4 TB/s). It is bound by HBM, with the vector ALUs behind
// (37 instructions per element and step, 6 of them transcendental: they issue in
// 70 % of the kernel's cycles). The backward of the first takes 250 us (1.17 GB,
// 4.7 TB/s; 70 instructions, 67 % of the cycles): its tile fills the registers
// at two waves per SIMD, too few to cover every load and wait.
#include "block.h"
#include "block_math.h"
#include "colsum.h"

namespace mscan {

namespace {

constexpr int kLanes = 64;
constexpr int kHeld = 32;   // earlier tiles' maps held while looking back

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
// from[-step], ... (`before` of them): back to the nearest state told, holding
// the maps on the way, and forward again through those. That takes the same
// products and sums in the same order as if each of those tiles had told its
// state already, so the result does not depend on who was first. A word not
// there yet is waited for: its tile started earlier than this one. One word
// is asked for at first, mostly a state already, then four together (four at
// once from the start: 134 against 127 us for 8 x 2048 x 5120 bf16, 86 against 87
// for 1 x 131072 x 256). With 16 maps held instead of 32, 1 x 131072 x 256 takes
// 108 us instead of 87, with 2 402; a copy of its 268 MB would take 51: in so narrow
// a sequence what takes the time is the state's way through the tiles.
__device__ __forceinline__ float state_before(const u64* from, int64_t step, int before, u64 (&held)[kHeld][kLanes]) {
  const int lane = threadIdx.x % kLanes;
  int n = 0;  // maps held: the words of the nearest n tiles
  float h = 0.0f;
  for (int ask = 1, found = 0; !found; ask = 4) {
    u64 w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = k < ask && n + k < before ? heard(from - (n + k) * step) : 0;
    bool more = true;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      more = more && w[k] != 0;
      if (!more) continue;
      if (is_state(w[k])) {
        h = low_of(w[k]);
        found = 1;
        more = false;
      } else if (n < kHeld) {
        held[n++][lane] = w[k];
      } else {
        more = false;
      }
    }
    if (!found && !more) __builtin_amdgcn_s_sleep(1);
  }
  while (n > 0) {
    const u64 w = held[--n][lane];
    h = through(map_of(w), low_of(w), h);
  }
  return h;
}

// The tiles' words and the counter that hands tiles out, cleared before each
// call by a kernel of its own.
__global__ __launch_bounds__(256) void clear_kernel(uint4* p, int64_t n) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * 256)
    p[i] = make_uint4(0, 0, 0, 0);
}

constexpr size_t kHeader = 256;  // bytes before the words: the counter

// Tiles are handed out in the order of a counter, all channels of all batch
// rows before the next span of time, one to a workgroup when it starts. A tile
// waits only for tiles handed out before it, whose workgroups are running:
// the first unfinished tile of all waits for nobody, so every wait ends,
// whatever the number of workgroups that run at once. (Workgroups that stay and
// ask for their next tile early were slower: 159 against 144 us for the forward
// of 8 x 2048 x 5120 bf16; fresh ones load while finished ones still store.)
struct Order {
  int per_span;   // tiles of one span of time
  int tiles;      // channel tiles of one batch row
  int spans;
};

// This workgroup's tile. Without a counter (one span: nobody waits) its own index.
__device__ __forceinline__ int take_tile(unsigned* counter, int* shared) {
  if (!counter) return static_cast<int>(blockIdx.x);
  if (threadIdx.x == 0) *shared = static_cast<int>(atomicAdd(counter, 1u));
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(*shared);
}

// First of a lane's V channels in a tile. Lanes past the last channel (and the
// last lane, when dim is not a multiple of V) take the last V channels: they
// compute what their owner does, and what both write is the same.
template <int V>
__device__ __forceinline__ uint32_t lane_channel(int tile, int64_t dim) {
  const uint32_t c = (tile * kLanes + threadIdx.x % kLanes) * V;
  const uint32_t last = static_cast<uint32_t>(dim) - V;
  return c < last ? c : last;
}
// Whether channel c is this lane's own (only the owner tells words: a later
// map of another tile's lane must not take the place of a state).
template <int V>
__device__ __forceinline__ bool owns(int tile, uint32_t c, int64_t dim) {
  return c >= (tile * kLanes + threadIdx.x % kLanes) * V && c < dim;
}

// A tile's place: its span of time (in the order the tiles are handed out),
// its batch row and its channels, and this wave's steps of it.
template <int V, int STEPS, int WAVES>
struct Place {
  int lane, wave, turn, steps, tile;
  int64_t b, t0, row;
  uint32_t c;
  __device__ __forceinline__ Place(int id, const Order& o, int64_t seqlen, int64_t dim, bool backwards) {
    lane = threadIdx.x % kLanes;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kLanes);
    turn = id / o.per_span;
    tile = id % o.per_span;
    b = tile / o.tiles;
    tile %= o.tiles;
    c = lane_channel<V>(tile, dim);
    t0 = static_cast<int64_t>(backwards ? o.spans - 1 - turn : turn) * (STEPS * WAVES) + wave * STEPS;
    const int64_t left = seqlen - t0;
    steps = left < 0 ? 0 : left < STEPS ? static_cast<int>(left) : STEPS;
    row = b * seqlen + t0;
  }
};

// Channel c of a row whose start is the same in every lane: scalar base, 32-bit
// lane offset. (For the stores only: the loads measured 1 % slower with it.)
template <class T>
__device__ __forceinline__ T* in_row(T* row, uint32_t c) {
  return reinterpret_cast<T*>(reinterpret_cast<char*>(row) + c * static_cast<uint32_t>(sizeof(T)));
}

// A wave's steps of one tensor, all loads in flight together. Past the end
// (never when PLAIN) the last step is loaded again; its values are not used.
template <bool PLAIN, bool LAST, class IO, int V, int STEPS>
__device__ __forceinline__ void load_steps(const void* base, int64_t row, int64_t stride, int c, int steps,
                                           Piece<IO, V> (&to)[STEPS]) {
  const typename IO::raw* p = static_cast<const typename IO::raw*>(base) + row * stride;
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    to[i].template load_if<LAST>(p + c);
    if (PLAIN || i + 1 < steps) p += stride;
  }
}

// What the waves of a tile share: their maps, the state that enters the tile,
// and what state_before holds.
template <int V, int WAVES>
struct Shared {
  float A[WAVES][V][kLanes], B[WAVES][V][kLanes], enter[V][kLanes];
  u64 held[V][kHeld][kLanes];
  int tile;
};

// For channel v of every lane, by one wave: joins the waves' maps (from the
// last wave to the first when BACKWARDS), tells the tile's map, finds the state
// that enters the tile (`first` for the first tile) and tells the one that
// leaves it, or gives it to the caller when no tile comes after: true then.
template <bool BACKWARDS, int V, int STEPS, int WAVES>
__device__ __forceinline__ bool pass_on(int v, const Place<V, STEPS, WAVES>& at, int spans, int64_t states,
                                        int64_t state, int64_t dim, u64* words, const float* first,
                                        Shared<V, WAVES>& sh, float& out) {
  float At = 1.0f, Bt = 0.0f;
#pragma unroll
  for (int i = 0; i < WAVES; ++i) {
    const int k = BACKWARDS ? WAVES - 1 - i : i;
    const float Ak = sh.A[k][v][at.lane];
    Bt = through(Ak, sh.B[k][v][at.lane], Bt);
    At = Ak == 0.0f || At == 0.0f ? 0.0f : joined(At, Ak);
  }
  const bool last = at.turn + 1 == spans, own = owns<V>(at.tile, at.c + v, dim);
  u64* word = words + at.turn * states + state + v;
  float h;
  if (at.turn > 0) {
    if (!last && own) tell(word, word_of_map(At, Bt));
    h = state_before(word - states, states, at.turn, sh.held[v]);
  } else {
    h = first ? first[state + v] : 0.0f;
  }
  sh.enter[v][at.lane] = h;
  out = through(At, Bt, h);
  if (!last && own) tell(word, word_of_state(out));
  return last;
}

// The resets of a wave's steps, as bits.
__device__ __forceinline__ uint32_t reset_bits(const uint8_t* reset, int64_t row, int steps) {
  if (!reset) return 0;
  const int lane = threadIdx.x % kLanes;
  const bool on = lane < steps && reset[row + lane] != 0;
  return static_cast<uint32_t>(__ballot(on));
}

// A tile: steps per wave, waves. Its fixed costs (a tile's ticket, two barriers,
// the words) want it large, the registers and the number of tiles small. On
// 8 x 2048 x 5120 and 1 x 131072 x 5120 bf16, two channels per lane: 16 x 8 steps
// 127 and 971 us, 8 x 8 156 and 1167, 8 x 16 174 and 1330, 16 x 4 158 and 1154,
// 16 x 16 150 and 1075, 32 x 4 135 and 975, 32 x 8 160 and 1134; 16 x 8 with one
// channel per lane 155 and 1117.
constexpr int kFwdSteps = 16, kFwdWaves = 8;
constexpr int kFwdSpan = kFwdSteps * kFwdWaves, kFwdThreads = kLanes * kFwdWaves;
static_assert(kGatedCheckpoint % kFwdSteps == 0, "a checkpoint is where a wave's steps start");

// A wave's steps as maps (a, u) in registers, and their joined map (A1, B1).
// PLAIN: all STEPS steps are there and none is a reset.
template <bool PLAIN, bool LAST, class IO, int V>
__device__ __forceinline__ void steps_to_maps(const GatedProblem& p, const Place<V, kFwdSteps, kFwdWaves>& at,
                                              uint32_t resets, float (&a)[kFwdSteps][V], float (&u)[kFwdSteps][V],
                                              float (&A1)[V], float (&B1)[V]) {
  Piece<IO, V> x[kFwdSteps], r[kFwdSteps], g[kFwdSteps];
  float rate[V];
#pragma unroll
  for (int v = 0; v < V; ++v) rate[v] = p.A[at.c + v] * kLog2e;
  load_steps<PLAIN, LAST>(p.r, at.row, p.sr, at.c, at.steps, r);
  load_steps<PLAIN, LAST>(p.g, at.row, p.sg, at.c, at.steps, g);
  load_steps<PLAIN, LAST>(p.x, at.row, p.sx, at.c, at.steps, x);
#pragma unroll
  for (int i = 0; i < kFwdSteps; ++i)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float w = decay_weight(rate[v], sigmoid_f(r[i].get(v)), a[i][v]);
      const bool on = !PLAIN && (resets >> i & 1), past = !PLAIN && i >= at.steps;
      if (on) w = 1.0f;
      u[i][v] = w * (sigmoid_f(g[i].get(v)) * x[i].get(v));
      if (past) {
        a[i][v] = 1.0f;
        u[i][v] = 0.0f;
      }
      B1[v] = on ? u[i][v] : fmaf(a[i][v], B1[v], u[i][v]);
      A1[v] = on || (!PLAIN && A1[v] == 0.0f) ? 0.0f : PLAIN ? A1[v] * a[i][v] : joined(A1[v], a[i][v]);
    }
  if (PLAIN)
#pragma unroll
    for (int v = 0; v < V; ++v) A1[v] = fmaxf(A1[v], 0x1p-149f);
}

// One tile: kFwdSpan steps of 64 V channels, kFwdSteps of them per wave. Each
// wave turns its steps into maps, kept in registers, and joins them; the waves'
// maps meet in LDS, one wave per channel of a lane tells the tile's map, finds
// the state that enters the tile and tells the one that leaves it; then every
// wave runs its steps from its own entering state.
template <class IO, int V, bool LAST>
__global__ __launch_bounds__(kFwdThreads) void gated_fwd_kernel(GatedProblem p, Order o, unsigned* counter,
                                                                u64* words) {
  using raw = typename IO::raw;
  __shared__ Shared<V, kFwdWaves> sh;
  const Place<V, kFwdSteps, kFwdWaves> at(take_tile(counter, &sh.tile), o, p.seqlen, p.dim, false);
  const int lane = at.lane, wave = at.wave, steps = at.steps;
  float a[kFwdSteps][V], u[kFwdSteps][V];
  float A1[V], B1[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    A1[v] = 1.0f;
    B1[v] = 0.0f;
  }
  const uint32_t resets = reset_bits(p.reset, at.row, steps);
  const bool plain = steps == kFwdSteps && resets == 0;
  if (plain)
    steps_to_maps<true, LAST, IO, V>(p, at, resets, a, u, A1, B1);
  else if (steps > 0)
    steps_to_maps<false, LAST, IO, V>(p, at, resets, a, u, A1, B1);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    sh.A[wave][v][lane] = A1[v];
    sh.B[wave][v][lane] = B1[v];
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
      const float Ak = sh.A[k][v][lane];
      B0[v] = through(Ak, sh.B[k][v][lane], B0[v]);
      A0[v] = Ak == 0.0f || A0[v] == 0.0f ? 0.0f : joined(A0[v], Ak);
    }
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (wave == kFwdWaves - 1 - v) {
      const int64_t state = at.b * p.dim + at.c;
      float out;
      if (pass_on<false>(v, at, o.spans, p.batch * p.dim, state, p.dim, words, p.h0, sh, out) && p.last_state)
        p.last_state[state + v] = out;
    }
  __syncthreads();
  if (steps == 0) return;
  float h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = through(A0[v], B0[v], sh.enter[v][lane]);
  if (p.checkpoints && at.t0 % kGatedCheckpoint == 0) {
    const int64_t marks = (p.seqlen + kGatedCheckpoint - 1) / kGatedCheckpoint;
#pragma unroll
    for (int v = 0; v < V; ++v)
      p.checkpoints[(at.b * marks + at.t0 / kGatedCheckpoint) * p.dim + at.c + v] = h[v];
  }
  raw* out = static_cast<raw*>(p.out) + at.row * p.so;
  if (plain) {
#pragma unroll
    for (int i = 0; i < kFwdSteps; ++i) {
      Piece<IO, V> y;
#pragma unroll
      for (int v = 0; v < V; ++v) h[v] = fmaf(a[i][v], h[v], u[i][v]);
      y.set(h);
      y.store(in_row(out, at.c));
      out += p.so;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < kFwdSteps; ++i) {
    if (i >= steps) continue;
    Piece<IO, V> y;
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = resets >> i & 1 ? u[i][v] : fmaf(a[i][v], h[v], u[i][v]);
    y.set(h);
    y.store(in_row(out, at.c));
    out += p.so;
  }
}

// The state after no steps.
__global__ __launch_bounds__(256) void gated_no_steps_kernel(const float* from, float* to, int64_t n) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i < n) to[i] = from ? from[i] : 0.0f;
}

// A tile of the backward, 16 steps in each of 4 waves. bf16 takes two channels
// per lane: 256 registers, two waves per SIMD, 440 us for a training step of
// 8 x 2048 x 5120 (385 since) against 478 with one channel (163 registers, three
// waves) and 534 with 8 steps in each of 8 waves. With fp32, whose pieces take twice the
// room, two channels do not fit, so it takes one.
constexpr int kBwdSteps = 16, kBwdWaves = 4;
constexpr int kBwdThreads = kLanes * kBwdWaves;
static_assert(kBwdSteps * kBwdWaves == kGatedCheckpoint, "a tile starts at a checkpoint");

// What the backward keeps of a wave's steps: the decay a, the input gate sg and
// its product with the weight p = w sg, the recurrence gate sr, and d, sr times
// the slope of h_t along log a: first sr a^2 / w sg x, then sr a h_{t-1} minus that.
// (sr / w stays in range where 1 / w need not.)
template <class IO, int V>
struct Steps {
  float a[kBwdSteps][V], p[kBwdSteps][V], sg[kBwdSteps][V], sr[kBwdSteps][V], d[kBwdSteps][V];
  Piece<IO, V> x[kBwdSteps], dy[kBwdSteps];
};

// Loads a wave's steps and joins their maps: (A1, B1) of the states, (A1, M1)
// of the adjoint, from the last step to the first.
template <bool PLAIN, bool LAST, class IO, int V>
__device__ __forceinline__ void bwd_maps(const GatedBwdProblem& p, const Place<V, kBwdSteps, kBwdWaves>& at,
                                         uint32_t resets, const float (&rate)[V], Steps<IO, V>& s, float (&A1)[V],
                                         float (&B1)[V], float (&M1)[V]) {
  Piece<IO, V> r[kBwdSteps], g[kBwdSteps];
  load_steps<PLAIN, LAST>(p.r, at.row, p.sr, at.c, at.steps, r);
  load_steps<PLAIN, LAST>(p.g, at.row, p.sg, at.c, at.steps, g);
  load_steps<PLAIN, LAST>(p.x, at.row, p.sx, at.c, at.steps, s.x);
  load_steps<PLAIN, LAST>(p.dout, at.row, p.so, at.c, at.steps, s.dy);
#pragma unroll
  for (int i = 0; i < kBwdSteps; ++i)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const bool on = !PLAIN && (resets >> i & 1), past = !PLAIN && i >= at.steps;
      const float sr = sigmoid_f(r[i].get(v)), sg = sigmoid_f(g[i].get(v)), xv = s.x[i].get(v);
      float a;
      bool near;
      const RateRoot A(rate[v]);
      const float gap = decay_gap<true>(rate[v] * kLog2e, sr, a, near);
      const float inv = gap >= 0x1p-126f ? __builtin_amdgcn_rsqf(gap) : 0.0f;  // no slope where the state is held
      float w = gap * inv, slope = inv * sr;  // w and sr / w
      if (near) {
        w *= A.root;
        slope *= A.inv;
      }
      if (on) w = 1.0f;
      if (past) {
        a = 1.0f;
        w = 0.0f;
      }
      const float pg = w * sg, u = past ? 0.0f : pg * xv;
      s.a[i][v] = a;
      s.p[i][v] = pg;
      s.sg[i][v] = sg;
      s.sr[i][v] = sr;
      s.d[i][v] = a * a * slope * (sg * xv);
      B1[v] = on ? u : fmaf(a, B1[v], u);
      A1[v] = on || (!PLAIN && A1[v] == 0.0f) ? 0.0f : PLAIN ? A1[v] * a : joined(A1[v], a);
    }
  if (PLAIN)
#pragma unroll
    for (int v = 0; v < V; ++v) A1[v] = fmaxf(A1[v], 0x1p-149f);
#pragma unroll
  for (int i = kBwdSteps - 1; i >= 0; --i)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!PLAIN && i >= at.steps) continue;
      M1[v] = !PLAIN && (resets >> i & 1) ? 0.0f : s.a[i][v] * (s.dy[i].get(v) + M1[v]);
    }
}

// The states before a wave's steps, from h before the first, into d.
template <bool PLAIN, class IO, int V>
__device__ __forceinline__ void bwd_states(int steps, uint32_t resets, float (&h)[V], Steps<IO, V>& s) {
#pragma unroll
  for (int i = 0; i < kBwdSteps; ++i)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!PLAIN && i >= steps) continue;
      const float u = s.p[i][v] * s.x[i].get(v), kept = s.a[i][v] * h[v];
      const bool on = !PLAIN && (resets >> i & 1);
      s.d[i][v] = on ? 0.0f : fmaf(kept, s.sr[i][v], -s.d[i][v]);
      h[v] = on ? u : kept + u;
    }
}

// A wave's gradients, from the adjoint m that enters its last step. Their stores
// take the non-temporal hint too where the call streams (a training step of
// 8 x 2048 x 5120 bf16 395 us without, 386 with it); the forward's output does not
// (1 x 131072 x 5120 996 us without, 1010 with it; 8 x 2048 x 5120 132 and 129).
template <bool PLAIN, bool LAST, class IO, int V>
__device__ __forceinline__ void bwd_grads(const GatedBwdProblem& p, const Place<V, kBwdSteps, kBwdWaves>& at,
                                          uint32_t resets, const float (&rate)[V], const Steps<IO, V>& s,
                                          float (&m)[V], float (&dA)[V]) {
  using raw = typename IO::raw;
  const int64_t end = at.row + at.steps - 1;
  raw* dxp = static_cast<raw*>(p.dx) + end * p.sdx;
  raw* drp = static_cast<raw*>(p.dr) + end * p.sdr;
  raw* dgp = static_cast<raw*>(p.dg) + end * p.sdg;
#pragma unroll
  for (int i = kBwdSteps - 1; i >= 0; --i) {
    if (!PLAIN && i >= at.steps) continue;
    float xs[V], rs[V], gs[V];
    const bool on = !PLAIN && (resets >> i & 1);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float lam = s.dy[i].get(v) + m[v], lp = lam * s.p[i][v];
      const float dvr = on ? 0.0f : lam * s.d[i][v];
      m[v] = on ? 0.0f : s.a[i][v] * lam;
      dA[v] += dvr;
      xs[v] = lp;
      gs[v] = lp * s.x[i].get(v) * (1.0f - s.sg[i][v]);
      rs[v] = on ? 0.0f : dvr * rate[v] * (1.0f - s.sr[i][v]);  // 0 whatever r is
    }
    Piece<IO, V> dx, dr, dg;
    dx.set(xs);
    dr.set(rs);
    dg.set(gs);
    dx.template store_if<LAST>(in_row(dxp, at.c));
    dr.template store_if<LAST>(in_row(drp, at.c));
    dg.template store_if<LAST>(in_row(dgp, at.c));
    dxp -= p.sdx;
    drp -= p.sdr;
    dgp -= p.sdg;
  }
}

// One tile of the backward, handed out from the last span to the first. The
// steps' maps give the states before them (from the checkpoint) and, run from
// the end, the adjoint: m -> a (dout + m) from step t to the one before, where
// m enters step t from the one after it, so that lam_t = dout_t + m. Each wave
// keeps its steps in registers, finds its entering state and adjoint as the
// forward does, and writes its steps' gradients. parts: one row of dA per span
// and batch row.
template <class IO, int V, bool LAST>
__global__ __launch_bounds__(kBwdThreads, 2) void gated_bwd_kernel(GatedBwdProblem p, Order o, unsigned* counter,
                                                                   u64* words, float* parts) {
  __shared__ Shared<V, kBwdWaves> sh;            // A and B of the adjoint
  __shared__ float mapB[kBwdWaves][V][kLanes];   // B of the states
  const Place<V, kBwdSteps, kBwdWaves> at(take_tile(counter, &sh.tile), o, p.seqlen, p.dim, true);
  const int lane = at.lane, wave = at.wave, span = o.spans - 1 - at.turn;
  const int64_t step = p.batch * p.dim, state = at.b * p.dim + at.c;
  Steps<IO, V> s;
  float rate[V], A1[V], B1[V], M1[V], h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    A1[v] = 1.0f;
    B1[v] = M1[v] = 0.0f;
    rate[v] = p.A[at.c + v];
    h[v] = p.checkpoints[(at.b * o.spans + span) * p.dim + at.c + v];
  }
  const uint32_t resets = reset_bits(p.reset, at.row, at.steps);
  const bool plain = at.steps == kBwdSteps && resets == 0;
  if (plain)
    bwd_maps<true, LAST>(p, at, resets, rate, s, A1, B1, M1);
  else if (at.steps > 0)
    bwd_maps<false, LAST>(p, at, resets, rate, s, A1, B1, M1);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    sh.A[wave][v][lane] = A1[v];
    mapB[wave][v][lane] = B1[v];
    sh.B[wave][v][lane] = M1[v];
  }
  __syncthreads();
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (wave == v) {
      float out;
      if (pass_on<true>(v, at, o.spans, step, state, p.dim, words, p.dlast, sh, out) && p.dh0) p.dh0[state + v] = out;
    }
  for (int k = 0; k < wave; ++k)
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = through(sh.A[k][v][lane], mapB[k][v][lane], h[v]);
  if (plain)
    bwd_states<true>(at.steps, resets, h, s);
  else
    bwd_states<false>(at.steps, resets, h, s);
  __syncthreads();
  float dA[V], m[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    dA[v] = 0.0f;
    m[v] = sh.enter[v][lane];
  }
  for (int k = kBwdWaves - 1; k > wave; --k)
#pragma unroll
    for (int v = 0; v < V; ++v) m[v] = through(sh.A[k][v][lane], sh.B[k][v][lane], m[v]);
  if (plain)
    bwd_grads<true, LAST>(p, at, resets, rate, s, m, dA);
  else if (at.steps > 0)
    bwd_grads<false, LAST>(p, at, resets, rate, s, m, dA);
  // the waves' parts of dA, added in their order (mapB is read no more)
#pragma unroll
  for (int v = 0; v < V; ++v) mapB[wave][v][lane] = dA[v];
  __syncthreads();
  if (wave == 0)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float sum = 0.0f;
#pragma unroll
      for (int k = 0; k < kBwdWaves; ++k) sum += mapB[k][v][lane];
      parts[at.turn * step + state + v] = sum;
    }
}

constexpr int kTokenRows = 4;   // batch rows per thread, loaded together

// One decode token: a channel of kTokenRows batch rows per thread. Bound by
// HBM: state in and out, three inputs, one output. 4096 x 5120 bf16: 63 us,
// 5.3 TB/s; with one, two or eight rows per thread 87, 62 and 64.5, and 1024 x 5120
// 24.1, 17.1 and 15.5 against 15.6. (Two channels per thread instead of one were
// 4 % slower, four 21 %: with plain loads and one output buffer for all calls.)
// The inputs carry the non-temporal hint at every size: 4096 x 5120 bf16 62.5 us
// against 66.2, 2048 rows 29.2 against 30.6, 1024 rows 15.6 against 14.0, 512 and
// fewer the same.
template <class IO>
__global__ __launch_bounds__(kLanes) void gated_update_kernel(GatedUpdateProblem p) {
  using raw = typename IO::raw;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kLanes + threadIdx.x;
  if (c >= p.dim) return;
  const float rate = p.A[c] * kLog2e;
  for (int64_t b0 = static_cast<int64_t>(blockIdx.y) * kTokenRows; b0 < p.batch;
       b0 += static_cast<int64_t>(gridDim.y) * kTokenRows) {
    Piece<IO, 1> x[kTokenRows], r[kTokenRows], g[kTokenRows];
    float h[kTokenRows];
#pragma unroll
    for (int i = 0; i < kTokenRows; ++i) {
      const int64_t b = b0 + i < p.batch ? b0 + i : p.batch - 1;  // past the end: not used
      h[i] = p.state[b * p.dim + c];
      x[i].load_last(static_cast<const raw*>(p.x) + b * p.sx + c);
      r[i].load_last(static_cast<const raw*>(p.r) + b * p.sr + c);
      g[i].load_last(static_cast<const raw*>(p.g) + b * p.sg + c);
    }
#pragma unroll
    for (int i = 0; i < kTokenRows; ++i) {
      const int64_t b = b0 + i;
      if (b >= p.batch) break;
      float a;
      const float w = decay_weight(rate, sigmoid_f(r[i].get(0)), a);
      const float next = fmaf(a, h[i], w * (sigmoid_f(g[i].get(0)) * x[i].get(0)));
      p.state[b * p.dim + c] = next;
      static_cast<raw*>(p.out)[b * p.so + c] = IO::from_f32(next);
    }
  }
}

Order order_of(int64_t batch, int64_t seqlen, int64_t dim, int V, int64_t span) {
  Order o;
  o.tiles = static_cast<int>((dim + kLanes * V - 1) / (kLanes * V));
  o.per_span = static_cast<int>(batch * o.tiles);
  o.spans = static_cast<int>((seqlen + span - 1) / span);
  return o;
}

dim3 grid_of(const Order& o) { return dim3(static_cast<unsigned>(o.per_span) * o.spans); }

size_t rounded_up(size_t bytes) { return (bytes + 255) / 256 * 256; }

// The counter and one word per channel of every span but the last; nothing for
// sequences of one span, whose tiles wait for nobody.
size_t words_bytes(int64_t batch, int64_t seqlen, int64_t dim, int64_t span) {
  const int64_t spans = (seqlen + span - 1) / span;
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
  const Order o = order_of(p.batch, p.seqlen, p.dim, V, kFwdSpan);
  const size_t bytes = words_bytes(p.batch, p.seqlen, p.dim, kFwdSpan);
  if (bytes) {
    const hipError_t e = clear_words(workspace, bytes, stream);
    if (e != hipSuccess) return e;
  }
  unsigned* counter = bytes ? static_cast<unsigned*>(workspace) : nullptr;
  u64* words = bytes ? reinterpret_cast<u64*>(static_cast<char*>(workspace) + kHeader) : nullptr;
  const auto kernel = streams(4 * p.batch * p.seqlen * p.dim * static_cast<int64_t>(sizeof(typename IO::raw)))
                          ? gated_fwd_kernel<IO, V, true>
                          : gated_fwd_kernel<IO, V, false>;
  hipLaunchKernelGGL(kernel, grid_of(o), dim3(kFwdThreads), 0, stream, p, o, counter, words);
  return hipGetLastError();
}

template <class IO, int V>
hipError_t launch_bwd(const GatedBwdProblem& p, void* workspace, hipStream_t stream) {
  const Order o = order_of(p.batch, p.seqlen, p.dim, V, kGatedCheckpoint);
  const size_t bytes = words_bytes(p.batch, p.seqlen, p.dim, kGatedCheckpoint);
  if (bytes) {
    const hipError_t e = clear_words(workspace, bytes, stream);
    if (e != hipSuccess) return e;
  }
  char* ws = static_cast<char*>(workspace);
  unsigned* counter = bytes ? reinterpret_cast<unsigned*>(ws) : nullptr;
  u64* words = bytes ? reinterpret_cast<u64*>(ws + kHeader) : nullptr;
  float* parts = reinterpret_cast<float*>(ws + bytes);
  const auto kernel = streams(7 * p.batch * p.seqlen * p.dim * static_cast<int64_t>(sizeof(typename IO::raw)))
                          ? gated_bwd_kernel<IO, V, true>
                          : gated_bwd_kernel<IO, V, false>;
  hipLaunchKernelGGL(kernel, grid_of(o), dim3(kBwdThreads), 0, stream, p, o, counter, words, parts);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return launch_colsum(parts, p.batch * o.spans, p.dim, StoreFlat{p.dA}, stream);
}

}  // namespace

size_t gated_fwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim) {
  return words_bytes(batch, seqlen, dim, kFwdSpan);
}

size_t gated_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim) {
  const int64_t spans = (seqlen + kGatedCheckpoint - 1) / kGatedCheckpoint;
  return words_bytes(batch, seqlen, dim, kGatedCheckpoint) + rounded_up(static_cast<size_t>(spans * batch * dim) * 4);
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
  return launch_bwd<F32Io, 1>(p, workspace, stream);
}

hipError_t launch_gated_update(const GatedUpdateProblem& p, hipStream_t stream) {
  const int64_t rows = (p.batch + kTokenRows - 1) / kTokenRows;
  const dim3 grid(static_cast<unsigned>((p.dim + kLanes - 1) / kLanes),
                  static_cast<unsigned>(rows < 65535 ? rows : 65535));
  if (p.io == kIoBf16)
    hipLaunchKernelGGL((gated_update_kernel<Bf16Io>), grid, dim3(kLanes), 0, stream, p);
  else
    hipLaunchKernelGGL((gated_update_kernel<F32Io>), grid, dim3(kLanes), 0, stream, p);
  return hipGetLastError();
}

}  // namespace mscan

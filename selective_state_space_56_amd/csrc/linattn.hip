// Linear attention with a decay for each head: how a call is cut into roles and
// segments, and the small kernels around the map's own (linattn.h).
#include "colsum.h"
#include "linattn_walk.h"

namespace mscan {

namespace {

// ---------------------------------------------------------------------------
// Segments. The state that enters segment p + 1 of a sequence is
// gone_p enter_p + local_p, of which local and gone are known by then, and local_p alone behind a
// cut, whatever enters; enter takes local's place. A thread takes four elements of one (sequence, head), and loads the next
// segments' before it needs them: bound by that latency (25 segments of 20 states of
// 128 x 128, 66 MB: 15 us).
constexpr int kJoinThreads = 256;
constexpr int kJoinAhead = 8;

__global__ __launch_bounds__(kJoinThreads) void join_kernel(MixCall w, int chunk, int64_t blocks) {
  const MixRole& r = w.role[blockIdx.y];
  const int64_t size = static_cast<int64_t>(r.K) * r.V;
  const int64_t e = ((blockIdx.x % blocks) * kJoinThreads + threadIdx.x) * 4;
  const int64_t sh = blockIdx.x / blocks;
  const int own_head = static_cast<int>(sh % w.some);
  const int64_t seq = sh / w.some;
  if (e >= size) return;
  const Sequence s = sequence_of(w.offsets, seq, w.seqlen, w.rows);
  const int64_t base = first_slot(s.begin, seq, static_cast<uint32_t>(w.per) * chunk);
  const int segs = segments_of(static_cast<int>((s.len + chunk - 1) / chunk), w.per);
  float cur[4] = {};
  if (r.s0) {
    const float* from = r.s0 + (seq * w.heads + w.head0 + own_head) * size;
    for (int k = 0; k < 4; ++k)
      cur[k] = r.s0_turned ? from[(e + k) % r.V * r.K + (e + k) / r.V] : from[e + k];
  }
  // kJoinAhead segments' loads go out together
  for (int p0 = 0; p0 < segs; p0 += kJoinAhead) {
    float own[kJoinAhead][4], gone[kJoinAhead];
#pragma unroll
    for (int i = 0; i < kJoinAhead; ++i) {
      Piece<F32Io, 4> piece = {};
      gone[i] = 0.0f;
      if (p0 + i + 1 < segs) {  // (nobody needs what the last one leaves)
        const int64_t at = (base + (r.reverse ? segs - 1 - p0 - i : p0 + i)) * w.some + own_head;
        piece.load(r.local + at * size + e);
        gone[i] = r.gone[at];
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) own[i][k] = piece.get(k);
    }
#pragma unroll
    for (int i = 0; i < kJoinAhead; ++i) {
      if (p0 + i >= segs) break;
      const int64_t at = (base + (r.reverse ? segs - 1 - p0 - i : p0 + i)) * w.some + own_head;
      Piece<F32Io, 4> piece;
      piece.set(cur);
      piece.store(r.local + at * size + e);
#pragma unroll
      for (int k = 0; k < 4; ++k) cur[k] = gone[i] < 0.0f ? own[i][k] : fmaf(gone[i], cur[k], own[i][k]);
    }
  }
}

// ---------------------------------------------------------------------------
// Gradients of the decays. dg_t is the sum of what crosses step t of a chunk,
//   dg_t = e^{ell_C} <S_in, dS_out> + sum_{s < t} a_s + sum_{u >= t} b_u + pairs_t
// with what the runs leave: the state S_in that enters the chunk and the gradient dS_out of the one
// that leaves it (dq's and dk's run, as V x K both), a_s = end_s k_s . (dS_out v_s),
// b_u = in_u scale q_u . (S_in dout_u), and the chunk's own pairs that t lies between. Every term is a part of
// dg_t itself and none is subtracted: the difference of q . dq and k . dk summed from the
// sequence's end, which is the same, or a product <S, dS> carried from chunk to chunk, leaves the
// rounding of what other tokens add, which is more than strong decays, early tokens or small
// gradients before large ones leave of dg_t.
// One workgroup for each chunk and head. Bound by HBM: both states are read (8 x 2048 steps of 20 heads of
// 128 x 128, bf16: 0.63 GB in 117 us, 5.4 TB/s; with four and eight pieces in flight per thread the training
// step of that size takes 671 and 710 us, with two 661).
constexpr int kDecayThreads = 256;
constexpr int kDecayAhead = 2;               // 16-byte pieces of each state in flight per thread
constexpr int64_t kDecayGroups = int64_t(1) << 16;  // workgroups at most; each takes every kDecayGroups-th chunk and head

struct DecayGrad {
  MixCall w;                 // sequences; per is not used
  const float* a;            // (tiles, heads, rows)
  const float* b;            // the same
  const float* pairs;        // the same
  const float* S;            // (chunk slots, some, size), in the runs' order of elements
  const float* dS;           // (inner slots, some, size), the same
  const float* dlast;        // (batch, heads, K, V): for a sequence's last chunk; or null
  bool first;                // whether a state enters a sequence's first chunk
  float* dg;                 // (rows, heads), or null:
  float* parts;              // (chunk slots, heads): sums over the chunk
  int64_t slots;
  int tiles, K, V;
  int64_t size;
};

// Where a run leaves its registers 4 j .. 4 j + 3: the first of four rows of a 32 x 32 tile.
template <int C>
__device__ __forceinline__ int quad_row(int j, int hi) { return C == 64 ? 16 * (j >> 1) + 8 * hi + 4 * (j & 1) : 8 * j + 4 * hi; }

// Sum over a wave, in each lane.
__device__ __forceinline__ double over_wave(double v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off);
  return v;
}

template <int C>
__global__ __launch_bounds__(kDecayThreads) void decay_grad_kernel(DecayGrad p) {
  const MixCall& w = p.w;
  constexpr int kWaves = kDecayThreads / 64;
  __shared__ double s_sum[2][kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int turn = 0;
  for (int64_t unit = blockIdx.x; unit < p.slots * w.some; unit += gridDim.x) {
    const int own = static_cast<int>(unit % w.some), head = w.head0 + own;
    const int64_t slot = unit / w.some;
    const int seq = w.offsets ? sequence_at(w.offsets, w.batch, w.seqlen, w.rows, C, slot)
                              : static_cast<int>(slot / ((w.seqlen + C - 1) / C));
    const Sequence s = sequence_of(w.offsets, seq, w.seqlen, w.rows);
    const int64_t chunks = (s.len + C - 1) / C, c = slot - chunk_slot(w.offsets, w.seqlen, s.begin, seq, 0, C);
    if (c < 0 || c >= chunks) {  // (a slot that no chunk has)
      if (p.parts && tid == 0) p.parts[slot * w.heads + head] = 0.0f;
      continue;
    }
    // every wave for itself, a step per lane
    const int64_t left = s.len - c * C, row = s.begin + c * C + lane;
    const bool on = lane < C && lane < left;
    const float g = on ? w.g[row * w.g_step + head] : 0.0f;
    const bool cut = on && g <= kNoDecay;
    const uint64_t cuts = __ballot(cut);
    const double total = over_wave(cut ? 0.0 : static_cast<double>(g));
    const bool through = passes(cuts != 0, total) && (c > 0 || p.first) && (c + 1 < chunks || p.dlast);
    // keys before the last cut reach nothing behind the chunk, and what entered it no query from the first on: what
    // stands there may be anything
    double a = 0.0, b = 0.0, pairs = 0.0;
    if (wave == 0 && on) {
      const bool keeps = (cuts >> lane >> 1) == 0, sees = (cuts & (~uint64_t(0) >> (63 - lane))) == 0;
      for (int k = 0; k < p.tiles; ++k) {
        const int64_t at = (static_cast<int64_t>(k) * w.heads + head) * w.rows + row;
        if (keeps) a += p.a[at];
        if (sees) b += p.b[at];
        pairs += p.pairs[at];
      }
    }
    double dot = 0.0;
    if (through) {
      using Quad = Words<float, 4, 16>;
      const Quad* S = reinterpret_cast<const Quad*>(p.S + unit * p.size);
      const bool inner = c + 1 < chunks;
      const int64_t at = inner ? inner_slot(w.offsets, w.seqlen, s.begin, seq, c, C) * w.some + own : 0;
      const Quad* dS = reinterpret_cast<const Quad*>(p.dS + at * p.size);
      const float* dlast = inner ? nullptr : p.dlast + (static_cast<int64_t>(seq) * w.heads + head) * p.K * p.V;
      const int quads = static_cast<int>(p.size / 4), down = (p.V + 31) / 32;
      for (int e0 = tid; e0 < quads; e0 += kDecayThreads * kDecayAhead) {
        Quad x[kDecayAhead] = {}, y[kDecayAhead] = {};
#pragma unroll
        for (int k = 0; k < kDecayAhead; ++k) {
          const int e = e0 + kDecayThreads * k;
          if (e >= quads) continue;
          x[k] = __builtin_nontemporal_load(S + e);
          if (inner) {
            y[k] = __builtin_nontemporal_load(dS + e);
          } else {  // from rows of keys, of any alignment
            const int key = e / 256 / down * 32 + e % 32, value = e / 256 % down * 32 + quad_row<C>(e / 64 % 4, e / 32 % 2);
            if (key < p.K && value < p.V) y[k] = *reinterpret_cast<const Words<float, 4, 4>*>(dlast + key * p.V + value);
          }
        }
#pragma unroll
        for (int k = 0; k < kDecayAhead; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i) dot = fma(static_cast<double>(x[k][i]), static_cast<double>(y[k][i]), dot);
      }
      dot = over_wave(dot);
    }
    turn ^= 1;  // (the sums of the barrier before may still be read)
    if (lane == 0) s_sum[turn][wave] = dot;
    __syncthreads();
    if (wave > 0) continue;
    // sums before and from each step on
    double pre = a, post = b;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const double u = __shfl_up(pre, off), v = __shfl_down(post, off);
      if (lane >= off) pre += u;
      if (lane + off < 64) post += v;
    }
    pre = __shfl_up(pre, 1);
    double grad = (lane == 0 ? 0.0 : pre) + post + pairs;
    if (through) {
      double sum = 0.0;
      for (int k = 0; k < kWaves; ++k) sum += s_sum[turn][k];
      grad += exp_exactly(total) * sum;
    }
    if (!on || cut) grad = 0.0;  // the gradient of a cut is 0
    if (p.dg && on) p.dg[row * w.heads + head] = static_cast<float>(grad);
    if (p.parts) {
      grad = over_wave(grad);
      if (lane == 0) p.parts[slot * w.heads + head] = static_cast<float>(grad);
    }
  }
}

// ---------------------------------------------------------------------------
// Gradients of shared queries and keys: the sum over a group's heads, in order, of
// the float32 rows that the heads have written, 8 values per thread. Bound by HBM (4000
// rows of 32 heads of 64 into 16, dq and dk: 13 us, 82 MB read, 6.3 TB/s from the last-level
// cache).
struct GroupSum {
  const float* part[2];      // (rows, heads, K)
  void* to[2];
  int64_t stride[2];
  const int64_t* offsets;
  int64_t rows, pieces;      // pieces: 8-value pieces of a row of `to`
  int heads, groups, K, batch;
};

template <class IO>
__global__ __launch_bounds__(256) void group_sum_kernel(GroupSum p) {
  const int64_t begin = p.offsets ? offset_of(p.offsets, 0, 0, p.rows) : 0;
  const int64_t end = p.offsets ? offset_of(p.offsets, p.batch, 0, p.rows) : p.rows;
  const int per = p.heads / p.groups;
  for (int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; id < p.rows * p.pieces;
       id += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t row = id / p.pieces;
    if (row < begin || row >= end) continue;
    const int x = static_cast<int>(id % p.pieces) * 8, group = x / p.K, c = x % p.K;
    const float* from = (blockIdx.y ? p.part[1] : p.part[0]) + (row * p.heads + static_cast<int64_t>(group) * per) * p.K + c;
    float sum[8] = {};
    for (int h = 0; h < per; ++h, from += p.K) {
      Piece<F32Io, 8> v;
      v.load(from);
#pragma unroll
      for (int k = 0; k < 8; ++k) sum[k] += v.get(k);
    }
    Piece<IO, 8> out;
    out.set(sum);
    out.store(static_cast<typename IO::raw*>(blockIdx.y ? p.to[1] : p.to[0]) +
              row * (blockIdx.y ? p.stride[1] : p.stride[0]) + x);
  }
}

// ---------------------------------------------------------------------------
// Zeros in the rows before the first and behind the last of packed sequences. Few or none as
// a rule, so few workgroups look (256: 1.9 us, 2048: 4.8).
struct RestRows {
  void* to[4];
  int64_t stride[4], bytes[4];  // in bytes; bytes: of a row, 0 for no tensor
  const int64_t* offsets;
  int64_t rows;
  int batch;
};

__global__ __launch_bounds__(256) void zero_rest_kernel(RestRows p) {
  const int64_t a = offset_of(p.offsets, 0, 0, p.rows);
  int64_t b = offset_of(p.offsets, p.batch, 0, p.rows);
  if (b < a) b = a;
  const int64_t rest = a + p.rows - b;
  for (int64_t i = blockIdx.x; i < rest; i += gridDim.x) {
    const int64_t row = i < a ? i : i - a + b;
    for (int k = 0; k < 4; ++k)
      for (int64_t x = 2 * threadIdx.x; x < p.bytes[k]; x += 512)
        *reinterpret_cast<uint16_t*>(static_cast<char*>(p.to[k]) + row * p.stride[k] + x) = 0;
  }
}

// ---------------------------------------------------------------------------

size_t r256(size_t v) { return (v + 255) / 256 * 256; }

int64_t compute_units() {
  int dev = 0, n = 0;
  if (hipGetDevice(&dev) != hipSuccess ||
      hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0)
    n = 256;
  return n;
}

// Steps of a chunk: what the kernels' tiles hold.
int chunk_of(const LinattnSizes& n) { return n.io == MAMBA_F32 ? 32 : 64; }
int64_t chunks_of(const LinattnSizes& n) { return (n.rows + chunk_of(n) - 1) / chunk_of(n); }

// Chunks of a segment, when `walks` workgroups walk each sequence. One segment per
// sequence reads everything once; more let few sequences fill the machine, planned as two
// workgroups for each compute unit (which hold one where a state has over 128 rows, and in float32 with
// four tiles, two waves and sums: half of those wait), at the price of reading keys and values twice and of
// the states between. Sequences of one length get as many segments as workgroups fit (one
// more would wait for a place: 131072 steps of 20 heads, 500 workgroups 1.25 ms, 520 1.32).
// Of packed sequences the lengths are not known here: they are cut as one would be, unless
// there are very many. Down to one chunk: at least 8, 4, 2 and 1 of them took 87, 57, 47
// and 54 us for 1 x 2048 steps of 16 heads (128 x 128 bf16), 49, 51, 36 and 31 for 512 of 8, and
// 675, 377, 218 and 145 for the gradients of 881 of 6 heads (40 x 72 fp32, in chunks of 64).
int per_of(const LinattnSizes& n, int64_t walks) {
  const int64_t chunks = chunks_of(n), want = 2 * compute_units(), whole = chunks + 1, units = n.batch * walks;
  if (n.packed) {
    if (units >= 16 * want) return static_cast<int>(whole);
    const int64_t per = (chunks * walks + want - 1) / want;
    return static_cast<int>(per < 1 ? 1 : per < whole ? per : whole);
  }
  if (units == 0 || 2 * units > want) return static_cast<int>(whole);
  const int64_t own = (n.seqlen + chunk_of(n) - 1) / chunk_of(n), segs = want / units;
  const int64_t per = segs > own ? 1 : (own + segs - 1) / segs;
  return static_cast<int>(per < 1 ? 1 : per);
}
bool split(const LinattnSizes& n, int per) { return per <= (n.packed ? chunks_of(n) : (n.seqlen - 1) / chunk_of(n)); }

MixCall call_of(const LinattnProblem& p) {
  MixCall w{};
  w.offsets = p.offsets;
  w.g = p.g;
  w.g_step = p.head_decay ? 0 : p.n.heads;
  w.seqlen = p.n.seqlen;
  w.rows = p.n.rows;
  w.batch = static_cast<int>(p.n.batch);
  w.heads = w.some = static_cast<int>(p.n.heads);
  return w;
}

void set_segments(MixCall& w, const LinattnSizes& n, int per) {
  w.per = per;
  w.slots = slots_of(n.rows, n.batch, static_cast<int64_t>(per) * chunk_of(n));
}

// What a run's segments need of the workspace: their states and decays.
struct SegmentBytes {
  size_t states, gone;
  size_t total() const { return states + gone; }
};
SegmentBytes segment_bytes(const LinattnSizes& n, int per, int64_t heads) {
  if (!split(n, per)) return {0, 0};
  const size_t at = static_cast<size_t>(slots_of(n.rows, n.batch, static_cast<int64_t>(per) * chunk_of(n))) * heads;
  return {r256(at * n.K * n.V * 4), r256(at * 4)};
}

void give_segments(MixRole& r, const SegmentBytes& s, char*& at) {
  r.local = reinterpret_cast<float*>(at);
  r.gone = reinterpret_cast<float*>(at + s.states);
  at += s.total();
}

hipError_t walk(const MixCall& w, int io, hipStream_t stream) {
  return io == MAMBA_BF16 ? launch_walk_bf16(w, stream) : launch_walk_f32(w, stream);
}

// The runs of w: with segments, first what each leaves, then what enters each.
hipError_t run(MixCall w, const LinattnSizes& n, bool cut, hipStream_t stream) {
  const int chunk = chunk_of(n);
  w.tiles = value_tiles(w.role[0].V);
  w.together = static_cast<uint32_t>(n.heads / n.groups * w.tiles * w.roles);
  if (cut) {
    hipError_t e = walk(w, n.io, stream);
    if (e != hipSuccess) return e;
    const int64_t blocks = (n.K * n.V / 4 + kJoinThreads - 1) / kJoinThreads;
    hipLaunchKernelGGL(join_kernel, dim3(static_cast<unsigned>(n.batch * w.some * blocks), w.roles), dim3(kJoinThreads),
                       0, stream, w, chunk, blocks);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  for (int k = 0; k < w.roles; ++k) {
    w.role[k].enter = w.role[k].local;
    w.role[k].local = nullptr;
  }
  return walk(w, n.io, stream);
}

hipError_t zero_rest(const RestRows& z, hipStream_t stream) {
  hipLaunchKernelGGL(zero_rest_kernel, dim3(static_cast<unsigned>(z.rows < 256 ? z.rows : 256)), dim3(256), 0, stream, z);
  return hipGetLastError();
}

// The backward's three runs go in one launch if their operands have one shape: they are the
// same rows. Else dv's is one and that of dk and dq another, each with segments of its own
// (forward and backward of 4 x 1000 steps of 32 heads of 64 x 128 took 260 us, with segments
// as for one launch of all 290; 279 since the decays' gradients take every chunk's states).
bool one_shape(const LinattnSizes& n) {
  return key_tiles(n.K) == key_tiles(n.V) && value_width(n.V) == value_width(n.K) && value_tiles(n.V) == value_tiles(n.K);
}
// For the decays' gradients a state and its gradient are kept for every chunk, as much as the io tensors of
// 128 x 128 heads together. Where they would take more than this, the backward goes through its heads in turn,
// some groups at a time, which fill the machine by segments.
constexpr int64_t kStatesBytes = int64_t(8) << 30;

int64_t state_bytes(const LinattnSizes& n, int64_t slots) { return slots * entering_size(n.V, n.K) * 4; }
int64_t heads_at_a_time(const LinattnSizes& n) {
  const int64_t share = n.heads / n.groups;
  const int64_t group = share * state_bytes(n, chunk_slots_of(n, chunk_of(n)) + inner_slots_of(n, chunk_of(n)));
  const int64_t fit = group > kStatesBytes ? 1 : group > 0 ? kStatesBytes / group : n.groups;
  if (fit >= n.groups) return n.heads;
  const int64_t turns = (n.groups + fit - 1) / fit;
  return (n.groups + turns - 1) / turns * share;
}
int dv_per(const LinattnSizes& n) { return per_of(n, heads_at_a_time(n) * value_tiles(n.V) * (one_shape(n) ? 3 : 1)); }
int dk_dq_per(const LinattnSizes& n) { return per_of(n, heads_at_a_time(n) * value_tiles(n.K) * (one_shape(n) ? 3 : 2)); }

// The backward's workspace.
struct BwdBytes {
  SegmentBytes dv, dk_dq;
  size_t S, dS, sums, part, parts;
  int64_t slots;             // of chunks
  size_t total() const { return dv.total() + 2 * dk_dq.total() + S + dS + 3 * sums + 2 * part + parts; }
};
BwdBytes bwd_bytes(const LinattnSizes& n, bool head_decay) {
  BwdBytes s;
  const int64_t some = heads_at_a_time(n);
  s.dv = segment_bytes(n, dv_per(n), some);
  s.dk_dq = segment_bytes(n, dk_dq_per(n), some);
  s.slots = chunk_slots_of(n, chunk_of(n));
  s.S = r256(some * state_bytes(n, s.slots));
  s.dS = r256(some * state_bytes(n, inner_slots_of(n, chunk_of(n))));
  s.sums = r256(static_cast<size_t>(value_tiles(n.K)) * n.heads * n.rows * 4);
  s.part = n.heads == n.groups ? 0 : r256(static_cast<size_t>(n.rows) * n.heads * n.K * 4);
  s.parts = head_decay ? r256(static_cast<size_t>(s.slots) * n.heads * 4) : 0;
  return s;
}

}  // namespace

size_t linattn_fwd_workspace_bytes(const LinattnSizes& n) {
  if (n.rows == 0 || n.heads == 0 || n.batch == 0) return 0;
  return segment_bytes(n, per_of(n, n.heads * value_tiles(n.V)), n.heads).total();
}

size_t linattn_bwd_workspace_bytes(const LinattnSizes& n, bool head_decay) {
  if (n.rows == 0 || n.heads == 0 || n.batch == 0) return 0;
  return bwd_bytes(n, head_decay).total();
}

hipError_t launch_linattn_fwd(const LinattnProblem& p, void* workspace, hipStream_t stream) {
  const LinattnSizes& n = p.n;
  const int eb = n.io == MAMBA_BF16 ? 2 : 4;
  if (p.zero_rest && n.rows > 0) {
    RestRows z{};
    z.to[0] = p.out;
    z.stride[0] = p.so * eb;
    z.bytes[0] = n.heads * n.V * eb;
    z.offsets = p.offsets;
    z.rows = n.rows;
    z.batch = static_cast<int>(n.batch);
    const hipError_t e = zero_rest(z, stream);
    if (e != hipSuccess) return e;
  }
  if (n.batch == 0) return hipSuccess;
  MixCall w = call_of(p);
  const int per = per_of(n, n.heads * value_tiles(n.V));
  set_segments(w, n, per);
  w.roles = 1;
  MixRole& r = w.role[0];
  r.q = p.q;
  r.k = p.k;
  r.v = p.v;
  r.o = p.out;
  r.sq = p.sq;
  r.sk = p.sk;
  r.sv = p.sv;
  r.so = p.so;
  r.qdiv = r.kdiv = static_cast<int>(n.heads / n.groups);
  r.vdiv = r.ediv = 1;
  r.K = static_cast<int>(n.K);
  r.V = static_cast<int>(n.V);
  r.s0 = p.h0;
  r.last = p.last_state;
  r.score = r.from = p.scale;
  r.to = 1.0f;
  const bool cut = n.rows > 0 && split(n, per);
  char* at = static_cast<char*>(workspace);
  if (cut) give_segments(r, segment_bytes(n, per, n.heads), at);
  return run(w, n, cut, stream);
}

hipError_t launch_linattn_bwd(const LinattnBwdProblem& p, void* workspace, hipStream_t stream) {
  const LinattnProblem& f = p.f;
  const LinattnSizes& n = f.n;
  const int64_t eb = n.io == MAMBA_BF16 ? 2 : 4;
  hipError_t e;
  if (f.zero_rest && n.rows > 0) {
    RestRows z{};
    void* to[4] = {p.dq, p.dk, p.dv, f.head_decay ? nullptr : p.dg};
    const int64_t stride[4] = {p.sdq * eb, p.sdk * eb, p.sdv * eb, n.heads * 4};
    const int64_t bytes[4] = {n.groups * n.K * eb, n.groups * n.K * eb, n.heads * n.V * eb, n.heads * 4};
    for (int k = 0; k < 4; ++k) {
      z.to[k] = to[k];
      z.stride[k] = stride[k];
      z.bytes[k] = to[k] ? bytes[k] : 0;
    }
    z.offsets = f.offsets;
    z.rows = n.rows;
    z.batch = static_cast<int>(n.batch);
    if ((e = zero_rest(z, stream)) != hipSuccess) return e;
  }
  const bool work = n.batch > 0 && n.rows > 0;
  const BwdBytes s = work ? bwd_bytes(n, f.head_decay) : BwdBytes{};
  char* at = static_cast<char*>(workspace);
  auto take = [&at](size_t bytes) {
    float* v = reinterpret_cast<float*>(at);
    at += bytes;
    return v;
  };
  if (n.batch > 0) {
    MixCall w = call_of(f);
    const int share = static_cast<int>(n.heads / n.groups), K = static_cast<int>(n.K), V = static_cast<int>(n.V);
    // dv: queries k, keys q, values dout, in reverse; the state is dS (K x V)
    MixRole dv{};
    dv.q = f.k;
    dv.sq = f.sk;
    dv.k = f.q;
    dv.sk = f.sq;
    dv.v = p.dout;
    dv.sv = f.so;
    dv.qdiv = dv.kdiv = share;
    dv.vdiv = dv.ediv = 1;
    dv.o = p.dv;
    dv.so = p.sdv;
    dv.K = K;
    dv.V = V;
    dv.s0 = p.dlast;
    dv.last = p.dh0;
    dv.reverse = true;
    dv.score = dv.to = f.scale;
    dv.from = 1.0f;
    // dk: queries v, keys dout, values q, in reverse; dS^T (V x K)
    MixRole dk{};
    dk.q = f.v;
    dk.sq = f.sv;
    dk.k = p.dout;
    dk.sk = f.so;
    dk.v = f.q;
    dk.sv = f.sq;
    dk.qdiv = dk.kdiv = 1;
    dk.vdiv = dk.ediv = share;
    dk.o = p.dk;
    dk.so = p.sdk;
    dk.K = V;
    dk.V = K;
    dk.s0 = p.dlast;
    dk.s0_turned = true;
    dk.reverse = true;
    dk.score = dk.to = f.scale;
    dk.from = 1.0f;
    // dq: queries dout, keys v, values k; S^T (V x K)
    MixRole dq = dk;
    dq.q = p.dout;
    dq.sq = f.so;
    dq.k = f.v;
    dq.sk = f.sv;
    dq.v = f.k;
    dq.sv = f.sk;
    dq.o = p.dq;
    dq.so = p.sdq;
    dq.s0 = f.h0;
    dq.reverse = false;
    dq.score = dq.from = f.scale;
    dq.to = 1.0f;
    const bool cut_dv = work && split(n, dv_per(n)), cut_dk_dq = work && split(n, dk_dq_per(n));
    if (cut_dv) give_segments(dv, s.dv, at);
    if (cut_dk_dq)
      for (MixRole* r : {&dk, &dq}) give_segments(*r, s.dk_dq, at);
    DecayGrad d{};
    if (work && p.dg) {
      dk.e = f.k;
      dk.se = f.sk;
      dk.entering = take(s.dS);
      dk.sums = take(s.sums);
      dq.e = f.q;
      dq.se = f.sq;
      dq.entering = take(s.S);
      dq.sums = take(s.sums);
      dq.pairs = take(s.sums);
      d.w = w;
      d.a = dk.sums;
      d.b = dq.sums;
      d.pairs = dq.pairs;
      d.S = dq.entering;
      d.dS = dk.entering;
      d.dlast = p.dlast;
      d.first = f.h0 != nullptr;
      d.dg = f.head_decay ? nullptr : p.dg;
      d.parts = f.head_decay ? take(s.parts) : nullptr;
      d.slots = s.slots;
      d.tiles = value_tiles(K);
      d.K = K;
      d.V = V;
      d.size = entering_size(V, K);
    }
    if (work && share > 1) {
      dq.part = take(s.part);
      dk.part = take(s.part);
    }
    const int some = static_cast<int>(work ? heads_at_a_time(n) : n.heads);
    for (int h = 0; h < n.heads; h += some) {
      w.head0 = h;
      w.some = n.heads - h < some ? static_cast<int>(n.heads) - h : some;
      set_segments(w, n, dv_per(n));
      w.role[0] = dv;
      w.roles = 1;
      if (one_shape(n)) {
        w.role[1] = dk;
        w.role[2] = dq;
        w.roles = 3;
      }
      if ((e = run(w, n, cut_dv, stream)) != hipSuccess) return e;
      if (!one_shape(n)) {
        set_segments(w, n, dk_dq_per(n));
        w.role[0] = dk;
        w.role[1] = dq;
        w.roles = 2;
        if ((e = run(w, n, cut_dk_dq, stream)) != hipSuccess) return e;
      }
      if (work && p.dg) {
        d.w.head0 = w.head0;
        d.w.some = w.some;
        const int64_t units = s.slots * w.some;
        const dim3 grid(static_cast<unsigned>(units < kDecayGroups ? units : kDecayGroups));
        if (chunk_of(n) == 64)
          hipLaunchKernelGGL((decay_grad_kernel<64>), grid, dim3(kDecayThreads), 0, stream, d);
        else
          hipLaunchKernelGGL((decay_grad_kernel<32>), grid, dim3(kDecayThreads), 0, stream, d);
        if ((e = hipGetLastError()) != hipSuccess) return e;
      }
    }
    if (work && share > 1) {
      GroupSum gs{};
      gs.part[0] = dq.part;
      gs.part[1] = dk.part;
      gs.to[0] = p.dq;
      gs.to[1] = p.dk;
      gs.stride[0] = p.sdq;
      gs.stride[1] = p.sdk;
      gs.offsets = f.offsets;
      gs.rows = n.rows;
      gs.pieces = n.groups * n.K / 8;
      gs.heads = static_cast<int>(n.heads);
      gs.groups = static_cast<int>(n.groups);
      gs.K = K;
      gs.batch = static_cast<int>(n.batch);
      const int64_t groups = (n.rows * gs.pieces + 255) / 256;
      const dim3 grid(static_cast<unsigned>(groups < (1 << 20) ? groups : 1 << 20), 2);
      if (n.io == MAMBA_BF16)
        hipLaunchKernelGGL((group_sum_kernel<Bf16Io>), grid, dim3(256), 0, stream, gs);
      else
        hipLaunchKernelGGL((group_sum_kernel<F32Io>), grid, dim3(256), 0, stream, gs);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (work && p.dg && f.head_decay) return launch_colsum(d.parts, s.slots, n.heads, StoreFlat{p.dg}, stream);
  }
  // no tokens: a decay that every token shares has the gradient 0
  if (!work && p.dg && f.head_decay) return launch_colsum(nullptr, 0, n.heads, StoreFlat{p.dg}, stream);
  return hipSuccess;
}

}  // namespace mscan

// Linear attention in float32 on the matrix cores (v_mfma_f32_32x32x2_f32): the
// map of linattn.h over the chunks of one segment, for one head and up to 128
// value channels per workgroup.
//
// Operand layouts (wave64, lane l): A (32 x 2): row l % 32, k = l / 32; B (2 x 32):
// column l % 32, k = l / 32; D (32 x 32): register r is row 8 (r / 4) + 4 (l / 32) +
// r % 4, column l % 32. A product's terms may come in any order, as long as both
// operands agree: taken as rows 8 j + 4 (l / 32) + e of the four instructions e,
// they make S and the scores usable as operands just as they stand in the
// registers of D, and four of A's values are one 16-byte read.
//
// Bound by the matrix cores: 8 x 2048 steps of 40 heads of 128 x 128 take 1.04 ms, 49
// TFLOP/s of 152 that a large product reaches, since 320 workgroups on 256 compute units are
// two rounds for some, and since one wave makes a chunk's scores while the others wait. Chunks of 32 steps, not 64 as with bf16: half the scores, and
// two workgroups fit a compute unit, one of which has products to issue while the other
// waits (64 steps and one workgroup, rows loaded when they were needed: 1.80 ms, its
// gradients 4.83 where they then took 2.76; 3.29 with every chunk's states for those of the decays). The next chunk's rows are loaded while one is worked on.
#include "linattn_walk.h"

namespace mscan {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x16 mfma(float a, float b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x2f32(a, b, c, 0, 0, 0);
}

constexpr int kC = 32;  // steps of a chunk

// Rows of D: see above.
struct Layout {
  static constexpr int kRows = 16, kLane = 4;
  static constexpr int row(int tile, int i) { return 32 * tile + 8 * (i >> 2) + (i & 3); }
};

// One operand's rows of a chunk, 8 values at a time: W per row (0 from `have` on and past
// the chunk's end), N pieces per thread.
template <int W, int THREADS>
struct Rows {
  static constexpr int kPer = W / 8, N = kC * kPer / THREADS;
  static_assert(kC * kPer % THREADS == 0, "whole rows of pieces");
  const float* base;
  int64_t stride;
  int have;
  bool back;

  __device__ __forceinline__ Rows(const void* p, int64_t first_row, int64_t stride_, int64_t first_col, int have_, bool reverse)
      : base(static_cast<const float*>(p) + first_row * stride_ + first_col), stride(stride_), have(have_), back(reverse) {}
  // rows of a chunk that starts c0 steps into the sequence and has n
  __device__ __forceinline__ void load(f32x4 (&to)[2 * N], int tid, int64_t c0, int n) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int id = tid + i * THREADS, row = id / kPer, x = 8 * (id % kPer);
      to[2 * i] = to[2 * i + 1] = f32x4{};
      if (row < n && x < have) {
        Piece<F32Io, 8> v;
        v.load(base + (c0 + (back ? n - 1 - row : row)) * stride + x);
        to[2 * i] = f32x4{v.get(0), v.get(1), v.get(2), v.get(3)};
        to[2 * i + 1] = f32x4{v.get(4), v.get(5), v.get(6), v.get(7)};
      }
    }
  }
  static __device__ __forceinline__ void keep(const f32x4 (&from)[2 * N], float* tile, int ld) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int id = threadIdx.x + i * THREADS;
      float* to = tile + id / kPer * ld + 8 * (id % kPer);
      *reinterpret_cast<f32x4*>(to) = from[2 * i];
      *reinterpret_cast<f32x4*>(to + 4) = from[2 * i + 1];
    }
  }
};

// Waves per SIMD that the kernels' registers are held to: two workgroups, where they fit.
constexpr int least_waves(int KT, int NW, bool sums) { return KT == 8 || (KT == 4 && NW == 2 && sums) ? 1 : 2; }

// KT: 32-row tiles of the state; NW: waves, 32 value channels each; SUMS: with the sums for
// the decays' gradients.
template <int KT, int NW, bool SUMS>
__global__ __launch_bounds__(64 * NW, least_waves(KT, NW, SUMS)) void walk_f32_kernel(MixCall w) {
  constexpr int C = kC, kK = 32 * KT, kV = 32 * NW, kThreads = 64 * NW;
  constexpr int ldk = kK + 4, ldv = kV + 4, ldp = C + 4;
  using RowsK = Rows<kK, kThreads>;
  using RowsV = Rows<kV, kThreads>;
  __shared__ Decays<C> dec;
  __shared__ __align__(16) float s_q[C][ldk], s_k[C][ldk], s_v[C][ldv], s_e[SUMS ? C : 1][ldv], s_p[C][ldp];
  __shared__ float s_red[SUMS ? NW : 1][C], s_row[C];
  Walk at;
  if (!at.find(w, C)) return;
  const MixRole& r = w.role[at.role];
  const int tid = threadIdx.x, lane = tid & 63, lo = lane & 31, hi = lane >> 5;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = at.tile * kV + 32 * wv + lo;  // this lane's value channel
  const int vw = r.V - at.tile * kV;            // value channels from this tile on
  const bool outputs = r.local == nullptr, sums = SUMS && r.sums, pairs = sums && r.pairs;

  f32x16 S[KT];
  at.enter_state<Layout>(w, r, S, col, hi);

  const RowsK rq(r.q, at.begin, r.sq, static_cast<int64_t>(at.head / r.qdiv) * r.K, r.K, at.reverse);
  const RowsK rk(r.k, at.begin, r.sk, static_cast<int64_t>(at.head / r.kdiv) * r.K, r.K, at.reverse);
  const RowsV rv(r.v, at.begin, r.sv, static_cast<int64_t>(at.head / r.vdiv) * r.V + at.tile * kV, vw, at.reverse);
  const RowsV re(r.e, at.begin, r.se, static_cast<int64_t>(at.head / r.ediv) * r.V + at.tile * kV, vw, at.reverse);
  f32x4 q[2 * RowsK::N], k[2 * RowsK::N], v[2 * RowsV::N], x[2 * RowsV::N];
  float g = 0.0f;
  auto tokens = [&](int c) {
    const int64_t left = at.len - static_cast<int64_t>(c) * C;
    return left < C ? static_cast<int>(left) : C;
  };
  auto fetch = [&](int c) {
    const int64_t c0 = static_cast<int64_t>(c) * C;
    const int n = tokens(c);
    int own = tid;
    if (SUMS) asm volatile("" : "+v"(own));  // (addresses formed here, not kept in registers around the loop)
    rk.load(k, own, c0, n);
    rv.load(v, own, c0, n);
    if (outputs) rq.load(q, own, c0, n);
    if (sums) re.load(x, own, c0, n);
    if (wv == NW - 1) g = lane < n ? w.g[(at.begin + at.token(lane, c0, n)) * w.g_step + at.head] : 0.0f;
  };

  Gone gone;
  if (at.first != at.stop) fetch(at.first);
  for (int c = at.first; c != at.stop; c += at.step) {
    const int64_t c0 = static_cast<int64_t>(c) * C;
    const int n = tokens(c), next = c + at.step;
    if (wv == NW - 1) chunk_decays<C>(dec, g, n, r.reverse, r.from, r.to, r.score);
    RowsK::keep(k, &s_k[0][0], ldk);
    RowsV::keep(v, &s_v[0][0], ldv);
    if (outputs) RowsK::keep(q, &s_q[0][0], ldk);
    if (sums) RowsV::keep(x, &s_e[0][0], ldv);
    if (next != at.stop) fetch(next);
    __syncthreads();
    if (outputs) {
      if (sums) at.leave_entering(w, r, S, c, dec, at.tile * NW + wv, 0, lane);
      // one wave makes the scores, transposed (earlier steps s as rows, steps t as columns),
      // and another what the other operands' rows give, each chunk the next ones
      const int scores = c % NW, others = (c + 1) % NW;
      f32x16 u = {};
      if (wv == scores) {
        f32x16 p = {};
#pragma unroll 4
        for (int j = 0; j < kK; j += 8) {
          const f32x4 a = *reinterpret_cast<const f32x4*>(&s_k[lo][j + 4 * hi]);
          const f32x4 b = *reinterpret_cast<const f32x4*>(&s_q[lo][j + 4 * hi]);
#pragma unroll
          for (int e = 0; e < 4; ++e) p = mfma(a[e], b[e], p);
        }
        const int from = dec.from[lo];
        const double ell = dec.ell[lo];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int s = 8 * (i >> 2) + 4 * hi + (i & 3);
          const float f = exp_of(ell - dec.ell[s]) * r.score;
          p[i] = where((s <= lo) & (s >= from), p[i] * f);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<f32x4*>(&s_p[lo][8 * i + 4 * hi]) = f32x4{p[4 * i], p[4 * i + 1], p[4 * i + 2], p[4 * i + 3]};
      }
      if (pairs && wv == others) {
#pragma unroll 4
        for (int j = 0; j < kV; j += 8) {
          const f32x4 a = *reinterpret_cast<const f32x4*>(&s_v[lo][j + 4 * hi]);
          const f32x4 b = *reinterpret_cast<const f32x4*>(&s_e[lo][j + 4 * hi]);
#pragma unroll
          for (int e = 0; e < 4; ++e) u = mfma(a[e], b[e], u);
        }
      }
      // what the state that enters gives
      f32x16 acc = {};
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const f32x4 a = *reinterpret_cast<const f32x4*>(&s_q[lo][32 * kt + 8 * j + 4 * hi]);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc = mfma(a[e], S[kt][4 * j + e], acc);
        }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int t = 8 * (i >> 2) + 4 * hi + (i & 3);
        acc[i] = where(dec.from[t] < 0, acc[i] * dec.in[t]);  // what a cut drops may be anything
        if (sums) {
          const float all = over_32(acc[i] * s_e[t][32 * wv + lo]);
          if (lo == 0) s_red[wv][t] = all;
        }
      }
      __syncthreads();
      if (pairs && wv == others) {
        // what crosses each step (sums only, as with bfloat16); the lane's places formed here, not
        // kept in registers around the loop
        int own = lane;
        asm volatile("" : "+v"(own));
        const int lo = own & 31, hi = own >> 5, from = dec.from[lo];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int s = 8 * (i >> 2) + 4 * hi + (i & 3);
          u[i] = where((s < lo) & (s >= from), u[i] * s_p[lo][s]);
        }
        prefix_of(u, hi);
#pragma unroll
        for (int i = 0; i < 16; ++i) u[i] = where(8 * (i >> 2) + 4 * hi + (i & 3) < lo, u[i]);
        const float crossing = over_columns(u, lo);
        if ((lo & 1) == 0) s_row[column_step(lo, hi)] = crossing;
      }
      const f32x16 before = acc;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x4 a = *reinterpret_cast<const f32x4*>(&s_p[lo][8 * j + 4 * hi]);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc = mfma(a[e], s_v[8 * j + 4 * hi + e][32 * wv + lo], acc);
      }
      // a score of 0 times a value that is not finite is NaN: where an output is not
      // finite, its steps are added one by one, those that it sees only
      float worst = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) worst = fmaf(acc[i], 0.0f, worst);
      if (__any(worst != 0.0f)) {
        acc = before;
        for (int s = 0; s < C; ++s) {
          const float value = s_v[s][32 * wv + lo];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int t = 8 * (i >> 2) + 4 * hi + (i & 3);
            const float more = fmaf(s_p[t][s], value, acc[i]);
            acc[i] = ((s <= t) & (s >= dec.from[t])) ? more : acc[i];
          }
        }
      }
      at.store<F32Io, Layout>(w, r, acc, 0, c0, n, col, hi);
      if (sums) {
        __syncthreads();
        if (tid < n) {
          float sum = 0.0f;
#pragma unroll
          for (int i = 0; i < NW; ++i) sum += s_red[i][tid];
          const int64_t to = (static_cast<int64_t>(at.tile) * w.heads + at.head) * w.rows + at.begin + at.token(tid, c0, n);
          r.sums[to] = sum;
          if (pairs) r.pairs[to] = tid > 0 ? s_row[tid - 1] : 0.0f;
        }
      }
    }
    const float all = dec.all;
    const bool cut = dec.cut;
    const int kept = dec.kept;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
#pragma unroll
      for (int i = 0; i < 16; ++i) S[kt][i] = where(!cut, S[kt][i] * all);
    }
    for (int s0 = 0; s0 < C; s0 += 8)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int s = s0 + 4 * hi + e;
        const float f = dec.end[s];
        const bool on = s >= kept;
        const float b = where(on, s_v[s][32 * wv + lo] * f);
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) S[kt] = mfma(where(on, s_k[s][32 * kt + lo]), b, S[kt]);
      }
    gone.add(dec.cut, dec.total);
    __syncthreads();  // the next chunk's rows take these places
  }
  at.leave_state<Layout>(w, r, S, gone, col, hi);
}

template <int KT, int NW>
hipError_t launch(const MixCall& w, hipStream_t stream) {
  bool sums = false;
  for (int k = 0; k < w.roles; ++k) sums |= w.role[k].sums != nullptr && !w.role[k].local;
  const dim3 grid(static_cast<unsigned>(walk_units(w)));
  if (sums)
    hipLaunchKernelGGL((walk_f32_kernel<KT, NW, true>), grid, dim3(64 * NW), 0, stream, w);
  else
    hipLaunchKernelGGL((walk_f32_kernel<KT, NW, false>), grid, dim3(64 * NW), 0, stream, w);
  return hipGetLastError();
}

template <int KT>
hipError_t by_values(const MixCall& w, hipStream_t stream) {
  // (two waves hold 64 channels, but with a state of 256 rows too few registers)
  return KT < 8 && value_width(w.role[0].V) == 64 ? launch<KT, KT < 8 ? 2 : 4>(w, stream) : launch<KT, 4>(w, stream);
}

}  // namespace

hipError_t launch_walk_f32(const MixCall& w, hipStream_t stream) {
  const int kt = key_tiles(w.role[0].K);
  return kt == 2 ? by_values<2>(w, stream) : kt == 4 ? by_values<4>(w, stream) : by_values<8>(w, stream);
}

}  // namespace mscan

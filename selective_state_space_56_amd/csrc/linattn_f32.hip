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
#include "linattn.h"
#include "linattn_walk.h"

namespace mscan {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x16 mfma(float a, float b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x2f32(a, b, c, 0, 0, 0);
}

// Rows of D: see above.
struct Layout {
  static constexpr int kRows = 16, kLane = 4;
  static constexpr int row(int tile, int i) { return 32 * tile + 8 * (i >> 2) + (i & 3); }
};

// KT: 32-row tiles of the state; NW: waves, 32 value channels each; CT: 32-step
// tiles of a chunk.
template <int KT, int NW, int CT>
__global__ __launch_bounds__(64 * NW, 1) void walk_f32_kernel(MixCall w) {
  constexpr int C = 32 * CT, kK = 32 * KT, kV = 32 * NW, kThreads = 64 * NW;
  constexpr int ldk = kK + 4, ldv = kV + 4, ldp = C + 4;
  __shared__ Decays<C> dec;
  __shared__ __align__(16) float s_q[C][ldk], s_k[C][ldk], s_v[C][ldv], s_e[C][ldv], s_p[C][ldp];
  __shared__ float s_red[NW][C], s_row[CT][C];
  Walk at;
  if (!at.find(w, C)) return;
  const MixRole& r = w.role[at.role];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, lo = lane & 31, hi = lane >> 5;
  const int col = at.tile * kV + 32 * wv + lo;  // this lane's value channel
  const int vw = r.V - at.tile * kV;            // value channels from this tile on

  f32x16 S[KT];
  at.enter_state<Layout>(w, r, S, col, hi);

  // rows of the chunk's tokens, 8 values at a time; 0 past its end and its channels
  auto stage = [&](float* to, int ld, int width, const void* from, int64_t stride, int64_t first_col, int have, int64_t c0,
                   int n) {
    const int per = width / 8;
    for (int id = tid; id < C * per; id += kThreads) {
      const int row = id / per, x = 8 * (id % per);
      f32x4 a = {}, b = {};
      if (row < n && x < have) {
        Piece<F32Io, 8> p;
        p.load(static_cast<const float*>(from) + (at.begin + at.token(row, c0, n)) * stride + first_col + x);
        a = f32x4{p.get(0), p.get(1), p.get(2), p.get(3)};
        b = f32x4{p.get(4), p.get(5), p.get(6), p.get(7)};
      }
      *reinterpret_cast<f32x4*>(to + row * ld + x) = a;
      *reinterpret_cast<f32x4*>(to + row * ld + x + 4) = b;
    }
  };

  Gone gone;
  for (int c = at.first; c != at.stop; c += at.step) {
    const int64_t c0 = static_cast<int64_t>(c) * C;
    const int n = at.len - c0 < C ? static_cast<int>(at.len - c0) : C;
    if (wv == 0) {
      const float g = lane < n ? w.g[(at.begin + at.token(lane, c0, n)) * w.g_step + at.head] : 0.0f;
      chunk_decays<C>(dec, g, n, r.reverse, r.from, r.to, r.score);
    }
    if (!r.local) stage(&s_q[0][0], ldk, kK, r.q, r.sq, (at.head / r.qdiv) * r.K, r.K, c0, n);
    stage(&s_k[0][0], ldk, kK, r.k, r.sk, (at.head / r.kdiv) * r.K, r.K, c0, n);
    stage(&s_v[0][0], ldv, kV, r.v, r.sv, static_cast<int64_t>(at.head / r.vdiv) * r.V + at.tile * kV, vw, c0, n);
    if (r.sums) stage(&s_e[0][0], ldv, kV, r.e, r.se, static_cast<int64_t>(at.head / r.ediv) * r.V + at.tile * kV, vw, c0, n);
    __syncthreads();
    if (!r.local) {
      at.leave_mark<Layout>(w, r, S, c, C, col, hi);
      // scores, transposed (earlier steps s as rows, steps t as columns), one 32 x 32
      // tile per wave at a time
      int turn = 0;
      for (int ti = 0; ti < CT; ++ti)
        for (int si = 0; si <= ti; ++si, ++turn) {
          if (turn % NW != wv) continue;
          f32x16 p = {};
#pragma unroll 4
          for (int x = 0; x < kK; x += 8) {
            const f32x4 a = *reinterpret_cast<const f32x4*>(&s_k[32 * si + lo][x + 4 * hi]);
            const f32x4 b = *reinterpret_cast<const f32x4*>(&s_q[32 * ti + lo][x + 4 * hi]);
#pragma unroll
            for (int e = 0; e < 4; ++e) p = mfma(a[e], b[e], p);
          }
          const int t = 32 * ti + lo, from = dec.from[t];
          const double ell = dec.ell[t];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int s = 32 * si + 8 * (i >> 2) + 4 * hi + (i & 3);
            const float f = exp_of(ell - dec.ell[s]) * r.score;
            p[i] = where((s <= t) & (s >= from), p[i] * f);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<f32x4*>(&s_p[t][32 * si + 8 * i + 4 * hi]) =
                f32x4{p[4 * i], p[4 * i + 1], p[4 * i + 2], p[4 * i + 3]};
          if (r.sums) {
            f32x16 u = {};
#pragma unroll 4
            for (int x = 0; x < kV; x += 8) {
              const f32x4 a = *reinterpret_cast<const f32x4*>(&s_v[32 * si + lo][x + 4 * hi]);
              const f32x4 b = *reinterpret_cast<const f32x4*>(&s_e[32 * ti + lo][x + 4 * hi]);
#pragma unroll
              for (int e = 0; e < 4; ++e) u = mfma(a[e], b[e], u);
            }
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int s = 32 * si + 8 * (i >> 2) + 4 * hi + (i & 3);
              u[i] = where((s < t) & (s >= from), u[i] * p[i]);
              sum += u[i];
            }
            sum += __shfl_xor(sum, 32);
            if (hi == 0) s_row[si][t] = sum;
          }
        }
      __syncthreads();
      for (int ti = 0; ti < CT; ++ti) {
        f32x16 acc = {};
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const f32x4 a = *reinterpret_cast<const f32x4*>(&s_q[32 * ti + lo][32 * kt + 8 * j + 4 * hi]);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc = mfma(a[e], S[kt][4 * j + e], acc);
          }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int t = 32 * ti + 8 * (i >> 2) + 4 * hi + (i & 3);
          const float f = dec.in[t];
          acc[i] = where(f != 0.0f, acc[i] * f);
          if (r.sums) {
            const float all = over_32(acc[i] * s_e[t][32 * wv + lo]);
            if (lo == 0) s_red[wv][t] = all;
          }
        }
        const f32x16 before = acc;
        for (int si = 0; si <= ti; ++si)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const f32x4 a = *reinterpret_cast<const f32x4*>(&s_p[32 * ti + lo][32 * si + 8 * j + 4 * hi]);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc = mfma(a[e], s_v[32 * si + 8 * j + 4 * hi + e][32 * wv + lo], acc);
          }
        // a score of 0 times a value that is not finite is NaN: where an output is not
        // finite, its steps are added one by one, those that it sees only
        float worst = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) worst = fmaf(acc[i], 0.0f, worst);
        if (__any(worst != 0.0f)) {
          acc = before;
          for (int s = 0; s < 32 * (ti + 1); ++s) {
            const float v = s_v[s][32 * wv + lo];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int t = 32 * ti + 8 * (i >> 2) + 4 * hi + (i & 3);
              const float more = fmaf(s_p[t][s], v, acc[i]);
              acc[i] = ((s <= t) & (s >= dec.from[t])) ? more : acc[i];
            }
          }
        }
        at.store<F32Io, Layout>(w, r, acc, 32 * ti, c0, n, col, hi);
      }
      if (r.sums) {
        __syncthreads();
        if (tid < n) {
          float sum = 0.0f, both = 0.0f;
#pragma unroll
          for (int i = 0; i < NW; ++i) sum += s_red[i][tid];
          for (int i = 0; i <= tid / 32; ++i) both += s_row[i][tid];
          float* to = r.sums + (static_cast<int64_t>(at.tile) * w.heads + at.head) * w.rows + at.begin + at.token(tid, c0, n);
          to[0] = sum;
          to[static_cast<int64_t>(w.tiles) * w.heads * w.rows] = both;
        }
      }
    }
    const float all = dec.all;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
#pragma unroll
      for (int i = 0; i < 16; ++i) S[kt][i] = where(all != 0.0f, S[kt][i] * all);
    }
    for (int s0 = 0; s0 < C; s0 += 8)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int s = s0 + 4 * hi + e;
        const float f = dec.end[s];
        const bool on = f != 0.0f;
        const float b = where(on, s_v[s][32 * wv + lo] * f);
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) S[kt] = mfma(where(on, s_k[s][32 * kt + lo]), b, S[kt]);
      }
    gone.add(dec.cut, dec.total);
    __syncthreads();  // the next chunk's rows take these places
  }
  at.leave_state<Layout>(w, r, S, gone, col, hi);
}

template <int KT, int NW, int CT>
hipError_t launch(const MixCall& w, hipStream_t stream) {
  hipLaunchKernelGGL((walk_f32_kernel<KT, NW, CT>), dim3(static_cast<unsigned>(walk_units(w))), dim3(64 * NW), 0,
                     stream, w);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_walk_f32(const MixCall& w, int chunk, hipStream_t stream) {
  const int kt = key_tiles(w.role[0].K), nw = value_width(MAMBA_F32, w.role[0].K, w.role[0].V) / 32;
  if (kt == 8) return launch<8, 2, 1>(w, stream);
  if (chunk == 32) {
    if (kt == 2) return nw == 2 ? launch<2, 2, 1>(w, stream) : launch<2, 4, 1>(w, stream);
    return nw == 2 ? launch<4, 2, 1>(w, stream) : launch<4, 4, 1>(w, stream);
  }
  if (kt == 2) return nw == 2 ? launch<2, 2, 2>(w, stream) : launch<2, 4, 2>(w, stream);
  return nw == 2 ? launch<4, 2, 2>(w, stream) : launch<4, 4, 2>(w, stream);
}

}  // namespace mscan

// Linear attention with bfloat16 io on the matrix cores: the map of linattn.h over
// the chunks of one segment, for one head and up to 128 value channels per
// workgroup, 32 of them per wave.
//
// Products take bf16 operands and accumulate in float32 (v_mfma_f32_32x32x16_bf16).
// q, k and v are bf16 as they come; what is float32 goes in as a sum of bf16 parts, one
// product each: the scores and the state in the outputs as two (2^-17 of each term),
// the weighted values that make the state as three (exact: 8 + 8 + 8 bits), so that
// the state is a float32 one; with the sums for the decays' gradients the state as
// three there too.
//
// Operand layouts (wave64, lane l): A (32 x 16): row l % 32, k = 8 (l / 32) .. + 7;
// B (16 x 32): column l % 32, the same k; D (32 x 32): register i is row
// 8 (i / 4) + 4 (l / 32) + i % 4, column l % 32. The state stays in registers as D
// and is used as B without moving: the rows of A that make it are taken in the
// order in which register i comes out as row 16 (i / 8) + 8 (l / 32) + i % 8.
// Operands whose k is the step come from LDS by the transposing load.
#include "linattn_walk.h"

namespace mscan {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4_ptr;

__device__ __forceinline__ f32x16 mfma(u32x4 a, u32x4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Two values rounded to bf16 in one word, a in the low half.
__device__ __forceinline__ uint32_t pack(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}
__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Two values as N bf16 parts each, in words as pack: with two, hi = bf16(v) and lo =
// bf16(v - hi); with three, the value's bits eight at a time, whose sum is the value.
template <int N>
__device__ __forceinline__ void split(float a, float b, uint32_t (&part)[N]) {
  if constexpr (N == 2) {
    part[0] = pack(a, b);
    part[1] = pack(a - low(part[0]), b - high(part[0]));
  } else {
    part[0] = __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302);
    a -= low(part[0]);
    b -= high(part[0]);
    part[1] = __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302);
    part[2] = __builtin_amdgcn_perm(__float_as_uint(b - high(part[1])), __float_as_uint(a - low(part[1])), 0x07060302);
  }
}

// Eight consecutive bf16 of an LDS row.
__device__ __forceinline__ u32x4 row8(const uint16_t* p) { return *reinterpret_cast<const u32x4*>(p); }

// Eight steps of a lane's column from a step-major LDS tile T (row stride ld): lane l
// receives T[8 (l / 32) + e][c], e = 0 .. 7. The transposing load works on 16 lanes: lane
// q names 4 consecutive elements of row q / 4 and receives column q of that 4 x 16
// block. c is l % 32, or with TURNED the state's row order above: the 4-column
// blocks (a, h) of each 16 columns taken as (h, a).
template <bool TURNED>
__device__ __forceinline__ u32x4 column8(const uint16_t* T, int ld, int lane) {
  const int grp = lane >> 4, q = lane & 15;
  const int block = TURNED ? ((q & 1) << 1) | ((q >> 1) & 1) : q & 3;
  const uint16_t* p = T + (8 * (grp >> 1) + (q >> 2)) * ld + 16 * (grp & 1) + 4 * block;
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_ptr)(p));
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_ptr)(p + 4 * ld));
  return __builtin_bit_cast(u32x4, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// The value of the lane N places round within its 16 lanes.
template <int N>
__device__ __forceinline__ float turned(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x120 + N, 0xf, 0xf, true));
}
// Sums over the 32 lanes of each half wave of two values: a's in lanes 0 .. 15 of the
// half, b's in lanes 16 .. 31.
__device__ __forceinline__ float over_32_of_two(float a, float b) {
  const auto w = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  float v = __uint_as_float(w[0]) + __uint_as_float(w[1]);
  v += turned<8>(v);
  v += turned<4>(v);
  v += turned<2>(v);
  return v + turned<1>(v);
}

// One operand's rows of a chunk, 16 bytes at a time: W values per row (0 from `have`
// on), N pieces per thread. A chunk's rows are one buffer resource that ends with its
// last row, so that rows past it read 0 and are not written without a condition (in
// reverse they lie before its first row, which as an offset is out of range too).
// Offsets stay below 2^31: rows are at most kMixMaxStride elements apart.
template <int W, int C, int THREADS>
struct Rows {
  static constexpr int kPer = W / 8, N = C * kPer / THREADS, kStep = THREADS / kPer;
  static_assert(C * kPer % THREADS == 0 && THREADS % kPer == 0, "whole rows of pieces");
  const uint16_t* base;
  int stride;             // of rows, in bytes
  uint32_t lane;          // this lane's offset
  int row, x, width;      // width: of a row, in bytes
  bool back;

  __device__ __forceinline__ Rows(const void* p, int64_t first_row, int64_t stride_, int64_t first_col, int have, bool reverse)
      : base(static_cast<const uint16_t*>(p) + first_row * stride_ + first_col), stride(static_cast<int>(2 * stride_)),
        width(2 * (have < W ? have : W)), back(reverse) {
    row = threadIdx.x / kPer;
    x = 8 * (threadIdx.x % kPer);
    lane = x < have ? static_cast<uint32_t>((reverse ? -row : row) * stride + 2 * x) : kOffNone;
  }
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t chunk(int64_t c0, int n) const {
    return make_rsrc(base + c0 * (stride / 2), static_cast<uint32_t>((n - 1) * stride + width));
  }
  // rows of a chunk that starts c0 steps into the sequence and has n
  __device__ __forceinline__ void load(u32x4 (&to)[N], int64_t c0, int n) const {
    const auto rs = chunk(c0, n);
    const int first = back ? (n - 1) * stride : 0, step = (back ? -kStep : kStep) * stride;
#pragma unroll
    for (int i = 0; i < N; ++i)
      to[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, lane + (first + i * step), 0, 0));
  }
  __device__ __forceinline__ void keep(const u32x4 (&from)[N], uint16_t* tile, int ld) const {
#pragma unroll
    for (int i = 0; i < N; ++i) *reinterpret_cast<u32x4*>(tile + (row + i * kStep) * ld + x) = from[i];
  }
};

// KT: 32-row tiles of a wave's state; KH: waves that share the state's rows, KT tiles
// each; NV: waves that share the value channels; CT: 32-step tiles of a chunk; SUMS: with
// the sums for the decays' gradients.
template <int KT, int KH, int NV, int CT, bool SUMS>
__global__ __launch_bounds__(64 * NV * KH, NV == 4 && !SUMS ? 2 : 1) void walk_bf16_kernel(MixCall w) {
  constexpr int NW = NV * KH, C = 32 * CT, kK = 32 * KT * KH, kV = 32 * NV, kThreads = 64 * NW;
  constexpr int kW = kK > kV ? kK : kV;  // widest rows that the queries' tile holds
  // row strides of the tiles: rows read along, 16 bytes per lane, start 4 banks apart;
  // rows read by the transposing load 16 (values) or 20 (keys, which are read both
  // ways) banks apart
  constexpr int ldq = kW + 8, ldk = kK + (kK == 64 ? 24 : 40), ldv = kV + 32, ldp = C + 8;
  constexpr int kParts = SUMS ? 3 : 2;
  __shared__ Decays<C> s_dec[2];
  __shared__ __align__(16) uint16_t s_q[C][ldq], s_k[C][ldk], s_v[C][ldv], s_p[2][C][ldp];
  __shared__ float s_red[SUMS ? NV : 1][C], s_row[CT][C], s_col[CT][C];
  __shared__ float s_half[KH > 1 ? NV : 1][KH > 1 ? CT * 16 : 1][64];
  Walk at;
  if (!at.find(w, C)) return;
  const MixRole& r = w.role[at.role];
  const int tid = threadIdx.x, lane = tid & 63, lo = lane & 31, hi = lane >> 5;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int vv = wv % NV, kh = wv / NV, k0 = 32 * KT * kh;  // this wave's channels and rows of the state
  const int col = at.tile * kV + 32 * vv + lo;             // this lane's value channel
  const int vw = r.V - at.tile * kV;
  const bool outputs = r.local == nullptr, sums = SUMS && r.sums;

  f32x16 S[KT];
  at.enter_state<KT, true>(w, r, S, col, hi, k0);

  const Rows<kK, C, kThreads> rq(r.q, at.begin, r.sq, static_cast<int64_t>(at.head / r.qdiv) * r.K, r.K, at.reverse);
  const Rows<kK, C, kThreads> rk(r.k, at.begin, r.sk, static_cast<int64_t>(at.head / r.kdiv) * r.K, r.K, at.reverse);
  const Rows<kV, C, kThreads> rv(r.v, at.begin, r.sv, static_cast<int64_t>(at.head / r.vdiv) * r.V + at.tile * kV, vw, at.reverse);
  const Rows<kV, C, kThreads> re(r.e, at.begin, r.se, static_cast<int64_t>(at.head / r.ediv) * r.V + at.tile * kV, vw, at.reverse);
  u32x4 q[rq.N], k[rk.N], v[rv.N], x[re.N];
  auto tokens = [&](int c) {
    const int64_t left = at.len - static_cast<int64_t>(c) * C;
    return left < C ? static_cast<int>(left) : C;
  };
  auto fetch = [&](int c) {
    const int64_t c0 = static_cast<int64_t>(c) * C;
    const int n = tokens(c);
    rk.load(k, c0, n);
    rv.load(v, c0, n);
  };
  auto gate = [&](int c) {
    const int n = tokens(c);
    return lane < n ? w.g[(at.begin + at.token(lane, static_cast<int64_t>(c) * C, n)) * w.g_step + at.head] : 0.0f;
  };

  Gone gone;
  int turn = 0;
  float g = 0.0f;
  if (at.first != at.stop) {
    fetch(at.first);
    if (outputs) rq.load(q, static_cast<int64_t>(at.first) * C, tokens(at.first));
    // the last wave, which has no scores to make, forms each chunk's decays one chunk ahead
    if (wv == NW - 1) {
      chunk_decays<C>(s_dec[0], gate(at.first), tokens(at.first), r.reverse, r.from, r.to);
      if (at.first + at.step != at.stop) g = gate(at.first + at.step);
    }
  }
  for (int c = at.first; c != at.stop; c += at.step, turn ^= 1) {
    const int64_t c0 = static_cast<int64_t>(c) * C;
    const int n = tokens(c), next = c + at.step;
    const Decays<C>& dec = s_dec[turn];
    rk.keep(k, &s_k[0][0], ldk);
    rv.keep(v, &s_v[0][0], ldv);
    if (outputs) rq.keep(q, &s_q[0][0], ldq);
    if (next != at.stop) fetch(next);
    if (sums) re.load(x, c0, n);
    __syncthreads();
    if (wv == NW - 1 && next != at.stop) {
      chunk_decays<C>(s_dec[turn ^ 1], g, tokens(next), r.reverse, r.from, r.to);
      if (next + at.step != at.stop) g = gate(next + at.step);
    }
    f32x16 acc[CT];
    if (outputs) {
      if (sums) at.leave_mark<KT, true>(w, r, S, c, C, col, hi, k0);
      // scores, transposed (earlier steps s as rows, steps t as columns)
      f32x16 p = {};
      constexpr int kTiles = CT * (CT + 1) / 2;
      const int tile = wv;  // of (0, 0), (1, 0), (1, 1)
      const int ti = tile > 0 ? 1 : 0, si = tile > 1 ? 1 : 0;
      auto score = [&](int ti, int si) {
        p = f32x16{};
#pragma unroll
        for (int j = 0; j < kK; j += 16)
          p = mfma(row8(&s_k[32 * si + lo][j + 8 * hi]), row8(&s_q[32 * ti + lo][j + 8 * hi]), p);
        const int t = 32 * ti + lo, from = dec.from[t];
        const double ell = dec.ell[t];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int s = 32 * si + 8 * (i >> 2) + 4 * hi + (i & 3);
          const float f = exp_of(ell - dec.ell[s]) * r.score;
          // -0 where t does not see s, and nowhere else
          p[i] = ((s <= t) & (s >= from)) ? p[i] * f + 0.0f : -0.0f;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t a[2], b[2];
          split<2>(p[4 * i], p[4 * i + 1], a);
          split<2>(p[4 * i + 2], p[4 * i + 3], b);
          const int s = 32 * si + 8 * i + 4 * hi;
          *reinterpret_cast<u32x2*>(&s_p[0][t][s]) = u32x2{a[0], b[0]};
          *reinterpret_cast<u32x2*>(&s_p[1][t][s]) = u32x2{a[1], b[1]};
        }
      };
      // pairs of steps: the scores times what the other operands' rows give, in float32
      auto pairs = [&](int ti, int si) {
        f32x16 u = {};
#pragma unroll
        for (int j = 0; j < kV; j += 16)
          u = mfma(row8(&s_v[32 * si + lo][j + 8 * hi]), row8(&s_q[32 * ti + lo][j + 8 * hi]), u);
        const int t = 32 * ti + lo, from = dec.from[t];
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int s = 32 * si + 8 * (i >> 2) + 4 * hi + (i & 3);
          u[i] = where((s < t) & (s >= from), u[i] * p[i]);
          sum += u[i];
        }
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const float two = over_32_of_two(u[i], u[i + 1]);
          if ((lo & 15) == 0) s_col[ti][32 * si + 8 * (i >> 2) + 4 * hi + (i & 3) + (lo >> 4)] = two;
        }
        sum += __shfl_xor(sum, 32);
        if (hi == 0) s_row[si][t] = sum;
      };
      // with two waves the second one has two of the three tiles: first (1, 0)
      constexpr bool kTwo = NW < kTiles;
      if (wv < kTiles) score(ti, si);
      f32x16 first = p;
      if (kTwo && wv == 1) score(1, 1);
      // what the state that enters gives
#pragma unroll
      for (int t = 0; t < CT; ++t) acc[t] = f32x16{};
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          u32x4 part[kParts];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t words[kParts];
            split<kParts>(S[kt][8 * j + 2 * e], S[kt][8 * j + 2 * e + 1], words);
#pragma unroll
            for (int m = 0; m < kParts; ++m) part[m][e] = words[m];
          }
#pragma unroll
          for (int t = 0; t < CT; ++t) {
            const u32x4 a = row8(&s_q[32 * t + lo][k0 + 32 * kt + 16 * j + 8 * hi]);
#pragma unroll
            for (int m = 0; m < kParts; ++m) acc[t] = mfma(a, part[m], acc[t]);
          }
        }
      // (not with the others: registers)
      if (next != at.stop) rq.load(q, static_cast<int64_t>(next) * C, tokens(next));
      static_assert(KH <= 2, "one wave adds one other's");
      if (KH > 1 && kh) {
#pragma unroll
        for (int i = 0; i < 16 * CT; ++i) s_half[vv][i][lane] = acc[i / 16][i % 16];
      }
      __syncthreads();
      if (KH > 1 && !kh) {
#pragma unroll
        for (int i = 0; i < 16 * CT; ++i) acc[i / 16][i % 16] += s_half[vv][i][lane];
      }
      const bool cut = __builtin_amdgcn_readfirstlane(dec.cut);
#pragma unroll
      for (int t = 0; t < CT; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[t][i] *= dec.in[32 * t + 8 * (i >> 2) + 4 * hi + (i & 3)];
      if (cut) {  // what a cut drops may be anything
#pragma unroll
        for (int t = 0; t < CT; ++t)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            acc[t][i] = where(dec.in[32 * t + 8 * (i >> 2) + 4 * hi + (i & 3)] != 0.0f, acc[t][i]);
      }
      if (sums) {
        re.keep(x, &s_q[0][0], ldq);  // the queries are done with
        __syncthreads();
        if (r.pairs) {
          if (kTwo && wv == 1) {
            pairs(1, 1);
            p = first;
          }
          if (wv < kTiles) pairs(ti, si);
        }
#pragma unroll
        for (int t = 0; t < CT && !kh; ++t)
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const int row = 32 * t + 8 * (i >> 2) + 4 * hi + (i & 3);
            const float two = over_32_of_two(acc[t][i] * Bf16Io::to_f32(s_q[row][32 * vv + lo]),
                                             acc[t][i + 1] * Bf16Io::to_f32(s_q[row + 1][32 * vv + lo]));
            if ((lo & 15) == 0) s_red[vv][row + (lo >> 4)] = two;
          }
        __syncthreads();  // the outputs take the rows' place
        if (tid < n) {
          float sum = 0.0f;
#pragma unroll
          for (int i = 0; i < NV; ++i) sum += s_red[i][tid];
          if (r.pairs) {
            for (int i = 0; i <= tid / 32; ++i) sum += s_row[i][tid];
            for (int i = tid / 32; i < CT; ++i) sum -= s_col[i][tid];
          }
          r.sums[(static_cast<int64_t>(at.tile) * w.heads + at.head) * w.rows + at.begin + at.token(tid, c0, n)] = sum;
        }
      }
      if (!kh) {
      // A score of 0 times a value that is not finite is NaN: with such a value among this
      // wave's, steps are added one by one, to the outputs that see them only (whose score
      // is not -0).
      u16x2 most = {};
#pragma unroll
      for (int j = 0; j < 2 * CT; ++j) {
        const u32x4 b = column8<false>(&s_v[16 * j][32 * vv], ldv, lane);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, b[e] & 0x7fff7fffu));
      }
      if (!__any((most[0] >= 0x7f80) | (most[1] >= 0x7f80))) {
#pragma unroll
        for (int j = 0; j < 2 * CT; ++j) {
          const u32x4 b = column8<false>(&s_v[16 * j][32 * vv], ldv, lane);
#pragma unroll
          for (int t = j / 2; t < CT; ++t) {
            acc[t] = mfma(row8(&s_p[0][32 * t + lo][16 * j + 8 * hi]), b, acc[t]);
            acc[t] = mfma(row8(&s_p[1][32 * t + lo][16 * j + 8 * hi]), b, acc[t]);
          }
        }
      } else {
#pragma unroll 1
        for (int s = 0; s < n; ++s) {
          const float value = Bf16Io::to_f32(s_v[s][32 * vv + lo]);
#pragma unroll
          for (int t = 0; t < CT; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int row = 32 * t + 8 * (i >> 2) + 4 * hi + (i & 3);
              const uint16_t score = s_p[0][row][s];
              const float more = fmaf(Bf16Io::to_f32(score) + Bf16Io::to_f32(s_p[1][row][s]), value, acc[t][i]);
              acc[t][i] = ((score != 0x8000) & (s < 32 * (t + 1))) ? more : acc[t][i];
            }
        }
      }
      if (r.part) {
#pragma unroll
        for (int t = 0; t < CT; ++t) at.store<Bf16Io>(w, r, acc[t], 32 * t, c0, n, col, hi);
      } else {
        // through the queries' place (this wave's columns of it), as pieces of rows
        uint16_t* to = &s_q[0][32 * vv];
#pragma unroll
        for (int t = 0; t < CT; ++t)
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const uint32_t two = pack(acc[t][i], acc[t][i + 1]);
            const int row = 32 * t + 8 * (i >> 2) + 4 * hi + (i & 3);
            to[row * ldq + lo] = static_cast<uint16_t>(two);
            to[(row + 1) * ldq + lo] = static_cast<uint16_t>(two >> 16);
          }
        __builtin_amdgcn_wave_barrier();
        const int piece = 8 * (lane & 3), stride = static_cast<int>(2 * r.so);
        const auto rs = make_rsrc(static_cast<uint16_t*>(r.o) + (at.begin + c0) * r.so + static_cast<int64_t>(at.head) * r.V +
                                      at.tile * kV + 32 * vv,
                                  static_cast<uint32_t>((n - 1) * stride + 2 * (vw - 32 * vv < 32 ? vw - 32 * vv : 32)));
        const uint32_t own =
            32 * vv + piece < vw ? static_cast<uint32_t>((at.reverse ? n - 1 - (lane >> 2) : lane >> 2) * stride + 2 * piece)
                                 : kOffNone;
#pragma unroll
        for (int i = 0; i < C / 16; ++i)
          __builtin_amdgcn_raw_buffer_store_b128(row8(to + (16 * i + (lane >> 2)) * ldq + piece), rs,
                                                 own + (at.reverse ? -16 : 16) * i * stride, 0, 0);
        __builtin_amdgcn_wave_barrier();
      }
      }
    }
    if (__builtin_amdgcn_readfirstlane(dec.cut)) {
      // the rows of steps that a later one cuts off, which may be anything, become 0
      __syncthreads();
      for (int id = tid; id < C * kK / 2; id += kThreads) {
        const int s = id / (kK / 2);
        if (dec.end[s] == 0.0f) *reinterpret_cast<uint32_t*>(&s_k[s][2 * (id % (kK / 2))]) = 0;
      }
      for (int id = tid; id < C * kV / 2; id += kThreads) {
        const int s = id / (kV / 2);
        if (dec.end[s] == 0.0f) *reinterpret_cast<uint32_t*>(&s_v[s][2 * (id % (kV / 2))]) = 0;
      }
      __syncthreads();
    }
    const float all = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(dec.all)));
    if (all != 0.0f) {
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) S[kt] *= all;
    } else {
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) S[kt] = f32x16{};
    }
#pragma unroll
    for (int j = 0; j < 2 * CT; ++j) {
      const u32x4 b = column8<false>(&s_v[16 * j][32 * vv], ldv, lane);
      const f32x4 f0 = *reinterpret_cast<const f32x4*>(&dec.end[16 * j + 8 * hi]);
      const f32x4 f1 = *reinterpret_cast<const f32x4*>(&dec.end[16 * j + 8 * hi + 4]);
      u32x4 part[3];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float a = e < 2 ? f0[2 * e] : f1[2 * e - 4], z = e < 2 ? f0[2 * e + 1] : f1[2 * e - 3];
        uint32_t words[3];
        split<3>(low(b[e]) * a, high(b[e]) * z, words);
#pragma unroll
        for (int m = 0; m < 3; ++m) part[m][e] = words[m];
      }
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        const u32x4 a = column8<true>(&s_k[16 * j][k0 + 32 * kt], ldk, lane);
#pragma unroll
        for (int m = 0; m < 3; ++m) S[kt] = mfma(a, part[m], S[kt]);
      }
    }
    gone.add(dec.cut, dec.total);
    __syncthreads();  // the next chunk's rows take these places
  }
  at.leave_state<KT, true>(w, r, S, gone, col, hi, k0);
}

template <int KT, int KH, int NV, int CT>
hipError_t launch(const MixCall& w, hipStream_t stream) {
  bool sums = false;
  for (int k = 0; k < w.roles; ++k) sums |= w.role[k].sums != nullptr && !w.role[k].local;
  const dim3 grid(static_cast<unsigned>(walk_units(w)));
  if (sums)
    hipLaunchKernelGGL((walk_bf16_kernel<KT, KH, NV, CT, true>), grid, dim3(64 * NV * KH), 0, stream, w);
  else
    hipLaunchKernelGGL((walk_bf16_kernel<KT, KH, NV, CT, false>), grid, dim3(64 * NV * KH), 0, stream, w);
  return hipGetLastError();
}

#ifdef ONLY
template __global__ void walk_bf16_kernel<ONLY, true>(MixCall);
template __global__ void walk_bf16_kernel<ONLY, false>(MixCall);
}  // namespace
#else
}  // namespace
hipError_t launch_walk_bf16(const MixCall& w, int chunk, hipStream_t stream) {
  const int kt = key_tiles(w.role[0].K), nw = value_waves(w.role[0].K, w.role[0].V);
  if (kt == 8) return launch<4, 2, 2, 1>(w, stream);
  if (chunk == 32) {
    if (kt == 2) return nw == 2 ? launch<2, 1, 2, 1>(w, stream) : launch<2, 1, 4, 1>(w, stream);
    return nw == 2 ? launch<4, 1, 2, 1>(w, stream) : launch<4, 1, 4, 1>(w, stream);
  }
  if (kt == 2) return nw == 2 ? launch<2, 1, 2, 2>(w, stream) : launch<2, 1, 4, 2>(w, stream);
  return nw == 2 ? launch<4, 1, 2, 2>(w, stream) : launch<4, 1, 4, 2>(w, stream);
}
#endif

}  // namespace mscan

// Linear attention with bfloat16 io on the matrix cores: the map of linattn.h over
// the chunks of one segment, for one head and up to 128 value channels per
// workgroup, 32 of them per wave.
//
// Products take bf16 operands and accumulate in float32 (v_mfma_f32_32x32x16_bf16).
// q, k and v are bf16 as they come; what is float32 goes in as a sum of bf16 parts, one
// product each: the scores and the state in the outputs as two (2^-17 of each term),
// the weighted values that make the state as three (exact: 8 + 8 + 8 bits), so that
// the state is a float32 one; with the sums for the decays' gradients the state as
// three there too. (Of a prompt's outputs 0.23 % are not the bf16 next to the exact value, where
// float32 sums leave 0.03 %. A third part of the scores would leave a compute unit room for one
// workgroup only: 84 KB of LDS at least.)
//
// Operand layouts (wave64, lane l): A (32 x 16): row l % 32, k = 8 (l / 32) .. + 7;
// B (16 x 32): column l % 32, the same k; D (32 x 32): register i is row
// 8 (i / 4) + 4 (l / 32) + i % 4, column l % 32. The state (rows: keys, columns: values)
// stays in registers as D and is an operand of the outputs without moving: the rows of A
// that make it are taken in the order in which register i comes out as row
// 16 (i / 8) + 8 (l / 32) + i % 8. Outputs are formed transposed (rows: values,
// columns: steps), so that a lane has one step: its factors are one value each, sums over
// the channels go along its registers, and its outputs leave four at a time. Operands
// whose k is the step come from LDS by the transposing load.
//
// Bound by issue: 8 x 2048 steps of 40 heads of 128 x 128 take 240 us, 2.9 TB/s of 5.3 that
// a copy reaches. The matrix products alone would take 67 us of them; splitting the state
// and the weighted values into parts, the scores' factors and LDS take the rest, and the
// vector and matrix instructions of a compute unit's eight waves hardly overlap. So the
// layout saves vector instructions: outputs formed as the state lies (steps as rows)
// took 374 us where transposed ones take 327 (packed prompts, 128 x 64), rows as
// buffer resources instead of conditions 287 -> 265.
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

// The leading 16 bits of two values, a's in the low half.
__device__ __forceinline__ uint32_t leading(float a, float b) {
  return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302);
}

// Two values as N bf16 parts each, in words as pack: with two, hi = bf16(v) and lo =
// bf16(v - hi); with three, the value's bits eight at a time, whose sum is the value.
template <int N>
__device__ __forceinline__ void split(float a, float b, uint32_t (&part)[N]) {
  if constexpr (N == 2) {
    part[0] = pack(a, b);
    part[1] = pack(a - low(part[0]), b - high(part[0]));
  } else {
    part[0] = leading(a, b);
    a -= low(part[0]);
    b -= high(part[0]);
    part[1] = leading(a, b);
    part[2] = leading(a - low(part[1]), b - high(part[1]));
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

// The sum of both half waves' values, in both.
__device__ __forceinline__ float over_halves(float v) {
  const auto w = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(w[0]) + __uint_as_float(w[1]);
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
  int stride, width;      // of rows, in bytes: their distance and what they hold
  bool back;

  __device__ __forceinline__ Rows(const void* p, int64_t first_row, int64_t stride_, int64_t first_col, int have, bool reverse)
      : base(static_cast<const uint16_t*>(p) + first_row * stride_ + first_col), stride(static_cast<int>(2 * stride_)),
        width(2 * (have < W ? have : W)), back(reverse) {}
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t chunk(int64_t c0, int n) const {
    return make_rsrc(base + c0 * (stride / 2), static_cast<uint32_t>((n - 1) * stride + width));
  }
  // the offset of thread tid's first piece, and what its further ones are apart
  __device__ __forceinline__ uint32_t first(int tid, int n) const {
    const int row = tid / kPer, x = 16 * (tid % kPer);
    return x < width ? static_cast<uint32_t>((back ? n - 1 - row : row) * stride + x) : kOffNone;
  }
  __device__ __forceinline__ int step() const { return (back ? -kStep : kStep) * stride; }
  static __device__ __forceinline__ int place(int tid, int i, int ld) {
    return (tid / kPer + i * kStep) * ld + 8 * (tid % kPer);
  }
  // rows of a chunk that starts c0 steps into the sequence and has n
  __device__ __forceinline__ void load(u32x4 (&to)[N], int tid, int64_t c0, int n) const {
    const auto rs = chunk(c0, n);
    const uint32_t at = first(tid, n);
#pragma unroll
    for (int i = 0; i < N; ++i)
      to[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, at + i * step(), 0, 0));
  }
  // to an LDS tile, and from one to memory
  static __device__ __forceinline__ void keep(const u32x4 (&from)[N], int tid, uint16_t* tile, int ld) {
#pragma unroll
    for (int i = 0; i < N; ++i) *reinterpret_cast<u32x4*>(tile + place(tid, i, ld)) = from[i];
  }
  __device__ __forceinline__ void store(int tid, const uint16_t* tile, int ld, int64_t c0, int n) const {
    const auto rs = chunk(c0, n);
    const uint32_t at = first(tid, n);
#pragma unroll
    for (int i = 0; i < N; ++i)
      __builtin_amdgcn_raw_buffer_store_b128(row8(tile + place(tid, i, ld)), rs, at + i * step(), 0, 0);
  }
};

// v, as if read anew: what is formed from it is formed where it stands, and not kept in
// registers through all of the loop around it.
__device__ __forceinline__ int fresh(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// v's values where the mask's bits are set, else 0, whatever they are. (As bits: chosen by
// a condition, or as a constant, they would be moved to other registers on all paths.)
__device__ __forceinline__ void drop(f32x16& v, uint32_t mask) {
  asm volatile("" : "+v"(mask));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(__float_as_uint(v[i]) & mask);
}

// Rows of the state's tiles.
struct StateRows {
  static constexpr int kRows = 16, kLane = 8;
  static constexpr int row(int tile, int i) { return 32 * tile + 16 * (i >> 3) + (i & 7); }
};

constexpr int kC = 64, kTT = kC / 32;          // steps of a chunk, and its tiles
constexpr int kTiles = kTT * (kTT + 1) / 2;    // of scores: (0, 0), (1, 0), (1, 1)

// Waves per SIMD that the kernels' registers are held to: two workgroups of four waves,
// where they fit.
constexpr int least_waves(int KT, int KH) { return KT * KH < 8 ? 2 : 1; }

// Four waves: NV of them side by side, 32 value channels each, and KH that share the
// state's rows, KT 32-row tiles each. (Up to 64 channels two waves would do, but leave half
// of a compute unit's registers and issue slots empty: with KH = 2 each makes half of the
// state's products and of the outputs what its rows give, and they add one tile of
// steps for each other.) SUMS: with the sums for the decays' gradients.
template <int KT, int KH, int NV, bool SUMS>
__global__ __launch_bounds__(64 * NV * KH, least_waves(KT, KH)) void walk_bf16_kernel(MixCall w) {
  constexpr int NW = NV * KH, C = kC, kK = 32 * KT * KH, kV = 32 * NV, kThreads = 64 * NW;
  static_assert(KH == 1 || KH == kTT, "a tile of steps for each wave that shares rows");
  // the widest rows that the queries' tile holds (with KH a tile of outputs for each wave)
  constexpr int kW = KH > 1 && kK < 128 ? 128 : kK > kV ? kK : kV;
  // row strides of the tiles: rows read along, 16 bytes per lane, start 4 banks apart;
  // rows read by the transposing load 16 (values) or 20 (keys, which are read both
  // ways) banks apart
  constexpr int ldq = kW + 8, ldk = kK + (kK == 64 ? 24 : 40), ldv = kV + 32, ldp = C + 8;
  constexpr int kParts = SUMS ? 3 : 2;
  using RowsK = Rows<kK, C, kThreads>;
  using RowsV = Rows<kV, C, kThreads>;
  __shared__ Decays<C> s_dec[2];
  __shared__ __align__(16) uint16_t s_q[C][ldq], s_k[C][ldk], s_v[C][ldv], s_p[2][C][ldp];
  // the waves' sums for the decays' gradients lie in the padding of the queries' and the
  // scores' rows (with room of their own only one workgroup would fit a compute unit)
  static_assert(4 * NV <= 2 * (ldq - kW) && 4 * kTT <= 2 * (ldp - C), "a float for each wave, and for each tile");
  auto s_red = [&](int t) { return reinterpret_cast<float*>(&s_q[t][kW]); };
  auto s_row = [&](int t) { return reinterpret_cast<float*>(&s_p[0][t][C]); };
  Walk at;
  if (!at.find(w, C)) return;
  const MixRole& r = w.role[at.role];
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int vv = wv % NV, kh = wv / NV, k0 = 32 * KT * kh;      // this wave's channels and rows of the state
  const int col = at.tile * kV + 32 * vv + (threadIdx.x & 31);  // this lane's value channel
  const int vw = r.V - at.tile * kV;
  const bool outputs = r.local == nullptr, sums = SUMS && r.sums, pairs = sums && r.pairs;

  f32x16 S[KT];
  at.enter_state<StateRows>(w, r, S, col, threadIdx.x % 64 / 32, k0);

  const RowsK rq(r.q, at.begin, r.sq, static_cast<int64_t>(at.head / r.qdiv) * r.K, r.K, at.reverse);
  const RowsK rk(r.k, at.begin, r.sk, static_cast<int64_t>(at.head / r.kdiv) * r.K, r.K, at.reverse);
  const RowsV rv(r.v, at.begin, r.sv, static_cast<int64_t>(at.head / r.vdiv) * r.V + at.tile * kV, vw, at.reverse);
  const RowsV re(r.e, at.begin, r.se, static_cast<int64_t>(at.head / r.ediv) * r.V + at.tile * kV, vw, at.reverse);
  const RowsV ro(r.o, at.begin, r.so, static_cast<int64_t>(at.head) * r.V + at.tile * kV, vw, at.reverse);
  u32x4 q[RowsK::N], k[RowsK::N], v[RowsV::N], x[RowsV::N];
  auto tokens = [&](int c) {
    const int64_t left = at.len - static_cast<int64_t>(c) * C;
    return left < C ? static_cast<int>(left) : C;
  };
  auto fetch = [&](int c) {
    const int64_t c0 = static_cast<int64_t>(c) * C;
    const int n = tokens(c), tid = fresh(threadIdx.x);
    rk.load(k, tid, c0, n);
    rv.load(v, tid, c0, n);
    if (outputs && !SUMS) rq.load(q, tid, c0, n);
  };
  // with the sums, apart: the registers are the other operand's until then
  auto fetch_q = [&](int c) {
    if (outputs && SUMS) rq.load(q, fresh(threadIdx.x), static_cast<int64_t>(c) * C, tokens(c));
  };
  auto gate = [&](int c) {
    const int n = tokens(c), lane = threadIdx.x & 63;
    return lane < n ? w.g[(at.begin + at.token(lane, static_cast<int64_t>(c) * C, n)) * w.g_step + at.head] : 0.0f;
  };
  // a chunk's outputs, left in the queries' place, as whole rows
  auto flush = [&](int c) {
    if (outputs && !r.part) ro.store(fresh(threadIdx.x), &s_q[0][0], ldq, static_cast<int64_t>(c) * C, tokens(c));
  };

  Gone gone;
  int turn = 0;
  float g = 0.0f;
  if (at.first != at.stop) {
    fetch(at.first);
    fetch_q(at.first);
    // the last wave, which has the fewest scores to make, forms each chunk's decays one chunk ahead
    if (wv == NW - 1) {
      chunk_decays<C>(s_dec[0], gate(at.first), tokens(at.first), r.reverse, r.from, r.to, r.score);
      if (at.first + at.step != at.stop) g = gate(at.first + at.step);
    }
  }
  for (int c = at.first; c != at.stop; c += at.step, turn ^= 1) {
    const int64_t c0 = static_cast<int64_t>(c) * C;
    const int n = tokens(c), next = c + at.step;
    const Decays<C>& dec = s_dec[turn];
    {
      const int tid = fresh(threadIdx.x);
      RowsK::keep(k, tid, &s_k[0][0], ldk);
      RowsV::keep(v, tid, &s_v[0][0], ldv);
      if (c != at.first) {
        flush(c - at.step);
        if (kK != kV) __syncthreads();  // (else each thread's queries take just its outputs' place)
      }
      if (outputs) RowsK::keep(q, tid, &s_q[0][0], ldq);
      if (next != at.stop) fetch(next);
      if (sums) re.load(x, tid, c0, n);
    }
    __syncthreads();
    if (wv == NW - 1 && next != at.stop) {
      chunk_decays<C>(s_dec[turn ^ 1], g, tokens(next), r.reverse, r.from, r.to, r.score);
      if (next + at.step != at.stop) g = gate(next + at.step);
    }
    if (outputs) {
      f32x16 acc[kTT];
      // scores, transposed (earlier steps s as rows, steps t as columns)
      constexpr int kEach = (kTiles + NW - 1) / NW;
      f32x16 p[kEach];
      {
        const int lane = fresh(threadIdx.x & 63), lo = lane & 31, hi = lane >> 5;
        if (sums) at.leave_entering(w, r, S, c, dec, at.tile * NV + vv, KT * kh, lane);
        const bool flat = __builtin_amdgcn_readfirstlane(dec.flat);
#pragma unroll
        for (int m = 0; m < kEach; ++m) {
          const int i = wv + m * NW, ti = i > 0, si = i > 1;
          p[m] = f32x16{};
          if (i >= kTiles) continue;
#pragma unroll
          for (int j = 0; j < kK; j += 16)
            p[m] = mfma(row8(&s_k[32 * si + lo][j + 8 * hi]), row8(&s_q[32 * ti + lo][j + 8 * hi]), p[m]);
          // times their decays, in the chunk's usual range as one factor of each step; 0 where t does not see s
          const int t = 32 * ti + lo, s0 = 32 * si + 4 * hi;
          if (flat) {
            const float up = dec.up[t];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const f32x4 down = *reinterpret_cast<const f32x4*>(&dec.down[s0 + 8 * i]);
#pragma unroll
              for (int e = 0; e < 4; ++e) p[m][4 * i + e] *= up * down[e];
            }
            if (ti == si) {
#pragma unroll
              for (int i = 0; i < 16; ++i) p[m][i] = where(8 * (i >> 2) + 4 * hi + (i & 3) <= lo, p[m][i]);
            }
          } else {
            const int from = dec.from[t];
            const double ell = dec.ell[t];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int s = s0 + 8 * (i >> 2) + (i & 3);
              const float f = exp_of(ell - dec.ell[s]) * r.score;
              p[m][i] = where((s <= t) & (s >= from), p[m][i] * f);
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t a[2], b[2];
            split<2>(p[m][4 * i], p[m][4 * i + 1], a);
            split<2>(p[m][4 * i + 2], p[m][4 * i + 3], b);
            *reinterpret_cast<u32x2*>(&s_p[0][t][s0 + 8 * i]) = u32x2{a[0], b[0]};
            *reinterpret_cast<u32x2*>(&s_p[1][t][s0 + 8 * i]) = u32x2{a[1], b[1]};
          }
        }
        // what the state that enters gives
#pragma unroll
        for (int t = 0; t < kTT; ++t) acc[t] = f32x16{};
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
            u32x4 b[kTT];
#pragma unroll
            for (int t = 0; t < kTT; ++t) b[t] = row8(&s_q[32 * t + lo][k0 + 32 * kt + 16 * j + 8 * hi]);
#pragma unroll
            for (int m = 0; m < kParts; ++m)
#pragma unroll
              for (int t = 0; t < kTT; ++t) acc[t] = mfma(part[m], b[t], acc[t]);
          }
        const bool cut = __builtin_amdgcn_readfirstlane(dec.cut);
#pragma unroll
        for (int t = 0; t < kTT; ++t) {
          const float f = dec.in[32 * t + lo];
          acc[t] *= f;
          if (cut) drop(acc[t], dec.from[32 * t + lo] < 0 ? 0xffffffffu : 0u);  // what a cut drops may be anything
        }
      }
      __syncthreads();
      if constexpr (KH > 1) {
        // each tile of steps is finished by one of the waves, in the queries' place
        const int lane = fresh(threadIdx.x & 63);
        f32x4* half = reinterpret_cast<f32x4*>(&s_q[0][0]) + lane;
        static_assert(sizeof(s_q) >= NW * 64 * 16 * sizeof(float), "a tile for each wave");
        const f32x16 give = acc[1 - kh];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          half[(4 * wv + i) * 64] = f32x4{give[4 * i], give[4 * i + 1], give[4 * i + 2], give[4 * i + 3]};
        __syncthreads();
        const int other = wv ^ NV;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x4 take = half[(4 * other + i) * 64];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            acc[0][4 * i + e] = (kh ? acc[1][4 * i + e] : acc[0][4 * i + e]) + take[e];
          }
        }
        __syncthreads();
      }
      // from here on acc[t] is tile first + t
      constexpr int kOwn = KH > 1 ? 1 : kTT;
      const int first = KH > 1 ? kh : 0;
      if (SUMS && !sums && next != at.stop) fetch_q(next);
      if (sums) {
        const int tid = fresh(threadIdx.x), lane = tid & 63, lo = lane & 31, hi = lane >> 5;
        RowsV::keep(x, tid, &s_q[0][0], ldq);  // the queries are done with
        if (next != at.stop) fetch_q(next);
        __syncthreads();
        // pairs of steps: the scores times what the other operands' rows give, in float32, and of
        // those what crosses each step (only sums of such pairs: a difference of sums over rows and
        // columns would lose what strong decays leave)
        if (pairs) {
#pragma unroll
          for (int m = 0; m < kEach; ++m) {
            const int i = wv + m * NW, ti = i > 0, si = i > 1;
            if (i >= kTiles) continue;
            f32x16 u = {};
#pragma unroll
            for (int j = 0; j < kV; j += 16)
              u = mfma(row8(&s_v[32 * si + lo][j + 8 * hi]), row8(&s_q[32 * ti + lo][j + 8 * hi]), u);
            const int t = 32 * ti + lo, from = dec.from[t];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int s = 32 * si + 8 * (i >> 2) + 4 * hi + (i & 3);
              u[i] = where((s < t) & (s >= from), u[i] * p[m][i]);
            }
            const float row = prefix_of(u, hi);
#pragma unroll
            for (int i = 0; i < 16; ++i) u[i] = where(32 * si + 8 * (i >> 2) + 4 * hi + (i & 3) < t, u[i]);
            const float crossing = over_columns(u, lo);
            // step s + 1 is crossed by tile (0, 0)'s and (1, 1)'s pairs, and up to step 32 by (1, 0)'s; those
            // after it by the latter's later rows
            if ((lo & 1) == 0) s_row(32 * si + column_step(lo, hi))[ti != si] = crossing;
            if (ti != si) {
              const float later = over_later(row, lo);
              if (hi == 0) s_row(t)[1] = later;
            }
          }
        }
        // and what the state that enters gives, with the same rows
#pragma unroll
        for (int t = 0; t < kOwn; ++t) {
          const int row = 32 * (first + t) + lo;
          float sum = 0.0f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const u32x2 e = *reinterpret_cast<const u32x2*>(&s_q[row][32 * vv + 8 * i + 4 * hi]);
            sum = fmaf(acc[t][4 * i], low(e[0]), sum);
            sum = fmaf(acc[t][4 * i + 1], high(e[0]), sum);
            sum = fmaf(acc[t][4 * i + 2], low(e[1]), sum);
            sum = fmaf(acc[t][4 * i + 3], high(e[1]), sum);
          }
          sum = over_halves(sum);
          if (hi == 0) s_red(row)[vv] = sum;
        }
        __syncthreads();  // the outputs take the rows' place
        if (tid < n) {
          float sum = 0.0f, crossing = 0.0f;
#pragma unroll
          for (int i = 0; i < NV; ++i) sum += s_red(tid)[i];
          if (pairs && tid > 0) crossing = s_row(tid - 1)[0] + s_row(tid > 32 ? tid : tid - 1)[1];
          const int64_t to = (static_cast<int64_t>(at.tile) * w.heads + at.head) * w.rows + at.begin + at.token(tid, c0, n);
          r.sums[to] = sum;
          if (pairs) r.pairs[to] = crossing;
        }
      }
      const int lane = fresh(threadIdx.x & 63), lo = lane & 31, hi = lane >> 5;
      // A score of 0 times a value that is not finite is NaN: with such a value among this
      // wave's, steps are added one by one, to the outputs that see them only (by their places: a
      // score that they see may be 0 too).
      u32x4 values[C / 16];
      u16x2 most = {};
#pragma unroll
      for (int j = 0; j < C / 16; ++j) {
        values[j] = column8<false>(&s_v[16 * j][32 * vv], ldv, lane);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, values[j][e] & 0x7fff7fffu));
      }
      if (__any((most[0] >= 0x7f80) | (most[1] >= 0x7f80))) {
#pragma unroll 1
        for (int s = 0; s < n; ++s) {
#pragma unroll
          for (int t = 0; t < kOwn; ++t) {
            const int row = 32 * (first + t) + lo;
            const float f = Bf16Io::to_f32(s_p[0][row][s]) + Bf16Io::to_f32(s_p[1][row][s]);
            if ((s <= row) & (s >= dec.from[row])) {
#pragma unroll
              for (int i = 0; i < 16; ++i)
                acc[t][i] = fmaf(f, Bf16Io::to_f32(s_v[s][32 * vv + 8 * (i >> 2) + 4 * hi + (i & 3)]), acc[t][i]);
            }
          }
        }
        // nothing is left for the products below (one path for both: see drop)
#pragma unroll
        for (int j = 0; j < C / 16; ++j) {
          uint32_t none = 0;
          asm volatile("" : "+v"(none));
          values[j] &= none;
        }
      }
#pragma unroll
      for (int j = 0; j < C / 16; ++j) {
        if (KH > 1 && j / 2 > first) break;
#pragma unroll
        for (int t = KH > 1 ? 0 : j / 2; t < kOwn; ++t) {
          const int row = 32 * (first + t) + lo;
          acc[t] = mfma(values[j], row8(&s_p[0][row][16 * j + 8 * hi]), acc[t]);
          acc[t] = mfma(values[j], row8(&s_p[1][row][16 * j + 8 * hi]), acc[t]);
        }
      }
      if (r.part) {
        // shared operands' gradients: a float32 row for each head
        const int channel = at.tile * kV + 32 * vv + 4 * hi;
        float* to = r.part + (at.begin + at.token(0, c0, n)) * w.heads * r.V + static_cast<int64_t>(at.head) * r.V + channel;
        const int64_t step = static_cast<int64_t>(at.reverse ? -w.heads : w.heads) * r.V;
#pragma unroll
        for (int t = 0; t < kOwn; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (32 * (first + t) + lo < n && channel + 8 * i < r.V)
              *reinterpret_cast<Words<float, 4, 4>*>(to + (32 * (first + t) + lo) * step + 8 * i) =
                  Words<float, 4, 4>{acc[t][4 * i], acc[t][4 * i + 1], acc[t][4 * i + 2], acc[t][4 * i + 3]};
      } else {
#pragma unroll
        for (int t = 0; t < kOwn; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<u32x2*>(&s_q[32 * (first + t) + lo][32 * vv + 8 * i + 4 * hi]) =
                u32x2{pack(acc[t][4 * i], acc[t][4 * i + 1]), pack(acc[t][4 * i + 2], acc[t][4 * i + 3])};
      }
    }
    if (__builtin_amdgcn_readfirstlane(dec.cut)) {
      // the rows of steps that a later one cuts off, which may be anything, become 0
      const int tid = fresh(threadIdx.x);
      __syncthreads();
      for (int id = tid; id < C * kK / 2; id += kThreads) {
        const int s = id / (kK / 2);
        if (s < dec.kept) *reinterpret_cast<uint32_t*>(&s_k[s][2 * (id % (kK / 2))]) = 0;
      }
      for (int id = tid; id < C * kV / 2; id += kThreads) {
        const int s = id / (kV / 2);
        if (s < dec.kept) *reinterpret_cast<uint32_t*>(&s_v[s][2 * (id % (kV / 2))]) = 0;
      }
      __syncthreads();
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) drop(S[kt], 0);
    }
    const int lane = fresh(threadIdx.x & 63), hi = lane >> 5;
    const float all = dec.all;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) S[kt] *= all;
#pragma unroll
    for (int j = 0; j < C / 16; ++j) {
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
      // products that follow one another go to different tiles, here and above (to one tile its
      // parts' three in a row: prompts 244 us where these took 237)
      constexpr int kSide = KT < 4 ? KT : 4;
#pragma unroll
      for (int kt = 0; kt < KT; kt += kSide) {
        u32x4 a[kSide];
#pragma unroll
        for (int i = 0; i < kSide; ++i) a[i] = column8<true>(&s_k[16 * j][k0 + 32 * (kt + i)], ldk, lane);
#pragma unroll
        for (int m = 0; m < 3; ++m)
#pragma unroll
          for (int i = 0; i < kSide; ++i) S[kt + i] = mfma(a[i], part[m], S[kt + i]);
      }
    }
    gone.add(dec.cut, dec.total);
    __syncthreads();  // the next chunk's rows take these places
  }
  if (at.first != at.stop) flush(at.stop - at.step);
  at.leave_state<StateRows>(w, r, S, gone, col, threadIdx.x % 64 / 32, k0);
}

template <int KT, int KH, int NV>
hipError_t launch(const MixCall& w, hipStream_t stream) {
  bool sums = false;
  for (int k = 0; k < w.roles; ++k) sums |= w.role[k].sums != nullptr && !w.role[k].local;
  const dim3 grid(static_cast<unsigned>(walk_units(w)));
  if (sums)
    hipLaunchKernelGGL((walk_bf16_kernel<KT, KH, NV, true>), grid, dim3(64 * NV * KH), 0, stream, w);
  else
    hipLaunchKernelGGL((walk_bf16_kernel<KT, KH, NV, false>), grid, dim3(64 * NV * KH), 0, stream, w);
  return hipGetLastError();
}

template <int KT>
hipError_t by_values(const MixCall& w, hipStream_t stream) {
  return value_width(w.role[0].V) == 64 ? launch<KT / 2, 2, 2>(w, stream)
                                                                 : launch<KT, 1, 4>(w, stream);
}

}  // namespace

hipError_t launch_walk_bf16(const MixCall& w, hipStream_t stream) {
  const int kt = key_tiles(w.role[0].K);
  return kt == 2 ? by_values<2>(w, stream) : kt == 4 ? by_values<4>(w, stream) : by_values<8>(w, stream);
}

}  // namespace mscan

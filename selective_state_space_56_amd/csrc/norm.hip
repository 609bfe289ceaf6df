// RMS norm of a block's entry: y = s rstd w with s = x + residual and
// rstd = 1 / sqrt(mean s^2 + eps), as an io output or as e4m3 with scales, and
// its backward.
//
// Bound by HBM: every element is read once and written once. Up to kRegDim
// channels a row stays in its workgroup's registers from the first load to the
// last store, 8 channels per lane, and the next row's loads are in flight while
// the current row is reduced and written. Wider rows are read again for each
// use (from the L2 cache, which holds them). Rows of any alignment take the same
// path (the last piece of a row element by element where the row is not whole
// pieces).
//
// Measured on an MI355X (a plain copy moves 5.3 TB/s): 16384 x 2560, bf16 with
// an fp32 stream, to 8 bits 85 us (461 MB, 5.4 TB/s); bf16 with a bf16 stream 60 us
// (336 MB, 5.6 TB/s), its backward 64 us and 5 for dweight (336 MB and 8 MB of
// parts, 5.4 TB/s). Away from such rows: up to 512 channels a launch of 16384 rows
// takes about 10 us whatever their number (a row takes a whole wave), and
// 4096 x 20000 bf16 155 us to 8 bits in groups and 461 a training step, where a copy of
// the same bytes takes 109 and 247 (each use of a wide row reads it again).
#include "block.h"
#include "block_math.h"
#include "colsum.h"

namespace mscan {

namespace {

constexpr int kPiece = 8;        // channels per lane and access
constexpr int kMaxWaves = 16;
constexpr int kRegDim = kMaxWaves * 64 * kPiece;
constexpr float kE4m3Max = 448.0f;
constexpr float kTiny = 0x1p-100f;

template <class IO>
using Row8 = Piece<IO, kPiece>;

template <class IO>
__device__ __forceinline__ void load8(Row8<IO>& to, const typename IO::raw* row, int d, int dim) {
  if (d + kPiece <= dim)
    to.load(row + d);
  else
    to.load_some(row + d, dim - d);
}

// The same for what is not read again: the backward's loads. A training step of
// 16384 x 2560 bf16 takes 130 us instead of 133.5, of 8192 rows 71.3 against 70.7, of
// 4096 38.6 against 41.4, of 2048 and fewer the same; of 16384 x 2560 fp32 273.5
// against 266.8. The forward's measured no better with it.
template <class IO>
__device__ __forceinline__ void load8_last(Row8<IO>& to, const typename IO::raw* row, int d, int dim) {
  if (d + kPiece <= dim)
    to.load_last(row + d);
  else
    to.load_some(row + d, dim - d);
}

template <class IO>
__device__ __forceinline__ void store8(const Row8<IO>& from, typename IO::raw* row, int d, int dim) {
  if (d + kPiece <= dim)
    from.store(row + d);
  else
    from.store_some(row + d, dim - d);
}

struct AddOp {
  static __device__ __forceinline__ float of(float a, float b) { return a + b; }
};
struct MaxOp {
  static __device__ __forceinline__ float of(float a, float b) { return fmaxf(a, b); }
};

// The value of the lane N places round within its 16 lanes.
template <int N>
__device__ __forceinline__ float turned(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x120 + N, 0xf, 0xf, true));
}

// Over 16 neighbouring lanes (the channels of one group of 128), in each of them.
template <class Op>
__device__ __forceinline__ float over_16(float v) {
  v = Op::of(v, turned<8>(v));
  v = Op::of(v, turned<4>(v));
  v = Op::of(v, turned<2>(v));
  return Op::of(v, turned<1>(v));
}

template <class Op>
__device__ __forceinline__ float over_wave(float v) {
  v = over_16<Op>(v);
  // swapping rows of 16 lanes, then halves, of two copies leaves each with one side's value
  const auto rows = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = Op::of(__uint_as_float(rows[0]), __uint_as_float(rows[1]));
  const auto halves = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return Op::of(__uint_as_float(halves[0]), __uint_as_float(halves[1]));
}

// N values over the workgroup, in every thread and the same in each (the waves'
// values are joined in their order). One barrier: two calls in a row use two
// different `scratch` arrays.
template <class Op, int N>
__device__ __forceinline__ void over_block(float (&v)[N], float (&scratch)[N][kMaxWaves]) {
  const int waves = blockDim.x / 64, wave = threadIdx.x / 64;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = over_wave<Op>(v[i]);
  if (waves == 1) return;
  if (threadIdx.x % 64 == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) scratch[i][wave] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = scratch[i][0];
    for (int k = 1; k < waves; ++k) v[i] = Op::of(v[i], scratch[i][k]);
  }
}

// 1 / sqrt(ss / dim + eps). The hardware's root takes values below its normal
// range as 0, so those are lifted by 2^64 first.
__device__ __forceinline__ float rstd_of(float ss, float inv_dim, float eps) {
  const float m = fmaf(ss, inv_dim, eps);
  return m < 0x1p-100f ? __builtin_amdgcn_rsqf(m * 0x1p64f) * 0x1p32f : __builtin_amdgcn_rsqf(m);
}

__device__ __forceinline__ float top_of(const float (&y)[kPiece]) {
  float top = kTiny;
#pragma unroll
  for (int j = 0; j < kPiece; ++j) top = fmaxf(top, fabsf(y[j]));
  return top;
}

// y / scale, rounded to float32 as a division does. For scales within kExact the
// correctly rounded reciprocal and two corrections by the remainder, which no
// number in them leaves float32's range for: the first makes the quotient one of
// the two floats around it, the second the nearer one. The compiler's division,
// which also holds at the ends of the range, costs more: 16384 x 2560 bf16 with an
// fp32 stream 84.6 us so, 86.5 with it (83.6 when y was multiplied by a rounded
// 1 / scale, which gave the neighbouring 8-bit value next to a middle).
constexpr float kExactFrom = 0x1p-60f, kExactTo = 0x1p100f;
__device__ __forceinline__ void divide(float (&y)[kPiece], float scale) {
  if (scale >= kExactFrom && scale <= kExactTo) {
    const float inv = 1.0f / scale;
#pragma unroll
    for (int j = 0; j < kPiece; ++j) {
      float q = y[j] * inv;
      q = fmaf(fmaf(-q, scale, y[j]), inv, q);
      y[j] = fmaf(fmaf(-q, scale, y[j]), inv, q);
    }
  } else {
#pragma unroll
    for (int j = 0; j < kPiece; ++j) y[j] /= scale;
  }
}

// 8 values as e4m3: the rounded float32 quotients by the scale that is stored.
// They are at most 448 and a rounding, which rounds to 448: nothing to saturate.
__device__ __forceinline__ void store_e4m3(float (&y)[kPiece], float scale, uint8_t* row, int d, int dim) {
  divide(y, scale);
  uint32_t q[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int word = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * h], y[4 * h + 1], 0, false);
    word = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * h + 2], y[4 * h + 3], word, true);
    q[h] = static_cast<uint32_t>(word);
  }
  if (d + kPiece <= dim)
    __builtin_memcpy(row + d, q, 8);
  else
#pragma unroll
    for (int j = 0; j < kPiece; ++j)
      if (d + j < dim) row[d + j] = static_cast<uint8_t>(q[j / 4] >> (8 * (j % 4)));
}

enum Out { kIo, kRowScale, kGroupScale };

// Rows blockIdx.x, blockIdx.x + gridDim.x, ..., channels 8 t .. 8 t + 7 in thread t.
template <class IO, class RES, int OUT>
__global__ __launch_bounds__(1024) void norm_kernel(NormProblem p) {
  using raw = typename IO::raw;
  using res_raw = typename RES::raw;
  __shared__ float sums[2][1][kMaxWaves], tops[2][1][kMaxWaves];
  const int dim = static_cast<int>(p.dim), d = static_cast<int>(threadIdx.x) * kPiece;
  const float inv_dim = 1.0f / static_cast<float>(dim);
  Row8<F32Io> w;
  load8(w, p.weight, d, dim);
  Row8<IO> x;
  Row8<RES> r;
  const auto load = [&](int64_t row) {
    load8(x, static_cast<const raw*>(p.x) + row * p.sx, d, dim);
    if (p.residual) load8(r, static_cast<const res_raw*>(p.residual) + row * p.sres, d, dim);
  };
  load(blockIdx.x);
  int turn = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
    float s[kPiece], ss[1] = {0.0f};
    if (p.residual) {
#pragma unroll
      for (int j = 0; j < kPiece; ++j) s[j] = x.get(j) + r.get(j);
      r.set(s);  // rounded to the stream's type here
#pragma unroll
      for (int j = 0; j < kPiece; ++j) s[j] = r.get(j);
      store8(r, static_cast<res_raw*>(p.sum) + row * p.ssum, d, dim);
    } else {
#pragma unroll
      for (int j = 0; j < kPiece; ++j) s[j] = x.get(j);
    }
    if (row + gridDim.x < p.rows) load(row + gridDim.x);
#pragma unroll
    for (int j = 0; j < kPiece; ++j) ss[0] = fmaf(s[j], s[j], ss[0]);
    over_block<AddOp>(ss, sums[turn]);
    const float rstd = rstd_of(ss[0], inv_dim, p.eps);
#pragma unroll
    for (int j = 0; j < kPiece; ++j) s[j] = s[j] * rstd * w.get(j);
    if constexpr (OUT == kIo) {
      Row8<IO> y;
      y.set(s);
      store8(y, static_cast<raw*>(p.out) + row * p.so, d, dim);
    } else {
      // channels past the end are 0 and do not raise a maximum
      float top[1] = {top_of(s)};
      float scale;
      if constexpr (OUT == kGroupScale) {
        scale = over_16<MaxOp>(top[0]) / kE4m3Max;
        if (threadIdx.x % 16 == 0 && d < dim) p.scale[row * ((dim + 127) / 128) + d / 128] = scale;
      } else {
        over_block<MaxOp>(top, tops[turn]);
        scale = top[0] / kE4m3Max;
        if (threadIdx.x == 0) p.scale[row] = scale;
      }
      store_e4m3(s, scale, static_cast<uint8_t*>(p.out) + row * p.so, d, dim);
    }
  }
}

// Rows of more than kRegDim channels, in turns of 1024 pieces.
template <class IO, class RES>
__global__ __launch_bounds__(1024) void norm_wide_kernel(NormProblem p) {
  using raw = typename IO::raw;
  using res_raw = typename RES::raw;
  __shared__ float sums[2][1][kMaxWaves], tops[2][1][kMaxWaves];
  const int dim = static_cast<int>(p.dim), first = static_cast<int>(threadIdx.x) * kPiece;
  const float inv_dim = 1.0f / static_cast<float>(dim);
  const int whole = (dim + kRegDim - 1) / kRegDim * kRegDim;  // every thread takes every turn
  int turn = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
    const raw* xr = static_cast<const raw*>(p.x) + row * p.sx;
    res_raw* sr = static_cast<res_raw*>(p.sum) + row * p.ssum;
    float ss[1] = {0.0f};
    for (int d = first; d < dim; d += kRegDim) {
      Row8<IO> x;
      load8(x, xr, d, dim);
      float s[kPiece];
#pragma unroll
      for (int j = 0; j < kPiece; ++j) s[j] = x.get(j);
      if (p.residual) {
        Row8<RES> r;
        load8(r, static_cast<const res_raw*>(p.residual) + row * p.sres, d, dim);
#pragma unroll
        for (int j = 0; j < kPiece; ++j) s[j] += r.get(j);
        r.set(s);
#pragma unroll
        for (int j = 0; j < kPiece; ++j) s[j] = r.get(j);
        store8(r, sr, d, dim);
      }
#pragma unroll
      for (int j = 0; j < kPiece; ++j) ss[0] = fmaf(s[j], s[j], ss[0]);
    }
    over_block<AddOp>(ss, sums[turn]);
    const float rstd = rstd_of(ss[0], inv_dim, p.eps);
    // y of a piece, from the stream that this same thread has stored (or x)
    const auto normed = [&](int d, float (&y)[kPiece]) {
      Row8<F32Io> w;
      load8(w, p.weight, d, dim);
      if (p.residual) {
        Row8<RES> r;
        load8(r, sr, d, dim);
#pragma unroll
        for (int j = 0; j < kPiece; ++j) y[j] = r.get(j) * rstd * w.get(j);
      } else {
        Row8<IO> x;
        load8(x, xr, d, dim);
#pragma unroll
        for (int j = 0; j < kPiece; ++j) y[j] = x.get(j) * rstd * w.get(j);
      }
    };
    float y[kPiece], top[1] = {kTiny}, scale = 0.0f;
    if (p.scale && !p.group) {
      for (int d = first; d < dim; d += kRegDim) {
        normed(d, y);
        top[0] = fmaxf(top[0], top_of(y));
      }
      over_block<MaxOp>(top, tops[turn]);
      scale = top[0] / kE4m3Max;
      if (threadIdx.x == 0) p.scale[row] = scale;
    }
    for (int d = first; d < whole; d += kRegDim) {
#pragma unroll
      for (int j = 0; j < kPiece; ++j) y[j] = 0.0f;
      if (d < dim) normed(d, y);
      if (p.scale && p.group) {
        scale = over_16<MaxOp>(top_of(y)) / kE4m3Max;
        if (threadIdx.x % 16 == 0 && d < dim) p.scale[row * ((dim + 127) / 128) + d / 128] = scale;
      }
      if (d >= dim) continue;
      if (p.scale) {
        store_e4m3(y, scale, static_cast<uint8_t*>(p.out) + row * p.so, d, dim);
      } else {
        Row8<IO> out;
        out.set(y);
        store8(out, static_cast<raw*>(p.out) + row * p.so, d, dim);
      }
    }
  }
}

// Rows blockIdx.x, blockIdx.x + gridDim.x, ..., each read once: both sums
// (s^2 and s u, u = w dout) in one reduction, then the row's gradient from the
// registers. Every workgroup keeps its rows' sum of dout s rstd: one row of parts.
template <class IO, class RES>
__global__ __launch_bounds__(1024, 5) void norm_bwd_kernel(NormBwdProblem p, float* parts) {
  using raw = typename IO::raw;
  using res_raw = typename RES::raw;
  __shared__ float sums[2][2][kMaxWaves];
  const int dim = static_cast<int>(p.dim), d = static_cast<int>(threadIdx.x) * kPiece;
  Row8<F32Io> w, dw;
  load8(w, p.weight, d, dim);
#pragma unroll
  for (int j = 0; j < kPiece; ++j) dw.v[j] = 0.0f;
  Row8<RES> s, ds;
  Row8<IO> dy;
  const auto load = [&](int64_t row) {
    load8_last(s, static_cast<const res_raw*>(p.sum) + row * p.ssum, d, dim);
    load8_last(dy, static_cast<const raw*>(p.dout) + row * p.so, d, dim);
    if (p.dsum) load8_last(ds, static_cast<const res_raw*>(p.dsum) + row * p.sdsum, d, dim);
  };
  load(blockIdx.x);
  int turn = 0;
  const float inv_dim = 1.0f / static_cast<float>(dim);
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
    Row8<RES> s0 = s, ds0;
    if (p.dsum) ds0 = ds;
    const Row8<IO> dy0 = dy;
    if (row + gridDim.x < p.rows) load(row + gridDim.x);
    float both[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < kPiece; ++j) {
      const float sv = s0.get(j);
      both[0] = fmaf(sv, sv, both[0]);
      both[1] = fmaf(sv, w.get(j) * dy0.get(j), both[1]);
    }
    over_block<AddOp>(both, sums[turn]);
    const float rstd = rstd_of(both[0], inv_dim, p.eps), mean = both[1] * rstd * inv_dim;
    float v[kPiece];
#pragma unroll
    for (int j = 0; j < kPiece; ++j) {
      const float norm = s0.get(j) * rstd, g = dy0.get(j);
      dw.v[j] = fmaf(g, norm, dw.v[j]);
      v[j] = rstd * fmaf(-norm, mean, w.get(j) * g);
      if (p.dsum) v[j] += ds0.get(j);
    }
    Row8<IO> dx;
    s0.set(v);
    dx.set(v);
    store8(s0, static_cast<res_raw*>(p.dresidual) + row * p.sdres, d, dim);
    if (p.dx) store8(dx, static_cast<raw*>(p.dx) + row * p.sdx, d, dim);
  }
  store8(dw, parts + static_cast<int64_t>(blockIdx.x) * dim, d, dim);
}

// Rows of more than kRegDim channels; the parts of dweight are kept in memory.
template <class IO, class RES>
__global__ __launch_bounds__(1024) void norm_bwd_wide_kernel(NormBwdProblem p, float* parts) {
  using raw = typename IO::raw;
  using res_raw = typename RES::raw;
  __shared__ float sums[2][2][kMaxWaves];
  const int dim = static_cast<int>(p.dim), first = static_cast<int>(threadIdx.x) * kPiece;
  float* part = parts + static_cast<int64_t>(blockIdx.x) * dim;
  const float inv_dim = 1.0f / static_cast<float>(dim);
  int turn = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
    const res_raw* sr = static_cast<const res_raw*>(p.sum) + row * p.ssum;
    const raw* yr = static_cast<const raw*>(p.dout) + row * p.so;
    float both[2] = {0.0f, 0.0f};
    for (int d = first; d < dim; d += kRegDim) {
      Row8<RES> s;
      Row8<IO> dy;
      Row8<F32Io> w;
      load8(s, sr, d, dim);
      load8(dy, yr, d, dim);
      load8(w, p.weight, d, dim);
#pragma unroll
      for (int j = 0; j < kPiece; ++j) {
        both[0] = fmaf(s.get(j), s.get(j), both[0]);
        both[1] = fmaf(s.get(j), w.get(j) * dy.get(j), both[1]);
      }
    }
    over_block<AddOp>(both, sums[turn]);
    const float rstd = rstd_of(both[0], inv_dim, p.eps), mean = both[1] * rstd * inv_dim;
    for (int d = first; d < dim; d += kRegDim) {
      Row8<RES> s, ds;
      Row8<IO> dy, dx;
      Row8<F32Io> w, dw;
      load8(s, sr, d, dim);
      load8(dy, yr, d, dim);
      load8(w, p.weight, d, dim);
      if (p.dsum) load8(ds, static_cast<const res_raw*>(p.dsum) + row * p.sdsum, d, dim);
      if (row != blockIdx.x) load8(dw, part, d, dim);
      float v[kPiece];
#pragma unroll
      for (int j = 0; j < kPiece; ++j) {
        const float norm = s.get(j) * rstd, g = dy.get(j);
        dw.v[j] = fmaf(g, norm, row != blockIdx.x ? dw.v[j] : 0.0f);
        v[j] = rstd * fmaf(-norm, mean, w.get(j) * g);
        if (p.dsum) v[j] += ds.get(j);
      }
      s.set(v);
      dx.set(v);
      store8(s, static_cast<res_raw*>(p.dresidual) + row * p.sdres, d, dim);
      if (p.dx) store8(dx, static_cast<raw*>(p.dx) + row * p.sdx, d, dim);
      store8(dw, part, d, dim);
    }
  }
}

// Threads of a row: one piece each, in whole waves.
unsigned threads_of(int64_t dim) {
  const int64_t waves = (dim + 64 * kPiece - 1) / (64 * kPiece);
  return static_cast<unsigned>(64 * (waves < kMaxWaves ? waves : kMaxWaves));
}

// Workgroups of a launch: what runs at once (of the backward four waves per
// SIMD, less what does not pack), each with the same number of rows but for the
// last. The backward takes two rows at least: a part of dweight per row is
// as much to write and read as half a row (1023 x 1541 fp32: 11.3 + 3.9 us with
// two, 12.0 + 6.2 with one, 13.3 + 3.9 with four).
unsigned grid_of(int64_t rows, int64_t dim, bool backward) {
  const int64_t waves = threads_of(dim) / 64;
  const int64_t per_cu = backward ? 16 / waves : (20 + waves - 1) / waves;
  const int64_t most = per_cu * device_cu_count(), least = backward ? 2 : 1;
  int64_t each = (rows + most - 1) / most;
  each = each < least ? least : each;
  return static_cast<unsigned>((rows + each - 1) / each);
}

template <class IO, class RES>
hipError_t launch_types(const NormProblem& p, hipStream_t stream) {
  const dim3 grid(grid_of(p.rows, p.dim, false)), block(threads_of(p.dim));
  if (p.dim > kRegDim)
    hipLaunchKernelGGL((norm_wide_kernel<IO, RES>), grid, block, 0, stream, p);
  else if (!p.scale)
    hipLaunchKernelGGL((norm_kernel<IO, RES, kIo>), grid, block, 0, stream, p);
  else if (p.group)
    hipLaunchKernelGGL((norm_kernel<IO, RES, kGroupScale>), grid, block, 0, stream, p);
  else
    hipLaunchKernelGGL((norm_kernel<IO, RES, kRowScale>), grid, block, 0, stream, p);
  return hipGetLastError();
}

template <class IO, class RES>
hipError_t launch_types(const NormBwdProblem& p, unsigned groups, float* parts, hipStream_t stream) {
  const dim3 grid(groups), block(threads_of(p.dim));
  if (p.dim > kRegDim)
    hipLaunchKernelGGL((norm_bwd_wide_kernel<IO, RES>), grid, block, 0, stream, p, parts);
  else
    hipLaunchKernelGGL((norm_bwd_kernel<IO, RES>), grid, block, 0, stream, p, parts);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm(const NormProblem& p, hipStream_t stream) {
  if (p.io == kIoF32) return launch_types<F32Io, F32Io>(p, stream);
  if (p.res == kIoF32) return launch_types<Bf16Io, F32Io>(p, stream);
  return launch_types<Bf16Io, Bf16Io>(p, stream);
}

size_t norm_bwd_workspace_bytes(int64_t rows, int64_t dim) {
  if (rows == 0 || dim == 0) return 0;
  return (static_cast<size_t>(grid_of(rows, dim, true)) * dim * 4 + 255) / 256 * 256;
}

hipError_t launch_norm_bwd(const NormBwdProblem& p, void* workspace, hipStream_t stream) {
  const unsigned groups = p.rows > 0 ? grid_of(p.rows, p.dim, true) : 0;
  float* parts = static_cast<float*>(workspace);
  if (groups > 0) {
    const hipError_t e = p.io == kIoF32    ? launch_types<F32Io, F32Io>(p, groups, parts, stream)
                         : p.res == kIoF32 ? launch_types<Bf16Io, F32Io>(p, groups, parts, stream)
                                           : launch_types<Bf16Io, Bf16Io>(p, groups, parts, stream);
    if (e != hipSuccess) return e;
  }
  return launch_colsum(parts, groups, p.dim, StoreFlat{p.dweight}, stream);
}

}  // namespace mscan

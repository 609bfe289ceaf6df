// Sums over the rows of a float32 matrix, one per column: the last step of the
// gradients that are shared by every token (decay, norm weight, convolution
// taps), whose per-workgroup parts are rows of a workspace. A workgroup takes 32
// columns and all rows: 4 to 7 us for 1500 columns and more; with few columns
// long rows of work fall to few workgroups (8192 x 320 of a convolution's backward
// over 4 x 131072 x 64: 14 us beside 79 of its main pass).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mscan {

constexpr int kColsumCols = 32;    // columns per workgroup: one 128-byte piece of a row
constexpr int kColsumRuns = 32;    // threads per column, each with its own rows
constexpr int kColsumAhead = 8;    // loads in flight per thread

// Workgroups of a launch at most; each takes every kColsumGroups-th group of
// columns. A launch holds fewer than 2^32 threads, and a convolution's backward may
// have 5 x 2^31 columns of sums.
constexpr int64_t kColsumGroups = int64_t(1) << 20;

// parts (rows, cols) -> out[column]; Store(column, sum) places it. Thread k of a
// column adds rows k, k + 32, ... in that order and one thread adds the 32 sums
// in order, so the result does not depend on how the waves run.
template <class Store>
__global__ __launch_bounds__(kColsumCols* kColsumRuns) void colsum_kernel(const float* parts, int64_t rows,
                                                                          int64_t cols, Store store) {
  __shared__ float sums[kColsumRuns][kColsumCols + 1];
  const int col = threadIdx.x % kColsumCols, run = threadIdx.x / kColsumCols;
  for (int64_t first = static_cast<int64_t>(blockIdx.x) * kColsumCols; first < cols;
       first += static_cast<int64_t>(gridDim.x) * kColsumCols) {
    const int64_t c = first + col;
    float s = 0.0f;
    if (c < cols) {
      const float* p = parts + c;
      int64_t r = run;
      for (; r + (kColsumAhead - 1) * kColsumRuns < rows; r += kColsumAhead * kColsumRuns) {
        float v[kColsumAhead];
#pragma unroll
        for (int k = 0; k < kColsumAhead; ++k) v[k] = p[(r + k * kColsumRuns) * cols];
#pragma unroll
        for (int k = 0; k < kColsumAhead; ++k) s += v[k];
      }
      for (; r < rows; r += kColsumRuns) s += p[r * cols];
    }
    sums[run][col] = s;
    __syncthreads();
    if (run == 0 && c < cols) {
      float t = 0.0f;
#pragma unroll
      for (int k = 0; k < kColsumRuns; ++k) t += sums[k][col];
      store(c, t);
    }
    __syncthreads();  // the next columns' sums take these places
  }
}

struct StoreFlat {
  float* out;
  __device__ __forceinline__ void operator()(int64_t c, float v) const { out[c] = v; }
};

template <class Store>
hipError_t launch_colsum(const float* parts, int64_t rows, int64_t cols, Store store, hipStream_t stream) {
  const int64_t groups = (cols + kColsumCols - 1) / kColsumCols;
  hipLaunchKernelGGL((colsum_kernel<Store>), dim3(static_cast<unsigned>(groups < kColsumGroups ? groups : kColsumGroups)),
                     dim3(kColsumCols * kColsumRuns), 0, stream, parts, rows, cols, store);
  return hipGetLastError();
}

}  // namespace mscan

// Sums over the rows of a float32 matrix, one per column: the last step of the
// gradients that are shared by every token (decay, norm weight, convolution
// taps), whose per-workgroup parts are rows of a workspace.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mscan {

constexpr int kColsumCols = 64;    // columns per workgroup, one per lane
constexpr int kColsumWaves = 16;   // waves per workgroup, each with its own rows

// parts (rows, cols) -> out[column]; Store(column, sum) places it. Each wave
// adds rows w, w + 16, ... in that order and wave 0 adds the waves' sums in
// order, so the result does not depend on how the waves run.
template <class Store>
__global__ __launch_bounds__(kColsumCols* kColsumWaves) void colsum_kernel(const float* parts, int64_t rows,
                                                                           int64_t cols, Store store) {
  __shared__ float sums[kColsumWaves][kColsumCols];
  const int lane = threadIdx.x % kColsumCols, wave = threadIdx.x / kColsumCols;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kColsumCols + lane;
  float s = 0.0f;
  if (c < cols)
    for (int64_t r = wave; r < rows; r += kColsumWaves) s += parts[r * cols + c];
  sums[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < cols) {
    float t = 0.0f;
#pragma unroll
    for (int k = 0; k < kColsumWaves; ++k) t += sums[k][lane];
    store(c, t);
  }
}

struct StoreFlat {
  float* out;
  __device__ __forceinline__ void operator()(int64_t c, float v) const { out[c] = v; }
};

template <class Store>
hipError_t launch_colsum(const float* parts, int64_t rows, int64_t cols, Store store, hipStream_t stream) {
  hipLaunchKernelGGL((colsum_kernel<Store>), dim3(static_cast<unsigned>((cols + kColsumCols - 1) / kColsumCols)),
                     dim3(kColsumCols * kColsumWaves), 0, stream, parts, rows, cols, store);
  return hipGetLastError();
}

}  // namespace mscan

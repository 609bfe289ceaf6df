// Drives the block operators' C ABI layer (api_block.cpp) on the host, with its
// launches replaced by counters: valid calls at small and extreme sizes, and
// refusals. Built with AddressSanitizer and UndefinedBehaviorSanitizer.
#include <cstdio>
#include <cstdlib>

#include "block.h"
#include "block/mamba_conv_bwd.h"
#include "block/mamba_gated.h"
#include "block/mamba_norm.h"

static int g_launched = 0;

namespace mscan {
size_t gated_fwd_workspace_bytes(int64_t b, int64_t, int64_t d) { return b * d > 0 ? 512 : 0; }
size_t gated_bwd_workspace_bytes(int64_t b, int64_t, int64_t d) { return b * d > 0 ? 512 : 0; }
size_t norm_bwd_workspace_bytes(int64_t r, int64_t d) { return r * d > 0 ? 256 : 0; }
size_t conv_bwd_workspace_bytes(int64_t b, int64_t, int64_t d, int) { return b * d > 0 ? 256 : 0; }
hipError_t launch_gated_fwd(const GatedProblem&, void*, hipStream_t) { return ++g_launched, hipSuccess; }
hipError_t launch_gated_bwd(const GatedBwdProblem&, void*, hipStream_t) { return ++g_launched, hipSuccess; }
hipError_t launch_gated_update(const GatedUpdateProblem&, hipStream_t) { return ++g_launched, hipSuccess; }
hipError_t launch_norm(const NormProblem&, hipStream_t) { return ++g_launched, hipSuccess; }
hipError_t launch_norm_bwd(const NormBwdProblem&, void*, hipStream_t) { return ++g_launched, hipErrorInvalidValue; }
hipError_t launch_conv_bwd(const ConvBwdProblem&, void*, hipStream_t) { return ++g_launched, hipSuccess; }
}  // namespace mscan

static void expect(int got, int want, const char* what) {
  if (got != want) {
    std::printf("%s: status %d, expected %d (%s)\n", what, got, want, mamba_last_error());
    std::exit(1);
  }
}

template <class T = void>
static T* at(uint64_t k) {
  return reinterpret_cast<T*>(uintptr_t(0x10000000000) + (k << 44));
}

static int fwd(const mamba_gated_desc& d, const mamba_gated_strides* s = nullptr, void* out = at(7)) {
  return mamba_gated_scan_fwd(&d, s, at(1), at(2), at(3), at<float>(4), at<float>(5), at<uint8_t>(6), out,
                              at<float>(8), at<float>(9), at(10), 512, nullptr);
}

static int bwd(const mamba_gated_desc& d, const mamba_gated_strides* s, void* dr, void* dg) {
  return mamba_gated_scan_bwd(&d, s, at(1), at(2), at(3), at<float>(4), at<uint8_t>(6), at<float>(5), at(7),
                              at<float>(8), at(9), dr, dg, at<float>(12), at<float>(13), at(14), 512, nullptr);
}

int main() {
  // sizes up to the limits: every product of sizes and strides stays in 64 bits
  const int64_t big = (int64_t(1) << 31) - 1;
  for (mamba_gated_desc d : {mamba_gated_desc{1, 1, 1, MAMBA_F32, 0}, mamba_gated_desc{(1 << 23) - 1, 1, 1, MAMBA_BF16, 0},
                             mamba_gated_desc{1, 100000000, 500, MAMBA_F32, 0}, mamba_gated_desc{1, 1, 1 << 26, MAMBA_F32, 0},
                             mamba_gated_desc{0, 5, 3, MAMBA_F32, 0}, mamba_gated_desc{2, 0, 3, MAMBA_F32, 0}})
    expect(fwd(d), MAMBA_OK, "gated forward");
  const int64_t extremes[] = {INT64_MIN, -1, INT64_MAX, int64_t(1) << 40, int64_t(1) << 32};
  for (int64_t v : extremes) {
    for (mamba_gated_desc d : {mamba_gated_desc{v, 2, 2, 0, 0}, mamba_gated_desc{2, v, 2, 0, 0}, mamba_gated_desc{2, 2, v, 0, 0}})
      expect(fwd(d), v < 0 ? MAMBA_ERR_INVALID_ARG : MAMBA_ERR_UNSUPPORTED, "gated size");
    const mamba_gated_desc d{2, 2, 2, 0, 0};
    const mamba_gated_strides s{0, v, 0, 0, 0, 0, 0};
    expect(fwd(d, &s), v < 0 ? MAMBA_ERR_INVALID_ARG : MAMBA_ERR_UNSUPPORTED, "gated stride");
  }
  const mamba_gated_desc d{2, 8, 16, MAMBA_BF16, 0};
  char* half = static_cast<char*>(at(10));
  const mamba_gated_strides wide{0, 0, 0, 0, 0, 32, 32};
  expect(bwd(d, &wide, half, half + 32), MAMBA_OK, "halves of one buffer");
  expect(bwd(d, &wide, half + 32, half), MAMBA_OK, "halves of one buffer, the other way round");
  expect(bwd(d, &wide, half, half + 31 * 2), MAMBA_ERR_INVALID_ARG, "halves that share a column");
  expect(bwd(d, &wide, half, half), MAMBA_ERR_INVALID_ARG, "the same half");
  expect(fwd(d, nullptr, nullptr), MAMBA_ERR_INVALID_ARG, "no output");
  const mamba_gated_desc one{3, 1, 16, MAMBA_BF16, 0};
  expect(mamba_gated_update(&one, nullptr, at<float>(1), at(2), at(3), at(4), at<float>(5), at(6), nullptr), MAMBA_OK,
         "token");

  mamba_norm_desc n{5, 40, 128, MAMBA_BF16, MAMBA_F32, 1e-6f, 0};
  expect(mamba_rmsnorm_quant_fwd(&n, nullptr, at(1), at(2), at<float>(3), at(4), at<float>(5), at(6), nullptr), MAMBA_OK,
         "8-bit norm");
  expect(mamba_rmsnorm_quant_fwd(&n, nullptr, at(1), at(2), at<float>(3), at(4), at<float>(5), at(2), nullptr), MAMBA_OK,
         "8-bit norm in place");
  n.group = 0;
  n.rows = big;
  n.dim = 512;
  expect(mamba_rmsnorm_fwd(&n, nullptr, at(1), at(2), at<float>(3), at(4), at(5), nullptr), MAMBA_OK, "most rows");
  expect(mamba_rmsnorm_bwd(&n, nullptr, at(1), at<float>(2), at(3), at(4), at(5), at(6), at<float>(7), at(8), 256, nullptr),
         MAMBA_ERR_HIP, "a failed launch");
  for (int64_t v : extremes) {
    mamba_norm_desc m = n;
    m.rows = v;
    expect(mamba_rmsnorm_fwd(&m, nullptr, at(1), at(2), at<float>(3), at(4), at(5), nullptr),
           v < 0 ? MAMBA_ERR_INVALID_ARG : MAMBA_ERR_UNSUPPORTED, "norm rows");
    m = n;
    m.dim = v;
    expect(mamba_rmsnorm_fwd(&m, nullptr, at(1), at(2), at<float>(3), at(4), at(5), nullptr),
           v < 0 ? MAMBA_ERR_INVALID_ARG : MAMBA_ERR_UNSUPPORTED, "norm dim");
  }

  mamba_conv_desc c{2, 9, 16, 4, MAMBA_BF16, 0};
  for (int64_t w = 1; w <= 4; ++w) {
    c.width = w;
    expect(mamba_conv1d_bwd(&c, at(1), at<float>(2), at<float>(3), at(4), at(5), at<float>(6), at(7), at<float>(8),
                            at<float>(9), at<float>(10), at(11), 256, nullptr),
           MAMBA_OK, "convolution backward");
  }
  expect(mamba_conv1d_bwd(&c, at(1), at<float>(2), at<float>(3), at(4), at(5), at<float>(6), at(7), at<float>(8),
                          at<float>(9), at<float>(10), at(11), 255, nullptr),
         MAMBA_ERR_INVALID_ARG, "a small workspace");
  std::printf("every case ran clean (%d launches)\n", g_launched);
  return 0;
}

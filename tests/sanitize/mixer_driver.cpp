// Drives the mixer operators' C ABI layer (api_mixer.cpp) on the host, with its
// launches replaced by counters: valid calls at small and extreme sizes, and
// refusals. Built with AddressSanitizer and UndefinedBehaviorSanitizer.
#include <cstdio>
#include <cstdlib>

#include "mixer.h"
#include "mixer/mamba_linattn.h"
#include "mixer/mamba_qknorm.h"

static int g_launched = 0;

namespace mscan {
size_t linattn_fwd_workspace_bytes(const LinattnSizes& n) { return n.rows * n.heads > 0 ? 512 : 0; }
size_t linattn_bwd_workspace_bytes(const LinattnSizes& n, bool) { return n.rows * n.heads > 0 ? 512 : 0; }
size_t qknorm_bwd_workspace_bytes(int64_t t, int64_t q, int64_t k, int64_t) { return t * (q + k) > 0 ? 256 : 0; }
hipError_t launch_linattn_fwd(const LinattnProblem&, void*, hipStream_t) { return ++g_launched, hipSuccess; }
hipError_t launch_linattn_bwd(const LinattnBwdProblem&, void*, hipStream_t) { return ++g_launched, hipSuccess; }
hipError_t launch_linattn_update(const LinattnUpdateProblem&, hipStream_t) { return ++g_launched, hipSuccess; }
hipError_t launch_qknorm_fwd(const QkNormProblem&, hipStream_t) { return ++g_launched, hipSuccess; }
hipError_t launch_qknorm_bwd(const QkNormProblem&, void*, hipStream_t) { return ++g_launched, hipErrorInvalidValue; }
}  // namespace mscan

static void expect(int got, int want, const char* what) {
  if (got != want) {
    std::printf("%s: status %d, expected %d (%s)\n", what, got, want, mamba_last_error());
    std::exit(1);
  }
}

template <class T = void>
static T* at(uint64_t k) {
  return reinterpret_cast<T*>(uintptr_t(0x10000000000) + (k << 50));
}

static int fwd(const mamba_linattn_desc& d, const mamba_linattn_strides* s = nullptr, size_t bytes = 512) {
  return mamba_linattn_fwd(&d, s, at(1), at(2), at(3), at<float>(4), at<float>(5),
                           d.flags & MAMBA_LINATTN_PACKED ? at<int64_t>(6) : nullptr, at(7), at<float>(8), at(9), bytes,
                           nullptr);
}

static int bwd(const mamba_linattn_desc& d, const mamba_linattn_strides* s, void* dq, void* dk, void* dv) {
  return mamba_linattn_bwd(&d, s, at(1), at(2), at(3), at<float>(4), at<float>(5),
                           d.flags & MAMBA_LINATTN_PACKED ? at<int64_t>(6) : nullptr, at(7), at<float>(8), dq, dk, dv,
                           at<float>(12), at<float>(13), at(14), 512, nullptr);
}

static int turn(const mamba_qknorm_desc& d, void* qo = at(7), void* ko = at(8)) {
  return mamba_qknorm_fwd(&d, nullptr, at(1), at(2), at<int64_t>(3), at<float>(4), at<float>(5), at<float>(6), qo, ko,
                          nullptr);
}

int main() {
  const int64_t most = (int64_t(1) << 31) - 1;
  // sizes up to the limits: every product of sizes and strides stays in 64 bits
  for (mamba_linattn_desc d :
       {mamba_linattn_desc{1, 1, 1, 1, 8, 8, MAMBA_F32, 0, 1.0f}, mamba_linattn_desc{1, most, 1, 1, 256, 256, MAMBA_BF16, 0, 1.0f},
        mamba_linattn_desc{1, 1, 1 << 15, 1, 8, 256, MAMBA_F32, MAMBA_LINATTN_HEAD_DECAY, 0.0f},
        mamba_linattn_desc{1 << 21, 1000, 1, 1, 8, 8, MAMBA_F32, 0, -1.0f},
        mamba_linattn_desc{1 << 21, most, 1, 1, 8, 8, MAMBA_F32, MAMBA_LINATTN_PACKED, 1.0f},
        mamba_linattn_desc{0, 9, 4, 2, 64, 64, MAMBA_F32, MAMBA_LINATTN_PACKED | MAMBA_LINATTN_ZERO_REST, 1.0f},
        mamba_linattn_desc{0, 5, 4, 2, 64, 64, MAMBA_F32, 0, 1.0f}, mamba_linattn_desc{2, 0, 4, 2, 64, 64, MAMBA_F32, 0, 1.0f}})
    expect(fwd(d), MAMBA_OK, "forward"), expect(bwd(d, nullptr, at(9), at(10), at(11)), MAMBA_OK, "backward");
  for (int64_t v : {INT64_MIN, int64_t(-1), INT64_MAX, int64_t(1) << 40, int64_t(1) << 32}) {
    const int want = v < 0 ? MAMBA_ERR_INVALID_ARG : MAMBA_ERR_UNSUPPORTED;
    const mamba_linattn_desc d{2, 2, 2, 2, 8, 8, 0, 0, 1.0f};
    mamba_linattn_desc e = d;
    e.batch = v;
    expect(fwd(e), want, "batch");
    e = d;
    e.seqlen = v;
    expect(fwd(e), want, "seqlen");
    e.flags = MAMBA_LINATTN_PACKED;
    expect(fwd(e), want, "packed rows");
    e = d;
    e.nheads = v < 0 ? v : v / 2 * 2;
    expect(fwd(e), want, "nheads");
    e = d;
    e.dkey = v;
    expect(fwd(e), want, "dkey");
    e = d;
    e.dvalue = v;
    expect(fwd(e), want, "dvalue");
    e = d;
    e.ngroups = v;
    expect(fwd(e), MAMBA_ERR_INVALID_ARG, "ngroups");
    const mamba_linattn_strides s{0, v, 0, 0, 0, 0, 0};
    expect(fwd(d, &s), want, "stride");
    mamba_qknorm_desc t{4, 2, 2, 64, 64, {32, 0, 0, 0}, 1, 0, 1e-6f, 0};
    t.tokens = v;
    expect(turn(t), want, "tokens");
    t.tokens = 4;
    t.qheads = v;
    expect(turn(t), want, "query heads");
    t.qheads = 2;
    t.kheads = v;
    expect(turn(t), want, "key heads");
    t.kheads = 2;
    t.headdim = v;
    expect(turn(t), want, "head size");
    t.headdim = 64;
    t.rotary = v;
    expect(turn(t), MAMBA_ERR_INVALID_ARG, "rotary");
    t.rotary = 64;
    t.sections[0] = v;
    expect(turn(t), MAMBA_ERR_INVALID_ARG, "section");
    t.sections[0] = 32;
    t.naxes = static_cast<int32_t>(v | 8);
    expect(turn(t), MAMBA_ERR_INVALID_ARG, "axes");
  }
  const mamba_linattn_desc d{2, 8, 2, 2, 8, 8, MAMBA_BF16, 0, 1.0f};
  char* buf = static_cast<char*>(at(9));
  const mamba_linattn_strides wide{0, 0, 0, 0, 48, 48, 48};
  expect(bwd(d, &wide, buf, buf + 32, buf + 64), MAMBA_OK, "thirds of one buffer");
  expect(bwd(d, &wide, buf + 64, buf, buf + 32), MAMBA_OK, "thirds of one buffer, in another order");
  expect(bwd(d, &wide, buf, buf + 30, buf + 64), MAMBA_ERR_INVALID_ARG, "thirds that share a column");
  expect(bwd(d, &wide, buf, buf, buf + 64), MAMBA_ERR_INVALID_ARG, "the same third");
  expect(fwd(d, nullptr, 511), MAMBA_ERR_INVALID_ARG, "a small workspace");
  const mamba_linattn_desc one{3, 1, 4, 2, 8, 16, MAMBA_BF16, 0, 1.0f};
  expect(mamba_linattn_update(&one, nullptr, at<float>(1), at(2), at(3), at(4), at<float>(5), at(6), nullptr), MAMBA_OK,
         "token");
  const mamba_qknorm_desc t{5, 3, 1, 128, 96, {16, 16, 16, 0}, 3, MAMBA_BF16, 0.0f, MAMBA_QKNORM_INTERLEAVED};
  expect(turn(t), MAMBA_OK, "rotation");
  expect(turn(t, at(1), at(2)), MAMBA_OK, "rotation in place");
  expect(turn(t, at(2), at(1)), MAMBA_ERR_INVALID_ARG, "each in the other's place");
  const mamba_qknorm_desc large{most / 4, 3, 1, 256, 0, {0, 0, 0, 0}, 1, MAMBA_F32, 0.0f, 0};
  expect(turn(large), MAMBA_OK, "most tokens");
  expect(mamba_qknorm_bwd(&t, nullptr, at(1), at(2), at<int64_t>(3), at<float>(4), at<float>(5), at<float>(6), at(7), at(8),
                          at(9), at(10), at<float>(11), at<float>(12), at(13), 256, nullptr),
         MAMBA_ERR_HIP, "a failed launch");
  expect(mamba_qknorm_bwd(&t, nullptr, at(1), at(2), at<int64_t>(3), at<float>(4), at<float>(5), at<float>(6), at(7), at(8),
                          at(9), at(10), at<float>(11), at<float>(12), at(13), 255, nullptr),
         MAMBA_ERR_INVALID_ARG, "a small workspace");
  std::printf("every case ran clean (%d launches)\n", g_launched);
  return 0;
}

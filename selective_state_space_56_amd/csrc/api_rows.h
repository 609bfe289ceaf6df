// Checks shared by the C ABI of operators whose tensors are rows that may be
// slices of wider ones: overlaps, alignment, strides, workspaces.
#pragma once

#include <hip/hip_runtime_api.h>

#include <initializer_list>

#include "api_util.h"

namespace mscan {

constexpr int64_t kMaxStride = int64_t(1) << 26;
constexpr int64_t kMaxElems = int64_t(1) << 40;

// A tensor of `rows` rows of `len` elements of `eb` bytes, `stride` elements apart.
struct Rows {
  const char* name;
  const void* p;
  int64_t rows, stride, len;
  size_t eb;
  Span span() const { return Span{name, p, len > 0 ? span_bytes(rows, stride, len, eb) : 0}; }
};

// Whether two row tensors share a byte. Tensors whose spans meet may still
// interleave (halves of one buffer's rows): with the same row distance the
// second one's rows must start where the first one's have ended.
inline bool collide(const Rows& a, const Rows& b) {
  if (!overlaps(a.span(), b.span())) return false;
  const int64_t step = a.stride * static_cast<int64_t>(a.eb);
  if (step != b.stride * static_cast<int64_t>(b.eb)) return true;
  const int64_t off = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.p)) -
                      static_cast<int64_t>(reinterpret_cast<uintptr_t>(a.p));
  const int64_t at = ((off % step) + step) % step;
  return at < a.len * static_cast<int64_t>(a.eb) || at > step - b.len * static_cast<int64_t>(b.eb);
}

inline Rows flat(const char* name, const void* p, int64_t elems, size_t eb) {
  return Rows{name, p, elems > 0 ? 1 : 0, elems, elems, eb};
}

inline mamba_status check_outputs(const char* who, std::initializer_list<Rows> in,
                           std::initializer_list<Rows> out) {
  for (auto o = out.begin(); o != out.end(); ++o) {
    for (const Rows& i : in)
      if (collide(*o, i)) return fail(MAMBA_ERR_INVALID_ARG, "%s: %s overlaps %s", who, o->name, i.name);
    for (auto q = o + 1; q != out.end(); ++q)
      if (collide(*o, *q)) return fail(MAMBA_ERR_INVALID_ARG, "%s: %s overlaps %s", who, o->name, q->name);
  }
  return MAMBA_OK;
}

inline mamba_status check_row_align(const char* who, std::initializer_list<Rows> tensors) {
  for (const Rows& t : tensors)
    if (t.p && reinterpret_cast<uintptr_t>(t.p) % t.eb)
      return fail(MAMBA_ERR_INVALID_ARG, "%s: %s is not %zu-byte aligned", who, t.name, t.eb);
  return MAMBA_OK;
}

inline mamba_status check_present(const char* who, std::initializer_list<Span> required) {
  for (const Span& r : required)
    if (!r.p) return fail(MAMBA_ERR_INVALID_ARG, "%s: %s is NULL", who, r.name);
  return MAMBA_OK;
}

// 0 means contiguous; any other stride must hold a row and stay addressable.
inline mamba_status resolve(const char* who, const char* name, int64_t given, int64_t dim, int64_t* to) {
  *to = dim;
  if (given == 0) return MAMBA_OK;
  if (given < dim)
    return fail(MAMBA_ERR_INVALID_ARG, "%s: %s stride %lld is below its row length %lld", who, name,
                (long long)given, (long long)dim);
  if (given > kMaxStride)
    return fail(MAMBA_ERR_UNSUPPORTED, "%s: %s stride %lld too large", who, name, (long long)given);
  *to = given;
  return MAMBA_OK;
}

inline mamba_status check_workspace(const char* who, const void* ws, size_t given, size_t need) {
  if (need == 0) return MAMBA_OK;
  if (!ws) return fail(MAMBA_ERR_INVALID_ARG, "%s: workspace is NULL but %zu bytes are needed", who, need);
  if (given < need)
    return fail(MAMBA_ERR_INVALID_ARG, "%s: workspace has %zu bytes, %zu needed", who, given, need);
  if (reinterpret_cast<uintptr_t>(ws) % 256)
    return fail(MAMBA_ERR_INVALID_ARG, "%s: workspace is not 256-byte aligned", who);
  return MAMBA_OK;
}

inline mamba_status check_io(const char* who, const char* name, int32_t io) {
  if (io != MAMBA_F32 && io != MAMBA_BF16)
    return fail(MAMBA_ERR_INVALID_ARG, "%s: %s %d is not MAMBA_F32 or MAMBA_BF16", who, name, (int)io);
  return MAMBA_OK;
}

inline mamba_status launched(const char* who, hipError_t e) {
  if (e != hipSuccess)
    return fail(MAMBA_ERR_HIP, "%s: launch failed: %s", who, hipGetErrorString(e));
  return ok();
}

}  // namespace mscan

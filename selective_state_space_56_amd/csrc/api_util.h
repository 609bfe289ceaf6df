// Helpers shared by the C ABI's source files: the thread's error message,
// overlap and alignment checks.
#pragma once

#include <cstdarg>
#include <cstdio>
#include <initializer_list>
#include <string>

#include <stddef.h>
#include <stdint.h>

#include "mamba_conv.h"
#include "mamba_scan.h"

namespace mscan {

// Detail of the last non-OK status returned on this thread (api.cpp).
std::string& last_error();

inline mamba_status fail(mamba_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  try {
    last_error() = buf;
  } catch (...) {  // out of memory: the status still tells, and nothing crosses the C boundary
  }
  return s;
}

inline mamba_status ok() {
  last_error().clear();
  return MAMBA_OK;
}

inline size_t io_bytes(int32_t io) { return io == MAMBA_BF16 ? 2 : 4; }

struct Span {
  const char* name;
  const void* p;
  size_t bytes;
};

inline bool overlaps(const Span& a, const Span& b) {
  if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
  const auto a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

inline mamba_status check_align(const char* who, std::initializer_list<Span> spans, size_t align) {
  for (const Span& s : spans)
    if (s.p && reinterpret_cast<uintptr_t>(s.p) % align)
      return fail(MAMBA_ERR_INVALID_ARG, "%s: %s is not %zu-byte aligned", who, s.name, align);
  return MAMBA_OK;
}

// Bytes spanned by `rows` rows of `len` elements `stride` elements apart.
inline size_t span_bytes(int64_t rows, int64_t stride, int64_t len, size_t eb) {
  return rows > 0 ? static_cast<size_t>((rows - 1) * stride + len) * eb : 0;
}

// Descriptor fields common to both convolution entry points.
inline mamba_status check_conv_desc(const mamba_conv_desc* d, const char* who) {
  if (!d) return fail(MAMBA_ERR_INVALID_ARG, "%s: desc is NULL", who);
  if (d->batch < 0 || d->seqlen < 0 || d->dim < 0)
    return fail(MAMBA_ERR_INVALID_ARG, "%s: negative size (batch=%lld seqlen=%lld dim=%lld)", who,
                (long long)d->batch, (long long)d->seqlen, (long long)d->dim);
  if (d->io_dtype != MAMBA_F32 && d->io_dtype != MAMBA_BF16)
    return fail(MAMBA_ERR_INVALID_ARG, "%s: io_dtype %d is not MAMBA_F32 or MAMBA_BF16", who,
                (int)d->io_dtype);
  if (d->width < 1) return fail(MAMBA_ERR_INVALID_ARG, "%s: width %lld < 1", who, (long long)d->width);
  if (d->width > 4)
    return fail(MAMBA_ERR_UNSUPPORTED, "%s: width %lld not supported (1 to 4)", who,
                (long long)d->width);
  if (d->flags != 0) return fail(MAMBA_ERR_INVALID_ARG, "%s: flags must be 0", who);
  const int64_t lim = int64_t(1) << 40;
  if (d->batch > 65535 || d->seqlen > lim || d->dim > (int64_t(1) << 31) ||
      (d->batch && d->dim > (int64_t(1) << 31) / d->batch) ||
      (d->batch * d->dim != 0 && d->seqlen > lim / (d->batch * d->dim)) ||
      (d->seqlen + 63) / 64 > 65535)
    return fail(MAMBA_ERR_UNSUPPORTED, "%s: problem too large", who);
  return MAMBA_OK;
}

}  // namespace mscan

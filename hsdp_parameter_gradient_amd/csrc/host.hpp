// What the host sides of the library's entry points share: the calling
// thread's error message and timing request, checked size arithmetic,
// pointer and overlap checks, and the guard that keeps C++ exceptions inside
// the C ABI.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include <algorithm>
#include <cstdarg>
#include <cstdio>
#include <exception>
#include <new>
#include <stdexcept>
#include <string>
#include <vector>

#include "fsdp_flat.h"

namespace fsdp {
namespace host {

inline thread_local std::string g_err;

inline int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  try {
    g_err = buf;
  } catch (...) {  // no memory for the message: the code still stands
    g_err.clear();
  }
  return code;
}

inline int ok() {
  g_err.clear();
  return FSDP_OK;
}

constexpr int64_t kMaxBytes = int64_t(1) << 60;

inline bool mul_ok(int64_t a, int64_t b, int64_t* out) {
  return !__builtin_mul_overflow(a, b, out) && *out <= kMaxBytes;
}
inline bool add_ok(int64_t a, int64_t b, int64_t* out) {
  return !__builtin_add_overflow(a, b, out) && *out <= kMaxBytes;
}

inline int elem_size(int32_t dtype) {
  switch (dtype) {
    case FSDP_F32: return 4;
    case FSDP_BF16: return 2;
    case FSDP_F16: return 2;
    default: return 0;
  }
}

// ---------------------------------------------------------------------------
// pointer checks
// ---------------------------------------------------------------------------

struct Span {
  uint64_t a, b;  // [a, b)
  int id;
};

inline int check_ptr(const void* p, int64_t nbytes, uint64_t align, const char* what, long idx) {
  if (nbytes == 0) return FSDP_OK;
  if (!p) return fail(FSDP_EINVAL, "%s[%ld] is NULL but holds %lld bytes", what, idx, (long long)nbytes);
  if ((uint64_t)p % align)
    return fail(FSDP_EALIGN, "%s[%ld] = %p is not %llu-byte aligned", what, idx, p, (unsigned long long)align);
  return FSDP_OK;
}

// Outputs must be pairwise disjoint and disjoint from every input.
inline int check_overlap(std::vector<Span> outs, const std::vector<Span>& ins) {
  outs.erase(std::remove_if(outs.begin(), outs.end(), [](const Span& s) { return s.a == s.b; }), outs.end());
  std::sort(outs.begin(), outs.end(), [](const Span& x, const Span& y) { return x.a < y.a; });
  for (size_t k = 1; k < outs.size(); ++k)
    if (outs[k].a < outs[k - 1].b)
      return fail(FSDP_EOVERLAP, "output buffers %d and %d overlap", outs[k - 1].id, outs[k].id);
  for (const Span& in : ins) {
    if (in.a == in.b) continue;
    // first output whose end is beyond in.a
    auto it = std::upper_bound(outs.begin(), outs.end(), in.a,
                               [](uint64_t v, const Span& s) { return v < s.b; });
    if (it != outs.end() && it->a < in.b)
      return fail(FSDP_EOVERLAP, "input buffer %d overlaps output buffer %d", in.id, it->id);
  }
  return FSDP_OK;
}

// Is `stream` being captured into a HIP graph?
inline bool capturing(hipStream_t stream) {
  hipStreamCaptureStatus st = hipStreamCaptureStatusNone;
  return hipStreamIsCapturing(stream, &st) == hipSuccess && st == hipStreamCaptureStatusActive;
}

// Events the calling thread's next kernel launch records at its start and
// end (fsdp_time_next_launch); taken by that launch.
inline thread_local void* g_time_start = nullptr;
inline thread_local void* g_time_stop = nullptr;

// No C++ exception may cross the C ABI: host allocation failures while
// planning become FSDP_ENOMEM, anything else FSDP_EINVAL.  Nothing has been
// enqueued when an exception is thrown (launches come last).
template <class F>
int guarded(F&& f) noexcept {
  try {
    return f();
  } catch (const std::bad_alloc&) {
    return fail(FSDP_ENOMEM, "out of host memory while planning the call");
  } catch (const std::length_error&) {
    return fail(FSDP_ENOMEM, "the call's host tables would exceed the largest allocation");
  } catch (const std::exception& e) {
    return fail(FSDP_EINVAL, "internal error: %s", e.what());
  } catch (...) {
    return fail(FSDP_EINVAL, "internal error");
  }
}

}  // namespace host
}  // namespace fsdp

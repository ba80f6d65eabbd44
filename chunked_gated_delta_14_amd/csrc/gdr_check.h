// Argument checks that the ABI's translation units around the recurrence share.
#pragma once

#include <stdint.h>

#include <cstdio>
#include <initializer_list>

#include "gdr.h"
#include "gdr_host.h"

namespace gdr {

constexpr int64_t kAlign = 256;
inline int64_t round_up(int64_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

inline int32_t invalid(const char *msg) { return host_status(GDR_ERR_INVALID_ARG, msg); }
inline int32_t unsupported(const char *msg) { return host_status(GDR_ERR_UNSUPPORTED, msg); }

inline bool is_dtype(int32_t d) { return d == GDR_BF16 || d == GDR_F32; }
inline bool element_aligned(const void *p, int32_t dtype) {
  return reinterpret_cast<uintptr_t>(p) % (dtype == GDR_BF16 ? 2 : 4) == 0;
}
// Stride of [T] rows `width` wide; rows of fewer than two tokens have none to check.
inline bool stride_ok(int64_t stride, int64_t width, int64_t T) { return T < 2 || stride >= width; }

// Whether one of a call's outputs is one of its inputs.  (Parts of one wider buffer,
// which rows may be, start at different addresses; other overlaps are the caller's.)
using Pointers = std::initializer_list<const void *>;
inline bool aliases(Pointers outs, Pointers ins) {
  for (const void *out : outs)
    for (const void *in : ins)
      if (out && out == in) return true;
  return false;
}

inline int32_t check_workspace(void *ws, int64_t have, int64_t need) {
  if (need > 0 && !ws) return host_status(GDR_ERR_WORKSPACE, "workspace is NULL");
  if (reinterpret_cast<uintptr_t>(ws) % kAlign) return host_status(GDR_ERR_WORKSPACE, "workspace is not 256-byte aligned");
  if (have < need) {
    char msg[96];
    std::snprintf(msg, sizeof msg, "workspace too small: need %lld bytes, got %lld", (long long)need, (long long)have);
    return host_status(GDR_ERR_WORKSPACE, msg);
  }
  return GDR_OK;
}

// Device check, then the launches of one call; a failing one ends the call.
template <class F>
inline int32_t launch(int kernel, void *stream, const char *what, F f) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  return host_hip(timed_launch(kernel, st, [&] { return f(st); }), what);
}

}  // namespace gdr

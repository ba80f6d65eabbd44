// Host-side services of the C-ABI layer shared by its translation units:
// the thread-local error message, the device check and the per-kernel timing.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdr {

// Timed kernels, in the order gdr_timing_read reports them.
enum TimedKernel {
  TK_FWD_PREP, TK_FWD_WALK, TK_BWD_WALK, TK_BWD_GRAD,
  TK_CONV_FWD, TK_CONV_BWD, TK_CONV_STEP, TK_GATE_FWD, TK_GATE_BWD, TK_STEP, TK_NORM_FWD, TK_NORM_BWD, TK_PARAM_SUM,
  TK_COUNT
};

// Record `msg` for gdr_last_error and return `code`; GDR_OK clears the message.
int32_t host_status(int32_t code, const char *msg);
int32_t host_check_device();
int32_t host_hip(hipError_t e, const char *what);

// Calls launch(ctx), which enqueues one kernel on st, bracketed by events when timing is on.
hipError_t host_timed(int kernel, hipStream_t st, hipError_t (*launch)(void *), void *ctx);
template <class F>
inline hipError_t timed_launch(int kernel, hipStream_t st, F &&f) {
  return host_timed(kernel, st, [](void *c) { return (*static_cast<F *>(c))(); }, &f);
}

}  // namespace gdr

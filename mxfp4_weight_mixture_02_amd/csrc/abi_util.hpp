// What the C entry points share: the thread's error message, argument
// checks and launches with optional event timing (defined in abi.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mxfp4_moe.h"

namespace mxmoe {

// Sets the thread's message and returns the code; ok() clears it.
int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int ok();

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline int hip_status(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(MXFP4_EHIP, "%s: %s", what, hipGetErrorString(e));
  return MXFP4_OK;
}

// Whether a launch can have so many workgroups of `threads` threads: 2^32 - 1
// threads in all.
inline bool launchable(int64_t blocks, int threads) { return blocks <= ((int64_t(1) << 32) - 1) / threads; }

// With mxfp4_moe_kernel_timing on, an event recorded on s before the launch
// (else nullptr), and the one after it.
hipEvent_t timing_begin(hipStream_t s);
void timing_end(hipEvent_t e0, const char* name, hipStream_t s);

// Enqueue one kernel; with timing on, bracket it with events on stream s.
template <class F>
int launch_timed(F&& enqueue, const char* name, hipStream_t s) {
  const hipEvent_t e0 = timing_begin(s);
  const int rc = hip_status(enqueue(), name);
  timing_end(e0, name, s);
  return rc;
}

#define LAUNCH(call, name)                                            \
  do {                                                                \
    int rc_ = mxmoe::launch_timed([&]() { return (call); }, name, s); \
    if (rc_ != MXFP4_OK) return rc_;                                  \
  } while (0)

}  // namespace mxmoe

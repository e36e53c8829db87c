// Launchers of the SwiGLU with 8-bit checkpoints (swiglu8.hip).  n8: groups
// of 8 elements of h (R * 2I / 8), a multiple of 4; a and h may be nullptr
// where they are outputs.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxmoe {

hipError_t launch_swiglu8_fwd(const uint16_t* h, int64_t n8, float alpha, float limit, uint16_t* a,
                              uint8_t* codes, uint8_t* scales, hipStream_t s);
hipError_t launch_swiglu8_bwd(const uint8_t* codes, const uint8_t* scales, const uint16_t* da,
                              int64_t n8, float alpha, float limit, uint16_t* dh, uint16_t* a,
                              hipStream_t s);
hipError_t launch_swiglu8_restore(const uint8_t* codes, const uint8_t* scales, int64_t n8,
                                  float alpha, float limit, uint16_t* h, uint16_t* a, hipStream_t s);

}  // namespace mxmoe

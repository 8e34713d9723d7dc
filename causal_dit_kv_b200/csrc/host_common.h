// What the host translation units share: error reporting, the driver's tensor-map
// encoder and the launch counter.
#pragma once

#include <cudaTypedefs.h>

#include "sdv2.h"
#include "sdv2_internal.h"

namespace sdv2 {

sdv2_status fail(sdv2_status st, const char *fmt, ...);
sdv2_status cuda_fail(cudaError_t e, const char *what);
PFN_cuTensorMapEncodeTiled_v12000 get_encode_fn();
sdv2_status check_device(int device);
void count_launch();
inline uint64_t align_up(uint64_t x, uint64_t a) { return (x + a - 1) / a * a; }
inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace sdv2

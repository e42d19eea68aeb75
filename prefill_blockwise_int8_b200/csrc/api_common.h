// Host helpers shared by the C entry points (tilemix_api.cu defines them):
// the per-thread error text, the device check and the tensor-map encoder.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <stddef.h>

#include "tilemix.h"

namespace tilemix {

// Records the text tilemix_last_error() returns on this thread.
tilemix_status fail(tilemix_status st, const char* fmt, ...);
tilemix_status ok();

bool aligned(const void* p, size_t a);

// TILEMIX_OK when the current device is an sm_100.
tilemix_status check_device();

PFN_cuTensorMapEncodeTiled_v12000 encode_fn();

}  // namespace tilemix

// api_internal.h -- what the C ABI's translation units share (defined in api.cu).
#pragma once

#include <cstdint>
#include <cuda.h>

#include "mmact.h"

namespace mmact {

// The current device: its SMs, its kernel status word and the bound on waits.
struct DeviceContext {
    int sm_count;
    unsigned int *status;
    unsigned long long wait_ns;
};
mmact_status device_context(DeviceContext *out);

// Tiled map over a row-major tensor (innermost dimension first, byte strides of
// the others), kept in the per-thread map cache.  Needs a device_context call
// before the first use.
bool encode_tensor_map(CUtensorMap *m, mmact_dtype dt, int rank, const void *ptr, const uint64_t *dims,
                       const uint64_t *strides_bytes, const uint32_t *box, bool swizzle);

}  // namespace mmact

// api_util.hpp -- what the two files of C entry points share: the export
// macro, the gfx950 check and small validation helpers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/mxq.h"

#define MXQ_API extern "C" __attribute__((visibility("default")))

namespace mxq {

// gfx950 check of the current device (cached per device); on success *cus is
// its compute-unit count.
mxq_status_t check_device(int* cus);

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline mxq_status_t launched(bool ok) {
    if (!ok) return MXQ_E_UNSUPPORTED;
    return hipGetLastError() == hipSuccess ? MXQ_OK : MXQ_E_LAUNCH;
}

inline hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

}  // namespace mxq

// kda_checks.hpp -- argument checks and status mapping shared by the C ABI
// layers (kda_api.hip, kda_hybrid_api.hip).  Host code only.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda.h"

namespace kda {

inline bool aligned_to(const void* p, unsigned n) { return ((uintptr_t)p & (n - 1u)) == 0; }
inline bool aligned16(const void* p) { return aligned_to(p, 16); }

// ptr must be non-null and 16-byte aligned when the array is non-empty
inline bool ok_ptr(const void* p, bool nonempty) { return !nonempty || (p != nullptr && aligned16(p)); }
// arrays read one element of n bytes at a time: natural alignment suffices
inline bool ok_elem(const void* p, bool nonempty, unsigned n) { return !nonempty || (p != nullptr && aligned_to(p, n)); }
inline bool ok_opt_ptr(const void* p) { return p == nullptr || aligned16(p); }

inline kda_status device_ready() {
    int dev = 0;
    return hipGetDevice(&dev) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

inline kda_status hip_status(hipError_t e) { return e == hipSuccess ? KDA_OK : KDA_ERR_HIP; }

}  // namespace kda

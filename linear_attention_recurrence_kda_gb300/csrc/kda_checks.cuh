// kda_checks.cuh -- the host-side argument checks that the C ABI's entry points share.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cstdlib>

#include <cuda_runtime.h>

#include "kda.h"

namespace kda {
namespace checks {

inline size_t io_size(kda_dtype_t dt) { return dt == KDA_BF16 ? 2 : 4; }

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct Range {
    uintptr_t lo, hi;  // [lo, hi)
};

inline Range range_of(const void* p, size_t bytes)
{
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return Range{lo, lo + bytes};
}

inline bool overlaps(Range a, Range b)
{
    if (a.lo == a.hi || b.lo == b.hi || a.lo == 0 || b.lo == 0) return false;
    return a.lo < b.hi && b.lo < a.hi;
}

// Device-accessible memory of the current device (or mapped pinned host memory).
inline kda_status_t check_device_pointer(const void* p)
{
    if (p == nullptr) return KDA_OK;
    cudaPointerAttributes attr;
    cudaError_t e = cudaPointerGetAttributes(&attr, p);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return e == cudaErrorInvalidValue ? KDA_ERR_INVALID_ARG : KDA_ERR_CUDA;
    }
    if (attr.devicePointer == nullptr) return KDA_ERR_INVALID_ARG;
    if (attr.type == cudaMemoryTypeDevice) {
        int dev = -1;
        if (cudaGetDevice(&dev) != cudaSuccess) return KDA_ERR_CUDA;
        if (attr.device != dev) return KDA_ERR_INVALID_ARG;
    }
    return KDA_OK;
}

// Tries of a kernel's hand-off waits before it gives up: `normal`, or fewer where KDA_DEBUG_HANDOFF_TRIES says so (a
// debugging aid, off unless set, read on every call: it exercises the timeout path).
inline uint32_t handoff_tries(uint32_t normal)
{
    if (const char* env = std::getenv("KDA_DEBUG_HANDOFF_TRIES")) {
        char* end = nullptr;
        const unsigned long v = std::strtoul(env, &end, 10);
        if (end != env && *end == '\0' && v < normal) return (uint32_t)v;
    }
    return normal;
}

}  // namespace checks
}  // namespace kda

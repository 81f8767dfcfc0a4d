// Host-side argument checks shared by the C ABI's translation units: byte ranges and their
// overlap, alignment, element sizes, and the status of a launch.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "bdssm.h"

namespace bdssm {

struct Range {
    uintptr_t lo, hi;  // [lo, hi)
};

inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi && a.lo != a.hi && b.lo != b.hi; }

inline Range rng(const void *p, int64_t bytes)
{
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return {lo, p ? lo + static_cast<uintptr_t>(bytes) : lo};
}

inline bool aligned(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

inline int elt(int dtype) { return dtype == BDSSM_BF16 ? 2 : 4; }

inline bdssm_status launched(hipError_t e) { return e == hipSuccess ? BDSSM_OK : BDSSM_ERR_HIP; }

}  // namespace bdssm

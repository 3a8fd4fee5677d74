// host.hpp -- host-side helpers shared by the entry points: pointer checks and
// the kernel launch.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "demo.h"

namespace demo {

inline uint64_t up256(uint64_t x) { return (x + 255u) & ~(uint64_t)255u; }

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

inline bool overlap(const void* a, uint64_t na, const void* b, uint64_t nb) {
    if (!a || !b || na == 0 || nb == 0) return false;
    const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    return a0 < b0 + nb && b0 < a0 + na;
}

template <class T>
struct same_type {
    using type = T;
};

// One kernel launch through hipLaunchKernel, whose return code belongs to this
// launch alone (hipGetLastError would also report an error that an earlier,
// unrelated HIP call left pending on the thread).  The parameter types come
// from the kernel; the arguments are converted to them.
template <class... P>
hipError_t launch(void (*kernel)(P...), dim3 grid, dim3 block, size_t lds, hipStream_t s,
                  typename same_type<P>::type... args) {
    void* argv[] = {static_cast<void*>(&args)...};
    return hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, block, argv, lds, s);
}

inline int status_of(hipError_t e) { return e == hipSuccess ? DEMO_OK : DEMO_EHIP; }

}  // namespace demo

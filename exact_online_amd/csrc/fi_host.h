// fi_host.h -- host helpers shared by the sources of the C ABI (fi_api.cpp,
// fi_operators.cpp).
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstring>

namespace fi {

int hip_fail(hipError_t e);   // records e for fi_strerror; FI_ERR_NOMEM or FI_ERR_HIP
int check_device();           // FI_OK on a gfx950 device

// A failed hipMalloc also leaves its error as the thread's "last error",
// which the next launch check (hipGetLastError) would then report as its own:
// take it back here, so a rejected fi_create leaves no trace for later calls.
template <typename T>
hipError_t dalloc(T **p, size_t bytes) {
    void *v = nullptr;
    hipError_t e = hipMalloc(&v, bytes < 256 ? 256 : bytes);
    if (e != hipSuccess) {
        (void)hipGetLastError();
        v = nullptr;
    }
    *p = static_cast<T *>(v);
    return e;
}

// The int a caller put in an enum-typed field or argument, read as its
// bytes: a value outside the enumeration is not one the enum type may hold,
// so it is never loaded as that type.
template <typename E>
int raw_int(const E &e) {
    static_assert(sizeof(E) == sizeof(int), "an int-sized enum");
    int v;
    std::memcpy(&v, &e, sizeof v);
    return v;
}

}  // namespace fi

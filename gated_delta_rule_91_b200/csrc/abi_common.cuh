// abi_common.cuh -- what the C entry points of both translation units share:
// the thread's last error text and the checks of pointers.
#pragma once
#include <stdarg.h>
#include <stdio.h>

#include <string>

#include "common.cuh"

namespace gdr {

inline thread_local std::string t_last_error;

__attribute__((format(printf, 2, 3))) inline gdr_status fail(gdr_status s, const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    t_last_error = buf;
    return s;
}

inline gdr_status cuda_fail(cudaError_t e, const char *where) {
    return fail(GDR_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

#define GDR_REQUIRE_PTR(p)                                                                   \
    do {                                                                                     \
        if ((p) == nullptr) return fail(GDR_ERR_INVALID_ARGUMENT, "%s: %s is NULL", fn, #p); \
        if (!aligned16(p))                                                                   \
            return fail(GDR_ERR_INVALID_ARGUMENT, "%s: %s is not 16-byte aligned", fn, #p);  \
    } while (0)
#define GDR_OPTIONAL_PTR(p)                                                                 \
    do {                                                                                    \
        if ((p) != nullptr && !aligned16(p))                                                \
            return fail(GDR_ERR_INVALID_ARGUMENT, "%s: %s is not 16-byte aligned", fn, #p); \
    } while (0)

// Reads the status word of the scan kernels' translation unit and clears it
// (each translation unit has its own g_status).
cudaError_t ssm_take_status(int *status);

}  // namespace gdr

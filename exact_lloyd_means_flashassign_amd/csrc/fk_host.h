// What the host-side entry points share: the calling thread's error message,
// the HIP error mapping and the argument checks.
#pragma once

#include <hip/hip_runtime.h>
#include <stdarg.h>
#include <stddef.h>
#include <stdint.h>
#include <stdio.h>

#include "fk.h"

namespace fk {

inline thread_local char g_err[512] = "";

inline fk_status fail(fk_status s, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof g_err, fmt, ap);
    va_end(ap);
    return s;
}

inline fk_status hip_fail(hipError_t e, const char *what) {
    (void)hipGetLastError();
    return fail(FK_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

#define FK_TRY(expr, what)                                  \
    do {                                                    \
        hipError_t e_ = (expr);                             \
        if (e_ != hipSuccess) return hip_fail(e_, (what));  \
    } while (0)

inline bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

inline bool overlap(const void *a, size_t an, const void *b, size_t bn) {
    const char *pa = (const char *)a, *pb = (const char *)b;
    return pa < pb + bn && pb < pa + an;
}

inline fk_status check_workspace(void *ws, size_t ws_bytes, size_t need) {
    if (ws == nullptr) return fail(FK_ERR_WORKSPACE, "workspace is NULL (%zu bytes needed)", need);
    if (!aligned(ws, 256)) return fail(FK_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    if (ws_bytes < need) return fail(FK_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", ws_bytes, need);
    return FK_OK;
}

inline fk_status check_device() {
    int n = 0;
    const hipError_t e = hipGetDeviceCount(&n);
    if (e != hipSuccess || n <= 0) {
        (void)hipGetLastError();
        return fail(FK_ERR_NO_DEVICE, "no HIP device is visible");
    }
    return FK_OK;
}

}  // namespace fk

// naju_host.h -- argument checks and error reporting shared by the files that
// hold C-ABI entry points (defined in naju_api.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/naju.h"

namespace naju {

// records the thread's error message and returns st
naju_status_t fail(naju_status_t st, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
naju_status_t hip_status(hipError_t e, const char *what);
// a required / optional pointer, aligned to `align` bytes
naju_status_t need(const void *p, const char *name, size_t align);
naju_status_t opt(const void *p, const char *name, size_t align);
// a caller's workspace of at least need_b bytes, 256-byte aligned
naju_status_t need_ws(const void *ws, size_t bytes, size_t need_b);

}  // namespace naju

#define NAJU_TRY(x)                                                                            \
    do {                                                                                       \
        naju_status_t _s = (x);                                                                \
        if (_s != NAJU_OK) return _s;                                                          \
    } while (0)

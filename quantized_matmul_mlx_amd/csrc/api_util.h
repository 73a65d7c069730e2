// What the C ABI's host checks share: the calling thread's error text, statuses of launches and
// pointer checks.
#pragma once

#include "qaff.h"

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>

namespace qaff {

// api.cpp: the calling thread's error text (qaff_last_error).
void set_error(const char* text) noexcept;

__attribute__((format(printf, 2, 3))) inline qaff_status fail(qaff_status st, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    set_error(buf);
    return st;
}

inline qaff_status after_launch(const char* op, hipError_t e, hipStream_t stream) {
    static const bool sync = [] {
        const char* v = std::getenv("QAFF_DEBUG_SYNC");
        return v && v[0] && std::strcmp(v, "0") != 0;
    }();
    if (e == hipErrorInvalidConfiguration)
        return fail(QAFF_ERR_UNSUPPORTED, "%s: more rows than one launch holds (2^32 threads)", op);
    if (e == hipSuccess && sync) e = hipStreamSynchronize(stream);
    if (e != hipSuccess) return fail(QAFF_ERR_DEVICE, "%s: %s", op, hipGetErrorString(e));
    return QAFF_OK;
}

inline bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// A pointer that a non-empty size needs: set and aligned.
inline qaff_status check_ptr(const char* op, const char* name, const void* p, uintptr_t a) {
    if (!p) return fail(QAFF_ERR_INVALID_ARGUMENT, "%s: null %s", op, name);
    if (!aligned(p, a)) return fail(QAFF_ERR_INVALID_ARGUMENT, "%s: %s must be %d-byte aligned", op, name, (int)a);
    return QAFF_OK;
}

}  // namespace qaff

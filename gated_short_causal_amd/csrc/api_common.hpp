// api_common.hpp -- error reporting and argument checks shared by the C entry
// points of api.cpp and api_hybrid.cpp.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cstdlib>

#include "lfm2sc.h"

namespace lfm2sc {

// Record the calling thread's error text / clear it; both return the status (api.cpp).
int fail(int code, const char* fmt, ...);
int ok();

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

inline bool check_mode() {
    static const bool on = [] {
        const char* e = std::getenv("LFM2SC_CHECK");
        return e != nullptr && e[0] == '1';
    }();
    return on;
}

constexpr int64_t kMaxRows = (int64_t)1 << 31;   // row offsets are int32

#define TRY(expr)                       \
    do {                                \
        const int rc_ = (expr);         \
        if (rc_ != LFM2SC_OK) return rc_; \
    } while (0)

inline int check_stride(const char* fn, const char* name, int64_t stride, int64_t min) {
    if (stride < min) return fail(LFM2SC_ERR_BAD_SHAPE, "%s: %s=%lld is below the minimum %lld", fn, name,
                                  (long long)stride, (long long)min);
    if (stride % 8 != 0) return fail(LFM2SC_ERR_ALIGNMENT, "%s: %s=%lld is not a multiple of 8 elements", fn, name,
                                     (long long)stride);
    return LFM2SC_OK;
}

inline int check_ptr(const char* fn, const char* name, const void* p, uintptr_t align) {
    if (p == nullptr) return fail(LFM2SC_ERR_NULL_POINTER, "%s: %s is NULL", fn, name);
    if (!aligned(p, align)) return fail(LFM2SC_ERR_ALIGNMENT, "%s: %s=%p is not %u-byte aligned", fn, name, p,
                                        (unsigned)align);
    return LFM2SC_OK;
}

inline int launched(const char* fn, hipError_t e) {
    if (e != hipSuccess) return fail(LFM2SC_ERR_HIP, "%s: HIP error %d (%s)", fn, (int)e, hipGetErrorString(e));
    return ok();
}

}  // namespace lfm2sc

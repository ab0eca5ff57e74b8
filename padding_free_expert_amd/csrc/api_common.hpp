// What the files of the C ABI share: error reporting (one message per calling
// thread), the architecture check and the argument-check macros.  Defined in
// api.cpp.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/xmoe.h"

namespace xmoe_api {

xmoe_status fail(xmoe_status st, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
xmoe_status ok();
xmoe_status hip_status(hipError_t e, const char *what);
xmoe_status check_device();
xmoe_status check_dtype(xmoe_dtype dt);

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline hipStream_t S(void *s) { return static_cast<hipStream_t>(s); }

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;

// a * b <= limit for a, b >= 0, without forming a product that could overflow
// (callers may pass any int64 size; the checks must stay defined for all)
inline bool within(int64_t a, int64_t b, int64_t limit) {
    return a >= 0 && b >= 0 && (b == 0 || a <= limit / b);
}

}  // namespace xmoe_api

#define REQUIRE(cond, st, ...)                     \
    do {                                           \
        if (!(cond)) return fail(st, __VA_ARGS__); \
    } while (0)

#define CHECK_DEVICE()                  \
    do {                                \
        xmoe_status _s = check_device(); \
        if (_s != XMOE_OK) return _s;   \
    } while (0)

#define TRY(expr)                     \
    do {                              \
        xmoe_status _s = (expr);      \
        if (_s != XMOE_OK) return _s; \
    } while (0)

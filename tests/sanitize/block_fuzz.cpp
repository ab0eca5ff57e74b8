// Random arguments from the edges of every parameter's range for the calls
// around the layer (norm, balance loss, 8-bit experts), with no-op launchers
// and no device: each call returns a documented status, with a message where it
// is not XMOE_OK, and the sanitizers stay silent.  Without a device a call whose
// arguments are accepted ends at the device check (XMOE_ERR_HIP).
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <limits>
#include <random>

#include "../../include/xmoe.h"

namespace {

std::mt19937_64 rng(12345);
int failures = 0;
long calls = 0, accepted = 0;

int64_t i64() {
    static const int64_t v[] = {0, 1, 2, 15, 16, 31, 32, 33, 64, 96, 128, 255, 256, 511, 512, 1000, 1024, 4096, 4097, 8192,
                                16384, 16392, 65536, 65568, 1 << 20, 1 << 24, (1 << 25) - 1, 1 << 25, 1 << 26,
                                (int64_t{1} << 26) + 1, (int64_t{1} << 31) - 1, int64_t{1} << 31, int64_t{1} << 34,
                                int64_t{1} << 40, int64_t{1} << 62, INT64_MAX, -1, -64, INT64_MIN};
    return v[rng() % (sizeof v / sizeof v[0])];
}
int64_t small() { return static_cast<int64_t>(rng() % 5000); }
int64_t size() { return rng() % 2 ? i64() : small(); }
int32_t i32() {
    const int64_t v = rng() % 3 ? small() / 8 * 8 : i64();
    return static_cast<int32_t>(v > INT32_MAX ? INT32_MAX : v < INT32_MIN ? INT32_MIN : v);
}
void *ptr() {
    static char *next = reinterpret_cast<char *>(uintptr_t{1} << 40);
    const int r = static_cast<int>(rng() % 40);
    if (r == 0) return nullptr;
    if (r == 1) return next + 8;
    if (r == 2) return reinterpret_cast<void *>(UINTPTR_MAX - 15);
    next += (int64_t{1} << 32) * static_cast<int64_t>(rng() % 16);
    return next;
}
const float *f() { return static_cast<const float *>(ptr()); }
float *fo() { return static_cast<float *>(ptr()); }
const int32_t *i() { return static_cast<const int32_t *>(ptr()); }
const uint8_t *u() { return rng() % 2 ? nullptr : static_cast<const uint8_t *>(ptr()); }
xmoe_dtype dt() {
    const int r = static_cast<int>(rng() % 20);
    return static_cast<xmoe_dtype>(r == 0 ? 7 : r % 2);
}
size_t bytes() { return rng() % 4 ? size_t{1} << 50 : static_cast<size_t>(rng() % 4096); }
float real() {
    static const float v[] = {0.0f, 1e-6f, 1.0f, -1.0f, 1e30f};
    const int r = static_cast<int>(rng() % 8);
    return r < 5 ? v[r] : r == 5 ? std::numeric_limits<float>::quiet_NaN() : std::numeric_limits<float>::infinity();
}

void seen(const char *what, xmoe_status s) {
    ++calls;
    const bool known = s == XMOE_OK || s == XMOE_ERR_INVALID_VALUE || s == XMOE_ERR_UNSUPPORTED ||
                       s == XMOE_ERR_WORKSPACE || s == XMOE_ERR_HIP;
    const bool told = (std::strlen(xmoe_last_error()) > 0) == (s != XMOE_OK);
    if (s == XMOE_ERR_HIP) ++accepted;
    if (!known || !told) {
        ++failures;
        std::printf("%s: status %d, message '%s'\n", what, static_cast<int>(s), xmoe_last_error());
    }
}

}  // namespace

int main() {
    for (int n = 0; n < 60000; ++n) {
        switch (n % 11) {
            case 0: seen("norm", xmoe_add_rmsnorm(ptr(), rng() % 2 ? ptr() : nullptr, ptr(), dt(), size(), i32(), real(), ptr(), ptr(), rng() % 2 ? ptr() : nullptr, ptr(), fo(), nullptr)); break;
            case 1: seen("norm_bwd", xmoe_add_rmsnorm_bwd(ptr(), ptr(), ptr(), ptr(), f(), dt(), size(), i32(), ptr(), fo(), ptr(), bytes(), nullptr)); break;
            case 2: seen("balance", xmoe_balance_loss(f(), i(), size(), i32(), i32(), i(), i32(), u(), real(), fo(), static_cast<int32_t *>(ptr()), fo(), ptr(), bytes(), nullptr)); break;
            case 3: seen("balance_bwd", xmoe_balance_loss_bwd(f(), f(), size(), i32(), i(), i32(), u(), f(), fo(), nullptr)); break;
            case 4: seen("route_bwd_balance", xmoe_route_bwd_balance(ptr(), ptr(), f(), i(), f(), i32(), f(), i(), i32(), u(), f(), dt(), size(), i32(), i32(), i32(), real(), 1, ptr(), fo(), ptr(), bytes(), nullptr)); break;
            case 5: seen("quantize", xmoe_mx8_quantize(ptr(), dt(), size(), i32(), ptr(), ptr(), nullptr)); break;
            case 6: seen("dequantize", xmoe_mx8_dequantize(ptr(), ptr(), dt(), size(), i32(), ptr(), nullptr)); break;
            case 7: seen("weights", xmoe_mx8_quantize_weights(ptr(), dt(), i32(), i32(), i32(), ptr(), ptr(), nullptr)); break;
            case 8: {
                const int64_t rows = size(), T = rng() % 2 ? rows : size();
                seen("up", xmoe_expert_ffn_up_mx8(ptr(), ptr(), rng() % 2 ? i() : nullptr, T, ptr(), ptr(), ptr(), ptr(), i(), i32(), rows, i32(), i32(), ptr(), ptr(), nullptr));
                break;
            }
            case 9: seen("down", xmoe_expert_ffn_down_mx8(ptr(), ptr(), ptr(), ptr(), i(), i32(), size(), i32(), i32(), ptr(), nullptr)); break;
            default:
                (void)xmoe_add_rmsnorm_bwd_workspace_size(size(), i32(), dt());
                (void)xmoe_balance_loss_workspace_size(size(), i32(), i32());
        }
    }
    if (accepted == 0) {
        ++failures;
        std::printf("no call was accepted\n");
    }
    std::printf("%ld calls, %ld accepted\nfuzz: %d failures\n", calls, accepted, failures);
    return failures != 0;
}

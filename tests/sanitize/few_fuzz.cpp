// Random arguments from the edges of every parameter's range for the layer for a few
// tokens and the FFN with 8-bit pre-activations, with no-op launchers and no device: each
// call returns a documented status, with a message where it is not XMOE_OK, and the
// sanitizers stay silent.  Without a device a call whose arguments are accepted ends at
// the device check (XMOE_ERR_HIP).
#include <climits>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <random>

#include "../../include/xmoe.h"

namespace {

std::mt19937_64 rng(54321);
int failures = 0;
long calls = 0, accepted[5] = {};

int64_t edge() {
    static const int64_t v[] = {0, 1, 7, 8, 16, 31, 32, 63, 64, 65, 128, 255, 256, 1000, 1024, 1032, 4096, 8192, 32768, 65536,
                                65568, 1 << 20, (1 << 20) + 8, 1 << 25, (int64_t{1} << 31) - 1, int64_t{1} << 31,
                                int64_t{1} << 33, int64_t{1} << 62, INT64_MAX, -1, -64, INT64_MIN};
    return v[rng() % (sizeof v / sizeof v[0])];
}
int64_t tokens() { return rng() % 3 ? static_cast<int64_t>(rng() % 66) : edge(); }
int64_t rows() { return rng() % 2 ? static_cast<int64_t>(rng() % 5000) : edge(); }
int32_t i32() {
    const int64_t v = rng() % 4 ? static_cast<int64_t>(rng() % 300) * 32 : edge();
    return static_cast<int32_t>(v > INT32_MAX ? INT32_MAX : v < INT32_MIN ? INT32_MIN : v);
}
int32_t experts() { return rng() % 4 ? static_cast<int32_t>(8 + rng() % 32 * 8) : i32(); }
int32_t choices() { return rng() % 4 ? static_cast<int32_t>(1 + rng() % 8) : i32(); }
int32_t shared_width() { return rng() % 2 ? 0 : i32(); }
void *ptr() {
    static char *next = reinterpret_cast<char *>(uintptr_t{1} << 40);
    const int r = static_cast<int>(rng() % 60);
    if (r == 0) return nullptr;
    if (r == 1) return next + 8;
    if (r == 2) return reinterpret_cast<void *>(UINTPTR_MAX - 15);
    next += (int64_t{1} << 24) * static_cast<int64_t>(rng() % 16);
    return next;
}
float *f() { return static_cast<float *>(ptr()); }
int32_t *i() { return static_cast<int32_t *>(ptr()); }
const int32_t *maybe() { return rng() % 2 ? i() : nullptr; }
xmoe_dtype dt() {
    const int r = static_cast<int>(rng() % 20);
    return static_cast<xmoe_dtype>(r == 0 ? 7 : r % 2);
}
size_t bytes() { return rng() % 4 ? size_t{1} << 60 : static_cast<size_t>(rng() % 4096); }

void seen(int which, const char *what, xmoe_status s) {
    ++calls;
    const bool known = s == XMOE_OK || s == XMOE_ERR_INVALID_VALUE || s == XMOE_ERR_UNSUPPORTED ||
                       s == XMOE_ERR_WORKSPACE || s == XMOE_ERR_HIP;
    const bool told = (std::strlen(xmoe_last_error()) > 0) == (s != XMOE_OK);
    if (s == XMOE_ERR_HIP) ++accepted[which];
    if (!known || !told) {
        ++failures;
        std::printf("%s: status %d, message '%s'\n", what, static_cast<int>(s), xmoe_last_error());
    }
}

xmoe_mx8_ffn ffn() { return {ptr(), ptr(), ptr(), ptr(), ptr(), ptr()}; }

}  // namespace

int main() {
    for (int n = 0; n < 60000; ++n) {
        switch (n % 6) {
            case 0:
                seen(0, "few", xmoe_layer_few(ptr(), ptr(), ptr(), ptr(), ptr(), ptr(), ptr(), ptr(), dt(), tokens(), i32(), experts(), choices(), i32(), shared_width(), 1.0f, f(), f(), i(), f(), f(), ptr(), ptr(), bytes(), nullptr));
                break;
            case 1: {
                const xmoe_mx8_ffn r = ffn(), s = ffn();
                seen(1, "few_mx8", xmoe_layer_few_mx8(ptr(), ptr(), ptr(), ptr(), rng() % 50 ? &r : nullptr, rng() % 3 ? &s : nullptr, tokens(), i32(), experts(), choices(), i32(), shared_width(), 1.0f, f(), f(), i(), f(), f(), ptr(), ptr(), bytes(), nullptr));
                break;
            }
            case 2: {
                const int64_t n_rows = rows();
                seen(2, "up_ckpt8", xmoe_expert_ffn_up_ckpt8(ptr(), maybe(), rng() % 2 ? n_rows : rows(), ptr(), ptr(), dt(), i(), experts(), n_rows, i32(), i32(), ptr(), ptr(), ptr(), nullptr));
                break;
            }
            case 3: seen(3, "dequantize", xmoe_ckpt8_dequantize(ptr(), ptr(), dt(), rows(), i32(), ptr(), nullptr)); break;
            case 4: {
                const int64_t n_rows = rows();
                seen(4, "dact_ckpt8", xmoe_expert_ffn_bwd_dact_ckpt8(ptr(), maybe(), rng() % 2 ? f() : nullptr, rng() % 2 ? n_rows : rows(), ptr(), ptr(), ptr(), dt(), i(), experts(), n_rows, i32(), i32(), ptr(), ptr(), maybe(), rng() % 2 ? f() : nullptr, ptr(), bytes(), nullptr));
                break;
            }
            default:
                (void)xmoe_layer_few_workspace_size(tokens(), i32(), experts(), choices(), i32(), shared_width(), dt());
                (void)xmoe_layer_few_mx8_workspace_size(tokens(), i32(), experts(), choices(), i32(), shared_width());
                (void)xmoe_expert_ffn_bwd_dact_ckpt8_workspace_size(rows(), i32());
        }
    }
    for (int which = 0; which < 5; ++which)
        if (accepted[which] == 0) {
            ++failures;
            std::printf("no call of kind %d was accepted\n", which);
        }
    std::printf("%ld calls\nfuzz: %d failures\n", calls, failures);
    return failures != 0;
}

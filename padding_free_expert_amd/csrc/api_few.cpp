// C ABI of the whole layer for a few tokens.  Argument validation as in api.cpp;
// semantics in xmoe.h.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "api_common.hpp"
#include "few.hpp"

using namespace xmoe_api;

namespace {

constexpr int32_t kMaxFewDim = 65536;
constexpr int64_t kMaxFewBytes = (int64_t(1) << 31) - 1;  // of one expert's matrix: 32-bit offsets

xmoe_status check_few_sizes(const xmoe::FewSizes &z) {
    const int32_t step = z.mx8 ? 32 : 8;
    const int64_t es = z.mx8 ? 1 : z.dt == XMOE_BF16 ? 2 : 4, gs = z.dt == XMOE_BF16 ? 2 : 4;
    REQUIRE(z.T >= 0 && z.d >= 1 && z.h >= 1 && z.hs >= 0, XMOE_ERR_INVALID_VALUE,
            "T and hs must be >= 0, d and h >= 1");
    REQUIRE(z.T <= xmoe::kFewTokens, XMOE_ERR_UNSUPPORTED, "T must be at most %d", xmoe::kFewTokens);
    REQUIRE(z.E >= 1 && z.E <= 1024, XMOE_ERR_INVALID_VALUE, "E must be in [1, 1024]");
    REQUIRE(z.k >= 1 && z.k <= z.E, XMOE_ERR_INVALID_VALUE, "k must be in [1, E]");
    REQUIRE(z.d % step == 0 && z.h % step == 0 && z.hs % step == 0, XMOE_ERR_UNSUPPORTED,
            "d, h and hs must be multiples of %d", step);
    REQUIRE(z.d <= kMaxFewDim && z.h <= kMaxFewDim && z.hs <= kMaxFewDim, XMOE_ERR_UNSUPPORTED,
            "d, h and hs must be at most %d", kMaxFewDim);
    REQUIRE(z.dt != XMOE_BF16 || z.E % 8 == 0, XMOE_ERR_UNSUPPORTED, "bf16 needs E a multiple of 8");
    REQUIRE(within(z.d, std::max(z.h, z.hs), kMaxFewBytes / es) && within(z.d, z.E, kMaxFewBytes / gs),
            XMOE_ERR_UNSUPPORTED, "one expert's matrix must have less than 2^31 bytes");
    return XMOE_OK;
}

xmoe_status run_few(const xmoe::FewSizes &z, const xmoe::FewTensors &t, size_t ws_bytes, void *stream, const char *what) {
    TRY(check_few_sizes(z));
    const auto scaled = [&](const xmoe::FewWeights &w) { return !z.mx8 || (w.w1s && w.w3s && w.w2s); };
    REQUIRE(t.wg && t.routed.w1 && t.routed.w3 && t.routed.w2 && scaled(t.routed), XMOE_ERR_INVALID_VALUE,
            "wg and the experts' weights are required");
    REQUIRE(z.hs == 0 || (t.shared.w1 && t.shared.w3 && t.shared.w2 && scaled(t.shared)), XMOE_ERR_INVALID_VALUE,
            "the shared experts' weights are required when hs > 0");
    REQUIRE(z.T == 0 || (t.x && t.ids && t.w && t.logits && t.y && (!z.mx8 || (t.xq && t.xs))), XMOE_ERR_INVALID_VALUE,
            "a required pointer is NULL");
    for (const void *p : {t.x, t.xq, t.xs, t.wg, static_cast<const void *>(t.y), t.routed.w1, t.routed.w3, t.routed.w2,
                          t.routed.w1s, t.routed.w3s, t.routed.w2s, t.shared.w1, t.shared.w3, t.shared.w2, t.shared.w1s,
                          t.shared.w3s, t.shared.w2s})
        REQUIRE(aligned16(p), XMOE_ERR_UNSUPPORTED, "matrices must be 16-byte aligned");
    REQUIRE(z.T == 0 || (t.ws && aligned16(t.ws)), XMOE_ERR_WORKSPACE, "workspace is NULL or not 16-byte aligned");
    REQUIRE(ws_bytes >= xmoe::few_workspace(z), XMOE_ERR_WORKSPACE, "workspace too small (see %s_workspace_size)", what);
    CHECK_DEVICE();
    return hip_status(xmoe::launch_layer_few(z, t, S(stream)), what);
}

}  // namespace

extern "C" {

size_t xmoe_layer_few_workspace_size(int64_t T, int32_t d, int32_t E, int32_t k, int32_t h, int32_t hs,
                                     xmoe_dtype dtype) {
    const xmoe::FewSizes z{dtype, false, T, d, E, k, h, hs};
    if ((dtype != XMOE_F32 && dtype != XMOE_BF16) || check_few_sizes(z) != XMOE_OK) return 0;
    return xmoe::few_workspace(z);
}

xmoe_status xmoe_layer_few(const void *x, const void *wg, const void *w1, const void *w3, const void *w2,
                           const void *s1, const void *s3, const void *s2, xmoe_dtype dtype, int64_t T, int32_t d,
                           int32_t E, int32_t k, int32_t h, int32_t hs, float inv_temperature, const float *logit_bias,
                           const float *select_bias, int32_t *topk_ids, float *topk_w, float *logits, void *y,
                           void *workspace, size_t ws_bytes, void *stream) {
    TRY(check_dtype(dtype));
    xmoe::FewTensors t{};
    t.x = x;
    t.wg = wg;
    t.routed = {w1, w3, w2, nullptr, nullptr, nullptr};
    if (hs > 0) t.shared = {s1, s3, s2, nullptr, nullptr, nullptr};
    t.scale = inv_temperature;
    t.lbias = logit_bias;
    t.sbias = select_bias;
    t.ids = topk_ids;
    t.w = topk_w;
    t.logits = logits;
    t.y = y;
    t.ws = workspace;
    return run_few({dtype, false, T, d, E, k, h, hs}, t, ws_bytes, stream, "xmoe_layer_few");
}

size_t xmoe_layer_few_mx8_workspace_size(int64_t T, int32_t d, int32_t E, int32_t k, int32_t h, int32_t hs) {
    const xmoe::FewSizes z{XMOE_BF16, true, T, d, E, k, h, hs};
    return check_few_sizes(z) == XMOE_OK ? xmoe::few_workspace(z) : 0;
}

xmoe_status xmoe_layer_few_mx8(const void *x, const void *xq, const void *xscale, const void *wg,
                               const xmoe_mx8_ffn *routed, const xmoe_mx8_ffn *shared, int64_t T, int32_t d, int32_t E,
                               int32_t k, int32_t h, int32_t hs, float inv_temperature, const float *logit_bias,
                               const float *select_bias, int32_t *topk_ids, float *topk_w, float *logits, void *y,
                               void *workspace, size_t ws_bytes, void *stream) {
    REQUIRE(routed && (hs <= 0 || shared), XMOE_ERR_INVALID_VALUE, "the experts' weights are required");
    const auto set = [](const xmoe_mx8_ffn &f) {
        return xmoe::FewWeights{f.w1, f.w3, f.w2, f.w1_scale, f.w3_scale, f.w2_scale};
    };
    xmoe::FewTensors t{};
    t.x = x;
    t.xq = xq;
    t.xs = xscale;
    t.wg = wg;
    t.routed = set(*routed);
    if (hs > 0) t.shared = set(*shared);
    t.scale = inv_temperature;
    t.lbias = logit_bias;
    t.sbias = select_bias;
    t.ids = topk_ids;
    t.w = topk_w;
    t.logits = logits;
    t.y = y;
    t.ws = workspace;
    return run_few({XMOE_BF16, true, T, d, E, k, h, hs}, t, ws_bytes, stream, "xmoe_layer_few_mx8");
}

}  // extern "C"

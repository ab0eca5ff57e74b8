// C ABI of the expert FFN with its pre-activations kept in 8 bits.  Argument
// validation as in api.cpp; semantics in xmoe.h.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "api_common.hpp"
#include "kernels.hpp"

using namespace xmoe_api;

namespace {

constexpr int32_t kMaxDim = 1 << 20;

xmoe_status check_sizes(int32_t E, int64_t rows, int32_t d, int32_t h) {
    REQUIRE(E >= 1 && E <= 1024, XMOE_ERR_INVALID_VALUE, "E must be in [1, 1024]");
    REQUIRE(rows >= 0 && rows <= kMaxRows, XMOE_ERR_INVALID_VALUE, "rows must be in [0, 2^31)");
    REQUIRE(d >= 1 && h >= 1, XMOE_ERR_INVALID_VALUE, "d and h must be >= 1");
    REQUIRE(d % 8 == 0 && h % 8 == 0, XMOE_ERR_UNSUPPORTED, "d and h must be multiples of 8");
    REQUIRE(d <= kMaxDim && h <= kMaxDim, XMOE_ERR_UNSUPPORTED, "d and h must be at most %d", kMaxDim);
    return XMOE_OK;
}

// rows of x (or dy): row r is x[token_ids[r]], or x[r]
xmoe_status check_source(const void *x, const int32_t *token_ids, int64_t T, int64_t rows, int32_t d,
                         xmoe_dtype dtype) {
    REQUIRE(T >= 0, XMOE_ERR_INVALID_VALUE, "T must be >= 0");
    REQUIRE(rows == 0 || x, XMOE_ERR_INVALID_VALUE, "a required pointer is NULL");
    REQUIRE(aligned16(x), XMOE_ERR_UNSUPPORTED, "matrices must be 16-byte aligned");
    if (!token_ids) {
        REQUIRE(T == rows, XMOE_ERR_INVALID_VALUE, "without token_ids T must be rows");
        return XMOE_OK;
    }
    REQUIRE(rows == 0 || T > 0, XMOE_ERR_INVALID_VALUE, "rows need tokens");
    REQUIRE(within(T, static_cast<int64_t>(d) * (dtype == XMOE_BF16 ? 2 : 4), (int64_t(1) << 31) - 1),
            XMOE_ERR_UNSUPPORTED, "T * d * element size must be < 2^31 with token_ids");
    return XMOE_OK;
}

size_t dact_workspace(int64_t rows, int32_t h) {
    return static_cast<size_t>((h + 63) / 64) * static_cast<size_t>(rows) * 4;
}

}  // namespace

extern "C" {

xmoe_status xmoe_expert_ffn_up_ckpt8(const void *x, const int32_t *token_ids, int64_t T, const void *w1,
                                     const void *w3, xmoe_dtype dtype, const int32_t *expert_offsets, int32_t E,
                                     int64_t rows, int32_t d, int32_t h, void *act, void *hq, void *hscale,
                                     void *stream) {
    TRY(check_dtype(dtype));
    REQUIRE(w1 && w3 && expert_offsets && (rows == 0 || (act && hq && hscale)), XMOE_ERR_INVALID_VALUE,
            "a required pointer is NULL");
    TRY(check_sizes(E, rows, d, h));
    TRY(check_source(x, token_ids, T, rows, d, dtype));
    REQUIRE(aligned16(w1) && aligned16(w3) && aligned16(act) && aligned16(hq) && aligned16(hscale), XMOE_ERR_UNSUPPORTED,
            "matrices must be 16-byte aligned");
    CHECK_DEVICE();
    return hip_status(xmoe::launch_ffn_up_ckpt8(dtype, x, token_ids, T, w1, w3, expert_offsets, E, rows, d, h, act, hq,
                                                hscale, S(stream)),
                      "xmoe_expert_ffn_up_ckpt8 launch");
}

xmoe_status xmoe_ckpt8_dequantize(const void *hq, const void *hscale, xmoe_dtype dtype, int64_t rows, int32_t h,
                                  void *h13, void *stream) {
    TRY(check_dtype(dtype));
    TRY(check_sizes(1, rows, 8, h));
    REQUIRE(within(rows, std::max(h / 4, 256), (int64_t(1) << 32) - 257), XMOE_ERR_INVALID_VALUE,
            "rows * max(h / 4, 256) must be < 2^32");
    REQUIRE(rows == 0 || (hq && hscale && h13), XMOE_ERR_INVALID_VALUE, "a required pointer is NULL");
    REQUIRE(aligned16(hq) && aligned16(hscale) && aligned16(h13), XMOE_ERR_UNSUPPORTED, "matrices must be 16-byte aligned");
    CHECK_DEVICE();
    return hip_status(xmoe::launch_ckpt8_dequantize(dtype, hq, hscale, rows, h, h13, S(stream)),
                      "xmoe_ckpt8_dequantize launch");
}

size_t xmoe_expert_ffn_bwd_dact_ckpt8_workspace_size(int64_t rows, int32_t h) {
    if (check_sizes(1, rows, 8, h) != XMOE_OK) return 0;
    return dact_workspace(rows, h);
}

xmoe_status xmoe_expert_ffn_bwd_dact_ckpt8(const void *dy, const int32_t *token_ids, const float *row_weights,
                                           int64_t T, const void *w2, const void *hq, const void *hscale,
                                           xmoe_dtype dtype, const int32_t *expert_offsets, int32_t E, int64_t rows,
                                           int32_t d, int32_t h, void *dh13, void *act, const int32_t *slot_to_row,
                                           float *dweights, void *workspace, size_t ws_bytes, void *stream) {
    TRY(check_dtype(dtype));
    REQUIRE(w2 && expert_offsets && (rows == 0 || (hq && hscale && dh13 && act)), XMOE_ERR_INVALID_VALUE,
            "a required pointer is NULL");
    TRY(check_sizes(E, rows, d, h));
    TRY(check_source(dy, token_ids, T, rows, d, dtype));
    REQUIRE(dweights || !slot_to_row, XMOE_ERR_INVALID_VALUE, "slot_to_row orders dweights, which is NULL");
    REQUIRE(aligned16(w2) && aligned16(hq) && aligned16(hscale) && aligned16(dh13) && aligned16(act),
            XMOE_ERR_UNSUPPORTED, "matrices must be 16-byte aligned");
    if (dweights && rows > 0) {
        REQUIRE(workspace && aligned16(workspace), XMOE_ERR_WORKSPACE, "workspace is NULL or not 16-byte aligned");
        REQUIRE(ws_bytes >= dact_workspace(rows, h), XMOE_ERR_WORKSPACE,
                "workspace too small (see xmoe_expert_ffn_bwd_dact_ckpt8_workspace_size)");
    }
    CHECK_DEVICE();
    return hip_status(xmoe::launch_ffn_bwd_dact_ckpt8(dtype, dy, token_ids, T, row_weights, w2, hq, hscale,
                                                      expert_offsets, E, rows, d, h, dh13, act, slot_to_row, dweights,
                                                      workspace, S(stream)),
                      "xmoe_expert_ffn_bwd_dact_ckpt8 launch");
}

}  // extern "C"

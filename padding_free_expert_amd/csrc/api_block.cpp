// C ABI of what stands around the expert layer: the residual addition with the
// root-mean-square norm, the gate's balance loss, and the experts' FFN on 8-bit
// rows.  Argument validation as in api.cpp; semantics in xmoe.h.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "api_common.hpp"
#include "kernels.hpp"

using namespace xmoe_api;

namespace {

constexpr int64_t kMaxElems = int64_t(1) << 34;     // rows * max(d, 512): the launch's threads stay below 2^32
constexpr int64_t kMaxMx8Elems = int64_t(1) << 33;  // the same for fp32 rows in whole waves (544: 192 threads a row)
constexpr int32_t kMaxNormDim = 16384;
constexpr int32_t kMaxMx8Dim = 65536;
constexpr int64_t kMaxBalanceTokens = int64_t(1) << 26;
constexpr int32_t kMaxSequences = 4096;

bool overlap(const void *a, int64_t na, const void *b, int64_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && x < y + static_cast<uintptr_t>(nb) && y < x + static_cast<uintptr_t>(na);
}
// the same buffer, or none of it
bool same_or_apart(const void *a, const void *b, int64_t bytes) { return a == b || !overlap(a, bytes, b, bytes); }

xmoe_status check_norm_sizes(int64_t T, int32_t d) {
    REQUIRE(T >= 0 && d >= 1, XMOE_ERR_INVALID_VALUE, "T must be >= 0 and d >= 1");
    REQUIRE(d % 8 == 0, XMOE_ERR_UNSUPPORTED, "d must be a multiple of 8");
    REQUIRE(d <= kMaxNormDim, XMOE_ERR_UNSUPPORTED, "d must be at most %d", kMaxNormDim);
    REQUIRE(within(T, std::max(d, 512), kMaxElems - 1), XMOE_ERR_INVALID_VALUE, "T * max(d, 512) must be < 2^34");
    return XMOE_OK;
}

xmoe_status check_balance(const float *logits, const int32_t *seq_offsets, int64_t T, int32_t E, int32_t S) {
    REQUIRE(T >= 0 && T <= kMaxBalanceTokens, XMOE_ERR_INVALID_VALUE, "T must be in [0, 2^26]");
    REQUIRE(E >= 1 && E <= 1024, XMOE_ERR_INVALID_VALUE, "E must be in [1, 1024]");
    REQUIRE(S >= 1 && S <= kMaxSequences, XMOE_ERR_INVALID_VALUE, "S must be in [1, %d]", kMaxSequences);
    REQUIRE(seq_offsets || S == 1, XMOE_ERR_INVALID_VALUE, "seq_offsets is required when S > 1");
    REQUIRE(T == 0 || logits, XMOE_ERR_INVALID_VALUE, "logits is NULL");
    REQUIRE(aligned16(logits), XMOE_ERR_UNSUPPORTED, "logits must be 16-byte aligned");
    return XMOE_OK;
}

xmoe_status check_mx8_rows(int64_t n, int32_t K) {
    REQUIRE(n >= 0 && K >= 1, XMOE_ERR_INVALID_VALUE, "n must be >= 0 and K >= 1");
    REQUIRE(K % 32 == 0, XMOE_ERR_UNSUPPORTED, "K must be a multiple of 32");
    REQUIRE(K <= kMaxMx8Dim, XMOE_ERR_UNSUPPORTED, "K must be at most %d", kMaxMx8Dim);
    REQUIRE(within(n, std::max(K, 512), kMaxMx8Elems - 1), XMOE_ERR_INVALID_VALUE, "n * max(K, 512) must be < 2^33");
    return XMOE_OK;
}

xmoe_status check_mx8_ffn(const int32_t *offsets, int32_t E, int64_t rows, int32_t d, int32_t h) {
    REQUIRE(offsets, XMOE_ERR_INVALID_VALUE, "expert_offsets is NULL");
    REQUIRE(E >= 1 && E <= 1024, XMOE_ERR_INVALID_VALUE, "E must be in [1, 1024]");
    REQUIRE(rows >= 0 && rows <= kMaxRows, XMOE_ERR_INVALID_VALUE, "rows must be in [0, 2^31)");
    REQUIRE(d >= 1 && h >= 1, XMOE_ERR_INVALID_VALUE, "d and h must be >= 1");
    REQUIRE(d % 32 == 0 && h % 32 == 0, XMOE_ERR_UNSUPPORTED, "d and h must be multiples of 32");
    REQUIRE(d <= kMaxMx8Dim && h <= kMaxMx8Dim, XMOE_ERR_UNSUPPORTED, "d and h must be at most %d", kMaxMx8Dim);
    REQUIRE(within(rows, std::max(std::max(d, h), 512), kMaxElems - 1), XMOE_ERR_INVALID_VALUE,
            "rows * max(d, h, 512) must be < 2^34");
    return XMOE_OK;
}

}  // namespace

extern "C" {

xmoe_status xmoe_add_rmsnorm(const void *x, const void *res, const void *gamma, xmoe_dtype dtype, int64_t T, int32_t d,
                             float eps, void *sum, void *y, void *q, void *scale, float *rstd, void *stream) {
    TRY(check_dtype(dtype));
    TRY(check_norm_sizes(T, d));
    REQUIRE(gamma && (T == 0 || (x && (y || q))), XMOE_ERR_INVALID_VALUE, "x, gamma and y or q are required");
    REQUIRE(!q || T == 0 || scale, XMOE_ERR_INVALID_VALUE, "scale is required with q");
    REQUIRE(eps >= 0.0f, XMOE_ERR_INVALID_VALUE, "eps must be >= 0");
    REQUIRE(!q || d % 32 == 0, XMOE_ERR_UNSUPPORTED, "an output in 8 bits needs d a multiple of 32");
    REQUIRE(aligned16(x) && aligned16(res) && aligned16(gamma) && aligned16(sum) && aligned16(y) && aligned16(q) &&
                aligned16(scale),
            XMOE_ERR_UNSUPPORTED, "matrices must be 16-byte aligned");
    const int64_t bytes = T * d * (dtype == XMOE_BF16 ? 2 : 4);
    for (const void *o : {static_cast<const void *>(sum), static_cast<const void *>(y)})
        REQUIRE(same_or_apart(o, x, bytes) && same_or_apart(o, res, bytes), XMOE_ERR_INVALID_VALUE,
                "sum and y may be x or res, but not overlap them otherwise");
    REQUIRE(!overlap(sum, bytes, y, bytes), XMOE_ERR_INVALID_VALUE, "sum and y must not overlap");
    for (const void *o : {x, res, static_cast<const void *>(sum), static_cast<const void *>(y)})
        REQUIRE(!overlap(q, T * d, o, bytes), XMOE_ERR_INVALID_VALUE, "q must not overlap x, res, sum or y");
    CHECK_DEVICE();
    return hip_status(xmoe::launch_add_rmsnorm(dtype, x, res, gamma, T, d, eps, sum, y, q, scale, rstd, S(stream)),
                      "xmoe_add_rmsnorm launch");
}

size_t xmoe_add_rmsnorm_bwd_workspace_size(int64_t T, int32_t d, xmoe_dtype dtype) {
    if ((dtype != XMOE_F32 && dtype != XMOE_BF16) || T < 0 || d < 1 || d % 8 || d > kMaxNormDim ||
        !within(T, std::max(d, 512), kMaxElems - 1))
        return 0;
    return xmoe::add_rmsnorm_bwd_workspace(T, d, dtype);
}

xmoe_status xmoe_add_rmsnorm_bwd(const void *dy, const void *dsum, const void *sum, const void *gamma,
                                 const float *rstd, xmoe_dtype dtype, int64_t T, int32_t d, void *dx, float *dgamma,
                                 void *workspace, size_t ws_bytes, void *stream) {
    TRY(check_dtype(dtype));
    TRY(check_norm_sizes(T, d));
    REQUIRE(gamma && dgamma && (T == 0 || (dy && sum && rstd && dx)), XMOE_ERR_INVALID_VALUE,
            "a required pointer is NULL");
    REQUIRE(aligned16(dy) && aligned16(dsum) && aligned16(sum) && aligned16(gamma) && aligned16(dx) &&
                aligned16(dgamma),
            XMOE_ERR_UNSUPPORTED, "matrices must be 16-byte aligned");
    const int64_t bytes = T * d * (dtype == XMOE_BF16 ? 2 : 4);
    REQUIRE(same_or_apart(dx, dy, bytes) && same_or_apart(dx, dsum, bytes) && same_or_apart(dx, sum, bytes),
            XMOE_ERR_INVALID_VALUE, "dx may be dy, dsum or sum, but not overlap them otherwise");
    REQUIRE(workspace && aligned16(workspace), XMOE_ERR_WORKSPACE, "workspace is NULL or not 16-byte aligned");
    REQUIRE(ws_bytes >= xmoe::add_rmsnorm_bwd_workspace(T, d, dtype), XMOE_ERR_WORKSPACE,
            "workspace too small (see xmoe_add_rmsnorm_bwd_workspace_size)");
    CHECK_DEVICE();
    return hip_status(xmoe::launch_add_rmsnorm_bwd(dtype, dy, dsum, sum, gamma, rstd, T, d, dx, dgamma, workspace,
                                                   S(stream)),
                      "xmoe_add_rmsnorm_bwd launch");
}

size_t xmoe_balance_loss_workspace_size(int64_t T, int32_t E, int32_t n_seq) {
    if (T < 0 || T > kMaxBalanceTokens || E < 1 || E > 1024 || n_seq < 1 || n_seq > kMaxSequences) return 0;
    return xmoe::balance_workspace(T, E, n_seq);
}

xmoe_status xmoe_balance_loss(const float *logits, const int32_t *topk_ids, int64_t T, int32_t E, int32_t k,
                              const int32_t *seq_offsets, int32_t n_seq, const uint8_t *token_mask, float alpha,
                              float *loss, int32_t *counts, float *coef, void *workspace, size_t ws_bytes,
                              void *stream) {
    TRY(check_balance(logits, seq_offsets, T, E, n_seq));
    REQUIRE(k >= 1 && k <= E, XMOE_ERR_INVALID_VALUE, "k must be in [1, E]");
    REQUIRE(loss && counts && coef && (T == 0 || topk_ids), XMOE_ERR_INVALID_VALUE, "a required pointer is NULL");
    REQUIRE(workspace && aligned16(workspace), XMOE_ERR_WORKSPACE, "workspace is NULL or not 16-byte aligned");
    REQUIRE(ws_bytes >= xmoe::balance_workspace(T, E, n_seq), XMOE_ERR_WORKSPACE,
            "workspace too small (see xmoe_balance_loss_workspace_size)");
    CHECK_DEVICE();
    return hip_status(xmoe::launch_balance_loss(logits, topk_ids, T, E, k, seq_offsets, n_seq, token_mask, alpha, loss,
                                                counts, coef, workspace, S(stream)),
                      "xmoe_balance_loss launch");
}

xmoe_status xmoe_balance_loss_bwd(const float *logits, const float *coef, int64_t T, int32_t E,
                                  const int32_t *seq_offsets, int32_t n_seq, const uint8_t *token_mask,
                                  const float *dloss, float *dlogits, void *stream) {
    TRY(check_balance(logits, seq_offsets, T, E, n_seq));
    REQUIRE(T == 0 || (coef && dlogits), XMOE_ERR_INVALID_VALUE, "coef and dlogits are required");
    REQUIRE(aligned16(dlogits), XMOE_ERR_UNSUPPORTED, "dlogits must be 16-byte aligned");
    CHECK_DEVICE();
    return hip_status(xmoe::launch_balance_loss_bwd(logits, T, E, {seq_offsets, n_seq, token_mask, coef, dloss},
                                                    dlogits, S(stream)),
                      "xmoe_balance_loss_bwd launch");
}

xmoe_status xmoe_route_bwd_balance(const void *x, const void *wg, const float *logits, const int32_t *topk_ids,
                                   const float *dtopk_w, int32_t ldw, const float *coef, const int32_t *seq_offsets,
                                   int32_t n_seq, const uint8_t *token_mask, const float *dloss, xmoe_dtype dtype,
                                   int64_t T, int32_t d, int32_t E, int32_t k, float inv_temperature,
                                   int32_t accumulate, void *dx, float *dwg, void *workspace, size_t ws_bytes,
                                   void *stream) {
    TRY(check_dtype(dtype));
    TRY(check_balance(logits, seq_offsets, T, E, n_seq));
    REQUIRE(wg && dwg && (T == 0 || (x && topk_ids && dtopk_w && dx && coef)), XMOE_ERR_INVALID_VALUE,
            "a required pointer is NULL");
    REQUIRE(d >= 1, XMOE_ERR_INVALID_VALUE, "d must be >= 1");
    REQUIRE(k >= 1 && k <= E && ldw >= k, XMOE_ERR_INVALID_VALUE, "k must be in [1, E] and ldw >= k");
    REQUIRE(within(T, ldw, kMaxRows), XMOE_ERR_INVALID_VALUE, "T*ldw must be < 2^31");
    if (dtype == XMOE_BF16) {
        REQUIRE(d % 8 == 0 && E % 8 == 0, XMOE_ERR_UNSUPPORTED, "the bf16 gate needs d and E multiples of 8");
        REQUIRE(aligned16(x) && aligned16(wg) && aligned16(dx), XMOE_ERR_UNSUPPORTED,
                "x, wg and dx must be 16-byte aligned");
    }
    REQUIRE(workspace && aligned16(workspace), XMOE_ERR_WORKSPACE, "workspace is NULL or not 16-byte aligned");
    REQUIRE(ws_bytes >= xmoe::route_bwd_workspace(T, d, E, dtype), XMOE_ERR_WORKSPACE,
            "workspace too small (see xmoe_route_bwd_workspace_size)");
    CHECK_DEVICE();
    return hip_status(xmoe::launch_route_bwd_balance(dtype, x, wg, logits, topk_ids, dtopk_w, ldw, T, d, E, k,
                                                     inv_temperature, accumulate != 0,
                                                     {seq_offsets, n_seq, token_mask, coef, dloss}, dx, dwg, workspace,
                                                     S(stream)),
                      "xmoe_route_bwd_balance launch");
}

xmoe_status xmoe_mx8_quantize(const void *x, xmoe_dtype dtype, int64_t n, int32_t K, void *q, void *scale,
                              void *stream) {
    TRY(check_dtype(dtype));
    TRY(check_mx8_rows(n, K));
    REQUIRE(n == 0 || (x && q && scale), XMOE_ERR_INVALID_VALUE, "x, q and scale are required");
    REQUIRE(aligned16(x) && aligned16(q) && aligned16(scale), XMOE_ERR_UNSUPPORTED, "matrices must be 16-byte aligned");
    REQUIRE(!overlap(q, n * K, x, n * K * (dtype == XMOE_BF16 ? 2 : 4)), XMOE_ERR_INVALID_VALUE,
            "q must not overlap x");
    CHECK_DEVICE();
    return hip_status(xmoe::launch_mx8_quantize(dtype, x, n, K, q, scale, S(stream)), "xmoe_mx8_quantize launch");
}

xmoe_status xmoe_mx8_dequantize(const void *q, const void *scale, xmoe_dtype dtype, int64_t n, int32_t K, void *out,
                                void *stream) {
    TRY(check_dtype(dtype));
    TRY(check_mx8_rows(n, K));
    REQUIRE(n == 0 || (q && scale && out), XMOE_ERR_INVALID_VALUE, "q, scale and out are required");
    REQUIRE(aligned16(q) && aligned16(scale) && aligned16(out), XMOE_ERR_UNSUPPORTED,
            "matrices must be 16-byte aligned");
    CHECK_DEVICE();
    return hip_status(xmoe::launch_mx8_dequantize(dtype, q, scale, n, K, out, S(stream)),
                      "xmoe_mx8_dequantize launch");
}

xmoe_status xmoe_mx8_quantize_weights(const void *w, xmoe_dtype dtype, int32_t E, int32_t K, int32_t N, void *q,
                                      void *scale, void *stream) {
    TRY(check_dtype(dtype));
    REQUIRE(w && q && scale, XMOE_ERR_INVALID_VALUE, "w, q and scale are required");
    REQUIRE(E >= 1 && E <= 1024 && K >= 1 && N >= 1, XMOE_ERR_INVALID_VALUE,
            "E must be in [1, 1024], K and N >= 1");
    REQUIRE(K % 32 == 0 && N % 32 == 0, XMOE_ERR_UNSUPPORTED, "K and N must be multiples of 32");
    REQUIRE(K <= kMaxMx8Dim && N <= kMaxMx8Dim, XMOE_ERR_UNSUPPORTED, "K and N must be at most %d", kMaxMx8Dim);
    // blocks of 128 x 64: their threads stay below 2^32
    REQUIRE(within(static_cast<int64_t>(E) * ((K + 127) / 128), (N + 63) / 64, (int64_t{1} << 24) - 1),
            XMOE_ERR_UNSUPPORTED, "E * ceil(K / 128) * ceil(N / 64) must be < 2^24");
    REQUIRE(aligned16(w) && aligned16(q) && aligned16(scale), XMOE_ERR_UNSUPPORTED, "matrices must be 16-byte aligned");
    CHECK_DEVICE();
    return hip_status(xmoe::launch_mx8_quantize_weights(dtype, w, E, K, N, q, scale, S(stream)),
                      "xmoe_mx8_quantize_weights launch");
}

xmoe_status xmoe_expert_ffn_up_mx8(const void *xq, const void *xscale, const int32_t *token_ids, int64_t T,
                                   const void *w1, const void *w1_scale, const void *w3, const void *w3_scale,
                                   const int32_t *expert_offsets, int32_t E, int64_t rows, int32_t d, int32_t h,
                                   void *act, void *act_scale, void *stream) {
    TRY(check_mx8_ffn(expert_offsets, E, rows, d, h));
    REQUIRE(w1 && w1_scale && w3 && w3_scale && (rows == 0 || (xq && xscale && act && act_scale)),
            XMOE_ERR_INVALID_VALUE, "a required pointer is NULL");
    if (token_ids) {
        REQUIRE(T >= 0 && (rows == 0 || T >= 1), XMOE_ERR_INVALID_VALUE,
                "T must be >= 1 when there are rows to gather");
        // gathered rows are addressed with 32-bit offsets
        REQUIRE(within(T, d, (int64_t{1} << 31) - 1), XMOE_ERR_UNSUPPORTED,
                "xq must be smaller than 2^31 bytes to be gathered");
    } else {
        REQUIRE(T == rows, XMOE_ERR_INVALID_VALUE, "without token_ids T must equal rows");
    }
    REQUIRE(aligned16(xq) && aligned16(xscale) && aligned16(w1) && aligned16(w1_scale) && aligned16(w3) &&
                aligned16(w3_scale) && aligned16(act) && aligned16(act_scale),
            XMOE_ERR_UNSUPPORTED, "matrices must be 16-byte aligned");
    CHECK_DEVICE();
    return hip_status(xmoe::launch_ffn_up_mx8(xq, xscale, token_ids, T, w1, w1_scale, w3, w3_scale, expert_offsets, E,
                                              rows, d, h, act, act_scale, S(stream)),
                      "xmoe_expert_ffn_up_mx8 launch");
}

xmoe_status xmoe_expert_ffn_down_mx8(const void *act, const void *act_scale, const void *w2, const void *w2_scale,
                                     const int32_t *expert_offsets, int32_t E, int64_t rows, int32_t d, int32_t h,
                                     void *ye, void *stream) {
    TRY(check_mx8_ffn(expert_offsets, E, rows, d, h));
    REQUIRE(w2 && w2_scale && (rows == 0 || (act && act_scale && ye)), XMOE_ERR_INVALID_VALUE,
            "a required pointer is NULL");
    REQUIRE(aligned16(act) && aligned16(act_scale) && aligned16(w2) && aligned16(w2_scale) && aligned16(ye),
            XMOE_ERR_UNSUPPORTED, "matrices must be 16-byte aligned");
    CHECK_DEVICE();
    return hip_status(xmoe::launch_ffn_down_mx8(act, act_scale, w2, w2_scale, expert_offsets, E, rows, d, h, ye,
                                                S(stream)),
                      "xmoe_expert_ffn_down_mx8 launch");
}

}  // extern "C"

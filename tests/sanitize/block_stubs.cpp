// No-op launchers of the calls around the layer (norm, balance loss, 8-bit
// experts), beside those of launch_stubs.cpp, so that api_block.cpp's host code
// can be built and run under the host sanitizers without any device code.
#include <hip/hip_runtime.h>

#include "../../padding_free_expert_amd/csrc/kernels.hpp"

namespace xmoe {

size_t balance_workspace(int64_t T, int E, int S) { return static_cast<size_t>((T / 16 + S) * E * 8 + 64); }
hipError_t launch_balance_loss(const float *, const int32_t *, int64_t, int, int, const int32_t *, int, const uint8_t *,
                               float, float *, int32_t *, float *, void *, hipStream_t) { return hipSuccess; }
hipError_t launch_balance_loss_bwd(const float *, int64_t, int, const BalanceArgs &, float *, hipStream_t) {
    return hipSuccess;
}
hipError_t launch_route_bwd_balance(int, const void *, const void *, const float *, const int32_t *, const float *, int,
                                    int64_t, int, int, int, float, bool, const BalanceArgs &, void *, float *, void *,
                                    hipStream_t) { return hipSuccess; }
hipError_t launch_add_rmsnorm(int, const void *, const void *, const void *, int64_t, int, float, void *, void *, void *,
                              void *, float *, hipStream_t) { return hipSuccess; }
size_t add_rmsnorm_bwd_workspace(int64_t, int d, int) { return static_cast<size_t>(d) * 4 * 64; }
hipError_t launch_add_rmsnorm_bwd(int, const void *, const void *, const void *, const void *, const float *, int64_t, int,
                                  void *, float *, void *, hipStream_t) { return hipSuccess; }
hipError_t launch_mx8_quantize(int, const void *, int64_t, int, void *, void *, hipStream_t) { return hipSuccess; }
hipError_t launch_mx8_dequantize(int, const void *, const void *, int64_t, int, void *, hipStream_t) {
    return hipSuccess;
}
hipError_t launch_mx8_quantize_weights(int, const void *, int, int, int, void *, void *, hipStream_t) {
    return hipSuccess;
}
hipError_t launch_ffn_up_mx8(const void *, const void *, const int32_t *, int64_t, const void *, const void *,
                             const void *, const void *, const int32_t *, int, int64_t, int, int, void *, void *,
                             hipStream_t) { return hipSuccess; }
hipError_t launch_ffn_down_mx8(const void *, const void *, const void *, const void *, const int32_t *, int, int64_t, int,
                               int, void *, hipStream_t) { return hipSuccess; }

}  // namespace xmoe

// No-op launchers of the layer for a few tokens and of the FFN with 8-bit
// pre-activations, so that api_few.cpp and api_ckpt8.cpp can be built and run under the
// host sanitizers without any device code.
#include <hip/hip_runtime.h>

#include "../../padding_free_expert_amd/csrc/few.hpp"
#include "../../padding_free_expert_amd/csrc/kernels.hpp"

namespace xmoe {

size_t few_workspace(const FewSizes &z) { return static_cast<size_t>(z.T) * (z.d + static_cast<int64_t>(z.k) * z.h) * 4; }
hipError_t launch_layer_few(const FewSizes &, const FewTensors &, hipStream_t) { return hipSuccess; }
hipError_t launch_ffn_up_ckpt8(int, const void *, const int32_t *, int64_t, const void *, const void *, const int32_t *,
                               int, int64_t, int, int, void *, void *, void *, hipStream_t) { return hipSuccess; }
hipError_t launch_ckpt8_dequantize(int, const void *, const void *, int64_t, int, void *, hipStream_t) {
    return hipSuccess;
}
hipError_t launch_ffn_bwd_dact_ckpt8(int, const void *, const int32_t *, int64_t, const float *, const void *,
                                     const void *, const void *, const int32_t *, int, int64_t, int, int, void *, void *,
                                     const int32_t *, float *, void *, hipStream_t) { return hipSuccess; }

}  // namespace xmoe

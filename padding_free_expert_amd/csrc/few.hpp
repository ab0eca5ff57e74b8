// The whole layer for a few tokens (few.hip): what its launcher takes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace xmoe {

constexpr int kFewTokens = 64;

struct FewSizes {
    int dt;      // rows, gate and output
    bool mx8;    // the experts' weights and their rows in 8 bits
    int64_t T;
    int d, E, k, h, hs;  // hs: width of the shared experts side by side, 0: none
};

struct FewWeights {
    const void *w1, *w3, *w2, *w1s, *w3s, *w2s;  // scales with 8 bits only
};

struct FewTensors {
    const void *x, *xq, *xs, *wg;
    FewWeights routed, shared;
    float scale;
    const float *lbias, *sbias;
    int32_t *ids;
    float *w, *logits;
    void *y, *ws;
};

size_t few_workspace(const FewSizes &z);
hipError_t launch_layer_few(const FewSizes &z, const FewTensors &t, hipStream_t s);

}  // namespace xmoe

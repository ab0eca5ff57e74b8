// Pre-activations kept in 8 bits for the backward ("ckpt8"): whole numbers of
// -127..127 times a power of two, one scale byte b = 2^(b - 127) for each 32
// consecutive columns of a row (the last block of a row may be shorter).
//
// The scale is the least power of two that brings the block's largest magnitude to at
// most 127; elements then take one round-to-nearest-even.  A whole number's step is the
// same for every element of a block, 1/127 to 1/63.5 of its largest: the backward
// multiplies H3 and the slope of silu(H1) with gradients, where an element's own error
// counts, not its relative one.  For normal values (columns of one size) a block's error
// is 0.6% of its norm, against 2.6% for e4m3 with the same scales and bytes.  Seven bits
// and a power of two are exact in bf16, too.  An all-zero block has b = 127; one that
// holds an infinity or a NaN has b = 255 and stands for NaNs.
#pragma once

#include "common.hpp"

namespace xmoe {

// Scale byte of a block from the largest bit pattern of its magnitudes (integer order:
// finite < infinity < NaN).  amax = m 2^x, 1 <= m < 2, and 127 = 1.984375 * 2^6: the
// exponent is x - 6, one more where m > 1.984375, clamped at 2^-127 (below which the
// step is 2^-127 itself).
__device__ __forceinline__ uint32_t ck8_scale_byte(uint32_t amax_bits) {
    const int e = static_cast<int>(amax_bits >> 23) - 6 + ((amax_bits & 0x7fffffu) > 0x7e0000u ? 1 : 0);
    uint32_t b = static_cast<uint32_t>(max(e, 0));
    b = amax_bits == 0u ? 127u : b;
    return amax_bits >= 0x7f800000u ? 255u : b;
}

// 2^(127 - b); for b = 255 anything finite (the block stands for NaNs by its scale)
__device__ __forceinline__ float ck8_inv_scale(uint32_t b) {
    return __uint_as_float(b == 255u ? 0u : (254u - b) << 23);
}

// 2^(b - 127); b = 0 is fp32's subnormal 2^-127, b = 255 a NaN
__device__ __forceinline__ float ck8_scale(uint32_t b) {
    return __uint_as_float(b == 255u ? 0x7fc00000u : b == 0u ? 0x00400000u : b << 23);
}

// Four elements -> four signed bytes (first in bits 0..7).  Adding 1.5 * 2^23 rounds the
// scaled value to a whole number (to nearest even, the product being exact) and leaves
// it in the low bits.
__device__ __forceinline__ uint32_t ck8_pack4(float a, float b, float c, float d, float inv) {
    const uint32_t x = __float_as_uint(__builtin_fmaf(a, inv, 12582912.0f)), y = __float_as_uint(__builtin_fmaf(b, inv, 12582912.0f));
    const uint32_t z = __float_as_uint(__builtin_fmaf(c, inv, 12582912.0f)), w = __float_as_uint(__builtin_fmaf(d, inv, 12582912.0f));
    return __builtin_amdgcn_perm(__builtin_amdgcn_perm(w, z, 0x0c0c0400u), __builtin_amdgcn_perm(y, x, 0x0c0c0400u), 0x05040100u);
}

// Four signed bytes times the scale, exact.
__device__ __forceinline__ void ck8_unpack4(uint32_t q, float s, float *f) {
    const uint32_t u = q ^ 0x80808080u;  // 128 more, without a sign
    f[0] = (static_cast<float>(u & 255u) - 128.0f) * s;
    f[1] = (static_cast<float>((u >> 8) & 255u) - 128.0f) * s;
    f[2] = (static_cast<float>((u >> 16) & 255u) - 128.0f) * s;
    f[3] = (static_cast<float>(u >> 24) - 128.0f) * s;
}

}  // namespace xmoe

// 8-bit rows with block scales ("mx8"): e4m3 elements (4 significant bits, at
// most 448), one scale byte b = 2^(b - 127) for each 32 consecutive elements of
// the summed axis -- the operand form of gfx950's scaled matrix instructions.
//
// The scale of a block is the least power of two that brings its largest
// magnitude to at most 448, so no element saturates; elements then take one
// round-to-nearest-even.  A power of two leaves the division exact, so that
// rounding is the only one.  A block whose elements are all zero has b = 127;
// one that holds an infinity or a NaN has b = 255 (the NaN of the scale format)
// and stands for NaNs.  Scales of n rows of K elements lie as
// [ceil(K / 128), n, 4]: the four bytes that a 128-deep k step of one row needs
// are one dword, and the dwords of consecutive rows are consecutive, so a
// matrix instruction's scale operand is one coalesced load.  The bytes past
// K / 32 in the last group are 127.
#pragma once

#include "common.hpp"

namespace xmoe {

constexpr int kMxBlock = 32;
constexpr uint32_t kMxOne = 127u;

// Scale byte of a block from the largest bit pattern of its magnitudes
// (integer order: finite < infinity < NaN).  With amax = m 2^x, 1 <= m < 2, and
// 448 = 1.75 * 2^8, the exponent is x - 8, one more where m > 1.75; it is
// clamped at 2^-127, where magnitudes below 448 * 2^-127 lose nothing but
// range that fp32 holds as subnormals.
__device__ __forceinline__ uint32_t mx8_scale_byte(uint32_t amax_bits) {
    const int e = static_cast<int>(amax_bits >> 23) - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    uint32_t b = static_cast<uint32_t>(max(e, 0));
    b = amax_bits == 0u ? kMxOne : b;
    return amax_bits >= 0x7f800000u ? 255u : b;
}

// 2^(127 - b), what the elements are multiplied by (b <= 247 in finite blocks);
// a NaN for b = 255, so that every element becomes one
__device__ __forceinline__ float mx8_inv_scale(uint32_t b) {
    return __uint_as_float(b == 255u ? 0x7fc00000u : (254u - b) << 23);
}

// 2^(b - 127); b = 0 is fp32's subnormal 2^-127, b = 255 a NaN
__device__ __forceinline__ float mx8_scale(uint32_t b) {
    return __uint_as_float(b == 255u ? 0x7fc00000u : b == 0u ? 0x00400000u : b << 23);
}

// four elements -> four e4m3 bytes (first in bits 0..7), already multiplied by 2^(127 - b)
__device__ __forceinline__ uint32_t mx8_pack4(float a, float b, float c, float d) {
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    v = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
    return static_cast<uint32_t>(v);
}

// V elements of one lane, 32 / V consecutive lanes holding a block: the block's
// scale byte (the same in its lanes) and the lane's V bytes in out[V / 4].
// Every lane of the wavefront takes part; a lane without elements passes zeros.
template <int V>
__device__ __forceinline__ uint32_t mx8_quant(const float (&f)[V], uint32_t (&out)[V / 4]) {
    uint32_t a = 0u;
#pragma unroll
    for (int i = 0; i < V; ++i) a = max(a, __float_as_uint(f[i]) & 0x7fffffffu);
#pragma unroll
    for (int off = 1; off < kMxBlock / V; off <<= 1) a = max(a, static_cast<uint32_t>(__shfl_xor(static_cast<int>(a), off, 64)));
    const uint32_t b = mx8_scale_byte(a);
    const float s = mx8_inv_scale(b);
#pragma unroll
    for (int i = 0; i < V; i += 4)
        out[i / 4] = mx8_pack4(f[i] * s, f[i + 1] * s, f[i + 2] * s, f[i + 3] * s);
    return b;
}

// The dword of four consecutive blocks' scale bytes, in every one of their
// 128 / V lanes (their first lane is a multiple of 128 / V).
template <int V>
__device__ __forceinline__ uint32_t mx8_scale_dword(uint32_t b, int lane) {
    constexpr int L = kMxBlock / V;  // lanes of a block
    int w = static_cast<int>(b << (8 * ((lane / L) & 3)));
    w |= __shfl_xor(w, L, 64);
    w |= __shfl_xor(w, 2 * L, 64);
    return static_cast<uint32_t>(w);
}

}  // namespace xmoe

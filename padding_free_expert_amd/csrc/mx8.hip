// Expert FFN on 8-bit rows and weights with block scales, and the kernels that
// bring values into that form and back (mx8.hpp describes it).
//
//   up    act = mx8(silu(x . W1) * (x . W3))   x rows gathered by token id
//   down  ye = act . W2                        bf16
// Weights are held [E, N, K] -- the summed axis last, where the scales group it
// and where both operands of a matrix instruction read 16 consecutive bytes.
//
// v_mfma_scale_f32_16x16x128 takes per lane 32 bytes of one row of each operand
// and one scale byte for each.  Lane l holds row l % 16; the 16-byte chunks of
// the row's 128 that it carries are l / 16 and 4 + l / 16, and the scale of the
// row's s-th 32 elements is the one that lane group s holds (both checked
// against the instruction on the card).  So one lane's dword of a row's four
// scales, shifted by 8 (l / 16), serves it.
#include <algorithm>

#include "common.hpp"
#include "gemm.hpp"
#include "kernels.hpp"
#include "mx8.hpp"

namespace xmoe {

namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

// ------------------------------------------------------- into and out of 8 bits

// One wave per row and 64 16-byte vectors; rows are independent.
template <typename T>
__global__ __launch_bounds__(256) void mx8_quantize_kernel(const T *__restrict__ x, int64_t n, int K, int segs,
                                                           uint8_t *__restrict__ q, uint8_t *__restrict__ scale) {
    constexpr int V = Elem<T>::kVec;
    const int lane = threadIdx.x & 63;
    const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
    const int64_t row = w / segs;
    if (row >= n) return;  // whole waves
    const int c = static_cast<int>(w - row * segs) * 64 + lane;
    const bool in = c < K / V;
    float f[V];
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] = 0.0f;
    if (in) Elem<T>::unpack(reinterpret_cast<const uint4 *>(x + row * K)[c], f);
    uint32_t o[V / 4];
    const uint32_t b = mx8_quant<V>(f, o);
    const uint32_t d = mx8_scale_dword<V>(in ? b : kMxOne, lane);
    if (!in) return;
    uint32_t *dst = reinterpret_cast<uint32_t *>(q + row * K + static_cast<int64_t>(c) * V);
    if constexpr (V == 8) *reinterpret_cast<uint2 *>(dst) = make_uint2(o[0], o[1]);
    else *dst = o[0];
    if (c % (128 / V) == 0)
        *reinterpret_cast<uint32_t *>(scale + (static_cast<int64_t>(c / (128 / V)) * n + row) * 4) = d;
}

// Four e4m3 values of a dword times the block's scale (exact in fp32, and in
// bf16, whose 8 significant bits hold the 4)
__device__ __forceinline__ void mx8_unpack4(uint32_t v, float s, float *f) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    const f2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(v), false);
    const f2 hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(v), true);
    f[0] = lo[0] * s; f[1] = lo[1] * s; f[2] = hi[0] * s; f[3] = hi[1] * s;
}

template <typename T>
__global__ __launch_bounds__(256) void mx8_dequantize_kernel(const uint8_t *__restrict__ q,
                                                             const uint8_t *__restrict__ scale, int64_t n, int K,
                                                             T *__restrict__ out) {
    constexpr int V = Elem<T>::kVec;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;  // 16 elements each
    const int per = K / 16;
    const int64_t row = i / per;
    if (row >= n) return;
    const int c = static_cast<int>(i - row * per);
    const int g = c / 2;  // 32-element block
    const float s = mx8_scale(scale[(static_cast<int64_t>(g >> 2) * n + row) * 4 + (g & 3)]);
    const uint4 v = reinterpret_cast<const uint4 *>(q + row * K)[c];
    float f[16];
    mx8_unpack4(v.x, s, f);
    mx8_unpack4(v.y, s, f + 4);
    mx8_unpack4(v.z, s, f + 8);
    mx8_unpack4(v.w, s, f + 12);
    uint4 *dst = reinterpret_cast<uint4 *>(out + row * K + static_cast<int64_t>(c) * 16);
#pragma unroll
    for (int j = 0; j < 16 / V; ++j) dst[j] = Elem<T>::pack(f + j * V);
}

// w [E, K, N] -> q [E, N, K]: a block takes 128 of K by 64 of N through LDS
// (rows of 65 floats: the column reads of 64 lanes then meet 64 banks); thread
// (column, 32-element block) forms one scale and 32 bytes.
template <typename T>
__global__ __launch_bounds__(256) void mx8_quantize_weights_kernel(const T *__restrict__ w, int K, int N,
                                                                   uint8_t *__restrict__ q,
                                                                   uint8_t *__restrict__ scale) {
    constexpr int V = Elem<T>::kVec;
    __shared__ float s[128][65];
    const int tn = (N + 63) / 64, tk = (K + 127) / 128;
    const int64_t b = blockIdx.x;
    const int e = static_cast<int>(b / (static_cast<int64_t>(tn) * tk));
    const int rem = static_cast<int>(b - static_cast<int64_t>(e) * tn * tk);
    const int k0 = (rem / tn) * 128, n0 = (rem % tn) * 64;
    const T *src = w + static_cast<int64_t>(e) * K * N;
    for (int i = threadIdx.x; i < 128 * 64 / V; i += 256) {
        const int k = i / (64 / V), n = (i % (64 / V)) * V;
        float f[V];
#pragma unroll
        for (int v = 0; v < V; ++v) f[v] = 0.0f;
        if (k0 + k < K && n0 + n < N)
            Elem<T>::unpack(*reinterpret_cast<const uint4 *>(src + static_cast<int64_t>(k0 + k) * N + n0 + n), f);
#pragma unroll
        for (int v = 0; v < V; ++v) s[k][n + v] = f[v];
    }
    __syncthreads();
    const int n = n0 + (threadIdx.x & 63), g = threadIdx.x >> 6;  // column, 32-element block
    if (n >= N) return;
    uint32_t a = 0u;
#pragma unroll
    for (int i = 0; i < 32; ++i) a = max(a, __float_as_uint(s[32 * g + i][threadIdx.x & 63]) & 0x7fffffffu);
    const bool in = k0 + 32 * g < K;
    const uint32_t byte = in ? mx8_scale_byte(a) : kMxOne;
    scale[((static_cast<int64_t>(e) * tk + k0 / 128) * N + n) * 4 + g] = static_cast<uint8_t>(byte);
    if (!in) return;
    const float m = mx8_inv_scale(byte);
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float *p = &s[32 * g + 4 * i][threadIdx.x & 63];
        o[i] = byte == 255u ? 0x7f7f7f7fu : mx8_pack4(p[0] * m, p[65] * m, p[130] * m, p[195] * m);
    }
    uint4 *dst = reinterpret_cast<uint4 *>(q + (static_cast<int64_t>(e) * N + n) * K + k0 + 32 * g);
    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

// ------------------------------------------------------------------ products

struct Mx8Args {
    GemmArgs g;                 // what resolve_tile reads: GM_ROWS, offsets, G, extent, N
    int K;
    const uint8_t *a, *as;      // rows [a_rows, K] and scales [ceil(K / 128), a_rows, 4]
    int64_t a_rows;
    const int32_t *map;         // row r of the experts' rows is row map[r] of a; nullptr: row r
    const uint8_t *b0, *b0s, *b1, *b1s;  // weights [G, N, K] and scales [G, ceil(K / 128), N, 4]
    uint8_t *q, *qs;            // up: act [rows, N] and its scales
    bf16_t *y;                  // down: ye [rows, N]
};

__device__ __forceinline__ i32x8_t frag8(uint4 lo, uint4 hi) {
    return i32x8_t{static_cast<int>(lo.x), static_cast<int>(lo.y), static_cast<int>(lo.z), static_cast<int>(lo.w),
                   static_cast<int>(hi.x), static_cast<int>(hi.y), static_cast<int>(hi.z), static_cast<int>(hi.w)};
}

// Few rows per expert: the weights are streamed past the rows once.  A block
// takes 16 MT rows by 32 columns of one expert (of W1 and of W3 for the
// up-projection, NB = 2) and its KW waves split the summed axis in 128-deep
// steps; operands go from memory straight to registers, since no other wave of
// the block needs them.  The waves' partial sums meet in LDS, added in wave
// order.
template <int NB, int MT, int KW>
__global__ __launch_bounds__(64 * KW) void mx8_stream_kernel(Mx8Args p) {
    constexpr int BM = 16 * MT, BN = 32;
    constexpr int NF = NB * 2 * MT;  // 16 x 16 results of a wave
    __shared__ f32x4_t part[KW][NF][64];
    static_assert(sizeof(part) <= 64 * 1024, "partial sums");
    static_assert(KW >= MT, "one wave for each 16 rows of the result");
    Tile t;
    if (!resolve_tile<BM, BN>(p.g, &t, blockIdx.x, gridDim.x)) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int l16 = lane & 15, quad = lane >> 4;
    const int N = p.g.N, K = p.K, kb = (K + 127) / 128;
    const int n0 = t.nt * BN;

    // this lane's rows of both operands
    const uint8_t *ap[MT], *asp[MT];
    bool arow[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int m = t.m0 + 16 * i + l16;
        arow[i] = m < t.Mg;
        int64_t r = arow[i] ? t.base + m : 0;
        if (arow[i] && p.map) {
            r = p.map[r];
            if (r < 0 || r >= p.a_rows) {  // outside the rows: a row of zeros
                arow[i] = false;
                r = 0;
            }
        }
        ap[i] = p.a + r * K + 16 * quad;
        asp[i] = p.as + r * 4;
    }
    const uint8_t *bp[NB][2], *bsp[NB][2];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int n = n0 + 16 * j + l16;
            bp[b][j] = (b ? p.b1 : p.b0) + (static_cast<int64_t>(t.g) * N + n) * K + 16 * quad;
            bsp[b][j] = (b ? p.b1s : p.b0s) + (static_cast<int64_t>(t.g) * kb * N + n) * 4;
        }
    f32x4_t acc[NB][2][MT];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < MT; ++i) acc[b][j][i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

    const uint4 zero = make_uint4(0, 0, 0, 0);
    auto load = [&](const uint8_t *q, int64_t k, bool lo, bool hi) {
        return frag8(lo ? *reinterpret_cast<const uint4 *>(q + k) : zero,
                     hi ? *reinterpret_cast<const uint4 *>(q + k + 64) : zero);
    };
    // one 128-deep step; TAIL: K ends inside it (elements past K are zeros)
    auto step = [&](int s, auto tail) {
        constexpr bool TAIL = decltype(tail)::value;
        const int64_t k = static_cast<int64_t>(s) * 128;
        const bool lo = !TAIL || k + 16 * quad < K, hi = !TAIL || k + 64 + 16 * quad < K;
        i32x8_t fb[NB][2], fa[MT];
        int sb[NB][2], sa[MT];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                fb[b][j] = load(bp[b][j], k, lo, hi);
                sb[b][j] = *reinterpret_cast<const int *>(bsp[b][j] + static_cast<int64_t>(s) * N * 4);
            }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            fa[i] = load(ap[i], k, lo && arow[i], hi && arow[i]);
            sa[i] = *reinterpret_cast<const int *>(asp[i] + static_cast<int64_t>(s) * p.a_rows * 4);
            if (!arow[i]) sa[i] = 0x7f7f7f7f;
        }
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < MT; ++i)
                    acc[b][j][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        fb[b][j], fa[i], acc[b][j][i], 0, 0, 0, sb[b][j] >> (8 * quad), 0, sa[i] >> (8 * quad));
    };
    const int full = K / 128;
    for (int s = wave; s < full; s += KW) step(s, std::false_type{});
    if (full < kb && full % KW == wave) step(full, std::true_type{});

#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < MT; ++i) part[wave][(b * 2 + j) * MT + i][lane] = acc[b][j][i];
    __syncthreads();
    if (wave >= MT) return;
    // wave i: rows 16 i .. 16 i + 15; lane l has row l % 16, columns 16 j + 4 (l / 16) + r
    const int m = t.m0 + 16 * wave + l16;
    const int64_t row = t.base + m;
    const bool live = m < t.Mg;
    f32x4_t v[NB][2];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int f = (b * 2 + j) * MT + wave;
            v[b][j] = part[0][f][lane];
#pragma unroll
            for (int w = 1; w < KW; ++w) v[b][j] += part[w][f][lane];
        }
    if constexpr (NB == 2) {
        float o[8];
        uint32_t a = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            o[i] = silu_f(v[0][i / 4][i % 4]) * v[1][i / 4][i % 4];
            a = max(a, __float_as_uint(o[i]) & 0x7fffffffu);
        }
        a = max(a, static_cast<uint32_t>(__shfl_xor(static_cast<int>(a), 16, 64)));
        a = max(a, static_cast<uint32_t>(__shfl_xor(static_cast<int>(a), 32, 64)));
        const uint32_t byte = mx8_scale_byte(a);
        const float sc = mx8_inv_scale(byte);
        if (live) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
                *reinterpret_cast<uint32_t *>(p.q + row * N + n0 + 16 * j + 4 * quad) =
                    byte == 255u ? 0x7f7f7f7fu
                                 : mx8_pack4(o[4 * j] * sc, o[4 * j + 1] * sc, o[4 * j + 2] * sc, o[4 * j + 3] * sc);
            // the scale byte of this block of 32 columns; the last block also fills its group
            const int blk = n0 / 32;
            const int at = (blk & 3) + quad;
            if (quad == 0 || (n0 + 32 >= N && at < 4))
                p.qs[(static_cast<int64_t>(blk >> 2) * p.g.extent + row) * 4 + at] =
                    static_cast<uint8_t>(quad == 0 ? byte : kMxOne);
        }
    } else if (live) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
            *reinterpret_cast<uint2 *>(p.y + row * N + n0 + 16 * j + 4 * quad) =
                make_uint2(pack_bf16x2(v[0][j][0], v[0][j][1]), pack_bf16x2(v[0][j][2], v[0][j][3]));
    }
}

template <int NB, int MT, int KW>
hipError_t launch_stream(const Mx8Args &p, hipStream_t s) {
    // no expert without rows has a tile: at most rows / BM whole ones and one
    // more for each expert that has rows
    const int64_t tiles = p.g.extent / (16 * MT) + std::min<int64_t>(p.g.G, p.g.extent);
    const int64_t grid = tiles * (p.g.N / 32);
    if (grid <= 0) return hipSuccess;
    hipLaunchKernelGGL((mx8_stream_kernel<NB, MT, KW>), dim3(static_cast<unsigned>(grid)), dim3(64 * KW), 0, s, p);
    return hipGetLastError();
}

Mx8Args rows_args(const int32_t *offsets, int E, int64_t rows, int N, int K) {
    Mx8Args p{};
    p.g.group_mode = GM_ROWS;
    p.g.offsets = offsets;
    p.g.G = E;
    p.g.extent = rows;
    p.g.nphase = 1;
    p.g.N = N;
    p.g.K = K;
    p.K = K;
    return p;
}

template <int NB>
hipError_t product(const Mx8Args &p, hipStream_t s) {
    return launch_stream<NB, 2, 8>(p, s);
}

}  // namespace

hipError_t launch_mx8_quantize(int dt, const void *x, int64_t n, int K, void *q, void *scale, hipStream_t s) {
    if (n <= 0) return hipSuccess;
    const int V = dt == kBF16 ? 8 : 4;
    const int segs = (K / V + 63) / 64;
    const dim3 grid(static_cast<unsigned>((n * segs + 3) / 4)), block(256);
    auto *qb = static_cast<uint8_t *>(q), *sb = static_cast<uint8_t *>(scale);
    if (dt == kBF16)
        hipLaunchKernelGGL(mx8_quantize_kernel<bf16_t>, grid, block, 0, s, static_cast<const bf16_t *>(x), n, K, segs, qb, sb);
    else
        hipLaunchKernelGGL(mx8_quantize_kernel<float>, grid, block, 0, s, static_cast<const float *>(x), n, K, segs, qb, sb);
    return hipGetLastError();
}

hipError_t launch_mx8_dequantize(int dt, const void *q, const void *scale, int64_t n, int K, void *out,
                                 hipStream_t s) {
    if (n <= 0) return hipSuccess;
    const dim3 grid(static_cast<unsigned>((n * (K / 16) + 255) / 256)), block(256);
    auto *qb = static_cast<const uint8_t *>(q), *sb = static_cast<const uint8_t *>(scale);
    if (dt == kBF16)
        hipLaunchKernelGGL(mx8_dequantize_kernel<bf16_t>, grid, block, 0, s, qb, sb, n, K, static_cast<bf16_t *>(out));
    else
        hipLaunchKernelGGL(mx8_dequantize_kernel<float>, grid, block, 0, s, qb, sb, n, K, static_cast<float *>(out));
    return hipGetLastError();
}

hipError_t launch_mx8_quantize_weights(int dt, const void *w, int E, int K, int N, void *q, void *scale,
                                       hipStream_t s) {
    const int64_t blocks = static_cast<int64_t>(E) * ((K + 127) / 128) * ((N + 63) / 64);
    const dim3 grid(static_cast<unsigned>(blocks)), block(256);
    auto *qb = static_cast<uint8_t *>(q), *sb = static_cast<uint8_t *>(scale);
    if (dt == kBF16)
        hipLaunchKernelGGL(mx8_quantize_weights_kernel<bf16_t>, grid, block, 0, s, static_cast<const bf16_t *>(w), K, N, qb, sb);
    else
        hipLaunchKernelGGL(mx8_quantize_weights_kernel<float>, grid, block, 0, s, static_cast<const float *>(w), K, N, qb, sb);
    return hipGetLastError();
}

hipError_t launch_ffn_up_mx8(const void *xq, const void *xscale, const int32_t *row_map, int64_t map_rows,
                             const void *w1, const void *w1s, const void *w3, const void *w3s, const int32_t *offsets,
                             int E, int64_t rows, int d, int h, void *act, void *act_scale, hipStream_t s) {
    Mx8Args p = rows_args(offsets, E, rows, h, d);
    p.a = static_cast<const uint8_t *>(xq);
    p.as = static_cast<const uint8_t *>(xscale);
    p.a_rows = row_map ? map_rows : rows;
    p.map = row_map;
    p.b0 = static_cast<const uint8_t *>(w1);
    p.b0s = static_cast<const uint8_t *>(w1s);
    p.b1 = static_cast<const uint8_t *>(w3);
    p.b1s = static_cast<const uint8_t *>(w3s);
    p.q = static_cast<uint8_t *>(act);
    p.qs = static_cast<uint8_t *>(act_scale);
    return product<2>(p, s);
}

hipError_t launch_ffn_down_mx8(const void *act, const void *act_scale, const void *w2, const void *w2s,
                               const int32_t *offsets, int E, int64_t rows, int d, int h, void *ye, hipStream_t s) {
    Mx8Args p = rows_args(offsets, E, rows, d, h);
    p.a = static_cast<const uint8_t *>(act);
    p.as = static_cast<const uint8_t *>(act_scale);
    p.a_rows = rows;
    p.b0 = static_cast<const uint8_t *>(w2);
    p.b0s = static_cast<const uint8_t *>(w2s);
    p.y = static_cast<bf16_t *>(ye);
    return product<1>(p, s);
}

}  // namespace xmoe

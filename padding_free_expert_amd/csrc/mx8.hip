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

typedef int i32x4_t __attribute__((ext_vector_type(4)));
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

// Many rows per expert: 256 x 256 results a block (NB = 2: 128 columns of W1 and
// the same of W3), four waves of 128 x 128, one block per compute unit.  Both
// operands come into an S-slot ring of shared memory by direct loads, 64 bytes
// of K a slot, in the layout and with the swizzle of the bf16 products (a
// 16-byte chunk here is 16 elements instead of 8); the scale dwords of 128 of K
// (two slots) come the same way.  Wave tiles this wide are what the rates ask
// for: per 64 of K a wave reads 16 KiB from shared memory for 16 products of 64
// cycles; 64 x 128 tiles would read 12 KiB for 8, and with the ring's own
// writes shared memory would be busy longer than the matrix cores.
//
// Step `it` multiplies slot it's fragments, already in registers, while those
// of slot it + 1 are read.  It starts with the one wait and barrier of the step:
// slot it + 1 has landed, and every wave has read slot it, which then takes the
// loads of it + S.
template <int NB, int S>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1))) void mx8_tile_kernel(Mx8Args p) {
    constexpr int BM = 256, BN = 256 / NB, WGM = 2, WGN = 2, NW = 4;
    constexpr int WTM = BM / WGM, WTN = BN / WGN, TM = WTM / 32, TN = WTN / 32, TT = NB * TN;
    static_assert(TM == 4 && TT == 4, "sixteen 32 x 32 results a wave");
    using PA = DmaPlan<BM, 32, true, NW>;  // in 2-byte units: 64 bytes of K
    using PB = DmaPlan<BN, 32, true, NW>;
    constexpr int kABytes = PA::kBytes, kBBytes = PB::kBytes, kStage = kABytes + NB * kBBytes;
    constexpr int kL = PA::kN + NB * PB::kN;         // operand loads of a wave per slot
    constexpr int kScales = 512 * 4, kScaleSlots = 4;  // scale dwords of 256 + 256 rows
    constexpr int kRing = S * kStage;
    static_assert(S == 4, "the waits count two slots behind the next, one of each parity");
    static_assert(kRing + kScaleSlots * kScales <= 160 * 1024 - 64, "one block per compute unit");
    __shared__ __align__(1024) char smem[kRing + kScaleSlots * kScales];

    Tile t;
    if (!resolve_tile<BM, BN>(p.g, &t, blockIdx.x, gridDim.x)) return;
    const int N = p.g.N, K = p.K, kb = (K + 127) / 128;
    const int m0 = t.m0, n0 = t.nt * BN;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WGN, wn = wave % WGN, half = lane >> 5;
    const uint32_t sbase = __builtin_amdgcn_readfirstlane(lds_addr(smem));
    const bool wact = m0 + wm * WTM < t.Mg && n0 + wn * WTN < N;
    const int total = (K + 63) / 64;

    // operand loads: rows past the group's or N, and K's end, load zeros
    PA pa;
    PB pb;
    __amdgpu_buffer_rsrc_t ra, rb[NB];
    const int32_t *map = p.map ? p.map + t.base + m0 : nullptr;
    if (map) {
        pa.init_mapped(wave, lane, K / 2, map, t.Mg - m0, K / 2);
#pragma unroll
        for (int i = 0; i < PA::kN; ++i) {  // ids outside the rows: zeros
            const int row = ((i * NW + wave) * 1024 + lane * 16) / PA::kRowBytes;
            const int id = row < t.Mg - m0 ? map[row] : 0;
            if (id < 0 || id >= p.a_rows) pa.lim[i] = INT_MIN;
        }
        ra = make_rsrc(p.a, p.a_rows * K);
    } else {
        pa.init(wave, lane, K / 2, 0, t.Mg - m0, K / 2);
        ra = make_rsrc(p.a + (t.base + m0) * K, static_cast<int64_t>(t.Mg - m0) * K);
    }
    pb.init(wave, lane, K / 2, 0, N - n0, K / 2);
#pragma unroll
    for (int b = 0; b < NB; ++b)
        rb[b] = make_rsrc((b ? p.b1 : p.b0) + (static_cast<int64_t>(t.g) * N + n0) * K, static_cast<int64_t>(N - n0) * K);
    // scale loads: wave w takes rows 64 w .. 64 w + 63 of A's 256 and of B's (of W1 and W3: 128 each)
    int as_off = kOob, bs_off = kOob;
    {
        const int row = 64 * wave + lane;
        if (row < t.Mg - m0) {
            const int64_t id = map ? map[row] : t.base + m0 + row;
            if (id >= 0 && id < p.a_rows) as_off = static_cast<int>(map ? id * 4 : row * 4);
        }
        const int col = NB == 2 ? row & 127 : row;
        if (n0 + col < N) bs_off = col * 4;
    }
    const int64_t as_first = map ? 0 : t.base + m0;
    const uint8_t *bsrc = (NB == 2 && wave >= 2) ? p.b1s : p.b0s;

    auto issue_part = [&](int st, int part) {  // operand load `part` of slot st
        const bool live = st < total;
        const int kc = live ? st * 32 : INT_MAX, kadd = st * 64;
        const uint32_t dst = sbase + (st & (S - 1)) * kStage;
        if (part < PA::kN) {
            pa.issue(ra, kc, kadd, dst, wave, part);
        } else {
            const int b = (part - PA::kN) / PB::kN, i = (part - PA::kN) % PB::kN;
            pb.issue(rb[b], kc, kadd, dst + kABytes + b * kBBytes, wave, i);
        }
    };
    auto issue_scales = [&](int st) {  // even slots: the scales of their 128 of K
        const bool live = st < total;
        const int64_t g = live ? st >> 1 : 0;
        const uint32_t dst = sbase + kRing + ((st >> 1) & (kScaleSlots - 1)) * kScales + wave * 256;
        const __amdgpu_buffer_rsrc_t rsa = make_rsrc(p.as + (g * p.a_rows + as_first) * 4, (p.a_rows - as_first) * 4);
        const __amdgpu_buffer_rsrc_t rsb = make_rsrc(bsrc + ((static_cast<int64_t>(t.g) * kb + g) * N + n0) * 4,
                                                     static_cast<int64_t>(N - n0) * 4);
        lds_dma4(rsa, live ? as_off : kOob, dst);
        lds_dma4(rsb, live ? bs_off : kOob, dst + 1024);
    };

    f32x16_t acc[NB][TM][TN];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[b][i][j][r] = 0.0f;

    // fragment addresses: lane l reads chunks l / 32 and 2 + l / 32 of row l % 32
    // (the swizzle goes by the row modulo 32, so whole 32-row blocks are immediates)
    const int row = lane & 31, sw = swz_kc(row, 4);
    const uint32_t flo = row * 64 + 16 * (half ^ sw), fhi = row * 64 + 16 * ((2 + half) ^ sw);
    i32x8_t fA[2][TM], fB[2][TT];
    int sA[2][TM], sB[2][TT];
    typedef __attribute__((address_space(3))) const i32x4_t lds_i32x4;
    auto frag = [&](uint32_t tile) {
        const i32x4_t lo = *reinterpret_cast<lds_i32x4 *>(static_cast<uintptr_t>(tile + flo));
        const i32x4_t hi = *reinterpret_cast<lds_i32x4 *>(static_cast<uintptr_t>(tile + fhi));
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    };
    auto read_unit = [&](int set, int st, int u) {
        const uint32_t sa = sbase + (st & (S - 1)) * kStage;
        if (u < TM) {
            fA[set][u] = frag(sa + (wm * WTM + 32 * u) * 64);
        } else {
            const int b = (u - TM) / TN, j = (u - TM) % TN;
            fB[set][u - TM] = frag(sa + kABytes + b * kBBytes + (wn * WTN + 32 * j) * 64);
        }
    };
    auto read_scales = [&](int set, int st) {  // the scales of slot st's 128 of K
        const uint32_t ss = sbase + kRing + ((st >> 1) & (kScaleSlots - 1)) * kScales;
#pragma unroll
        for (int i = 0; i < TM; ++i) sA[set][i] = lds_read_i32(ss + (wm * WTM + 32 * i + row) * 4) >> (8 * half);
#pragma unroll
        for (int u = 0; u < TT; ++u)
            sB[set][u] = lds_read_i32(ss + 1024 + ((u / TN) * BN + wn * WTN + 32 * (u % TN) + row) * 4) >> (8 * half);
    };

#pragma unroll
    for (int st = 0; st < S; ++st) {
        if (st % 2 == 0) issue_scales(st);
#pragma unroll
        for (int u = 0; u < kL; ++u) issue_part(st, u);
    }
    wait_vmem<3 * kL + 2>();  // slot 0 has landed (slot 2 brings scales too)
    __syncthreads();
    auto k_loop = [&](auto active) {
        constexpr bool ACT = decltype(active)::value;
        if constexpr (ACT) {
            read_scales(0, 0);
#pragma unroll
            for (int u = 0; u < TM + TT; ++u) read_unit(0, 0, u);
        }
        // P: parity of the slot; Q: of its 128 of K (register sets)
        auto step = [&](int it, auto par, auto grp) {
            constexpr int P = decltype(par)::value, Q = decltype(grp)::value;
            wait_vmem<2 * kL + 2>();  // slots it + 2 and it + 3 may be in flight
            __syncthreads();
            if constexpr (P == 0) issue_scales(it + S);
            if constexpr (ACT && P == 1) read_scales(Q ^ 1, it + 1);
#pragma unroll
            for (int q = 0; q < TM * TT; ++q) {
                const int u = q / TM, i = q % TM;
                if constexpr (ACT) {
                    if (q < TM + TT) read_unit(P ^ 1, it + 1, q);
                    acc[u / TN][i][u % TN] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                        fB[P][u], fA[P][i], acc[u / TN][i][u % TN], 0, 0, 2 * P, sB[Q][u], 2 * P, sA[Q][i]);
                }
                if (q % 2 == 0 && q / 2 < kL) issue_part(it + S, q / 2);
            }
        };
        constexpr std::integral_constant<int, 0> c0{};
        constexpr std::integral_constant<int, 1> c1{};
        for (int it = 0; it < total; it += 4) {
            step(it, c0, c0);
            if (it + 1 < total) step(it + 1, c1, c0);
            if (it + 2 < total) step(it + 2, c0, c1);
            if (it + 3 < total) step(it + 3, c1, c1);
        }
    };
    if (wact) k_loop(std::true_type{});
    else k_loop(std::false_type{});
    wait_vmem<0>();  // no load may still target the ring
    if constexpr (NB == 1) {
        GroupPtrs<bf16_t> q{};
        q.crow = t.base;
        gemm_epilogue<BM, BN, WGM, WGN, 1, kRing, EPI_STORE, bf16_t>(p.g, t, q, acc, smem, sbase, m0, n0, lane, wave);
    } else {
        // lane l: row 32 i + l % 32, columns 32 j + 8 g + 4 (l / 32) + r; a block of
        // 32 columns lies in lanes l and l ^ 32.  The bytes leave through the ring
        // (rows of 144 bytes), 16 at a time, a row's four scale bytes as one dword.
        constexpr int LDC = BN + 16;
        char *const sc = smem + BM * LDC;
        static_assert(BM * LDC + BM * 4 <= kRing, "staging");
        __syncthreads();
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                float o[16];
                uint32_t a = 0u;
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const float h1 = acc[0][i][j][r];
                    o[r] = h1 * __builtin_amdgcn_rcpf(1.0f + __expf(-h1)) * acc[1][i][j][r];
                    a = max(a, __float_as_uint(o[r]) & 0x7fffffffu);
                }
                a = max(a, static_cast<uint32_t>(__shfl_xor(static_cast<int>(a), 32, 64)));
                const uint32_t byte = mx8_scale_byte(a);
                const float s = mx8_inv_scale(byte);
                const int m = wm * WTM + 32 * i + row, c = wn * WTN + 32 * j;
#pragma unroll
                for (int r = 0; r < 16; r += 4)
                    *reinterpret_cast<uint32_t *>(smem + m * LDC + c + 2 * r + 4 * half) =
                        byte == 255u ? 0x7f7f7f7fu : mx8_pack4(o[r] * s, o[r + 1] * s, o[r + 2] * s, o[r + 3] * s);
                // past N: the byte that fills the last group (a NaN row is NaN there too)
                if (half == 0) sc[m * 4 + c / 32] = static_cast<char>(n0 + c < N ? byte : kMxOne);
            }
        __syncthreads();
        const int rows = min(BM, t.Mg - m0);
        for (int c = threadIdx.x; c < rows * (BN / 16); c += 256) {
            const int m = c / (BN / 16), n = 16 * (c % (BN / 16));
            if (n0 + n < N)
                *reinterpret_cast<uint4 *>(p.q + (t.base + m0 + m) * N + n0 + n) =
                    *reinterpret_cast<const uint4 *>(smem + m * LDC + n);
        }
        if (static_cast<int>(threadIdx.x) < rows)
            *reinterpret_cast<uint32_t *>(p.qs + (static_cast<int64_t>(n0 / 128) * p.g.extent + t.base + m0 + threadIdx.x) * 4) =
                *reinterpret_cast<const uint32_t *>(sc + 4 * threadIdx.x);
    }
}

template <int NB>
hipError_t launch_tile(const Mx8Args &p, hipStream_t s) {
    constexpr int BM = 256, BN = 256 / NB;
    const int64_t tiles = p.g.extent / BM + std::min<int64_t>(p.g.G, p.g.extent);
    const int64_t grid = tiles * ((p.g.N + BN - 1) / BN);
    if (grid <= 0) return hipSuccess;
    hipLaunchKernelGGL((mx8_tile_kernel<NB, 4>), dim3(static_cast<unsigned>(grid)), dim3(256), 0, s, p);
    return hipGetLastError();
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
    // few rows per expert: the weights' bytes bound it
    if (p.g.extent <= 48 * static_cast<int64_t>(p.g.G)) return launch_stream<NB, 2, 8>(p, s);
    return launch_tile<NB>(p, s);
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
    p.g.C0 = ye;
    p.g.ldc = d;
    return product<1>(p, s);
}

}  // namespace xmoe

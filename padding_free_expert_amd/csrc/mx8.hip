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
// scales, shifted by 8 (l / 16), serves it.  The 32x32x64 form has row l % 32 and
// chunks l / 32 and 2 + l / 32.
//
// The instruction adds eight products at a time, each cut at 2^-13 of the power
// of two of the largest, and the eights' sums in fp32 (measured): a sum is off by
// less than 2^-10 of its products' magnitudes, by about 2^-14 of itself in
// practice.  About 0.17% of act's bytes become the neighbouring value by it.
#include <algorithm>

#include "common.hpp"
#include "gemm.hpp"
#include "kernels.hpp"
#include "mx8.hpp"
#include "mx8_choice.hpp"

namespace xmoe {

namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

// ------------------------------------------------------- into and out of 8 bits

// One wave per row and 64 16-byte vectors; rows are independent.  Memory-bound:
// 16384 x 4096 bf16 (203 MB) 42 us, 4.8 TB/s.
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

// Memory-bound: 8192 x 7168 to bf16 (178 MB) 35 us, 5.1 TB/s.
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
// (column, 32-element block) forms one scale and 32 bytes.  64 x 2048 x 1408
// bf16 (560 MB) 133 us, 4.2 TB/s.
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
        o[i] = mx8_pack4(p[0] * m, p[65] * m, p[130] * m, p[195] * m);
    }
    uint4 *dst = reinterpret_cast<uint4 *>(q + (static_cast<int64_t>(e) * N + n) * K + k0 + 32 * g);
    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

// ------------------------------------------------------------------ products

// one block of the tile kernel for each (a multiple of the XCDs' number)
constexpr int kComputeUnits = kMxComputeUnits;

// two fp32 -> packed bf16, round to nearest even
__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi) {
    typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
    typedef float f2 __attribute__((ext_vector_type(2)));
    const f2 v = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf2));
}

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

// The tile of this block for launches whose blocks take one tile each: every
// wave finds it by itself from the offsets, lane l counting the row tiles of
// groups per * l .. + per - 1.  Tiles as in resolve_tile; false: no tile.
template <int BM>
__device__ __forceinline__ bool wave_tile(const GemmArgs &p, int v, int tiles_n, Tile *t) {
    const int lane = threadIdx.x & 63;
    const int per = (p.G + 63) / 64, g0 = lane * per;
    const int mt = v / tiles_n;
    int64_t lo = 0, hi = 0;
    int cnt = 0;
    for (int i = 0; i < per; ++i) {
        if (g0 + i < p.G) {
            seg_bounds(p, g0 + i, &lo, &hi);
            cnt += static_cast<int>((hi - lo + BM - 1) / BM);
        }
    }
    int inc = cnt;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int u = __shfl_up(inc, off, 64);
        if (lane >= off) inc += u;
    }
    const unsigned long long past = __ballot(inc <= mt);
    if (past == ~0ull) return false;
    const int owner = __popcll(past);  // the first lane whose groups reach the tile
    int first = __shfl(inc - cnt, owner, 64), g = owner * per, n;
    for (int i = 0; ; ++i) {
        if (per > 1) seg_bounds(p, g + i, &lo, &hi);
        else lo = __shfl(static_cast<int>(lo), owner, 64), hi = __shfl(static_cast<int>(hi), owner, 64);
        n = static_cast<int>((hi - lo + BM - 1) / BM);
        if (mt < first + n) {
            g += i;
            break;
        }
        first += n;
    }
    const int local = v - first * tiles_n;
    t->g = __builtin_amdgcn_readfirstlane(g);
    t->m0 = __builtin_amdgcn_readfirstlane((local % n) * BM);
    t->nt = __builtin_amdgcn_readfirstlane(local / n);
    const int base = __builtin_amdgcn_readfirstlane(static_cast<int>(lo));
    t->base = base;
    t->Mg = __builtin_amdgcn_readfirstlane(static_cast<int>(hi)) - base;
    return true;
}

// Few rows per expert: the weights are streamed past the rows once.  A block
// takes 16 MT rows of one expert by 64 weight rows (32 of W1 and the same of W3
// for the up-projection, NB = 2) and its four waves split the summed axis in
// 128-deep steps.  The waves' partial sums meet in LDS, added in wave order.
// Bound by the weights' bytes: what counts is whole lines in flight, so operands
// come as lines through a piece of shared memory of each wave's own (with loads in
// the instruction's order, 96 tokens of 64 experts of d = 2048, h = 1408, top-6
// took 78 + 44 us up and down, now 60 + 33: 6.2 and 5.6 TB/s), and registers are
// kept few enough for four blocks on a compute unit (eight waves a block 65 + 38, a
// second step's loads ahead 65 + 38).  Weights are loaded past the caches (else 67
// + 38), rows are not (4 experts of 64 rows 13.9 + 11.1 against 16.1 + 12.3 us).  One
// token 11.5 + 8.1 us, of which 3.7 and 3.0 are launch and the tile's search.
template <int NB, int MT>
__global__ __launch_bounds__(256) void mx8_stream_kernel(Mx8Args p) {
    constexpr int KW = 4, NC = 4 / NB, BM = 16 * MT, BN = 16 * NC;
    constexpr int NF = 4 * MT;  // 16 x 16 results of a wave
    __shared__ f32x4_t part[KW][NF][64];
    static_assert(sizeof(part) <= 32 * 1024, "four blocks on a compute unit");
    static_assert(KW >= MT * (NB == 1 ? 2 : 1), "a wave for each 16 rows (and 32 columns) of the result");
    const int N = p.g.N, K = p.K, kb = (K + 127) / 128;
    Tile t;
    if (!wave_tile<BM>(p.g, xcd_tile_order(blockIdx.x, gridDim.x), (N + BN - 1) / BN, &t)) return;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, quad = lane >> 4;
    const int n0 = t.nt * BN;

    // Operands come as whole 128-byte lines, eight rows a load (lane l: chunk l % 8 of
    // row l / 8, then of row 8 + l / 8), and go through a piece of shared memory of
    // the wave's own into the order of the instruction, whose 16 neighbouring lanes
    // hold 16 rows: asked for in that order, a load would touch 16 lines for 16 bytes
    // each.  Uniform bases that move with k; columns past N read the tile's first.
    const uint8_t *wb[2], *ws[2];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        wb[b] = (b ? p.b1 : p.b0) + (static_cast<int64_t>(t.g) * N + n0) * K;
        ws[b] = (b ? p.b1s : p.b0s) + (static_cast<int64_t>(t.g) * kb * N + n0) * 4;
    }
    uint32_t aoff[MT][2], asoff[MT];
    const uint32_t boff = static_cast<uint32_t>(lane >> 3) * static_cast<uint32_t>(K) + 16 * (lane & 7);
    int col[NC];
#pragma unroll
    for (int j = 0; j < NC; ++j) col[j] = n0 + 16 * j < N ? 16 * j : 0;
    // rows past the group's end read its first row and are not stored; ids outside
    // the rows load zeros
    const uint8_t *const ab = p.map ? p.a : p.a + (t.base + t.m0) * K;
    const uint8_t *const as = p.map ? p.as : p.as + (t.base + t.m0) * 4;
    bool zero[MT][2], szero[MT];
    auto row_of = [&](int r, bool *none) {
        const int m = t.m0 + r < t.Mg ? r : 0;
        const int id = p.map ? p.map[t.base + t.m0 + m] : m;
        *none = p.map && (id < 0 || id >= p.a_rows);
        return *none ? 0u : static_cast<uint32_t>(id);
    };
#pragma unroll
    for (int i = 0; i < MT; ++i) {
#pragma unroll
        for (int y = 0; y < 2; ++y)
            aoff[i][y] = row_of(16 * i + 8 * y + (lane >> 3), &zero[i][y]) * static_cast<uint32_t>(K) + 16 * (lane & 7);
        asoff[i] = 4u * row_of(16 * i + l16, &szero[i]);
    }
    f32x4_t acc[NB][NC][MT];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
            for (int i = 0; i < MT; ++i) acc[b][j][i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

    struct Step {
        i32x4_t b[NB][NC][2];
        i32x4_t a[MT][2];
        int bs[NB][NC], as[MT];
    };
    auto fetch = [&](int s, Step &f) {
        const int64_t k = static_cast<int64_t>(s) * 128;
        const bool whole = k + 128 <= K;  // else K ends inside: elements past it are zeros
        const bool in = whole || k + 16 * (lane & 7) < K;
        auto line = [&](const uint8_t *q) {
            const i32x4_t z = {0, 0, 0, 0};
            return in ? __builtin_nontemporal_load(reinterpret_cast<const i32x4_t *>(q + boff)) : z;
        };
#pragma unroll
        for (int i = 0; i < MT; ++i) {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const i32x4_t z = {0, 0, 0, 0};
                f.a[i][y] = in && !zero[i][y] ? *reinterpret_cast<const i32x4_t *>(ab + k + aoff[i][y]) : z;
            }
            f.as[i] = szero[i] ? 0 : *reinterpret_cast<const int *>(as + static_cast<int64_t>(s) * p.a_rows * 4 + asoff[i]);
        }
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int j = 0; j < NC; ++j) {
                const uint8_t *const q = wb[b] + static_cast<int64_t>(col[j]) * K + k;
                f.b[b][j][0] = line(q);
                f.b[b][j][1] = line(q + 8 * static_cast<int64_t>(K));
                f.bs[b][j] = *reinterpret_cast<const int *>(ws[b] + (static_cast<int64_t>(s) * N + col[j]) * 4 + 4 * l16);
            }
    };
    // two slots of 2 KB in the wave's part of `part`, chunk c of row r at c ^ (r % 8)
    char *const stage = reinterpret_cast<char *>(&part[wave][0][0]);
    static_assert(NF * 64 * sizeof(f32x4_t) >= 4096, "two slots");
    char *const put = stage + (lane >> 3) * 128 + 16 * ((lane & 7) ^ (lane >> 3));
    const char *const lo_at = stage + l16 * 128 + 16 * (quad ^ (l16 & 7));
    const char *const hi_at = stage + l16 * 128 + 16 * ((4 + quad) ^ (l16 & 7));
    auto turn = [&](const i32x4_t (&v)[2], int at) {
        *reinterpret_cast<i32x4_t *>(put + at) = v[0];
        *reinterpret_cast<i32x4_t *>(put + at + 1024) = v[1];
        // a wave's accesses to shared memory are served in order
        __builtin_amdgcn_wave_barrier();
        const i32x4_t lo = *reinterpret_cast<const i32x4_t *>(lo_at + at);
        const i32x4_t hi = *reinterpret_cast<const i32x4_t *>(hi_at + at);
        __builtin_amdgcn_wave_barrier();
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    };
    auto multiply = [&](const Step &f) {
        i32x8_t a[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) a[i] = turn(f.a[i], (i & 1) * 2048);
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int j = 0; j < NC; ++j) {
                const i32x8_t w = turn(f.b[b][j], ((b * NC + j) & 1) * 2048);
#pragma unroll
                for (int i = 0; i < MT; ++i)
                    acc[b][j][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        w, a[i], acc[b][j][i], 0, 0, 0, f.bs[b][j] >> (8 * quad), 0, f.as[i] >> (8 * quad));
            }
    };
#pragma unroll 1
    for (int s = wave; s < kb; s += KW) {
        Step f;
        fetch(s, f);
        multiply(f);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
            for (int i = 0; i < MT; ++i) part[wave][(b * NC + j) * MT + i][lane] = acc[b][j][i];
    __syncthreads();
    // wave i (and, for the down-projection, MT + i for the upper 32 columns): rows
    // 16 i .. 16 i + 15; lane l has row l % 16, columns 16 j + 4 (l / 16) + r
    if (wave >= MT * (NB == 1 ? 2 : 1)) return;
    const int mi = wave % MT, j0 = 2 * (wave / MT);
    const int c0 = n0 + 16 * j0;
    const int m = t.m0 + 16 * mi + l16;
    const int64_t row = t.base + m;
    const bool live = m < t.Mg && c0 < N;
    f32x4_t v[NB][2];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int f = (b * NC + j0 + j) * MT + mi;
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
                *reinterpret_cast<uint32_t *>(p.q + row * N + c0 + 16 * j + 4 * quad) =
                    mx8_pack4(o[4 * j] * sc, o[4 * j + 1] * sc, o[4 * j + 2] * sc, o[4 * j + 3] * sc);
            // the scale byte of this block of 32 columns; the last block also fills its group
            const int blk = c0 / 32;
            const int at = (blk & 3) + quad;
            if (quad == 0 || (c0 + 32 >= N && at < 4))
                p.qs[(static_cast<int64_t>(blk >> 2) * p.g.extent + row) * 4 + at] =
                    static_cast<uint8_t>(quad == 0 ? byte : kMxOne);
        }
    } else if (live) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
            *reinterpret_cast<uint2 *>(p.y + row * N + c0 + 16 * j + 4 * quad) =
                make_uint2(cvt_bf16x2(v[0][j][0], v[0][j][1]), cvt_bf16x2(v[0][j][2], v[0][j][3]));
    }
}

// A value that the compiler takes as new at this point: what follows from it is
// computed here instead of being kept in registers across the loop around it.
__device__ __forceinline__ uint32_t fresh(uint32_t v) {
    asm volatile("" : "+v"(v));
    return v;
}

// direct-to-LDS loads as those of gemm.hpp, with a scalar offset; NT: past the
// caches
template <bool NT = false>
__device__ __forceinline__ void lds_dma16(__amdgpu_buffer_rsrc_t rs, uint32_t voff, uint32_t soff, uint32_t lds) {
    if constexpr (NT)
        asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %3 offen nt lds"
                     :
                     : "v"(voff), "s"(rs), "s"(lds), "s"(soff)
                     : "memory");
    else
        asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %3 offen lds"
                     :
                     : "v"(voff), "s"(rs), "s"(lds), "s"(soff)
                     : "memory");
}
__device__ __forceinline__ void lds_dma4(__amdgpu_buffer_rsrc_t rs, uint32_t voff, uint32_t soff, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dword %0, %1, %3 offen lds"
                 :
                 : "v"(voff), "s"(rs), "s"(lds), "s"(soff)
                 : "memory");
}

// A buffer over `bytes` from `base`; none where there is nothing (offsets with
// bit 31 set must be out of range, so a size never wraps).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t over(const void *base, int64_t bytes) {
    return make_rsrc(base, bytes > 0 ? bytes : 0);
}

// The tiles of a launch, found from the device-side offsets once per block and
// kept in shared memory.
struct TileTable {
    int end[1024];        // row tiles up to and including the expert's; INT_MAX past the last expert
    int lo[1024];         // first row
    uint16_t last[1024];  // rows of its last tile
    int wave_sum[4];
};

// Fills the table (256 threads; ends with a barrier).  Returns the row tiles.
template <int BM>
__device__ __forceinline__ int build_table(const GemmArgs &p, TileTable &tt) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int cnt[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int g = 4 * threadIdx.x + i;
        int64_t lo = 0, hi = 0;
        if (g < p.G) seg_bounds(p, g, &lo, &hi);
        const int n = static_cast<int>((hi - lo + BM - 1) / BM);
        tt.lo[g] = static_cast<int>(lo);
        tt.last[g] = static_cast<uint16_t>(n > 0 ? hi - lo - static_cast<int64_t>(n - 1) * BM : 0);
        sum += n;
        cnt[i] = sum;
    }
    int inc = sum;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int v = __shfl_up(inc, off, 64);
        if (lane >= off) inc += v;
    }
    if (lane == 63) tt.wave_sum[wave] = inc;
    __syncthreads();
    int before = inc - sum, total = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        if (w < wave) before += tt.wave_sum[w];
        total += tt.wave_sum[w];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int g = 4 * threadIdx.x + i;
        tt.end[g] = g < p.G ? before + cnt[i] : INT_MAX;
    }
    __syncthreads();
    return total;
}

// A tile of the tile kernel: rows [row, row + rows) of the experts' rows, all of
// expert g, and columns from n0.
struct TileAt {
    int g, n0, rows;
    int64_t row;
};

// Tile number v of the launch in the order of resolve_tile: an expert's tiles
// together, its row tiles fastest.  Every wave searches by itself (64 lanes over
// 16 entries each, then over those 16).
template <int BM, int BN>
__device__ __forceinline__ TileAt find_tile(const TileTable &tt, int v, int tiles_n) {
    const int lane = threadIdx.x & 63;
    const int mt = v / tiles_n;
    const int blk = __popcll(__ballot(tt.end[16 * lane + 15] <= mt));
    const int g = __builtin_amdgcn_readfirstlane(
        16 * blk + __popcll(__ballot(lane < 16 && tt.end[16 * blk + (lane & 15)] <= mt)));
    const int first = g > 0 ? tt.end[g - 1] : 0, n = tt.end[g] - first;
    const int local = v - first * tiles_n;
    TileAt t;
    t.g = g;
    t.n0 = __builtin_amdgcn_readfirstlane(local / n * BN);
    t.row = __builtin_amdgcn_readfirstlane(tt.lo[g] + local % n * BM);
    t.rows = __builtin_amdgcn_readfirstlane(local % n == n - 1 ? static_cast<int>(tt.last[g]) : BM);
    return t;
}

// Many rows per expert: 256 x 256 results a tile (NB = 2: 128 columns of W1 and
// the same of W3), four waves of 128 x 128, one block per compute unit that
// takes one tile after another.  Both operands come into two slots of shared
// memory by direct loads, 128 bytes of K a slot, with the swizzle of the bf16
// products (a 16-byte chunk here is 16 elements instead of 8); the scale dwords
// of the same 128 of K come the same way.  Wave tiles this wide are what the
// rates ask for: per 64 of K a wave reads 16 KiB from shared memory for 16
// products of 64 cycles.  Slots of 128 bytes of K let each load ask L2 for whole
// lines (with 64 bytes and four slots: twice the requests).
//
// A block of 128 of K is two steps of 64.  Step 0 multiplies fragments that are
// in registers while those of step 1 are read; a barrier in its middle then
// frees the slot, and the loads of two blocks ahead go out, spread over both
// steps.  Step 1 starts with the wait and barrier for the next block, whose
// first fragments are read under its products.  The next tile's first two
// blocks are loaded under the last two of this one, and results leave without a
// barrier, so that a tile's end costs its arithmetic and the issue of its stores
// only.
//
// Bound by the matrix cores: 131072 rows on 96 experts of d = 4096, h = 1024 take
// 950 us up (2.3 PFLOP/s) and 620 us down (1.8 PFLOP/s, 1.07 GB of results), where
// an 8192^3 fp8 product of the library reaches 2.9 PFLOP/s.  What is lost: rows
// that pad an expert's last tile, the clock under load, and silu with the
// quantization between tiles (without it 899 us up), which one wave on a SIMD
// cannot hide.  24576 rows on 64 experts of d = 2048, h = 1408: 176 + 90 us.
template <int NB, bool MAP, bool NT>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1))) void mx8_tile_kernel(Mx8Args p) {
    constexpr int BM = 256, BN = 256 / NB, WGN = 2, NW = 4, S = 2;
    constexpr int WTM = 128, WTN = BN / WGN, TM = WTM / 32, TN = WTN / 32;
    static_assert(TM == 4 && NB * TN == 4, "sixteen 32 x 32 results a wave");
    constexpr int kABytes = BM * 128, kBBytes = BN * 128, kStage = kABytes + NB * kBBytes;
    constexpr int kL = kStage / (NW * 1024);  // operand loads of a wave per block
    static_assert(kL == 16, "seven in step 0, nine in step 1");
    constexpr int kScales = 512 * 4;          // scale dwords of 256 + 256 rows
    constexpr int kRing = S * kStage;
    static_assert(kRing + S * kScales + sizeof(TileTable) + 4 * 4096 <= 160 * 1024, "one block per compute unit");
    __shared__ __align__(1024) char smem[kRing + S * kScales];
    __shared__ TileTable tt;
    __shared__ __align__(16) char stage[NB == 1 ? 4 * 4096 : 16];

    const int N = p.g.N, K = p.K, kb = (K + 127) / 128, kbe = max(kb, 2);  // blocks, two at least
    const int tiles_n = (N + BN - 1) / BN;
    const int tiles = build_table<BM>(p.g, tt) * tiles_n;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WGN, wn = wave % WGN, half = lane >> 5;
    const uint32_t sbase = __builtin_amdgcn_readfirstlane(lds_addr(smem));
    // Turn u of the launch.  Runs of consecutive tiles to an XCD as in
    // xcd_tile_order (this grid's 32 blocks of an XCD make a run in each round),
    // turned by one from round to round: an expert's last row tile is often
    // shorter, and with two row tiles an expert the same blocks would have all
    // the long ones.  Where the last round has tiles for at most half the blocks,
    // two blocks take 128 rows each of one (2048 rows on 4 experts of d = 2048,
    // h = 1408: 39 + 23 -> 36 + 20 us).
    constexpr int W = kXcds * kXcdRun;
    static_assert(kComputeUnits == W, "a round is one run on each XCD");
    const int whole = tiles / W * W, rest = tiles - whole;
    const bool split = 2 * rest <= W;
    const int turns = whole + (split ? 2 * rest : rest);
    auto take = [&](int u) {
        const int round = u / W, b = u % W;
        if (u < whole)
            return find_tile<BM, BN>(tt, round * W + b % kXcds * kXcdRun + (b / kXcds + round) % kXcdRun, tiles_n);
        TileAt t = find_tile<BM, BN>(tt, split ? whole + (u - whole) / 2 : u, tiles_n);
        if (split) {
            // a short tile's second half is empty and starts at its end
            const int from = min((u - whole) % 2 * WTM, t.rows);
            t.row += from;
            t.rows = min(t.rows - from, WTM);
        }
        return t;
    };
    int v = blockIdx.x;
    if (v >= turns) return;
    TileAt t = take(v);

    // Operand loads: load i of wave w fills tile rows 32 i + 8 w .. + 7, lane l
    // the chunk l % 8 of row 8 w + l / 8, which holds the row's chunk c (the
    // swizzle goes by the row modulo 16, so c is the same for all i).  A buffer
    // spans the tile's rows (MAP: all rows of a), so a lane's offset is its
    // row's, the block's k goes into the scalar offset, and rows past the
    // group's end or N are out of range and load zeros; so do offsets with bit 31
    // set: ids outside the rows and, in the last block, chunks past K.
    constexpr uint32_t kOut = 0x80000000u;
    const int lrow = 8 * wave + (lane >> 3), c16 = 16 * ((lane & 7) ^ swz_kc(lrow, 8));
    const uint32_t boff = static_cast<uint32_t>(lrow * K + c16), step32 = 32u * static_cast<uint32_t>(K);
    struct Source {  // what the loads of a tile need
        __amdgpu_buffer_rsrc_t a, b0, b1, as, bs;
        uint32_t aoff[MAP ? 8 : 1], as_off, bs_off;
    };
    auto source = [&](const TileAt &u) {
        Source q;
        // An empty tile (half of a short one) loads the row in front of it: range
        // checks take the scalar offset from the buffer's size, which for an empty
        // buffer would leave what is below zero.
        const int rows = max(u.rows, 1), n0 = u.n0;
        const int64_t r0 = u.row - (u.rows > 0 ? 0 : 1);
        const int m = 64 * wave + lane;  // scales: wave w takes rows 64 w .. + 63 of A's 256 and of B's
        q.as_off = m < rows ? 4u * m : kOut;
        if constexpr (MAP) {
            auto id_of = [&](int mm) {
                const int id = mm < rows ? p.map[r0 + mm] : -1;
                return id >= 0 && id < p.a_rows ? id : -1;
            };
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int id = id_of(32 * i + lrow);
                q.aoff[i] = id >= 0 ? static_cast<uint32_t>(id) * static_cast<uint32_t>(K) + c16 : kOut;
            }
            const int id = id_of(m);
            q.as_off = id >= 0 ? 4u * id : kOut;
            q.a = over(p.a, p.a_rows * K);
            q.as = over(p.as, p.a_rows * kb * 4);
        } else {
            q.a = over(p.a + r0 * K, static_cast<int64_t>(rows) * K);
            q.as = over(p.as + r0 * 4, (p.a_rows * kb - r0) * 4);
        }
        const int64_t b_at = (static_cast<int64_t>(u.g) * N + n0) * K;
        const int64_t bbytes = static_cast<int64_t>(min(N - n0, BN)) * K;
        q.b0 = over(p.b0 + b_at, bbytes);
        q.b1 = over((NB == 2 ? p.b1 : p.b0) + b_at, bbytes);
        const int col = NB == 2 ? m & 127 : m;  // B's: of W1 and W3 128 each
        q.bs_off = n0 + col < N ? 4u * col : kOut;
        const int64_t bs_at = static_cast<int64_t>(u.g) * kb * N + n0;
        q.bs = over(((NB == 2 && wave >= 2) ? p.b1s : p.b0s) + bs_at * 4, (static_cast<int64_t>(kb) * N - n0) * 4);
        return q;
    };
    // blocks past the end load zeros, so that the count of loads in flight stays the same
    struct Plan {
        uint32_t k, as, bs;  // scalar offsets of the block
        uint32_t row;        // offset of this lane's chunk in the tile's first rows
        uint32_t out;        // bit 31 set in lanes whose chunk is past K
        uint32_t sout;       // bit 31 set where the block has no scales
    };
    auto plan = [&](int blk, bool live) {
        live = live && blk < kb;
        const uint32_t g = live ? blk : 0;
        Plan q;
        q.k = g * 128u;
        q.as = g * static_cast<uint32_t>(p.a_rows) * 4u;
        q.bs = g * static_cast<uint32_t>(N) * 4u;
        q.row = fresh(boff);
        q.out = live && static_cast<int>(q.k) + c16 < K ? 0u : kOut;
        q.sout = live ? 0u : kOut;
        return q;
    };
    auto issue_part = [&](const Source &c, const Plan &q, int slot, int part) {
        const uint32_t dst = sbase + slot * kStage + wave * 1024;
        if (part < 8) {
            lds_dma16(c.a, (MAP ? c.aoff[MAP ? part : 0] : q.row + part * step32) | q.out, q.k, dst + part * 4096);
        } else {
            const int b = (part - 8) / (8 / NB), i = (part - 8) % (8 / NB);
            lds_dma16<NT>(b ? c.b1 : c.b0, (q.row + i * step32) | q.out, q.k, dst + kABytes + b * kBBytes + i * 4096);
        }
    };
    auto issue_scales = [&](const Source &c, const Plan &q, int slot) {
        const uint32_t dst = sbase + kRing + slot * kScales + wave * 256;
        lds_dma4(c.as, c.as_off | q.sout, q.as, dst);
        lds_dma4(c.bs, c.bs_off | q.sout, q.bs, dst + 1024);
    };

    // fragment addresses: of the eight chunks of row l % 32, lane l reads chunks
    // 4 s + l / 32 and 4 s + 2 + l / 32 in step s (the swizzle goes by the row
    // modulo 32, so whole 32-row blocks are immediates)
    const int row = lane & 31, sw = swz_kc(row, 8);
    uint32_t fad[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) fad[c] = row * 128 + 16 * ((2 * c + half) ^ sw);
    f32x16_t acc[NB][TM][TN];
    i32x8_t fA[2][TM], fB[2][4];
    int sA[2][TM], sB[2][4];
    typedef __attribute__((address_space(3))) const i32x4_t lds_i32x4;
    struct Frags {  // addresses of a step's fragments: one add each, the rest immediates
        uint32_t alo, ahi, blo, bhi;
    };
    auto frags = [&](int s, int slot, int arow, int bcol) {
        const uint32_t sa = sbase + slot * kStage + arow * 128;
        const uint32_t sb = sbase + slot * kStage + kABytes + bcol * 128;
        return Frags{fresh(sa + fad[2 * s]), fresh(sa + fad[2 * s + 1]), fresh(sb + fad[2 * s]), fresh(sb + fad[2 * s + 1])};
    };
    auto read_a = [&](const Frags &f, int s, int i) {
        const i32x4_t lo = *reinterpret_cast<lds_i32x4 *>(static_cast<uintptr_t>(f.alo + 4096 * i));
        const i32x4_t hi = *reinterpret_cast<lds_i32x4 *>(static_cast<uintptr_t>(f.ahi + 4096 * i));
        fA[s][i] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    };
    auto read_b = [&](const Frags &f, int s, int u, int off) {
        const i32x4_t lo = *reinterpret_cast<lds_i32x4 *>(static_cast<uintptr_t>(f.blo + off));
        const i32x4_t hi = *reinterpret_cast<lds_i32x4 *>(static_cast<uintptr_t>(f.bhi + off));
        fB[s][u] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    };

    Source src = source(t);
#pragma unroll
    for (int blk = 0; blk < S; ++blk) {
        const Plan pl = plan(blk, true);
        issue_scales(src, pl, blk);
#pragma unroll
        for (int u = 0; u < kL; ++u) issue_part(src, pl, blk, u);
    }
    wait_vmem<kL + 2>();  // block 0 has landed
    __syncthreads();
    int slot = 0;
    while (true) {
        const int nv = v + static_cast<int>(gridDim.x);
        const bool more = nv < turns;
        const TileAt next = more ? take(nv) : t;
        const Source nsrc = source(next);
        // One tile.  HALF: at most 128 rows, which all four waves share, each with
        // half the columns it has otherwise (128 x 64 of the 128 x 256 results).  1800
        // rows on 64 experts of d = 2048, h = 1408: 100 + 46 -> 91 + 44 us.
        auto tile = [&](auto half_tag) {
            constexpr bool HALF = decltype(half_tag)::value;
            constexpr int TJ = HALF ? TN / 2 : TN;        // column blocks of 32 of each matrix
            constexpr int TT = NB * TJ, NQ = TM * TT;     // B fragments, products of a step
            const int arow = HALF ? 0 : wm * WTM;
            const int bcol = HALF ? wave * 32 * TJ : wn * WTN;
            // fragment u of B: matrix u / TJ, column block u % TJ
            auto read_unit = [&](const Frags &f, int s, int u) {
                if (u < TM) read_a(f, s, u);
                else read_b(f, s, u - TM, ((u - TM) / TJ) * kBBytes + ((u - TM) % TJ) * 4096);
            };
            auto read_scales = [&](int set, int sl) {
                const uint32_t ss = sbase + kRing + sl * kScales;
                const uint32_t sa = fresh(ss + (arow + row) * 4), sb = fresh(ss + 1024 + (bcol + row) * 4);
#pragma unroll
                for (int i = 0; i < TM; ++i) sA[set][i] = lds_read_i32(sa + 128 * i) >> (8 * half);
#pragma unroll
                for (int u = 0; u < TT; ++u) sB[set][u] = lds_read_i32(sb + 4 * (u / TJ) * BN + 128 * (u % TJ)) >> (8 * half);
            };
            {
                read_scales(0, slot);
                const Frags f = frags(0, slot, arow, bcol);
#pragma unroll
                for (int u = 0; u < TM + TT; ++u) read_unit(f, 0, u);
            }
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int j = 0; j < TJ; ++j)
#pragma unroll
                        for (int r = 0; r < 16; ++r) acc[b][i][j][r] = 0.0f;
            // product q of step s.  The order around it is pinned: left to itself
            // the compiler puts all reads in front of the products, which then
            // wait for shared memory.
            auto product = [&](int s, int q) {
                const int u = q / TM, i = q % TM;
                if (s == 0)
                    acc[u / TJ][i][u % TJ] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                        fB[0][u], fA[0][i], acc[u / TJ][i][u % TJ], 0, 0, 0, sB[0][u], 0, sA[0][i]);
                else
                    acc[u / TJ][i][u % TJ] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                        fB[1][u], fA[1][i], acc[u / TJ][i][u % TJ], 0, 0, 2, sB[0][u], 2, sA[0][i]);
            };
            constexpr int kParts0 = 7;             // loads in step 0, the rest in step 1
            constexpr int kBar = HALF ? 4 : 8;     // the product whose turn frees the slot
            for (int blk = 0; blk < kbe; ++blk) {
                const bool ahead = blk + 2 >= kbe;  // the loads are the next tile's first two blocks
                if (blk + 2 == kbe) src = nsrc;
                const Plan pl = plan(ahead ? blk + 2 - kbe : blk + 2, !ahead || more);
                const Frags f1 = frags(1, slot, arow, bcol);
#pragma unroll
                for (int q = 0; q < NQ; ++q) {
                    product(0, q);
                    if constexpr (HALF) {
                        if (q < 3) {
                            read_unit(f1, 1, 2 * q);
                            read_unit(f1, 1, 2 * q + 1);
                        }
                    } else {
                        if (q < TM + TT) read_unit(f1, 1, q);
                    }
                    if (q == kBar) {
                        __syncthreads();  // every wave has read this block: its slot is free
                        issue_scales(src, pl, slot);
                    }
                    if constexpr (HALF) {
                        if (q > kBar) {
                            issue_part(src, pl, slot, 2 * (q - kBar - 1));
                            issue_part(src, pl, slot, 2 * (q - kBar - 1) + 1);
                            if (q == NQ - 1) issue_part(src, pl, slot, 6);
                        }
                    } else {
                        if (q > kBar) issue_part(src, pl, slot, q - kBar - 1);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                wait_vmem<2 + kParts0>();  // the next block has landed (what is out is of the one after)
                __syncthreads();
                read_scales(1, slot ^ 1);
                const Frags f0 = frags(0, slot ^ 1, arow, bcol);
#pragma unroll
                for (int q = 0; q < NQ; ++q) {
                    product(1, q);
                    if constexpr (HALF) {
                        if (q < TM + TT) read_unit(f0, 0, q);
                        if (q < 4) issue_part(src, pl, slot, kParts0 + 2 * q + 1);
                        if (q < 5) issue_part(src, pl, slot, kParts0 + 2 * q);
                    } else {
                        if (q % 2 == 0) read_unit(f0, 0, q / 2);
                        if (q < kL - kParts0) issue_part(src, pl, slot, q + kParts0);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
#pragma unroll
                for (int i = 0; i < TM; ++i) sA[0][i] = sA[1][i];
#pragma unroll
                for (int u = 0; u < TT; ++u) sB[0][u] = sB[1][u];
                slot ^= 1;
            }
            // the sums stay in the accumulation registers until their turn
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int j = 0; j < TJ; ++j) asm volatile("" : "+a"(acc[b][i][j]));
            // lane l: row 32 i + l % 32, columns 32 j + 8 g + 4 (l / 32) + r.  Stores go
            // through buffers that end with the tile's rows and with bit 31 set past
            // N, so that nothing branches and each result stays in its accumulator
            // until its turn.
            typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
            if constexpr (NB == 1) {
                // 32 rows by 64 columns at a time through a piece of shared memory of
                // the wave's own (chunk c of row m at c ^ (m % 8)): the stores then
                // cover 128 consecutive bytes of a row instead of 32 (down-projection
                // of 131072 rows, d = 4096, h = 1024: 655 -> 620 us)
                char *const st = stage + wave * 4096;
                const __amdgpu_buffer_rsrc_t ry = over(p.y + t.row * N, static_cast<int64_t>(t.rows) * N * 2);
                const int wrow = static_cast<int>(fresh(row)), rrow = static_cast<int>(fresh(lane >> 3)), rch = lane & 7;
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int j = 0; j < TJ; j += 2) {
#pragma unroll
                        for (int g = 0; g < 8; ++g) {
                            const f32x16_t &a = acc[0][i][j + g / 4];
                            const int e = 4 * (g % 4);
                            *reinterpret_cast<uint2 *>(st + wrow * 128 + 16 * (g ^ (wrow & 7)) + 8 * half) =
                                make_uint2(cvt_bf16x2(a[e], a[e + 1]), cvt_bf16x2(a[e + 2], a[e + 3]));
                        }
                        __builtin_amdgcn_wave_barrier();
                        const int c = t.n0 + bcol + 32 * j + 8 * rch;
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            const int m = 8 * h + rrow;
                            const u32x4_t v = *reinterpret_cast<const u32x4_t *>(st + m * 128 + 16 * (rch ^ (m & 7)));
                            const uint32_t at = static_cast<uint32_t>((arow + 32 * i + m) * N + c) * 2u;
                            __builtin_amdgcn_raw_buffer_store_b128(v, ry, static_cast<int>(c < N ? at : kOut), 0, 0);
                        }
                        __builtin_amdgcn_wave_barrier();
                        __builtin_amdgcn_sched_barrier(0);  // one piece at a time: registers
                    }
            } else {
                // swapping the lanes' halves gives each 16 consecutive bytes of its row
                const __amdgpu_buffer_rsrc_t rq = over(p.q + t.row * N, static_cast<int64_t>(t.rows) * N);
                const __amdgpu_buffer_rsrc_t rs =
                    over(p.qs + (static_cast<int64_t>(t.n0 / 128) * p.g.extent + t.row) * 4, t.rows * 4);
                const int erow = static_cast<int>(fresh(arow + row));
#pragma unroll
                for (int i = 0; i < TM; ++i) {
                    const int m = erow + 32 * i;
                    uint32_t bytes = 0u;
#pragma unroll
                    for (int j = 0; j < TJ; ++j) {
                        const int c = t.n0 + bcol + 32 * j;
                        f32x16_t h1 = acc[0][i][j], h3 = acc[1][i][j];
                        asm volatile("" : "+v"(h1), "+v"(h3));
                        float o[16];
                        uint32_t a = 0u;
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            o[e] = h1[e] * __builtin_amdgcn_rcpf(1.0f + __expf(-h1[e])) * h3[e];
                            a = max(a, __float_as_uint(o[e]) & 0x7fffffffu);
                        }
                        const auto other = __builtin_amdgcn_permlane32_swap(a, a, false, false);
                        a = max(other[0], other[1]);
                        const uint32_t byte = mx8_scale_byte(a);
                        const float s = mx8_inv_scale(byte);
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 16; e += 4)
                            w[e / 4] = mx8_pack4(o[e] * s, o[e + 1] * s, o[e + 2] * s, o[e + 3] * s);
                        const auto x = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
                        const auto y = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
                        __builtin_amdgcn_raw_buffer_store_b128(u32x4_t{x[0], x[1], y[0], y[1]}, rq,
                                                               static_cast<int>(c < N ? m * N + c + 16 * half : kOut), 0, 0);
                        // past N: the byte that fills the last group (a NaN row is NaN there too)
                        bytes |= (c < N ? byte : kMxOne) << (8 * j);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    const int at = static_cast<int>(half ? kOut : m * 4u + bcol / 32u);
                    if constexpr (HALF) __builtin_amdgcn_raw_buffer_store_b8(static_cast<uint8_t>(bytes), rs, at, 0, 0);
                    else __builtin_amdgcn_raw_buffer_store_b16(static_cast<uint16_t>(bytes), rs, at, 0, 0);
                }
            }
        };
        if (t.rows <= WTM) tile(std::true_type{});
        else tile(std::false_type{});
        if (!more) break;
        t = next;
        v = nv;
    }
    wait_vmem<0>();  // no load may still target the slots when the block ends
}

template <int NB, bool MAP>
hipError_t launch_tile(const Mx8Args &p, bool once, hipStream_t s) {
    constexpr int BM = 256, BN = 256 / NB;
    const int64_t cols = (p.g.N + BN - 1) / BN, active = std::min<int64_t>(p.g.G, p.g.extent);
    const int64_t grid = std::min<int64_t>(2 * (p.g.extent / BM + active) * cols, kComputeUnits);
    if (grid <= 0) return hipSuccess;
    if (once) hipLaunchKernelGGL((mx8_tile_kernel<NB, MAP, true>), dim3(static_cast<unsigned>(grid)), dim3(256), 0, s, p);
    else hipLaunchKernelGGL((mx8_tile_kernel<NB, MAP, false>), dim3(static_cast<unsigned>(grid)), dim3(256), 0, s, p);
    return hipGetLastError();
}

template <int NB, int MT>
hipError_t launch_stream(const Mx8Args &p, hipStream_t s) {
    // no expert without rows has a tile: at most rows / BM whole ones and one
    // more for each expert that has rows
    const int64_t tiles = p.g.extent / (16 * MT) + std::min<int64_t>(p.g.G, p.g.extent);
    const int64_t grid = tiles * ((p.g.N + 64 / NB - 1) / (64 / NB));
    if (grid <= 0) return hipSuccess;
    hipLaunchKernelGGL((mx8_stream_kernel<NB, MT>), dim3(static_cast<unsigned>(grid)), dim3(256), 0, s, p);
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
    const Mx8Choice c = mx8_choose(p.g.extent, p.g.G, p.g.N, NB);
    if (c.stream == 1) return launch_stream<NB, 1>(p, s);
    if (c.stream == 2) return launch_stream<NB, 2>(p, s);
    if constexpr (NB == 2) {
        if (p.map) return launch_tile<2, true>(p, c.once, s);
    }
    return launch_tile<NB, false>(p, c.once, s);
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

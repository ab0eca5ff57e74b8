// The whole layer for a few tokens (at most 64): gate, top-k, experts, shared
// experts and combine.
//
// The layer's other path sorts rows by expert and multiplies 128-row tiles; with a
// token or two for each expert its time is launches, searches for tiles and rows that
// are not there.  Here the weights that the tokens chose are streamed past their rows
// once, and what one product leaves for the next stays in the caches:
//   1  partial logits of the gate, and the shared experts' H1, H3 (they need no
//      routing): K split over blocks
//   2  softmax and top-k, a wave for each token
//   3  H1, H3 of the chosen experts
//   4  the down-projections, silu(H1) * H3 formed on the way in
//   5  y = sum_j p_j (parts of slot j) + parts of the shared experts
// Slot t k + j is token t's j-th choice; a unit of work is one expert (a chosen one or
// the shared ones side by side), a strip of its columns and a part of its rows.
// Every sum over parts runs in part order: no atomics, the same bits each time.
//
// A block's row tiles (one of 16 rows, or two) are a template argument, and which of the
// two instances runs is decided in front of its loop: with a branch around the second
// tile's products hipcc leaves too few waits between a matrix instruction and the copy of
// its result that a branch jumps to (ROCm 7.2, fp32: four columns of 64 were wrong).
//
// Products: the weights are the first operand of the matrix instruction (16 columns),
// the rows the second (16 rows), so that a row costs nothing up to 16 of them and rows
// that are not there may hold anything: a row's results depend on it alone.
#include <algorithm>

#include "common.hpp"
#include "few.hpp"
#include "gemm.hpp"
#include "kernels.hpp"
#include "mx8.hpp"

namespace xmoe {

namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int kFewWaves = 4;
constexpr int kFewThreads = 64 * kFewWaves;

// One set of experts: the routed ones, or the shared ones as a single expert.
struct FewFfn {
    const void *w1, *w3, *w2;            // [n, K, N], or 8 bits [n, N, K]
    const uint8_t *w1s, *w3s, *w2s;      // 8 bits: scales [n, ceil(K / 128), N, 4]
    int h;
    int slots;                           // rows of the partial sums
    int up_parts, up_len, down_parts, down_len;
    float *hp;                           // [up_parts, slots, 2h]  parts of H1 | H3
    float *yp;                           // [down_parts, slots, d] parts of the outputs
};

struct FewArgs {
    const void *x;                       // [T, d]
    const uint8_t *xq, *xs;              // 8 bits: the rows of the experts' products
    const void *wg;
    int T, d, E, k;
    float scale;
    const float *lbias, *sbias;
    int32_t *ids;
    float *w, *logits;
    void *y;
    int gate_parts, gate_len;
    float *zp;                           // [gate_parts, T, E]
    FewFfn r, s;                         // s.h == 0: no shared experts
};

// ------------------------------------------------------------------ products

// Weights in the layer's layout [K, N] (bf16 or fp32).  A wave's step is 32 of K by
// 16 chunks of 16 bytes (BN columns): lane l loads chunk l % 16 of the eight rows
// 8 (l / 16) + j, 256 bytes of each row by 16 lanes.  Column i of every chunk makes one
// product of 16 columns, column CV m + i being its m-th: two registers of neighbouring
// rows give a register of an operand (bf16), or are operands as they are (fp32, where
// the four lane groups hold the rows 8 (l / 16) + j of one product).  Lane l's results
// are then columns 4 CV (l / 16) + CV r + i of row l % 16: 4 CV in a row.  Reads past
// the matrix's end give zeros (K's tail); past a row's end they give the next row's
// values, which only reach columns that are not stored.
template <typename T>
struct PlainCore {
    using Elt = T;
    static constexpr bool kMx = false;
    static constexpr int CV = 16 / static_cast<int>(sizeof(T)), BN = 16 * CV, STEP = 32;
    static constexpr int kStage = 16;  // no staging
    struct X {
        i32x4_t v[sizeof(T) / 2];  // eight elements of a row
    };

    // acc[b][mt][i]; rows come from rowf(mt, k): the eight elements at k of row 16 mt + l % 16
    template <int NB, int MT, class Rows>
    __device__ static __forceinline__ void run(const void *const (&w)[NB], const uint8_t *const (&)[NB], int K, int N,
                                               int n0, int ka, int kb, Rows rowf, char *, int lane, int wave,
                                               f32x4_t (&acc)[NB][MT][CV]) {
        __amdgpu_buffer_rsrc_t rs[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) rs[b] = make_rsrc(w[b], static_cast<int64_t>(K) * N * static_cast<int>(sizeof(T)));
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < CV; ++i) acc[b][m][i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        const int quad = lane >> 4;
        const int rowb = N * static_cast<int>(sizeof(T));
        const int col = (n0 + CV * (lane & 15)) * static_cast<int>(sizeof(T));
        struct Step {
            i32x4_t w[NB][8];
            X x[MT];
        };
        auto fetch = [&](int k, Step &s) {
            const int at = (k + 8 * quad) * rowb + col;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    s.w[b][j] = __builtin_bit_cast(i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rs[b], at + j * rowb, 0, 0));
#pragma unroll
            for (int m = 0; m < MT; ++m)
                s.x[m] = rowf(m, k + 8 * quad);
        };
        auto multiply = [&](const Step &s) {
            if constexpr (sizeof(T) == 2) {
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int i = 0; i < CV; ++i) {
                        i32x4_t o;
#pragma unroll
                        for (int p = 0; p < 4; ++p)
                            o[p] = static_cast<int>(__builtin_amdgcn_perm(static_cast<uint32_t>(s.w[b][2 * p + 1][i / 2]),
                                                                          static_cast<uint32_t>(s.w[b][2 * p][i / 2]),
                                                                          i % 2 ? 0x07060302u : 0x05040100u));
#pragma unroll
                        for (int m = 0; m < MT; ++m)
                            acc[b][m][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                __builtin_bit_cast(bf16x8_t, o), __builtin_bit_cast(bf16x8_t, s.x[m].v[0]), acc[b][m][i], 0, 0,
                                0);
                    }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int i = 0; i < CV; ++i)
#pragma unroll
                            for (int m = 0; m < MT; ++m)
                                acc[b][m][i] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                                    __builtin_bit_cast(float, static_cast<int>(s.w[b][j][i])),
                                    __builtin_bit_cast(float, static_cast<int>(s.x[m].v[j / 4][j % 4])), acc[b][m][i], 0, 0, 0);
            }
        };
        constexpr int D = STEP * kFewWaves;
        Step p, q;
        int k = ka + STEP * wave;
        if (k < kb) fetch(k, p);
        while (k < kb) {
            if (k + D < kb) fetch(k + D, q);
            multiply(p);
            if (k + D >= kb) break;
            if (k + 2 * D < kb) fetch(k + 2 * D, p);
            multiply(q);
            k += 2 * D;
        }
    }

    // sum over the waves: thread (row, chunk) = (tid / 16, tid % 16) gets its CV columns
    __device__ static __forceinline__ void put(float (*red)[BN + 4], const f32x4_t (&acc)[CV], int lane) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int i = 0; i < CV; i += 4)
                *reinterpret_cast<f32x4_t *>(&red[lane & 15][4 * CV * (lane >> 4) + CV * r + i]) =
                    f32x4_t{acc[i][r], acc[i + 1][r], acc[i + 2][r], acc[i + 3][r]};
    }
};

// 8-bit weights [N, K] with scales: a wave's step is 128 of K by 64 columns (each
// matrix), as whole 128-byte lines through a piece of shared memory of the wave's own
// into the order of the instruction (mx8.hip says why).  Lane l's results are columns
// 16 j + 4 (l / 16) + r of row l % 16.
struct Mx8Core {
    using Elt = uint8_t;
    static constexpr bool kMx = true;
    static constexpr int CV = 4, BN = 64, STEP = 128;
    static constexpr int kStage = kFewWaves * 4096;
    struct X {
        i32x8_t v;   // chunks l / 16 and 4 + l / 16 of the row's 128 bytes
        int s;       // the row's scale dword
    };

    template <int NB, int MT, class Rows>
    __device__ static __forceinline__ void run(const void *const (&w)[NB], const uint8_t *const (&ws)[NB], int K, int N,
                                               int n0, int ka, int kb, Rows rowf, char *stage, int lane, int wave,
                                               f32x4_t (&acc)[NB][MT][CV]) {
        const int l16 = lane & 15, quad = lane >> 4;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < CV; ++i) acc[b][m][i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        int col[4];  // column tiles past N read the strip's first
#pragma unroll
        for (int j = 0; j < 4; ++j) col[j] = n0 + 16 * j < N ? 16 * j : 0;
        const uint32_t boff = static_cast<uint32_t>(lane >> 3) * static_cast<uint32_t>(K) + 16 * (lane & 7);
        struct Step {
            i32x4_t w[NB][4][2];
            int s[NB][4];
            X x[MT];
        };
        auto fetch = [&](int k, Step &f) {
            const bool in = k + 16 * (lane & 7) < K;  // K may end inside: zeros behind it
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint8_t *const q = static_cast<const uint8_t *>(w[b]) + static_cast<int64_t>(n0 + col[j]) * K + k;
                    const i32x4_t z = {0, 0, 0, 0};
                    f.w[b][j][0] = in ? __builtin_nontemporal_load(reinterpret_cast<const i32x4_t *>(q + boff)) : z;
                    f.w[b][j][1] =
                        in ? __builtin_nontemporal_load(reinterpret_cast<const i32x4_t *>(q + 8 * static_cast<int64_t>(K) + boff)) : z;
                    f.s[b][j] = *reinterpret_cast<const int *>(ws[b] + (static_cast<int64_t>(k >> 7) * N + n0 + col[j] + l16) * 4);
                }
#pragma unroll
            for (int m = 0; m < MT; ++m)
                f.x[m] = rowf(m, k);
        };
        char *const mine = stage + wave * 4096;
        char *const put = mine + (lane >> 3) * 128 + 16 * ((lane & 7) ^ (lane >> 3));
        const char *const lo_at = mine + l16 * 128 + 16 * (quad ^ (l16 & 7));
        const char *const hi_at = mine + l16 * 128 + 16 * ((4 + quad) ^ (l16 & 7));
        auto turn = [&](const i32x4_t (&v)[2], int at) {
            *reinterpret_cast<i32x4_t *>(put + at) = v[0];
            *reinterpret_cast<i32x4_t *>(put + at + 1024) = v[1];
            __builtin_amdgcn_wave_barrier();  // a wave's accesses to shared memory are served in order
            const i32x4_t lo = *reinterpret_cast<const i32x4_t *>(lo_at + at);
            const i32x4_t hi = *reinterpret_cast<const i32x4_t *>(hi_at + at);
            __builtin_amdgcn_wave_barrier();
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        };
        auto multiply = [&](const Step &f) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const i32x8_t v = turn(f.w[b][j], (j & 1) * 2048);
#pragma unroll
                    for (int m = 0; m < MT; ++m)
                        acc[b][m][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            v, f.x[m].v, acc[b][m][j], 0, 0, 0, f.s[b][j] >> (8 * quad), 0, f.x[m].s >> (8 * quad));
                }
        };
#pragma unroll 1
        for (int k = ka + STEP * wave; k < kb; k += STEP * kFewWaves) {
            Step f;
            fetch(k, f);
            multiply(f);
        }
    }

    __device__ static __forceinline__ void put(float (*red)[BN + 4], const f32x4_t (&acc)[CV], int lane) {
#pragma unroll
        for (int j = 0; j < 4; ++j) *reinterpret_cast<f32x4_t *>(&red[lane & 15][16 * j + 4 * (lane >> 4)]) = acc[j];
    }
};

// What a block keeps in shared memory beside its activations.
template <class C>
struct FewShared {
    float red[kFewWaves][16][C::BN + 4];
    __align__(16) char stage[C::kStage];
    int slot[64];
    uint32_t used[32];
    int expert;
};

// The waves' parts of 16 rows x BN columns, added in wave order: thread tid has row
// tid / 16, columns CV (tid % 16) ..
template <class C>
__device__ __forceinline__ void sum_waves(FewShared<C> &sh, const f32x4_t (&acc)[C::CV], int lane, int wave,
                                          float (&out)[C::CV]) {
    __syncthreads();
    C::put(sh.red[wave], acc, lane);
    __syncthreads();
    const int row = threadIdx.x >> 4, c0 = C::CV * (threadIdx.x & 15);
#pragma unroll
    for (int i = 0; i < C::CV; ++i) out[i] = sh.red[0][row][c0 + i];
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w)
#pragma unroll
        for (int i = 0; i < C::CV; ++i) out[i] += sh.red[w][row][c0 + i];
}

// The a-th chosen expert in ascending order and its slots by ascending token, from the
// ids of all tokens; the number of rows, 0 where fewer experts are chosen.  Ends with a
// barrier.
template <class C>
__device__ __forceinline__ int find_unit(const FewArgs &p, int a, FewShared<C> &sh, int *expert) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (threadIdx.x < 32) sh.used[threadIdx.x] = 0u;
    __syncthreads();
    for (int i = threadIdx.x; i < p.T * p.k; i += kFewThreads) {
        const int e = p.ids[i];
        atomicOr(&sh.used[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
    const uint32_t bits = lane < 32 ? sh.used[lane] : 0u;
    const int cnt = __popc(bits);
    int inc = cnt;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up(inc, off, 64);
        if (lane >= off) inc += v;
    }
    const unsigned long long past = __ballot(lane < 32 && inc <= a);
    const int word = __popcll(past);
    if (word >= 32) return 0;
    uint32_t b = __shfl(static_cast<int>(bits), word, 64);
    for (int n = a - __shfl(inc - cnt, word, 64); n > 0; --n) b &= b - 1;
    const int e = 32 * word + __ffs(b) - 1;
    int slot = -1;
    if (lane < p.T)
        for (int j = 0; j < p.k; ++j)
            if (p.ids[lane * p.k + j] == e) slot = lane * p.k + j;
    const unsigned long long has = __ballot(slot >= 0);
    if (wave == 0 && slot >= 0) sh.slot[__popcll(has & ((1ull << lane) - 1))] = slot;
    __syncthreads();
    *expert = __builtin_amdgcn_readfirstlane(e);
    return __popcll(has);
}

template <class C>
__device__ __forceinline__ const void *expert_at(const void *w, int64_t e, int64_t K, int64_t N) {
    return static_cast<const typename C::Elt *>(w) + e * K * N;
}
__device__ __forceinline__ const uint8_t *scales_at(const uint8_t *s, int64_t e, int64_t K, int64_t N) {
    return s + e * ((K + 127) / 128) * N * 4;
}

// The rows of x as operands.
template <class C>
struct RowsOfX {
    const FewArgs &p;
    const int *slot;   // nullptr: row r is token r
    int n, r0, per, lane;
    __device__ __forceinline__ int token(int m) const {
        const int r = r0 + 16 * m + (lane & 15);
        if (!slot) return r < n ? r : 0;
        return slot[r < n ? r : 0] / per;
    }
    __device__ __forceinline__ typename C::X operator()(int m, int k) const {
        typename C::X v;
        const int t = token(m);
        if constexpr (C::kMx) {
            const uint8_t *row = p.xq + static_cast<int64_t>(t) * p.d + k;
            const int quad = lane >> 4;
            const i32x4_t z = {0, 0, 0, 0};
            const i32x4_t lo = k + 16 * quad < p.d ? *reinterpret_cast<const i32x4_t *>(row + 16 * quad) : z;
            const i32x4_t hi = k + 64 + 16 * quad < p.d ? *reinterpret_cast<const i32x4_t *>(row + 64 + 16 * quad) : z;
            v.v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
            v.s = *reinterpret_cast<const int *>(p.xs + (static_cast<int64_t>(k >> 7) * p.T + t) * 4);
        } else {
            const auto *row = static_cast<const typename C::Elt *>(p.x) + static_cast<int64_t>(t) * p.d + k;
#pragma unroll
            for (int i = 0; i < static_cast<int>(sizeof(v) / 16); ++i)
                v.v[i] = k < p.d ? reinterpret_cast<const i32x4_t *>(row)[i] : i32x4_t{0, 0, 0, 0};
        }
        return v;
    }
};

// f(tiles, first row) for n rows: MT tiles of 16 rows at a time, one where they suffice.
template <int MT, class F>
__device__ __forceinline__ void by_tiles(int n, F f) {
    for (int r0 = 0; r0 < n; r0 += 16 * MT) {
        if (MT == 1 || n - r0 <= 16) f(std::integral_constant<int, 1>{}, r0);
        else f(std::integral_constant<int, MT>{}, r0);
    }
}

// H1 and H3 of one expert's rows: a strip of columns, a part of K.
template <class C, int MT>
__device__ __forceinline__ void up_unit(const FewArgs &p, const FewFfn &f, int e, int n, const int *slot, int per,
                                        int strip, int part, FewShared<C> &sh) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = strip * C::BN;
    const void *const w[2] = {expert_at<C>(f.w1, e, p.d, f.h), expert_at<C>(f.w3, e, p.d, f.h)};
    const uint8_t *const ws[2] = {C::kMx ? scales_at(f.w1s, e, p.d, f.h) : nullptr,
                                  C::kMx ? scales_at(f.w3s, e, p.d, f.h) : nullptr};
    const int ka = part * f.up_len, kb = min(p.d, ka + f.up_len);
    by_tiles<MT>(n, [&](auto tiles, int r0) {
        constexpr int M = decltype(tiles)::value;
        f32x4_t acc[2][M][C::CV];
        C::template run<2, M>(w, ws, p.d, f.h, n0, ka, kb, RowsOfX<C>{p, slot, n, r0, per, lane}, sh.stage, lane, wave, acc);
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const int r = r0 + 16 * m + (threadIdx.x >> 4), c = n0 + C::CV * (threadIdx.x & 15);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                float v[C::CV];
                sum_waves<C>(sh, acc[b][m], lane, wave, v);
                if (r < n && c < f.h) {
                    const int sl = slot ? slot[r] : r;
                    float *o = f.hp + (static_cast<int64_t>(part) * f.slots + sl) * 2 * f.h + b * f.h + c;
#pragma unroll
                    for (int i = 0; i < C::CV; i += 4)
                        *reinterpret_cast<float4 *>(o + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                }
            }
        }
    });
}

// ------------------------------------------------------------------- kernels

// 1: the gate's blocks first (what follows waits for them), then the shared experts'
template <class C, class G, int MT>
__global__ __launch_bounds__(kFewThreads) void few_gate_kernel(FewArgs p) {
    __shared__ union { FewShared<C> c; FewShared<G> g; } sh;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int strips = (p.E + G::BN - 1) / G::BN;
    int b = static_cast<int>(blockIdx.x);
    if (b >= strips * p.gate_parts) {
        b -= strips * p.gate_parts;
        up_unit<C, MT>(p, p.s, 0, p.T, nullptr, 1, b / p.s.up_parts, b % p.s.up_parts, sh.c);
        return;
    }
    const int n0 = (b / p.gate_parts) * G::BN, part = b % p.gate_parts;
    const void *const w[1] = {p.wg};
    const uint8_t *const ws[1] = {nullptr};
    const int ka = part * p.gate_len, kb = min(p.d, ka + p.gate_len);
    by_tiles<MT>(p.T, [&](auto tiles, int r0) {
        constexpr int M = decltype(tiles)::value;
        f32x4_t acc[1][M][G::CV];
        G::template run<1, M>(w, ws, p.d, p.E, n0, ka, kb, RowsOfX<G>{p, nullptr, p.T, r0, 1, lane}, sh.g.stage, lane, wave,
                              acc);
#pragma unroll
        for (int m = 0; m < M; ++m) {
            float v[G::CV];
            sum_waves<G>(sh.g, acc[0][m], lane, wave, v);
            const int t = r0 + 16 * m + (threadIdx.x >> 4), c = n0 + G::CV * (threadIdx.x & 15);
#pragma unroll
            for (int i = 0; i < G::CV; ++i)
                if (t < p.T && c + i < p.E) p.zp[(static_cast<int64_t>(part) * p.T + t) * p.E + c + i] = v[i];
        }
    });
}

// Order of fp32 values as whole numbers (ascending, -0 as 0), never 0; NaN above all.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    if ((u & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// 2: a wave for each token; lane l holds the experts l, l + 64, ...  k rounds of an
// arg-max under (value descending, index ascending).  Whatever the logits hold, the k
// ids are distinct and in range.
template <int QQ>
__global__ __launch_bounds__(64) void few_topk_kernel(FewArgs p) {
    const int lane = threadIdx.x, t = blockIdx.x;
    float s[QQ], mx = -INFINITY;
    uint32_t key[QQ];
#pragma unroll
    for (int q = 0; q < QQ; ++q) {
        const int e = lane + 64 * q;
        s[q] = -INFINITY;
        key[q] = 0u;
        if (e < p.E) {
            float z = p.zp[static_cast<int64_t>(t) * p.E + e];
            for (int i = 1; i < p.gate_parts; ++i) z += p.zp[(static_cast<int64_t>(i) * p.T + t) * p.E + e];
            z = __fmul_rn(z, p.scale);
            if (p.lbias) z = __fadd_rn(z, p.lbias[e]);
            s[q] = z;
            p.logits[static_cast<int64_t>(t) * p.E + e] = z;
            key[q] = order_key(p.sbias ? __fadd_rn(z, p.sbias[e]) : z);
            mx = fmaxf(mx, z);
        }
    }
    mx = wave_max(mx);
    float den = 0.0f;
#pragma unroll
    for (int q = 0; q < QQ; ++q)
        if (lane + 64 * q < p.E) den += expf(s[q] - mx);
    den = wave_sum(den);
    for (int j = 0; j < p.k; ++j) {
        uint32_t best = 0u;
        int at = 0;
#pragma unroll
        for (int q = 0; q < QQ; ++q)
            if (key[q] > best) {
                best = key[q];
                at = q;
            }
        uint32_t top = best;
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), off, 64)));
        int e = best == top ? lane + 64 * at : 0x7fffffff;
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) e = min(e, __shfl_xor(e, off, 64));
        if ((e & 63) == lane) {
#pragma unroll
            for (int q = 0; q < QQ; ++q)
                if (q == e >> 6) {
                    key[q] = 0u;
                    p.ids[t * p.k + j] = e;
                    p.w[t * p.k + j] = expf(s[q] - mx) / den;
                }
        }
    }
}

// 3
template <class C, int MT>
__global__ __launch_bounds__(kFewThreads) void few_up_kernel(FewArgs p) {
    __shared__ FewShared<C> sh;
    const int strips = (p.r.h + C::BN - 1) / C::BN;
    const int per = strips * p.r.up_parts;
    const int a = static_cast<int>(blockIdx.x) / per, rem = static_cast<int>(blockIdx.x) % per;
    int e;
    const int n = find_unit<C>(p, a, sh, &e);
    if (n == 0) return;
    up_unit<C, MT>(p, p.r, e, n, sh.slot, p.k, rem / p.r.up_parts, rem % p.r.up_parts, sh);
}

// The activations of a block's rows in shared memory: 16 MT rows of a part of h, in the
// weights' dtype (rows of LD bytes), or in 8 bits with their scale dwords.
template <class C, int MT, int KP>
struct ActTile {
    static constexpr int LD = KP * static_cast<int>(sizeof(typename C::Elt)) + 16;  // 16 more: neighbouring rows on other banks
    __align__(16) char v[16 * MT][LD];
    uint32_t s[C::kMx ? KP / 128 : 1][16 * MT];
};
template <class C, int MT, int KP>
struct RowsOfAct {
    const ActTile<C, MT, KP> &t;
    int ka, lane;
    __device__ __forceinline__ typename C::X operator()(int m, int k) const {
        typename C::X v;
        const int r = 16 * m + (lane & 15);
        const char *row = t.v[r] + (k - ka) * static_cast<int>(sizeof(typename C::Elt));
        if constexpr (C::kMx) {
            const int quad = lane >> 4;
            v.v = __builtin_shufflevector(*reinterpret_cast<const i32x4_t *>(row + 16 * quad),
                                          *reinterpret_cast<const i32x4_t *>(row + 64 + 16 * quad), 0, 1, 2, 3, 4, 5, 6, 7);
            v.s = static_cast<int>(t.s[(k - ka) >> 7][r]);
        } else {
#pragma unroll
            for (int i = 0; i < static_cast<int>(sizeof(v) / 16); ++i) v.v[i] = reinterpret_cast<const i32x4_t *>(row)[i];
        }
        return v;
    }
};

// 4: the chosen experts' units first, then the shared ones'
template <class C, int MT, int KP>
__global__ __launch_bounds__(kFewThreads) void few_down_kernel(FewArgs p, int units) {
    __shared__ FewShared<C> sh;
    __shared__ ActTile<C, MT, KP> act;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int strips = (p.d + C::BN - 1) / C::BN;
    int b = static_cast<int>(blockIdx.x);
    const bool shared = b >= units;
    if (shared) b -= units;
    const FewFfn &f = shared ? p.s : p.r;
    const int part = b % f.down_parts, strip = (b / f.down_parts) % strips;
    int e = 0, n = p.T;
    const int *slot = nullptr;
    if (!shared) {
        n = find_unit<C>(p, b / (f.down_parts * strips), sh, &e);
        slot = sh.slot;
        if (n == 0) return;
    }
    const void *const w[1] = {expert_at<C>(f.w2, e, f.h, p.d)};
    const uint8_t *const ws[1] = {C::kMx ? scales_at(f.w2s, e, f.h, p.d) : nullptr};
    const int ka = part * f.down_len, kb = min(f.h, ka + f.down_len);
    const int len = (kb - ka + C::STEP - 1) / C::STEP * C::STEP;  // zeros behind h
    by_tiles<MT>(n, [&](auto tiles, int r0) {
        constexpr int M = decltype(tiles)::value;
        const int nr = min(n - r0, 16 * M);
        __syncthreads();  // the rows before have been read
        for (int i = threadIdx.x; i < nr * (len / 4); i += kFewThreads) {
            const int r = i / (len / 4), c = 4 * (i % (len / 4));
            float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (ka + c < kb) {
                const float *src = f.hp + static_cast<int64_t>(slot ? slot[r0 + r] : r0 + r) * 2 * f.h + ka + c;
                float4 h1 = *reinterpret_cast<const float4 *>(src), h3 = *reinterpret_cast<const float4 *>(src + f.h);
                for (int q = 1; q < f.up_parts; ++q) {
                    src += static_cast<int64_t>(f.slots) * 2 * f.h;
                    const float4 a = *reinterpret_cast<const float4 *>(src), g = *reinterpret_cast<const float4 *>(src + f.h);
                    h1.x += a.x; h1.y += a.y; h1.z += a.z; h1.w += a.w;
                    h3.x += g.x; h3.y += g.y; h3.z += g.z; h3.w += g.w;
                }
                v[0] = silu_f(h1.x) * h3.x; v[1] = silu_f(h1.y) * h3.y; v[2] = silu_f(h1.z) * h3.z; v[3] = silu_f(h1.w) * h3.w;
            }
            if constexpr (C::kMx) {
                // len is a multiple of 128, so that a row's four values in 32 lanes are
                // whole groups, all of them taking part or none
                uint32_t o[1];
                const uint32_t byte = mx8_quant<4>(v, o);
                const uint32_t dw = mx8_scale_dword<4>(ka + c < kb ? byte : kMxOne, lane);
                *reinterpret_cast<uint32_t *>(act.v[r] + c) = o[0];
                if ((c & 127) == 0) act.s[c >> 7][r] = dw;
            } else if constexpr (sizeof(typename C::Elt) == 2) {
                *reinterpret_cast<uint2 *>(act.v[r] + 2 * c) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
            } else {
                *reinterpret_cast<float4 *>(act.v[r] + 4 * c) = make_float4(v[0], v[1], v[2], v[3]);
            }
        }
        __syncthreads();
        f32x4_t acc[1][M][C::CV];
        C::template run<1, M>(w, ws, f.h, p.d, strip * C::BN, ka, kb, RowsOfAct<C, MT, KP>{act, ka, lane}, sh.stage, lane, wave,
                              acc);
#pragma unroll
        for (int m = 0; m < M; ++m) {
            float v[C::CV];
            sum_waves<C>(sh, acc[0][m], lane, wave, v);
            const int r = r0 + 16 * m + (threadIdx.x >> 4), c = strip * C::BN + C::CV * (threadIdx.x & 15);
            if (r < n && c < p.d) {
                float *o = f.yp + (static_cast<int64_t>(part) * f.slots + (slot ? slot[r] : r)) * p.d + c;
#pragma unroll
                for (int i = 0; i < C::CV; i += 4)
                    *reinterpret_cast<float4 *>(o + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
            }
        }
    });
}

// 5: a thread for four columns of a token
template <typename T>
__global__ __launch_bounds__(256) void few_combine_kernel(FewArgs p) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int per = p.d / 4;
    if (i >= static_cast<int64_t>(p.T) * per) return;
    const int t = static_cast<int>(i / per), c = 4 * static_cast<int>(i % per);
    float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    auto parts = [&](const FewFfn &f, int slot, float w) {
        const float *src = f.yp + static_cast<int64_t>(slot) * p.d + c;
        float4 s = *reinterpret_cast<const float4 *>(src);
        for (int q = 1; q < f.down_parts; ++q) {
            src += static_cast<int64_t>(f.slots) * p.d;
            const float4 a = *reinterpret_cast<const float4 *>(src);
            s.x += a.x; s.y += a.y; s.z += a.z; s.w += a.w;
        }
        y[0] = __builtin_fmaf(w, s.x, y[0]); y[1] = __builtin_fmaf(w, s.y, y[1]);
        y[2] = __builtin_fmaf(w, s.z, y[2]); y[3] = __builtin_fmaf(w, s.w, y[3]);
    };
    for (int j = 0; j < p.k; ++j) parts(p.r, t * p.k + j, p.w[t * p.k + j]);
    if (p.s.h) parts(p.s, t, 1.0f);
    T *o = static_cast<T *>(p.y) + static_cast<int64_t>(t) * p.d + c;
    if constexpr (sizeof(T) == 2)
        *reinterpret_cast<uint2 *>(o) = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
    else
        *reinterpret_cast<float4 *>(o) = make_float4(y[0], y[1], y[2], y[3]);
}

// ---------------------------------------------------------------- the launches

struct Plan {
    FewArgs a;
    int64_t gate, shared, up, down, down_shared;  // blocks
    size_t bytes;
};

// parts of K so that `units` units make about `blocks` blocks: lengths are multiples of
// `quantum`, at most `most`
void split(int K, int64_t units, int64_t blocks, int quantum, int most, int *parts, int *len) {
    const int64_t want = std::max<int64_t>(1, blocks / std::max<int64_t>(1, units));
    int64_t l = (K + want - 1) / want;
    l = (l + quantum - 1) / quantum * quantum;
    l = std::min<int64_t>(l, most);
    *len = static_cast<int>(l);
    *parts = static_cast<int>((K + l - 1) / l);
}

template <class C, class G>
Plan make_plan(const FewSizes &z, int KP, char *ws) {
    Plan pl{};
    FewArgs &a = pl.a;
    a.T = static_cast<int>(z.T);
    a.d = z.d;
    a.E = z.E;
    a.k = z.k;
    size_t at = 0;
    auto take = [&](int64_t floats) {
        float *p = reinterpret_cast<float *>(reinterpret_cast<uintptr_t>(ws) + at);
        at += (static_cast<size_t>(floats) * 4 + 255) & ~static_cast<size_t>(255);
        return p;
    };
    constexpr int kBlocks = 512;
    constexpr int Q = C::STEP * kFewWaves;
    const int64_t gs = (z.E + G::BN - 1) / G::BN;
    split(z.d, gs, 64, G::STEP * kFewWaves, 1 << 30, &a.gate_parts, &a.gate_len);
    pl.gate = gs * a.gate_parts;
    a.zp = take(static_cast<int64_t>(a.gate_parts) * a.T * a.E);
    const int64_t active = std::min<int64_t>(static_cast<int64_t>(a.T) * a.k, a.E);
    const int64_t ds = (z.d + C::BN - 1) / C::BN;
    auto ffn = [&](FewFfn &f, int h, int64_t units, int slots, int64_t *up, int64_t *down) {
        f.h = h;
        f.slots = slots;
        const int64_t hs = (h + C::BN - 1) / C::BN;
        split(z.d, units * hs, kBlocks, Q, 1 << 30, &f.up_parts, &f.up_len);
        split(h, units * ds, kBlocks, Q, KP, &f.down_parts, &f.down_len);
        f.hp = take(static_cast<int64_t>(f.up_parts) * slots * 2 * h);
        f.yp = take(static_cast<int64_t>(f.down_parts) * slots * z.d);
        *up = units * hs * f.up_parts;
        *down = units * ds * f.down_parts;
    };
    ffn(a.r, z.h, active, a.T * a.k, &pl.up, &pl.down);
    if (z.hs) ffn(a.s, z.hs, 1, a.T, &pl.shared, &pl.down_shared);
    pl.bytes = at;
    return pl;
}

// K of a down-projection part: what its activations may take of shared memory
constexpr int kPartPlain = 512, kPartF32 = 256, kPartMx = 1024;

template <class C, class G, int MT, int KP>
hipError_t launch_as(Plan &pl, hipStream_t s) {
    const FewArgs &a = pl.a;
    hipLaunchKernelGGL((few_gate_kernel<C, G, MT>), dim3(static_cast<unsigned>(pl.gate + pl.shared)), dim3(kFewThreads), 0, s, a);
    const dim3 tokens(static_cast<unsigned>(a.T));
    if (a.E <= 64) hipLaunchKernelGGL((few_topk_kernel<1>), tokens, dim3(64), 0, s, a);
    else if (a.E <= 256) hipLaunchKernelGGL((few_topk_kernel<4>), tokens, dim3(64), 0, s, a);
    else hipLaunchKernelGGL((few_topk_kernel<16>), tokens, dim3(64), 0, s, a);
    hipLaunchKernelGGL((few_up_kernel<C, MT>), dim3(static_cast<unsigned>(pl.up)), dim3(kFewThreads), 0, s, a);
    hipLaunchKernelGGL((few_down_kernel<C, MT, KP>), dim3(static_cast<unsigned>(pl.down + pl.down_shared)), dim3(kFewThreads), 0,
                       s, a, static_cast<int>(pl.down));
    const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(a.T) * (a.d / 4) + 255) / 256));
    if constexpr (std::is_same<C, PlainCore<float>>::value)
        hipLaunchKernelGGL((few_combine_kernel<float>), grid, dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((few_combine_kernel<bf16_t>), grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

template <class C, class G, int KP>
hipError_t launch_core(const FewSizes &z, const FewTensors &t, hipStream_t s) {
    Plan pl = make_plan<C, G>(z, KP, static_cast<char *>(t.ws));
    FewArgs &a = pl.a;
    a.x = t.x;
    a.xq = static_cast<const uint8_t *>(t.xq);
    a.xs = static_cast<const uint8_t *>(t.xs);
    a.wg = t.wg;
    a.scale = t.scale;
    a.lbias = t.lbias;
    a.sbias = t.sbias;
    a.ids = t.ids;
    a.w = t.w;
    a.logits = t.logits;
    a.y = t.y;
    auto set = [](FewFfn &f, const FewWeights &w) {
        f.w1 = w.w1; f.w3 = w.w3; f.w2 = w.w2;
        f.w1s = static_cast<const uint8_t *>(w.w1s);
        f.w3s = static_cast<const uint8_t *>(w.w3s);
        f.w2s = static_cast<const uint8_t *>(w.w2s);
    };
    set(a.r, t.routed);
    set(a.s, t.shared);
    return z.T <= 16 ? launch_as<C, G, 1, KP>(pl, s) : launch_as<C, G, 2, KP>(pl, s);
}

}  // namespace

size_t few_workspace(const FewSizes &z) {
    if (z.mx8) return make_plan<Mx8Core, PlainCore<bf16_t>>(z, kPartMx, nullptr).bytes;
    return z.dt == kBF16 ? make_plan<PlainCore<bf16_t>, PlainCore<bf16_t>>(z, kPartPlain, nullptr).bytes
                         : make_plan<PlainCore<float>, PlainCore<float>>(z, kPartF32, nullptr).bytes;
}

hipError_t launch_layer_few(const FewSizes &z, const FewTensors &t, hipStream_t s) {
    if (z.T <= 0) return hipSuccess;
    if (z.mx8) return launch_core<Mx8Core, PlainCore<bf16_t>, kPartMx>(z, t, s);
    return z.dt == kBF16 ? launch_core<PlainCore<bf16_t>, PlainCore<bf16_t>, kPartPlain>(z, t, s)
                         : launch_core<PlainCore<float>, PlainCore<float>, kPartF32>(z, t, s);
}

}  // namespace xmoe

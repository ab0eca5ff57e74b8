// The whole layer for a few tokens (at most 64): gate, top-k, experts, shared
// experts and combine.
//
// The layer's other path sorts rows by expert and multiplies 128-row tiles; with a
// token or two for each expert its time is launches, searches for tiles and rows that
// are not there.  Here the weights that the tokens chose are streamed past their rows,
// once for each 16 (or 32) rows of an expert, and what one product leaves for the next
// stays in the caches:
//   1  partial logits of the gate, and the shared experts' H1, H3 (they need no
//      routing): K split over blocks
//   2  softmax and top-k, a wave for each token (up to four tokens: at the start of 3)
//   3  H1, H3 of the chosen experts
//   4  the down-projections, silu(H1) * H3 formed on the way in
//   5  y = sum_j p_j (parts of slot j) + parts of the shared experts
// Slot t k + j is token t's j-th choice; a unit of work is one expert (a chosen one or
// the shared ones side by side), a strip of its columns and a part of its rows.
// Every sum over parts runs in part order: no atomics, the same bits each time.
//
// Bound by the weights' bytes, which a plain read of as much takes 7 TB/s for (1 GB; 64 MB
// 5.9, 24 MB 4.5, launches in a row), and for one token by four launches' starts and the
// waits from one to the next.  Measured as layers, replayed from a graph (d = 2048, 64
// experts of h = 1408, top-6, two shared; bf16 / 8-bit weights behind the norm; the layer's
// sequence in brackets): 1 token 45 / 39 us (135 / 73, for 138 and 71 MB), 4 90 / 63 (148 /
// 91), 16 180 / 113 (241 / 133), 64 226 / 139 us (259 / 148, for 1.1 and 0.57 GB).  64 tokens
// on 160 experts of d = 4096, h = 1024, top-8 658 us (762), of which the up-projection is
// 409: 6.3 TB/s.
// The sequence wins where experts have many rows: with 8-bit weights and few experts from
// about 32 tokens on (16 experts, top-4: 55 against 61 us at 16 tokens, 62 against 62 at 32,
// 78 against 65 at 64), with bf16 where 64 tokens take every expert (16 experts of 64 rows:
// 188 against 143; 8 experts: 99 against 110), and by far where many tokens meet on a few
// experts of many (64 tokens on 8 of those 160: 608 against 218 us; 12 tokens on them: 83
// against 211), since further passes over a part's weights come from memory again.
//
// A block's row tiles (one of 16 rows, or two) are a template argument, and which of the
// two instances runs is decided in front of its loop: with a branch around the second
// tile's products hipcc leaves too few waits between a matrix instruction and the copy of
// its result that a branch jumps to (ROCm 7.2, fp32: four columns of 64 were wrong).
// Two tiles at a time where experts have more than 8 rows on average (see make_plan).  An
// expert with more rows than that takes further passes over its weights.
//
// Products: the weights are the first operand of the matrix instruction (16 columns),
// the rows the second (16 rows), so that a row costs nothing up to 16 of them and rows
// that are not there may hold anything: a row's results depend on it alone.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "common.hpp"
#include "few.hpp"
#include "gemm.hpp"
#include "kernels.hpp"
#include "mx8.hpp"

namespace xmoe {

namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int kFewWaves = 4;
constexpr int kFewThreads = 64 * kFewWaves;
// Weights pass the caches by: with an even choice of experts nothing reads them again soon
// (64 tokens on 160 experts 650 -> 716 us without, in 8 bits 372 -> 415).  All 64 on the
// same 8 of them, four passes over the same weights, would gain from the caches (671 ->
// 505 us, in 8 bits 279 -> 232).
constexpr int kNt = 2;
// Blocks that a small launch is cut into: two on a compute unit, where four would fit (384,
// 512, 640, 1024: one token in bf16 42.9, 41.8, 43.7, 42.4 us, in 8 bits 36.1, 34.5, 34.9,
// 34.9; 5 fp32 tokens of 30 experts 34.4, 31.2, 31.3, 31.2), and one of long parts (2048:
// 4 tokens of 32 8-bit experts 237 -> 245 us, 1280: 12 tokens 112.5 -> 117).
constexpr int kFewBlocks = 512, kBlocks = 1536;
constexpr int kGateParts = 16;    // of the gate's sums: what the top-k reads for each logit
constexpr int kPartRows = 16;     // see make_plan
// Strips (times parts) from which each is a wave's own (see few_down_kernel): 64 tokens of 64
// bf16 experts, 1.5 times as many, 207 us so and 215 by blocks, 12 tokens of them 149, 151.
constexpr int kManyStrips = 2048;
// Tokens and slots whose top-k the up-projection's blocks find themselves: a wave for each
// token, no launch (4.5 us) between the gate and the experts.
constexpr int kInlineTokens = kFewWaves, kInlineSlots = 64;

// One set of experts: the routed ones, or the shared ones as a single expert.
struct FewFfn {
    const void *w1, *w3, *w2;            // [n, K, N], or 8 bits [n, N, K]
    const uint8_t *w1s, *w3s, *w2s;      // 8 bits: scales [n, ceil(K / 128), N, 4]
    int h;
    int slots;                           // rows of the partial sums
    int up_parts, up_len, down_parts, down_len;
    int down_strips;                     // strips that a block of the down-projection takes
    float *hp;                           // [up_parts, slots, 2h]  parts of H1 | H3
    float *yp;                           // [down_parts, slots, d] parts of the outputs
    void *act;                           // [slots, h] activations, where a launch of their own forms them; or nullptr
    int chunks;                          // blocks that share a unit's rows, 16 (or 32) each
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
//
// A core multiplies a strip of BN columns of a matrix with M tiles of 16 rows over K in
// [ka, kb).  WK of the block's waves take the steps of K in turn (the up-projection's
// waves are two for W1 and two for W3, so that a wave's registers leave room for four
// on a SIMD: what counts is how many loads are under way); each holds sums of its own,
// added in wave order at the end.  start() asks for the weights of a wave's first step
// before anything that they do not need (with the rows, where these come from memory:
// Rows::kEarly); finish() runs the steps.

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
    // An activation is held in 32 bits: fp32, or for bf16's products as the sum of two
    // bf16 values, 2^-17 from it (rounded to one it adds an error of y's own rounding's
    // size, 1.4 times as much in all; the second product waits for no memory: level).
    // Eight of them are eight first halves, then eight second ones.
    struct Pair {
        bf16_t v[2];
    };
    using Act = std::conditional_t<sizeof(T) == 2, Pair, float>;
    static constexpr bool kMx = false;
    static constexpr int CV = 16 / static_cast<int>(sizeof(T)), BN = 16 * CV, STEP = 32;
    static constexpr int kStage = 16;  // no staging
    static constexpr int kLeast = 384;
    // K of a down-projection part at most: what its activations may take of shared memory
    static constexpr int kPart = 1024 / static_cast<int>(sizeof(T));
    struct X {
        i32x4_t v[sizeof(T) / 2];  // eight elements of a row
    };
    struct XAct {
        i32x4_t v[2];              // eight activations
    };
    // of x [rows, d]: the eight elements at k + 8 (l / 16)
    struct Raw {
        X x;
    };
    __device__ static __forceinline__ void load_row(const FewArgs &p, int t, int k, int lane, Raw &r) {
        const int at = k + 8 * (lane >> 4);
        const T *row = static_cast<const T *>(p.x) + t * p.d + at;  // 64 * 65536 elements at most
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(X) / 16); ++i)
            r.x.v[i] = at < p.d ? reinterpret_cast<const i32x4_t *>(row)[i] : i32x4_t{0, 0, 0, 0};
    }
    __device__ static __forceinline__ void open_row(const Raw &r, X &x) { x = r.x; }
    // of a row of activations in shared memory, k from the part's start
    __device__ static __forceinline__ void act_row(const char *row, int k, int lane, XAct &x) {
#pragma unroll
        for (int i = 0; i < 2; ++i) x.v[i] = reinterpret_cast<const i32x4_t *>(row + (k + 8 * (lane >> 4)) * 4)[i];
    }
    // bytes from a row's start to the activations c, c + 1, ...
    __device__ static __forceinline__ int act_at(int c) { return sizeof(T) == 2 ? 32 * (c >> 3) + 2 * (c & 7) : 4 * c; }

    template <int M, int WK, class Rows>
    struct Product {
        struct Step {
            i32x4_t w[8];
            Raw x[Rows::kEarly ? M : 1];
        };
        __amdgpu_buffer_rsrc_t rs;
        uint32_t rowb, col;
        int lane, kb, k0, k;
        Step p;
        f32x4_t acc[M][CV];

        __device__ __forceinline__ void fetch(int at_k, Step &s, const Rows &rows) const {
            // a step past the part reads nothing
            const uint32_t at = at_k < kb ? static_cast<uint32_t>(at_k + 8 * (lane >> 4)) * rowb + col : kOob;
            const uint32_t row = at_k < kb ? rowb : 0u;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                s.w[j] = __builtin_bit_cast(
                    i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rs, static_cast<int>(at + j * row), 0, kNt));
            if constexpr (Rows::kEarly)
#pragma unroll
                for (int m = 0; m < M; ++m) rows.load(m, at_k, s.x[m]);
        }
        __device__ __forceinline__ Product(const void *w, const uint8_t *, int K, int N, int ka, int kb_, int lane_, int wk,
                                           char *)
            : rowb(static_cast<uint32_t>(N) * static_cast<uint32_t>(sizeof(T))), lane(lane_), kb(kb_), k0(ka + STEP * wk) {
            rs = make_rsrc(w, static_cast<int64_t>(K) * N * static_cast<int>(sizeof(T)));
        }
        __device__ __forceinline__ void start(int n0, const Rows &rows) {
            col = static_cast<uint32_t>(n0 + CV * (lane & 15)) * static_cast<uint32_t>(sizeof(T));
            k = k0;
            fetch(k, p, rows);
        }
        __device__ __forceinline__ void multiply(const Step &s, int at_k, const Rows &rows) {
            typename Rows::X x[M];
#pragma unroll
            for (int m = 0; m < M; ++m) {
                if constexpr (Rows::kEarly) open_row(s.x[m], x[m]);
                else rows.read(m, at_k, x[m]);
            }
            if constexpr (sizeof(T) == 2) {
#pragma unroll
                for (int i = 0; i < CV; ++i) {
                    __builtin_amdgcn_sched_barrier(0);  // else the operands of all products are made first and spill
                    i32x4_t o;
#pragma unroll
                    for (int z = 0; z < 4; ++z)
                        o[z] = static_cast<int>(__builtin_amdgcn_perm(static_cast<uint32_t>(s.w[2 * z + 1][i / 2]),
                                                                      static_cast<uint32_t>(s.w[2 * z][i / 2]),
                                                                      i % 2 ? 0x07060302u : 0x05040100u));
#pragma unroll
                    for (int h = 0; h < static_cast<int>(sizeof(x[0].v) / 16); ++h)
#pragma unroll
                        for (int m = 0; m < M; ++m)
                            acc[m][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                __builtin_bit_cast(bf16x8_t, o), __builtin_bit_cast(bf16x8_t, x[m].v[h]), acc[m][i], 0, 0, 0);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int i = 0; i < CV; ++i)
#pragma unroll
                        for (int m = 0; m < M; ++m)
                            acc[m][i] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                                __builtin_bit_cast(float, static_cast<int>(s.w[j][i])),
                                __builtin_bit_cast(float, static_cast<int>(x[m].v[j / 4][j % 4])), acc[m][i], 0, 0, 0);
                }
            }
        }
        __device__ __forceinline__ void finish(const Rows &rows) {
#pragma unroll
            for (int m = 0; m < M; ++m)
#pragma unroll
                for (int i = 0; i < CV; ++i) acc[m][i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
            while (k < kb) {
                multiply(p, k, rows);
                k += STEP * WK;
                fetch(k, p, rows);
            }
        }
    };

    // f(column of the strip, four results from it) for the lane's results
    template <class F>
    __device__ static __forceinline__ void each(const f32x4_t (&acc)[CV], int lane, F f) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int i = 0; i < CV; i += 4)
                f(4 * CV * (lane >> 4) + CV * r + i, f32x4_t{acc[i][r], acc[i + 1][r], acc[i + 2][r], acc[i + 3][r]});
    }
};

// 16 e4m3 bytes times 2^(b - 127) as bf16, exact (values below bf16's smallest normal
// number, 2^-126, count as zeros); b = 255: NaNs
__device__ __forceinline__ void open8(const i32x4_t &v, int b, i32x4_t (&o)[2]) {
    typedef __bf16 bf2_t __attribute__((ext_vector_type(2)));
    const float s = mx8_scale(static_cast<uint32_t>(b) & 255u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bf2_t lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(static_cast<uint32_t>(v[i]), s, false);
        const bf2_t hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(static_cast<uint32_t>(v[i]), s, true);
        o[i / 2][2 * (i % 2)] = __builtin_bit_cast(int, lo);
        o[i / 2][2 * (i % 2) + 1] = __builtin_bit_cast(int, hi);
    }
}

// 8-bit weights [N, K] with scales: a wave's step is 128 of K by 64 columns (of each
// matrix), read as whole 128-byte lines, eight rows a load, and turned in a piece of
// shared memory of the wave's own so that lane l gets the 32 bytes 32 (l / 16) of row
// l % 16: one scale block.  They become bf16, which holds them exactly, and four
// products of 32 of K (lane group q has bytes 32 q + 8 z of the z-th): the scaled matrix
// instruction would take them as they are, but cuts its products at 2^-13 of the largest
// of eight, which turns one in 600 activations to the next byte (one token's error 3.8e-3
// against 1.7e-3), and here it has nothing to win: both wait for the weights.
// Lane l's results are columns 16 j + 4 (l / 16) + r of row l % 16.
struct Mx8Core {
    using Elt = uint8_t;
    using Act = bf16_t;   // activations rounded to 8 bits, held as bf16
    static constexpr bool kMx = true;
    static constexpr int CV = 4, BN = 64, STEP = 128;
    static constexpr int kStage = kFewWaves * 4096;
    static constexpr int kLeast = 1024, kPart = 512;
    struct X {
        i32x4_t v[4];   // elements 32 (l / 16) + 8 z of the row's 128
    };
    using XAct = X;
    struct Raw {
        i32x4_t v[2];
        int s;
    };
    __device__ static __forceinline__ void load_row(const FewArgs &p, int t, int k, int lane, Raw &r) {
        const int at = k + 32 * (lane >> 4);
        const bool in = at < p.d;
        const i32x4_t z = {0, 0, 0, 0};
        const i32x4_t *row = reinterpret_cast<const i32x4_t *>(p.xq + t * p.d + at);
        r.v[0] = in ? row[0] : z;
        r.v[1] = in ? row[1] : z;
        r.s = in ? p.xs[(static_cast<int64_t>(k >> 7) * p.T + t) * 4 + (lane >> 4)] : 127;
    }
    __device__ static __forceinline__ void open_row(const Raw &r, X &x) {
        i32x4_t o[2];
        open8(r.v[0], r.s, o);
        x.v[0] = o[0];
        x.v[1] = o[1];
        open8(r.v[1], r.s, o);
        x.v[2] = o[0];
        x.v[3] = o[1];
    }
    __device__ static __forceinline__ void act_row(const char *row, int k, int lane, X &x) {
#pragma unroll
        for (int z = 0; z < 4; ++z) x.v[z] = *reinterpret_cast<const i32x4_t *>(row + 2 * (k + 32 * (lane >> 4) + 8 * z));
    }
    __device__ static __forceinline__ int act_at(int c) { return 2 * c; }

    template <int M, int WK, class Rows>
    struct Product {
        struct Step {
            i32x4_t w[4][2];
            int s[4];
            Raw x[Rows::kEarly ? M : 1];
        };
        __amdgpu_buffer_rsrc_t rw, rsc;
        int K, N, kb, k0, k, lane, boff;
        int col[4];
        char *mine;
        Step p;
        f32x4_t acc[M][CV];

        __device__ __forceinline__ void fetch(int at_k, Step &f, const Rows &rows) const {
            // K may end inside a step (zeros behind it); a step past the part reads nothing
            const bool in = at_k < kb && at_k + 16 * (lane & 7) < K;
            const int sc = at_k < kb ? ((at_k >> 7) * N + (lane & 15)) * 4 : kOob;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int at = in ? col[j] * K + at_k + boff : kOob, at8 = in ? at + 8 * K : kOob;
                f.w[j][0] = __builtin_bit_cast(i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rw, at, 0, kNt));
                f.w[j][1] = __builtin_bit_cast(i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rw, at8, 0, kNt));
                f.s[j] = static_cast<int>(__builtin_amdgcn_raw_buffer_load_b32(rsc, at_k < kb ? sc + 4 * col[j] : kOob, 0, 0));
            }
            if constexpr (Rows::kEarly)
#pragma unroll
                for (int m = 0; m < M; ++m) rows.load(m, at_k, f.x[m]);
        }
        __device__ __forceinline__ Product(const void *w, const uint8_t *s, int K_, int N_, int ka, int kb_, int lane_, int wk,
                                           char *stage)
            : K(K_), N(N_), kb(kb_), k0(ka + STEP * wk), lane(lane_), mine(stage) {
            rw = make_rsrc(w, static_cast<int64_t>(N_) * K_);
            rsc = make_rsrc(s, static_cast<int64_t>((K_ + 127) / 128) * N_ * 4);
            boff = (lane >> 3) * K + 16 * (lane & 7);
        }
        __device__ __forceinline__ void start(int n0, const Rows &rows) {
#pragma unroll
            for (int j = 0; j < 4; ++j) col[j] = n0 + 16 * j < N ? n0 + 16 * j : n0;  // past N: the strip's first
            k = k0;
            fetch(k, p, rows);
        }
        __device__ __forceinline__ void multiply(const Step &f, int at_k, const Rows &rows) {
            const int l16 = lane & 15, quad = lane >> 4;
            char *const put = mine + (lane >> 3) * 128 + 16 * ((lane & 7) ^ (lane >> 3));
            const char *const lo_at = mine + l16 * 128 + 16 * ((2 * quad) ^ (l16 & 7));
            const char *const hi_at = mine + l16 * 128 + 16 * ((2 * quad + 1) ^ (l16 & 7));
            X x[M];
#pragma unroll
            for (int m = 0; m < M; ++m) {
                if constexpr (Rows::kEarly) open_row(f.x[m], x[m]);
                else rows.read(m, at_k, x[m]);
            }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    __builtin_amdgcn_sched_barrier(0);
                    const int at = (j & 1) * 2048;
                    *reinterpret_cast<i32x4_t *>(put + at) = f.w[j][0];
                    *reinterpret_cast<i32x4_t *>(put + at + 1024) = f.w[j][1];
                    __builtin_amdgcn_wave_barrier();  // a wave's accesses to shared memory are served in order
                    const i32x4_t lo = *reinterpret_cast<const i32x4_t *>(lo_at + at);
                    const i32x4_t hi = *reinterpret_cast<const i32x4_t *>(hi_at + at);
                    __builtin_amdgcn_wave_barrier();
                    const int sc = f.s[j] >> (8 * quad);
                    i32x4_t o[4], u[2];
                    open8(lo, sc, u);
                    o[0] = u[0];
                    o[1] = u[1];
                    open8(hi, sc, u);
                    o[2] = u[0];
                    o[3] = u[1];
#pragma unroll
                    for (int z = 0; z < 4; ++z)
#pragma unroll
                        for (int m = 0; m < M; ++m)
                            acc[m][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                __builtin_bit_cast(bf16x8_t, o[z]), __builtin_bit_cast(bf16x8_t, x[m].v[z]), acc[m][j], 0, 0, 0);
                }
        }
        __device__ __forceinline__ void finish(const Rows &rows) {
#pragma unroll
            for (int m = 0; m < M; ++m)
#pragma unroll
                for (int i = 0; i < CV; ++i) acc[m][i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
            while (k < kb) {
                multiply(p, k, rows);
                k += STEP * WK;
                fetch(k, p, rows);
            }
        }
    };

    template <class F>
    __device__ static __forceinline__ void each(const f32x4_t (&acc)[CV], int lane, F f) {
#pragma unroll
        for (int j = 0; j < 4; ++j) f(16 * j + 4 * (lane >> 4), acc[j]);
    }
};

// What a block keeps in shared memory beside its activations.
template <class C>
struct FewStage {
    __align__(16) char stage[C::kStage];
    int slot[kFewTokens];
};
template <class C>
struct FewShared : FewStage<C> {
    float red[kFewWaves][16][C::BN + 4];
};

// A value that the compiler takes as new at this point: the addresses made from it are
// made here, instead of in front of the loops around it and kept (they spilled).
__device__ __forceinline__ int fresh(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

// The waves' parts of 16 rows x BN columns, those of each WK waves added in wave order:
// thread tid has row tid / 16, columns CV (tid % 16) ..
template <class C, int WK, class Shared>
__device__ __forceinline__ void sum_waves(Shared &sh, const f32x4_t (&acc)[C::CV], int lane, int wave,
                                          float (&out)[kFewWaves / WK][C::CV]) {
    __syncthreads();
    C::each(acc, fresh(lane), [&](int c, f32x4_t v) { *reinterpret_cast<f32x4_t *>(&sh.red[wave][lane & 15][c]) = v; });
    __syncthreads();
    const int tid = fresh(threadIdx.x), row = tid >> 4, c0 = C::CV * (tid & 15);
#pragma unroll
    for (int b = 0; b < kFewWaves / WK; ++b) {
#pragma unroll
        for (int i = 0; i < C::CV; ++i) out[b][i] = sh.red[b * WK][row][c0 + i];
#pragma unroll
        for (int w = 1; w < WK; ++w)
#pragma unroll
            for (int i = 0; i < C::CV; ++i) out[b][i] += sh.red[b * WK + w][row][c0 + i];
    }
}

// Unit a of the chosen experts: with fewer slots than experts, the expert of slot a if
// no earlier slot chose it, else expert a.  Its slots by ascending token go to
// sh.slot (ends with a barrier); returns the number of rows, 0: no such unit.
template <class C>
__device__ __forceinline__ int find_unit(const FewArgs &p, const int32_t *ids, int a, FewStage<C> &sh, int *expert) {
    const int lane = threadIdx.x & 63;
    const bool by_slot = p.T * p.k <= p.E;
    const int e = __builtin_amdgcn_readfirstlane(by_slot ? ids[a] : a);
    int slot = -1;
    if (lane < p.T) {
        const int32_t *mine = ids + lane * p.k;
#pragma unroll 8
        for (int j = 0; j < p.k; ++j) slot = mine[j] == e ? lane * p.k + j : slot;
    }
    const unsigned long long has = __ballot(slot >= 0);
    if (has == 0) return 0;
    if (by_slot && __shfl(slot, __ffsll(has) - 1, 64) != a) return 0;
    if (threadIdx.x < 64 && slot >= 0) sh.slot[__popcll(has & ((1ull << lane) - 1))] = slot;
    __syncthreads();
    *expert = e;
    return __popcll(has);
}

template <class C>
__device__ __forceinline__ const void *expert_at(const void *w, int64_t e, int64_t K, int64_t N) {
    return static_cast<const typename C::Elt *>(w) + e * K * N;
}
__device__ __forceinline__ const uint8_t *scales_at(const uint8_t *s, int64_t e, int64_t K, int64_t N) {
    return s + e * ((K + 127) / 128) * N * 4;
}

// The rows of x as operands, asked for with the weights; slot nullptr: row r is token r.
template <class C, int M>
struct RowsOfX {
    using X = typename C::X;
    static constexpr bool kEarly = true;
    const FewArgs &p;
    int t[M], lane;
    __device__ __forceinline__ RowsOfX(const FewArgs &p_, const int *slot, int n, int r0, int lane_) : p(p_), lane(lane_) {
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const int r = r0 + 16 * m + (lane & 15), at = r < n ? r : 0;
            t[m] = slot ? slot[at] / p.k : at;
        }
    }
    __device__ __forceinline__ void load(int m, int k, typename C::Raw &raw) const { C::load_row(p, t[m], k, lane, raw); }
};

// f(tiles, first row) for the rows of one of `chunks` blocks: MT tiles of 16 rows at a
// time, one where they suffice.
template <int MT, class F>
__device__ __forceinline__ void by_tiles(int n, int chunk, int chunks, F f) {
    for (int r0 = 16 * MT * chunk; r0 < n; r0 += 16 * MT * chunks) {
        if (MT == 1 || n - r0 <= 16) f(std::integral_constant<int, 1>{}, r0);
        else f(std::integral_constant<int, MT>{}, r0);
    }
}

// H1 and H3 of one expert's rows: a strip of columns, a part of K.
template <class C, int MT>
__device__ __forceinline__ void up_unit(const FewArgs &p, const FewFfn &f, int e, int n, const int *slot, int at,
                                        FewShared<C> &sh) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int part = at % f.up_parts, chunk = at / f.up_parts % f.chunks;
    const int n0 = at / (f.up_parts * f.chunks) * C::BN;
    // waves 0, 1: W1; waves 2, 3: W3
    const bool second = wave >= 2;
    const void *const w = expert_at<C>(second ? f.w3 : f.w1, e, p.d, f.h);
    const uint8_t *const ws = C::kMx ? scales_at(second ? f.w3s : f.w1s, e, p.d, f.h) : nullptr;
    const int ka = part * f.up_len, kb = min(p.d, ka + f.up_len);
    by_tiles<MT>(n, chunk, f.chunks, [&](auto tiles, int r0) {
        constexpr int M = decltype(tiles)::value;
        const RowsOfX<C, M> rows(p, slot, n, r0, fresh(lane));
        typename C::template Product<M, 2, RowsOfX<C, M>> pr(w, ws, p.d, f.h, ka, kb, fresh(lane), wave & 1,
                                                             sh.stage + (C::kMx ? wave * 4096 : 0));
        pr.start(n0, rows);
        pr.finish(rows);
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const int tid = fresh(threadIdx.x), r = r0 + 16 * m + (tid >> 4), c = n0 + C::CV * (tid & 15);
            float v[2][C::CV];
            sum_waves<C, 2>(sh, pr.acc[m], lane, wave, v);
            if (r < n && c < f.h) {
                const int sl = slot ? slot[r] : r;
                float *o = f.hp + (static_cast<int64_t>(part) * f.slots + sl) * 2 * f.h + c;
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int i = 0; i < C::CV; i += 4)
                        *reinterpret_cast<float4 *>(o + b * f.h + i) = make_float4(v[b][i], v[b][i + 1], v[b][i + 2], v[b][i + 3]);
            }
        }
    });
}

// ------------------------------------------------------------------- kernels

// Waves a SIMD that the registers are kept for (bf16's down-projection with two row tiles
// has 66 KB of shared memory and runs two blocks on a compute unit, two waves a SIMD)
constexpr int few_occ(int row_tiles) { return row_tiles == 1 ? 4 : 3; }

// 1: the gate's blocks first (what follows waits for them), then the shared experts'
template <class C, class G, int MT>
__global__ __launch_bounds__(kFewThreads, few_occ(MT)) void few_gate_kernel(FewArgs p) {
    __shared__ union { FewShared<C> c; FewShared<G> g; } sh;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int strips = (p.E + G::BN - 1) / G::BN;
    int b = static_cast<int>(blockIdx.x);
    if (b >= strips * p.gate_parts) {
        b -= strips * p.gate_parts;
        up_unit<C, MT>(p, p.s, 0, p.T, nullptr, b, sh.c);
        return;
    }
    const int n0 = (b / p.gate_parts) * G::BN, part = b % p.gate_parts;
    const int ka = part * p.gate_len, kb = min(p.d, ka + p.gate_len);
    by_tiles<MT>(p.T, 0, 1, [&](auto tiles, int r0) {
        constexpr int M = decltype(tiles)::value;
        const RowsOfX<G, M> rows(p, nullptr, p.T, r0, fresh(lane));
        typename G::template Product<M, kFewWaves, RowsOfX<G, M>> pr(p.wg, nullptr, p.d, p.E, ka, kb, fresh(lane), wave,
                                                                     sh.g.stage);
        pr.start(n0, rows);
        pr.finish(rows);
#pragma unroll
        for (int m = 0; m < M; ++m) {
            float v[1][G::CV];
            sum_waves<G, kFewWaves>(sh.g, pr.acc[m], lane, wave, v);
            const int tid = fresh(threadIdx.x), t = r0 + 16 * m + (tid >> 4), c = n0 + G::CV * (tid & 15);
#pragma unroll
            for (int i = 0; i < G::CV; ++i)
                if (t < p.T && c + i < p.E) p.zp[(static_cast<int64_t>(part) * p.T + t) * p.E + c + i] = v[0][i];
        }
    });
}

// Order of fp32 values as whole numbers (ascending, -0 as 0), never 0; NaN above all.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    if ((u & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// Over the wave, by data-parallel moves (a shuffle through shared memory takes ten times
// as long): lane 63 ends up with the whole, which every lane gets.
template <int CTRL>
__device__ __forceinline__ int dpp(int none, int v) {
    return __builtin_amdgcn_update_dpp(none, v, CTRL, 0xf, 0xf, false);
}
template <class Op>
__device__ __forceinline__ int wave_all(int v, int none, Op op) {
    v = op(v, dpp<0x111>(none, v));  // row_shr:1
    v = op(v, dpp<0x112>(none, v));
    v = op(v, dpp<0x114>(none, v));
    v = op(v, dpp<0x118>(none, v));
    v = op(v, dpp<0x142>(none, v));  // row_bcast:15
    v = op(v, dpp<0x143>(none, v));  // row_bcast:31
    return __builtin_amdgcn_readlane(v, 63);
}
__device__ __forceinline__ uint32_t wave_top(uint32_t v) {
    return static_cast<uint32_t>(wave_all(static_cast<int>(v), 0, [](int a, int b) {
        return static_cast<int>(max(static_cast<uint32_t>(a), static_cast<uint32_t>(b)));
    }));
}
__device__ __forceinline__ float wave_largest(float v) {
    return __uint_as_float(wave_all(static_cast<int>(__float_as_uint(v)), static_cast<int>(0xff800000u), [](int a, int b) {
        return static_cast<int>(__float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b))));
    }));
}
__device__ __forceinline__ float wave_total(float v) {
    return __uint_as_float(wave_all(static_cast<int>(__float_as_uint(v)), 0, [](int a, int b) {
        return static_cast<int>(__float_as_uint(__uint_as_float(a) + __uint_as_float(b)));
    }));
}

// Softmax and top-k of token t by one wave; lane l holds the experts l, l + 64, ...
// k rounds of an arg-max under (value descending, index ascending).  Whatever the
// logits hold, the k ids are distinct and in range.  ids, w: the token's k; logits: its
// E, or nullptr.
template <int QQ>
__device__ __forceinline__ void topk_token(const FewArgs &p, int t, int lane, int32_t *ids, float *w, float *logits) {
    float s[QQ], mx = -INFINITY;
    uint32_t key[QQ];
#pragma unroll
    for (int q = 0; q < QQ; ++q) s[q] = 0.0f;
    // the parts in order, B of them in flight
    constexpr int B = QQ == 1 ? 16 : QQ == 4 ? 8 : 1;
    for (int i0 = 0; i0 < p.gate_parts; i0 += B) {
        float z[B][QQ];
#pragma unroll
        for (int i = 0; i < B; ++i)
#pragma unroll
            for (int q = 0; q < QQ; ++q) {
                const int e = lane + 64 * q;
                z[i][q] = i0 + i < p.gate_parts && e < p.E ? p.zp[(static_cast<int64_t>(i0 + i) * p.T + t) * p.E + e] : 0.0f;
            }
#pragma unroll
        for (int i = 0; i < B; ++i)
#pragma unroll
            for (int q = 0; q < QQ; ++q) s[q] += z[i][q];
    }
#pragma unroll
    for (int q = 0; q < QQ; ++q) {
        const int e = lane + 64 * q;
        key[q] = 0u;
        if (e < p.E) {
            float z = __fmul_rn(s[q], p.scale);
            if (p.lbias) z = __fadd_rn(z, p.lbias[e]);
            s[q] = z;
            if (logits) logits[e] = z;
            key[q] = order_key(p.sbias ? __fadd_rn(z, p.sbias[e]) : z);
            mx = fmaxf(mx, z);
        }
    }
    mx = wave_largest(mx);
    float den = 0.0f;
#pragma unroll
    for (int q = 0; q < QQ; ++q)
        if (lane + 64 * q < p.E) den += expf(s[q] - mx);
    den = wave_total(den);
    for (int j = 0; j < p.k; ++j) {
        uint32_t best = 0u;
        int at = 0;
#pragma unroll
        for (int q = 0; q < QQ; ++q)
            if (key[q] > best) {
                best = key[q];
                at = q;
            }
        const uint32_t top = wave_top(best);
        const unsigned long long tie = __ballot(best == top);
        int e = __ffsll(tie) - 1;
        if constexpr (QQ > 1) {
            e += 64 * __builtin_amdgcn_readlane(at, e);
            if (__popcll(tie) > 1)  // the lowest index: the largest of its complement
                e = static_cast<int>(~wave_top(best == top ? ~static_cast<uint32_t>(lane + 64 * at) : 0u));
        }
        if ((e & 63) == lane) {
#pragma unroll
            for (int q = 0; q < QQ; ++q)
                if (q == e >> 6) {
                    key[q] = 0u;
                    ids[j] = e;
                    w[j] = expf(s[q] - mx) / den;
                }
        }
    }
}

// 3.  QQ > 0: at most kInlineTokens tokens, whose softmax and top-k every block finds for
// itself (the first one writes them down): no launch between the gate and the experts
template <class C, int MT, int QQ>
__global__ __launch_bounds__(kFewThreads, few_occ(MT)) void few_up_kernel(FewArgs p) {
    __shared__ FewShared<C> sh;
    __shared__ int32_t own_ids[QQ > 0 ? kInlineSlots : 1];
    const int32_t *ids = p.ids;
    if constexpr (QQ > 0) {
        __shared__ float own_w[kInlineSlots];
        const int t = threadIdx.x >> 6;
        if (t < p.T)
            topk_token<QQ>(p, t, threadIdx.x & 63, own_ids + t * p.k, own_w + t * p.k,
                           blockIdx.x == 0 ? p.logits + static_cast<int64_t>(t) * p.E : nullptr);
        __syncthreads();
        if (blockIdx.x == 0)
            for (int i = threadIdx.x; i < p.T * p.k; i += kFewThreads) {
                p.ids[i] = own_ids[i];
                p.w[i] = own_w[i];
            }
        ids = own_ids;
    }
    const int strips = (p.r.h + C::BN - 1) / C::BN;
    const int per = strips * p.r.up_parts * p.r.chunks;
    const int a = static_cast<int>(blockIdx.x) / per, rem = static_cast<int>(blockIdx.x) % per;
    int e;
    const int n = find_unit<C>(p, ids, a, sh, &e);
    if (n == 0) return;
    up_unit<C, MT>(p, p.r, e, n, sh.slot, rem, sh);
}

// The activations of a block's rows in shared memory: 16 MT rows of a part of h.
template <class C, int MT, int KP>
struct ActTile {
    static constexpr int LD = KP * static_cast<int>(sizeof(typename C::Act)) + 16;  // 16 more: neighbouring rows on other banks
    __align__(16) char v[16 * MT][LD];
};
// What a block of the down-projection keeps there; its waves' sums take the activations'
// place, which are read by then.
template <class C, int MT, int KP, int WK>
struct DownShared : FewStage<C> {
    union {
        ActTile<C, MT, KP> act;
        float red[WK == 1 ? 1 : kFewWaves][16][C::BN + 4];
    };
};
template <class C, int MT, int KP>
struct RowsOfAct {
    using X = typename C::XAct;
    static constexpr bool kEarly = false;
    const ActTile<C, MT, KP> &t;
    int ka, lane;
    __device__ __forceinline__ void read(int m, int k, X &x) const {
        C::act_row(t.v[16 * m + (lane & 15)], k - ka, lane, x);
    }
};

// Four activations of slot `sl` from column c on (zeros unless `in`) from the parts of H1
// and H3.  8 bits: rounded to them and opened again; the eight lanes of a block of 32
// columns all take part.
template <class C>
__device__ __forceinline__ void form_act(const FewFfn &f, int sl, int c, bool in, char *out) {
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (in) {
        const float *src = f.hp + static_cast<int64_t>(sl) * 2 * f.h + c;
        float4 h1 = *reinterpret_cast<const float4 *>(src), h3 = *reinterpret_cast<const float4 *>(src + f.h);
#pragma unroll 4
        for (int q = 1; q < f.up_parts; ++q) {
            const float *const at = src + static_cast<int64_t>(q) * f.slots * 2 * f.h;
            const float4 a = *reinterpret_cast<const float4 *>(at), g = *reinterpret_cast<const float4 *>(at + f.h);
            h1.x += a.x; h1.y += a.y; h1.z += a.z; h1.w += a.w;
            h3.x += g.x; h3.y += g.y; h3.z += g.z; h3.w += g.w;
        }
        v[0] = silu_f(h1.x) * h3.x; v[1] = silu_f(h1.y) * h3.y; v[2] = silu_f(h1.z) * h3.z; v[3] = silu_f(h1.w) * h3.w;
    }
    if constexpr (C::kMx) {
        uint32_t o[1];
        const uint32_t byte = mx8_quant<4>(v, o);
        i32x4_t u[2];
        open8(i32x4_t{static_cast<int>(o[0]), 0, 0, 0}, static_cast<int>(byte), u);
        *reinterpret_cast<uint2 *>(out) = make_uint2(static_cast<uint32_t>(u[0][0]), static_cast<uint32_t>(u[0][1]));
    } else if constexpr (sizeof(typename C::Elt) == 2) {
        const uint2 hi = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
        const float of[4] = {__uint_as_float(hi.x << 16), __uint_as_float(hi.x & 0xffff0000u), __uint_as_float(hi.y << 16),
                             __uint_as_float(hi.y & 0xffff0000u)};
        float lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo[i] = v[i] - of[i];
            if (!(fabsf(lo[i]) < INFINITY)) lo[i] = 0.0f;  // behind an infinity or a NaN
        }
        *reinterpret_cast<uint2 *>(out) = hi;
        *reinterpret_cast<uint2 *>(out + 16) = make_uint2(pack_bf16x2(lo[0], lo[1]), pack_bf16x2(lo[2], lo[3]));
    } else {
        *reinterpret_cast<float4 *>(out) = make_float4(v[0], v[1], v[2], v[3]);
    }
}

// A wave: 256 columns of a slot's activations
template <class C>
__device__ __forceinline__ void act_wave(const FewFfn &f, int b) {
    const int per = (f.h + 255) / 256, sl = b / per, c = 256 * (b % per) + 4 * static_cast<int>(threadIdx.x);
    // whole blocks of 32 columns (8 bits) are in or out
    if (c < f.h)
        form_act<C>(f, sl, c, true, static_cast<char *>(f.act) + sizeof(typename C::Act) * static_cast<int64_t>(sl) * f.h + C::act_at(c));
}

// between 3 and 4, where few experts with many rows each are cut into many parts
template <class C>
__global__ __launch_bounds__(64) void few_act_kernel(FewArgs p) {
    act_wave<C>(p.r, blockIdx.x);
}

// 2: a wave for each token; behind them the shared experts' activations
template <class C, int QQ>
__global__ __launch_bounds__(64) void few_topk_kernel(FewArgs p) {
    const int b = blockIdx.x;
    if (b < p.T) {
        topk_token<QQ>(p, b, threadIdx.x, p.ids + b * p.k, p.w + b * p.k, p.logits + static_cast<int64_t>(b) * p.E);
        return;
    }
    act_wave<C>(p.s, b - p.T);
}

// 4: the chosen experts' units first, then the shared ones'.  WK = 4: the waves split a
// part's steps and meet after each strip; WK = 1: a wave takes every fourth strip over the
// whole part and stores its sums, for launches with more strips than waves that run at once
// (112 8-bit experts of 768 x 2048 with two rows each: 65 -> 43 us, 4.3 TB/s, the meetings'
// waits being gone)
template <class C, int MT, int KP, int WK>
__global__ __launch_bounds__(kFewThreads, few_occ(MT)) void few_down_kernel(FewArgs p, int units) {
    __shared__ DownShared<C, MT, KP, WK> sh;
    ActTile<C, MT, KP> &act = sh.act;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int b = static_cast<int>(blockIdx.x);
    const bool shared = b >= units;
    if (shared) b -= units;
    const FewFfn &f = shared ? p.s : p.r;
    const int part = b % f.down_parts, chunk = b / f.down_parts % f.chunks;
    const int width = f.down_strips * C::BN, groups = (p.d + width - 1) / width;
    b /= f.down_parts * f.chunks;
    const int n0 = b % groups * width, n1 = min(p.d, n0 + width);
    int e = 0, n = p.T;
    const int *slot = nullptr;
    if (!shared) {
        n = find_unit<C>(p, p.ids, b / groups, sh, &e);
        slot = sh.slot;
        if (n == 0) return;
    }
    const void *const w = expert_at<C>(f.w2, e, f.h, p.d);
    const uint8_t *const ws = C::kMx ? scales_at(f.w2s, e, f.h, p.d) : nullptr;
    const int ka = part * f.down_len, kb = min(f.h, ka + f.down_len);
    const int len = (kb - ka + C::STEP - 1) / C::STEP * C::STEP;  // zeros behind h
    by_tiles<MT>(n, chunk, f.chunks, [&](auto tiles, int r0) {
        constexpr int M = decltype(tiles)::value;
        const int nr = min(n - r0, 16 * M);
        const RowsOfAct<C, MT, KP> rows{act, ka, fresh(lane)};
        typename C::template Product<M, WK, RowsOfAct<C, MT, KP>> pr(w, ws, f.h, p.d, ka, kb, fresh(lane), wave % WK,
                                                                                   sh.stage + (C::kMx ? wave * 4096 : 0));
        constexpr int kNext = kFewWaves / WK * C::BN;  // from a wave's strip to its next
        const int first = n0 + (WK == 1 ? wave * C::BN : 0);
        if (first < n1) pr.start(first, rows);
        __syncthreads();  // the rows before have been read, and their sums
        using Act = typename C::Act;
        if (f.act) {
            constexpr int V = 16 / static_cast<int>(sizeof(Act));
            for (int i = threadIdx.x; i < nr * (len / V); i += kFewThreads) {
                const int r = i / (len / V), c = V * (i % (len / V));
                const Act *src = static_cast<const Act *>(f.act) + static_cast<int64_t>(slot ? slot[r0 + r] : r0 + r) * f.h + ka + c;
                *reinterpret_cast<i32x4_t *>(act.v[r] + sizeof(Act) * c) =
                    ka + c < kb ? *reinterpret_cast<const i32x4_t *>(src) : i32x4_t{0, 0, 0, 0};
            }
        } else {
            for (int i = threadIdx.x; i < nr * (len / 4); i += kFewThreads) {
                const int r = i / (len / 4), c = 4 * (i % (len / 4));
                form_act<C>(f, slot ? slot[r0 + r] : r0 + r, ka + c, ka + c < kb, act.v[r] + C::act_at(c));
            }
        }
        __syncthreads();
        if constexpr (WK == 1) {
            for (int c0 = first; c0 < n1; c0 += kNext) {
                pr.finish(rows);
                f32x4_t sum[M][C::CV];
#pragma unroll
                for (int m = 0; m < M; ++m)
#pragma unroll
                    for (int i = 0; i < C::CV; ++i) sum[m][i] = pr.acc[m][i];
                if (c0 + kNext < n1) pr.start(c0 + kNext, rows);  // under way while the sums leave
#pragma unroll
                for (int m = 0; m < M; ++m) {
                    const int l = fresh(lane), r = r0 + 16 * m + (l & 15);
                    float *const o = f.yp + (static_cast<int64_t>(part) * f.slots + (r < n ? (slot ? slot[r] : r) : 0)) * p.d + c0;
                    C::each(sum[m], l, [&](int c, f32x4_t v) {
                        if (r < n && c0 + c < p.d) *reinterpret_cast<f32x4_t *>(o + c) = v;
                    });
                }
            }
        } else {
            // one strip
            pr.finish(rows);
#pragma unroll
            for (int m = 0; m < M; ++m) {
                float v[1][C::CV];
                sum_waves<C, WK>(sh, pr.acc[m], lane, wave, v);
                const int tid = fresh(threadIdx.x), r = r0 + 16 * m + (tid >> 4), c = n0 + C::CV * (tid & 15);
                if (r < n && c < p.d) {
                    float *o = f.yp + (static_cast<int64_t>(part) * f.slots + (slot ? slot[r] : r)) * p.d + c;
#pragma unroll
                    for (int i = 0; i < C::CV; i += 4)
                        *reinterpret_cast<float4 *>(o + i) = make_float4(v[0][i], v[0][i + 1], v[0][i + 2], v[0][i + 3]);
                }
            }
        }
    });
}

// 5: four columns of a token by four threads, each with a quarter of the terms (term z to
// thread z % 4, eight of its terms in flight), whose sums meet in shared memory
constexpr int kCombineCols = 16;
template <typename T>
__global__ __launch_bounds__(4 * kCombineCols) void few_combine_kernel(FewArgs p) {
    __shared__ float4 part[4][kCombineCols];
    const int g = threadIdx.x / kCombineCols, u0 = threadIdx.x % kCombineCols;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kCombineCols + u0;
    const int per = p.d / 4;
    const bool live = i < static_cast<int64_t>(p.T) * per;
    const int t = live ? static_cast<int>(i / per) : 0, c = live ? 4 * static_cast<int>(i % per) : 0;
    float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    // term z: part z % parts of slot z / parts, the shared experts' parts behind them
    const int routed = p.k * p.r.down_parts, terms = routed + (p.s.h ? p.s.down_parts : 0);
    for (int z0 = g; z0 < terms; z0 += 32) {
        float4 v[8];
        float w[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int z = z0 + 4 * u < terms ? z0 + 4 * u : g;
            const bool own = z < routed;
            const int j = own ? z / p.r.down_parts : 0;
            const float *const src = own ? p.r.yp + (static_cast<int64_t>(z - j * p.r.down_parts) * p.r.slots + t * p.k + j) * p.d
                                         : p.s.yp + (static_cast<int64_t>(z - routed) * p.s.slots + t) * p.d;
            v[u] = *reinterpret_cast<const float4 *>(src + c);
            w[u] = own ? p.w[t * p.k + j] : 1.0f;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (z0 + 4 * u < terms) {
                y[0] = __builtin_fmaf(w[u], v[u].x, y[0]); y[1] = __builtin_fmaf(w[u], v[u].y, y[1]);
                y[2] = __builtin_fmaf(w[u], v[u].z, y[2]); y[3] = __builtin_fmaf(w[u], v[u].w, y[3]);
            }
    }
    part[g][u0] = make_float4(y[0], y[1], y[2], y[3]);
    __syncthreads();
    if (g != 0 || !live) return;
#pragma unroll
    for (int q = 1; q < 4; ++q) {
        const float4 a = part[q][u0];
        y[0] += a.x; y[1] += a.y; y[2] += a.z; y[3] += a.w;
    }
    T *o = static_cast<T *>(p.y) + static_cast<int64_t>(t) * p.d + c;
    if constexpr (sizeof(T) == 2)
        *reinterpret_cast<uint2 *>(o) = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
    else
        *reinterpret_cast<float4 *>(o) = make_float4(y[0], y[1], y[2], y[3]);
}

// ---------------------------------------------------------------- the launches

struct Plan {
    FewArgs a;
    int64_t gate, shared, act, up, down, down_shared;  // blocks
    int down_chunks;                                   // of the shared experts
    bool own_topk, tokens2, rows2, wave_strips;
    size_t bytes;
};

// Parts of K for `units` strips, in multiples of `quantum`, at most `most` long: so many
// that the launch has kBlocks blocks, but none shorter than `least` (what a part adds is
// sums written and read again, and a block's start), except that a small launch is cut
// until two blocks run on each compute unit.  No more than `cap` parts unless `most` asks.
void split(int K, double units, int quantum, int least, int most, int cap, int *parts, int *len) {
    const auto parts_of = [&](int64_t l) { return std::max<int64_t>(1, (K + l - 1) / l); };
    const int64_t few = static_cast<int64_t>(kFewBlocks / units);
    const int64_t many = std::min(static_cast<int64_t>(kBlocks / units), static_cast<int64_t>(K / least));
    const int64_t n = std::max({int64_t(1), std::min<int64_t>(std::max(few, many), cap), parts_of(most)});
    const int64_t l = std::min<int64_t>(((K + n - 1) / n + quantum - 1) / quantum * quantum, most);
    *len = static_cast<int>(l);
    *parts = static_cast<int>(parts_of(l));
}

template <class C, class G>
Plan make_plan(const FewSizes &z, char *ws) {
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
    const int64_t gs = (z.E + G::BN - 1) / G::BN;
    split(z.d, static_cast<double>(gs), G::STEP * kFewWaves, std::max(z.d / kGateParts, 128), 1 << 30, kGateParts, &a.gate_parts,
          &a.gate_len);
    pl.gate = gs * a.gate_parts;
    a.zp = take(static_cast<int64_t>(a.gate_parts) * a.T * a.E);
    const int64_t ds = (z.d + C::BN - 1) / C::BN;
    pl.own_topk = !(a.T <= kInlineTokens && a.T * a.k <= kInlineSlots && a.E <= 256);
    // two row tiles at a time: the tokens of the gate and of the shared experts'
    // up-projection, and the chosen experts' rows where they have more than 8 on average
    // (12.8 rows: 232 us so and 262 by single tiles in bf16, 107 and 118 in 8 bits, 162 and
    // 189 in fp32; 5 to 8 rows: level, 302 to 306 in bf16; 24 tokens of 9 rows 81 and 74)
    pl.tokens2 = a.T > 16;
    pl.rows2 = pl.tokens2 && static_cast<int64_t>(a.T) * a.k > 8 * static_cast<int64_t>(a.E);
    const int64_t units = std::min<int64_t>(static_cast<int64_t>(a.T) * a.k, a.E), slots = static_cast<int64_t>(a.T) * a.k;
    // how many experts evenly routed tokens choose
    const double busy = z.E * (1.0 - std::pow(1.0 - static_cast<double>(z.k) / z.E, static_cast<double>(z.T)));
    auto ffn = [&](FewFfn &f, int h, double units_busy, int64_t rows, bool routed, int up_rows, int down_rows) {
        f.h = h;
        f.slots = static_cast<int>(rows);
        const int64_t hs = (h + C::BN - 1) / C::BN;
        // Every strip of the down-projection reads the parts of its rows, a part costing as
        // much as 1 / 64 of the weights for each row of an expert: with many rows the
        // activations are formed before, the shared experts' by the top-k's launch, if there
        // is one, the chosen experts' by one of their own.  Where the chosen ones' border
        // lies, by cap, 2 cap and 4 cap: 40 bf16 experts of 13 rows 235, 235, 247 us; 16
        // 8-bit experts of 8 rows 34.4, 33.4, 36.2, but of 16 rows 66, 77, 77
        const int cap = std::max(1, static_cast<int>(kPartRows * units_busy / rows));
        split(z.d, units_busy * hs * up_rows, 2 * C::STEP, C::kLeast, 1 << 30, 1 << 30, &f.up_parts, &f.up_len);
        const bool own_act = routed ? f.up_parts > 2 * cap : pl.own_topk;
        if (!own_act) split(z.d, units_busy * hs * up_rows, 2 * C::STEP, C::kLeast, 1 << 30, cap, &f.up_parts, &f.up_len);
        split(h, units_busy * ds * down_rows, C::STEP * kFewWaves, C::kLeast, C::kPart, 1 << 30, &f.down_parts, &f.down_len);
        f.hp = take(static_cast<int64_t>(f.up_parts) * rows * 2 * h);
        f.yp = take(static_cast<int64_t>(f.down_parts) * rows * z.d);
        if (own_act) f.act = take((rows * h * static_cast<int64_t>(sizeof(typename C::Act)) + 3) / 4);
    };
    const int64_t hs = (z.h + C::BN - 1) / C::BN, ss = (z.hs + C::BN - 1) / C::BN;
    a.r.chunks = 1;  // (a block for each 32 rows of a chosen expert: 64 tokens of two, 8 experts 53 -> 65 us)
    ffn(a.r, z.h, busy, slots, true, 1, 1);
    pl.up = units * hs * a.r.up_parts;
    pl.down = units * ds * a.r.down_parts;
    if (z.hs) {
        // the shared experts' rows are shared out, too: every token has one
        a.s.chunks = (a.T + (pl.tokens2 ? 31 : 15)) / (pl.tokens2 ? 32 : 16);
        pl.down_chunks = (a.T + (pl.rows2 ? 31 : 15)) / (pl.rows2 ? 32 : 16);
        ffn(a.s, z.hs, 1.0, a.T, false, a.s.chunks, pl.down_chunks);
        pl.shared = ss * a.s.up_parts * a.s.chunks;
        pl.down_shared = ds * a.s.down_parts;
        if (pl.own_topk) pl.act = static_cast<int64_t>(a.T) * ((z.hs + 255) / 256);  // beside the top-k
    }
    // Launches with more strips than the compute units' waves take at once: a wave a strip,
    // and several of them a block, whose activations are formed once for all.  Two strips a
    // wave from 8192 on, within 5% of one strip on either side (a third of that in bf16 207
    // us with one, 212 with two; 6144 of 8 bits 128 and 122; 14336 255 and 257; 114688 1686 and 1673)
    const int64_t strips = pl.down + pl.down_shared;
    pl.wave_strips = strips >= kManyStrips;
    a.r.down_strips = pl.wave_strips ? kFewWaves * (strips >= 4 * kManyStrips ? 2 : 1) : 1;
    a.s.down_strips = pl.wave_strips ? kFewWaves : 1;
    pl.down = pl.down / ds * ((ds + a.r.down_strips - 1) / a.r.down_strips);
    pl.down_shared = pl.down_shared / ds * ((ds + a.s.down_strips - 1) / a.s.down_strips) * pl.down_chunks;
    pl.bytes = at;
    return pl;
}

template <class C, int MT>
void launch_up(const Plan &pl, hipStream_t s) {
    const FewArgs &a = pl.a;
    const dim3 grid(static_cast<unsigned>(pl.up)), block(kFewThreads), tokens(static_cast<unsigned>(a.T + pl.act));
    if constexpr (MT == 1)
        if (!pl.own_topk) {
            if (a.E <= 64) hipLaunchKernelGGL((few_up_kernel<C, 1, 1>), grid, block, 0, s, a);
            else hipLaunchKernelGGL((few_up_kernel<C, 1, 4>), grid, block, 0, s, a);
            return;
        }
    if (a.E <= 64) hipLaunchKernelGGL((few_topk_kernel<C, 1>), tokens, dim3(64), 0, s, a);
    else if (a.E <= 256) hipLaunchKernelGGL((few_topk_kernel<C, 4>), tokens, dim3(64), 0, s, a);
    else hipLaunchKernelGGL((few_topk_kernel<C, 16>), tokens, dim3(64), 0, s, a);
    hipLaunchKernelGGL((few_up_kernel<C, MT, 0>), grid, block, 0, s, a);
}

template <class C, int MT>
void launch_down(Plan &pl, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(pl.down + pl.down_shared)), block(kFewThreads);
    const int units = static_cast<int>(pl.down);
    pl.a.s.chunks = pl.down_chunks;
    if (pl.wave_strips) hipLaunchKernelGGL((few_down_kernel<C, MT, C::kPart, 1>), grid, block, 0, s, pl.a, units);
    else hipLaunchKernelGGL((few_down_kernel<C, MT, C::kPart, kFewWaves>), grid, block, 0, s, pl.a, units);
}

template <class C, class G>
hipError_t launch_all(Plan &pl, hipStream_t s) {
    const FewArgs &a = pl.a;
    const dim3 first(static_cast<unsigned>(pl.gate + pl.shared)), block(kFewThreads);
    if (pl.tokens2) hipLaunchKernelGGL((few_gate_kernel<C, G, 2>), first, block, 0, s, a);
    else hipLaunchKernelGGL((few_gate_kernel<C, G, 1>), first, block, 0, s, a);
    if (pl.rows2) launch_up<C, 2>(pl, s);
    else launch_up<C, 1>(pl, s);
    if (a.r.act)
        hipLaunchKernelGGL((few_act_kernel<C>), dim3(static_cast<unsigned>(a.r.slots * ((a.r.h + 255) / 256))), dim3(64), 0, s, a);
    if (pl.rows2) launch_down<C, 2>(pl, s);
    else launch_down<C, 1>(pl, s);
    const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(a.T) * (a.d / 4) + kCombineCols - 1) / kCombineCols));
    if constexpr (std::is_same<C, PlainCore<float>>::value)
        hipLaunchKernelGGL((few_combine_kernel<float>), grid, dim3(4 * kCombineCols), 0, s, a);
    else
        hipLaunchKernelGGL((few_combine_kernel<bf16_t>), grid, dim3(4 * kCombineCols), 0, s, a);
    return hipGetLastError();
}

template <class C, class G>
hipError_t launch_core(const FewSizes &z, const FewTensors &t, hipStream_t s) {
    Plan pl = make_plan<C, G>(z, static_cast<char *>(t.ws));
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
    return launch_all<C, G>(pl, s);
}

}  // namespace

size_t few_workspace(const FewSizes &z) {
    if (z.T <= 0) return 0;
    if (z.mx8) return make_plan<Mx8Core, PlainCore<bf16_t>>(z, nullptr).bytes;
    return z.dt == kBF16 ? make_plan<PlainCore<bf16_t>, PlainCore<bf16_t>>(z, nullptr).bytes
                         : make_plan<PlainCore<float>, PlainCore<float>>(z, nullptr).bytes;
}

hipError_t launch_layer_few(const FewSizes &z, const FewTensors &t, hipStream_t s) {
    if (z.T <= 0) return hipSuccess;
    if (z.mx8) return launch_core<Mx8Core, PlainCore<bf16_t>>(z, t, s);
    return z.dt == kBF16 ? launch_core<PlainCore<bf16_t>, PlainCore<bf16_t>>(z, t, s)
                         : launch_core<PlainCore<float>, PlainCore<float>>(z, t, s);
}

}  // namespace xmoe

// Balance loss of the gate: per-expert counts, loss and gradient.
//
// For sequence s with n_s counted tokens, c_{s,e} of whose slots chose expert e,
// and p = softmax(logits) (the gate's probabilities):
//   f_{s,e} = E c_{s,e} / (k n_s),  P_{s,e} = (1 / n_s) sum_t p_{t,e}
//   loss = alpha / S' * sum_s sum_e f_{s,e} P_{s,e}
// over the S' sequences that count any token.  The counts carry no gradient, so
//   coef_{s,e} = d loss / d p_{t,e} = alpha E c_{s,e} / (k n_s^2 S')
//   d loss / d logits_{t,e} = p_{t,e} (coef_{s,e} - sum_e' p_{t,e'} coef_{s,e'})
//
// Forward: one kernel reads the logits once; a block forms the probabilities of
// a chunk of tokens and the sums and counts of each sequence's piece of it.
// Piece (chunk b, sequence s) has row b + s of the partial sums: chunks and
// sequences both only go forward, so no two pieces share a row and the rows
// number at most chunks + S.  A second kernel adds a sequence's rows in order and
// writes counts and coef; its last block to end, or of many blocks a third kernel,
// adds the blocks' losses in order.  Nothing depends on the order in which blocks
// run.  S' comes from the counted tokens of every sequence, whose pieces are added
// side by side, since a sequence may be masked over any number of them: 2^20
// tokens of 16 experts in two sequences 51 us, one of them masked or not (379 and
// 50 where a thread looked for a sequence's first counted piece).
//
// The logits are read once here, once in the backward, which writes the gradient.
// Bound by latency: 4096 tokens of 64 experts take 3.7 + 6.5 us and 3.6 us back,
// the second kernel's two blocks a chain of loads that wait for each other
// (offsets, counts, rows) and the ticket; 32768 of 160 experts in 24 sequences (63
// MB in all) 11.2 + 5.6 + 1.8 and 11.5 us (logits out of memory; 10 where the
// last-level cache holds them).
#include <algorithm>

#include "balance.hpp"
#include "common.hpp"
#include "kernels.hpp"

namespace xmoe {

namespace {

constexpr int kWaves = 4;

// Tokens per block: about 512 blocks, two on each compute unit, at least one
// step of every wave; at most 128, so that a sum of p has few terms in sequence.
// More and smaller blocks leave the second kernel more rows: against 2048 blocks
// 16384 tokens of 64 experts 11.1 and 12.9 us (both kernels), 32768 of 160 in 24
// sequences 17.6 and 19.3, 131072 of 64 19.3 and 23.2; 65536 of 64 in 8
// sequences 15.6 and 15.0.
inline int chunk_tokens(int64_t T) {
    int c = 16;
    while (c < 128 && T > static_cast<int64_t>(c) * 512) c *= 2;
    return c;
}
// experts per block of the second kernel: its 32 row groups share a sequence's rows
constexpr int kFinalExperts = 32;
inline int final_blocks(int E) { return (E + kFinalExperts - 1) / kFinalExperts; }
inline size_t align256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

// S' needs the counted tokens of all sequences in every block of the second
// kernel.  It adds them up itself, 16 lanes a sequence, where that is few loads;
// else a kernel between the two does, once.
constexpr int kFewSequences = 64;
constexpr int64_t kFewChunks = 512;
inline bool counts_itself(int64_t T, int S) {
    return S == 1 || (S <= kFewSequences && T <= kFewChunks * chunk_tokens(T));
}

struct BalanceWs {
    float *psum;      // [rows, E]
    int32_t *csum;    // [rows, E]
    int32_t *nsum;    // [rows]
    double *part_loss; // [S, blocks of experts]
    int32_t *ticket;  // [1]
    int32_t *nseq;    // [S]; nullptr: the second kernel counts by itself
    size_t bytes;
};
BalanceWs balance_ws(void *ws, int64_t T, int E, int S) {
    const int64_t rows = (T + chunk_tokens(T) - 1) / chunk_tokens(T) + S;
    BalanceWs b;
    size_t at = 0;
    char *p = static_cast<char *>(ws);
    auto take = [&](size_t n) {
        char *q = p + at;
        at += align256(n);
        return q;
    };
    b.psum = reinterpret_cast<float *>(take(rows * E * 4));
    b.csum = reinterpret_cast<int32_t *>(take(rows * E * 4));
    b.nsum = reinterpret_cast<int32_t *>(take(rows * 4));
    b.part_loss = reinterpret_cast<double *>(take(static_cast<size_t>(S) * final_blocks(E) * 8));
    b.ticket = reinterpret_cast<int32_t *>(take(4));
    b.nseq = counts_itself(T, S) ? nullptr : reinterpret_cast<int32_t *>(take(static_cast<size_t>(S) * 4));
    b.bytes = at;
    return b;
}

// One token's logits in its LT lanes: lane r holds QQ experts, the 16-byte chunks
// r, r + LT, ... of the row (expert of value q: 4 (r + LT (q / 4)) + q % 4).
// Experts past E and dead tokens hold -infinity.
template <int LT, int QQ>
__device__ __forceinline__ void load_token(const float *row, bool live, int r, int E, float (&p)[QQ]) {
    auto ex = [&](int q) { return 4 * (r + LT * (q >> 2)) + (q & 3); };
#pragma unroll
    for (int q = 0; q < QQ; ++q) p[q] = -INFINITY;
    if (!live) return;
    if (E % 4 == 0) {
#pragma unroll
        for (int q = 0; q < QQ; q += 4)
            if (ex(q) < E) {
                const float4 v = *reinterpret_cast<const float4 *>(row + ex(q));
                p[q] = v.x; p[q + 1] = v.y; p[q + 2] = v.z; p[q + 3] = v.w;
            }
    } else {
#pragma unroll
        for (int q = 0; q < QQ; ++q)
            if (ex(q) < E) p[q] = row[ex(q)];
    }
}

// Logits -> probabilities in place (dead tokens: 0).  exp(x - max) is taken as
// 2^((x - max) L), L = log2(e): with expf and its range checks the arithmetic,
// not the loads, bound these kernels (44 vector instructions an element).  The
// difference comes first: x L - max L in one multiply-add saves an instruction,
// but max L leaves fp32's range in a row of the type's lowest values.  One
// division a token.
template <int LT, int QQ>
__device__ __forceinline__ void token_softmax(bool live, float (&p)[QQ]) {
    constexpr float kLog2e = 1.44269504f;
    float mx = -INFINITY;
#pragma unroll
    for (int q = 0; q < QQ; ++q) mx = fmaxf(mx, p[q]);
#pragma unroll
    for (int off = LT / 2; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor(mx, off, 64));
    float den = 0.0f;
#pragma unroll
    for (int q = 0; q < QQ; ++q) {  // 0 past E, where the logits are -infinity
        p[q] = __builtin_amdgcn_exp2f((p[q] - mx) * kLog2e);
        den += p[q];
    }
#pragma unroll
    for (int off = LT / 2; off > 0; off >>= 1) den += __shfl_xor(den, off, 64);
    const float inv = 1.0f / den;
#pragma unroll
    for (int q = 0; q < QQ; ++q) p[q] = live ? p[q] * inv : 0.0f;
}

template <int LT, int QQ>
__global__ __launch_bounds__(64 * kWaves) void balance_part_kernel(const float *__restrict__ logits,
                                                                   const int32_t *__restrict__ ids, int64_t T, int E,
                                                                   int k, const int32_t *__restrict__ off, int S,
                                                                   const uint8_t *__restrict__ mask, int chunk,
                                                                   BalanceWs ws) {
    constexpr int TPW = 64 / LT, TPB = kWaves * TPW;
    __shared__ float sp[kWaves][LT * QQ];
    __shared__ int32_t sc[LT * QQ];
    __shared__ int32_t sn[kWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = lane % LT, slot = wave * TPW + lane / LT;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * chunk;
    const int64_t t1 = t0 + chunk < T ? t0 + chunk : T;
    if (blockIdx.x == 0 && threadIdx.x == 0) *ws.ticket = 0;
    auto ex = [&](int q) { return 4 * (r + LT * (q >> 2)) + (q & 3); };
    // the first step's logits are on their way during the search: the first piece
    // starts with the chunk unless the chunk starts in front of the first sequence
    float next[QQ];
    load_token<LT, QQ>(logits + (t0 + slot) * E, t0 + slot < T, r, E, next);
    int nid = t0 + slot < T && r < k ? ids[(t0 + slot) * k + r] : -1;
    uint8_t nmask = mask && t0 + slot < T ? mask[t0 + slot] : 1;
    bool ahead = true;
    // the sequences that this chunk meets, in order (the same in every thread)
    int s = 0;
    if (off) s = max(find_sequence<64>(off, S, t0), 0);
    for (; s < S; ++s) {
        int64_t lo = 0, hi = T;
        if (off) {
            lo = off[s];
            hi = off[s + 1];
            if (lo >= t1) break;
        }
        lo = lo < t0 ? t0 : lo;
        hi = hi > t1 ? t1 : hi;
        if (lo >= hi) continue;  // an empty sequence: no row
        for (int e = threadIdx.x; e < LT * QQ; e += 64 * kWaves) sc[e] = 0;
        float acc[QQ];
        int n = 0;
#pragma unroll
        for (int q = 0; q < QQ; ++q) acc[q] = 0.0f;
        __syncthreads();
        // the next step's logits are on their way while this one's are worked on
        auto ask = [&](int64_t t) {
            nmask = mask && t < hi ? mask[t] : 1;
            nid = t < hi && r < k ? ids[t * k + r] : -1;
            load_token<LT, QQ>(logits + t * E, t < hi, r, E, next);
        };
        if (!(ahead && lo == t0)) ask(lo + slot);
        ahead = false;
        for (int64_t tb = lo; tb < hi; tb += TPB) {
            const int64_t t = tb + slot;
            const bool live = t < hi && nmask != 0;
            const int id = nid;
            float p[QQ];
#pragma unroll
            for (int q = 0; q < QQ; ++q) p[q] = next[q];
            ask(t + TPB);
            token_softmax<LT, QQ>(live, p);
#pragma unroll
            for (int q = 0; q < QQ; ++q) acc[q] += p[q];
            if (live) {
                n += r == 0 ? 1 : 0;
                if (id >= 0 && id < E) atomicAdd(&sc[id], 1);
                for (int j = r + LT; j < k; j += LT) {
                    const int e = ids[t * k + j];
                    if (e >= 0 && e < E) atomicAdd(&sc[e], 1);
                }
            }
        }
#pragma unroll
        for (int q = 0; q < QQ; ++q)
#pragma unroll
            for (int o = LT; o < 64; o <<= 1) acc[q] += __shfl_xor(acc[q], o, 64);
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) n += __shfl_xor(n, o, 64);
        if (lane < LT) {
#pragma unroll
            for (int q = 0; q < QQ; ++q) sp[wave][ex(q)] = acc[q];
        }
        if (lane == 0) sn[wave] = n;
        __syncthreads();
        const int64_t row = static_cast<int64_t>(blockIdx.x) + s;
        for (int e = threadIdx.x; e < E; e += 64 * kWaves) {
            float v = sp[0][e];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) v += sp[w][e];
            ws.psum[row * E + e] = v;
            ws.csum[row * E + e] = sc[e];
        }
        if (threadIdx.x == 0) {
            int v = sn[0];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) v += sn[w];
            ws.nsum[row] = v;
        }
        __syncthreads();
    }
}

// the rows [lo, hi) of sequence s in the partial sums
__device__ __forceinline__ void piece_rows(const int32_t *off, int s, int64_t T, int chunk, int64_t *lo, int64_t *hi) {
    int64_t a = 0, b = T;
    if (off) {
        a = off[s];
        b = off[s + 1];
    }
    a = a < 0 ? 0 : a;
    b = b > T ? T : b;
    *lo = a < b ? a / chunk + s : 0;
    *hi = a < b ? (b - 1) / chunk + s + 1 : 0;
}

// Counted tokens of each sequence, a block each, where the second kernel does not
// add them up by itself.
__global__ __launch_bounds__(256) void balance_count_kernel(int64_t T, const int32_t *off, int chunk, BalanceWs ws) {
    __shared__ int32_t wn[4];
    int64_t lo, hi;
    piece_rows(off, blockIdx.x, T, chunk, &lo, &hi);
    int32_t n = 0;
#pragma unroll 4
    for (int64_t b = lo + threadIdx.x; b < hi; b += 256) n += ws.nsum[b];
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) n += __shfl_xor(n, o, 64);
    if (threadIdx.x % 64 == 0) wn[threadIdx.x / 64] = n;
    __syncthreads();
    if (threadIdx.x == 0) ws.nseq[blockIdx.x] = wn[0] + wn[1] + wn[2] + wn[3];
}

// A block per sequence and 32 experts.  The rows' values are asked for first;
// what the counts need (n_s, S') comes beside them.
__global__ __launch_bounds__(1024) void balance_final_kernel(int64_t T, int E, int k, const int32_t *off, int S,
                                                             int chunk, float alpha, BalanceWs ws, bool hand_over,
                                                             float *loss, int32_t *counts, float *coef) {
    __shared__ bool last;
    __shared__ double red[32];
    __shared__ int32_t wn[16], wsome[16];
    __shared__ double sp[kFinalExperts][33];
    __shared__ int32_t sc[kFinalExperts][33];
    constexpr int W = kFinalExperts, parts = 1024 / W;
    static_assert(W == 32 && parts == 32, "half a wave for each expert");
    const int eb = static_cast<int>(gridDim.x) / S;  // blocks of a sequence
    const int s = blockIdx.x / eb;
    const int e = (blockIdx.x % eb) * W + threadIdx.x % W, part = threadIdx.x / W;
    int64_t lo, hi;
    piece_rows(off, s, T, chunk, &lo, &hi);
    double p = 0.0;
    int32_t c = 0, n = 0;
    if (e < E) {
#pragma unroll 4
        for (int64_t b = lo + part; b < hi; b += parts) {
            p += ws.psum[b * E + e];
            c += ws.csum[b * E + e];
        }
    }
    int some = 0;  // S': sequences that count a token
    if (S == 1) {
        for (int64_t b = lo + threadIdx.x; b < hi; b += 1024) n += ws.nsum[b];
    } else if (ws.nseq) {
        for (int i = threadIdx.x; i < S; i += 1024) {
            const int32_t v = ws.nseq[i];
            some += v > 0;
            n = i == s ? v : n;
        }
    } else {
        constexpr int L = 1024 / kFewSequences;  // lanes of a sequence
        const int i = threadIdx.x / L;
        int64_t a = 0, z = 0;
        if (i < S) piece_rows(off, i, T, chunk, &a, &z);
        int32_t v = 0;
#pragma unroll 4
        for (a += threadIdx.x % L; a < z; a += L) v += ws.nsum[a];
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
        if (threadIdx.x % L == 0) {
            some = v > 0;
            n = i == s ? v : 0;
        }
    }
    sp[threadIdx.x % W][part] = p;
    sc[threadIdx.x % W][part] = c;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        n += __shfl_xor(n, o, 64);
        some += __shfl_xor(some, o, 64);
    }
    if (threadIdx.x % 64 == 0) {
        wn[threadIdx.x / 64] = n;
        wsome[threadIdx.x / 64] = some;
    }
    __syncthreads();
    n = 0;
    some = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
        n += wn[w];
        some += wsome[w];
    }
    if (S == 1) some = 1;
    // half a wave adds an expert's 32 row groups
    const int re = (blockIdx.x % eb) * W + threadIdx.x / 32;
    p = sp[threadIdx.x / 32][threadIdx.x % 32];
    c = sc[threadIdx.x / 32][threadIdx.x % 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        p += __shfl_xor(p, o, 64);
        c += __shfl_xor(c, o, 64);
    }
    double l = 0.0;
    if (threadIdx.x % 32 == 0 && re < E) {
        const double nn = n;
        const double f = n > 0 ? static_cast<double>(alpha) * E * c / (k * nn * nn * some) : 0.0;
        counts[static_cast<int64_t>(s) * E + re] = c;
        coef[static_cast<int64_t>(s) * E + re] = static_cast<float>(f);
        l = n > 0 ? f * p : 0.0;
    }
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = l;
    __syncthreads();
    auto sum32 = [&](double v) {  // lanes 0 .. 31, in a fixed order
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
        return v;
    };
    if (threadIdx.x < 64) l = sum32(red[threadIdx.x % 32]);
    if (gridDim.x == 1) {
        if (threadIdx.x == 0) *loss = static_cast<float>(l);
        return;
    }
    if (threadIdx.x == 0) {
        ws.part_loss[blockIdx.x] = l;
        if (hand_over)
            last = __hip_atomic_fetch_add(ws.ticket, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
                   static_cast<int>(gridDim.x) - 1;
    }
    if (!hand_over) return;
    // The last block to come adds the blocks' losses in order; nobody waits for
    // anybody.  Taking the ticket releases the block's loss and acquires those of the
    // blocks before it, the barrier hands that on to the first wave.
    __syncthreads();
    if (!last || threadIdx.x >= 64) return;
    l = 0.0;
    if (threadIdx.x < 32)
        for (int i = threadIdx.x; i < static_cast<int>(gridDim.x); i += 32) l += ws.part_loss[i];
    l = sum32(l);
    if (threadIdx.x == 0) *loss = static_cast<float>(l);
}

// The blocks' losses, added in order, where there are more blocks than this.  Each
// release writes an XCD's L2 back and the blocks take the ticket one by one: 32768
// tokens of 512 experts in 4, 8, 12 and 60 sequences (64, 128, 192, 960 blocks) 24.8,
// 25.8, 30.1 and (relaxed) 44 us by the ticket, 24.2, 23.7, 26.0 and 33 with this kernel;
// 4096 tokens of 64 experts (2 blocks) 10.2 and 10.9, and a launch less on the host.
constexpr int64_t kHandOverBlocks = 64;
__global__ __launch_bounds__(1024) void balance_loss_kernel(const double *__restrict__ part, int n,
                                                            float *__restrict__ loss) {
    __shared__ double s[16];
    double l = 0.0;
#pragma unroll 4
    for (int i = threadIdx.x; i < n; i += 1024) l += part[i];
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) l += __shfl_xor(l, o, 64);
    if (threadIdx.x % 64 == 0) s[threadIdx.x / 64] = l;
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (int w = 1; w < 16; ++w) l += s[w];
    *loss = static_cast<float>(l);
}

template <int LT, int QQ>
__global__ __launch_bounds__(64 * kWaves) void balance_bwd_kernel(const float *__restrict__ logits, int64_t T, int E,
                                                                  BalanceArgs b, float *__restrict__ dlogits) {
    constexpr int TPW = 64 / LT;
    const int lane = threadIdx.x & 63;
    const int r = lane % LT;
    const int64_t t = (static_cast<int64_t>(blockIdx.x) * kWaves + (threadIdx.x >> 6)) * TPW + lane / LT;
    auto ex = [&](int q) { return 4 * (r + LT * (q >> 2)) + (q & 3); };
    float p[QQ], g[QQ];
    load_token<LT, QQ>(logits + t * E, t < T, r, E, p);  // on its way during the search
    const int s = b.seq_offsets ? find_sequence<LT>(b.seq_offsets, b.S, t) : 0;
    const bool live = t < T && s >= 0 && s < b.S && (!b.mask || b.mask[t] != 0);
    token_softmax<LT, QQ>(live, p);
    const float *co = b.coef + static_cast<int64_t>(live ? s : 0) * E;
    const float up = b.dloss ? *b.dloss : 1.0f;
    float c = 0.0f;
#pragma unroll
    for (int q = 0; q < QQ; ++q) {
        g[q] = live && ex(q) < E ? co[ex(q)] : 0.0f;
        c = __builtin_fmaf(p[q], g[q], c);
    }
#pragma unroll
    for (int o = LT / 2; o > 0; o >>= 1) c += __shfl_xor(c, o, 64);
    if (t >= T) return;
    // tokens that do not count get zeros, whatever their logits
    float *row = dlogits + t * E;
#pragma unroll
    for (int q = 0; q < QQ; ++q) g[q] = live ? up * p[q] * (g[q] - c) : 0.0f;
    if (E % 4 == 0) {
#pragma unroll
        for (int q = 0; q < QQ; q += 4)
            if (ex(q) < E) *reinterpret_cast<float4 *>(row + ex(q)) = make_float4(g[q], g[q + 1], g[q + 2], g[q + 3]);
    } else {
#pragma unroll
        for (int q = 0; q < QQ; ++q)
            if (ex(q) < E) row[ex(q)] = g[q];
    }
}

// Lanes per token and experts per lane: at most 16 experts a lane up to 512.
// Forward, 32768 tokens of 160 experts, both kernels: 16 lanes 21.4 us, 8 lanes
// 26.6, 32 lanes 22.2 (one sequence).
#define XMOE_BALANCE_SHAPE(E, CALL)      \
    do {                                 \
        if ((E) <= 32) CALL(8, 4);       \
        else if ((E) <= 64) CALL(16, 4); \
        else if ((E) <= 128) CALL(16, 8); \
        else if ((E) <= 192) CALL(16, 12); \
        else if ((E) <= 256) CALL(16, 16); \
        else if ((E) <= 512) CALL(32, 16); \
        else CALL(32, 32);               \
    } while (0)
// With many tokens 8 lanes a token, fewer steps between lanes.  Backward, up to
// 256 experts (32768 tokens of 64, 160, 256 experts 5.2, 9.5, 14.8 us against 6.0,
// 11.2, 16.7; 16384 of 160 6.6 against 7.0; 8192 of 160 5.2 against 4.9; 32768 of
// 512 29.3 against 28.0); forward, up to 128, whose lanes hold the sums too (32768
// tokens of 64 and 128 11.6 and 13.4 us against 12.9 and 13.7; 131072 of 64 17.5
// against 19.8, of 160 in 64 sequences 30.3 against 29.9).
constexpr int64_t kManyTokens = 16384;

}  // namespace

size_t balance_workspace(int64_t T, int E, int S) { return balance_ws(nullptr, T, E, S).bytes; }

hipError_t launch_balance_loss(const float *logits, const int32_t *ids, int64_t T, int E, int k,
                               const int32_t *seq_offsets, int S, const uint8_t *mask, float alpha, float *loss,
                               int32_t *counts, float *coef, void *ws, hipStream_t st) {
    const BalanceWs w = balance_ws(ws, T, E, S);
    const int chunk = chunk_tokens(T);
    // one block at least: it clears the ticket
    const unsigned blocks = static_cast<unsigned>(std::max<int64_t>((T + chunk - 1) / chunk, 1));
#define XMOE_BALANCE_PART(LT, QQ)                                                                                  \
    hipLaunchKernelGGL((balance_part_kernel<LT, QQ>), dim3(blocks), dim3(64 * kWaves), 0, st, logits, ids, T, E, k, \
                       seq_offsets, S, mask, chunk, w)
    const bool many = T >= kManyTokens && E > 32;
    if (many && E <= 64) XMOE_BALANCE_PART(8, 8);
    else if (many && E <= 128) XMOE_BALANCE_PART(8, 16);
    else XMOE_BALANCE_SHAPE(E, XMOE_BALANCE_PART);
#undef XMOE_BALANCE_PART
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (w.nseq) {
        hipLaunchKernelGGL(balance_count_kernel, dim3(static_cast<unsigned>(S)), dim3(256), 0, st, T, seq_offsets, chunk, w);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    const int64_t final = static_cast<int64_t>(S) * final_blocks(E);
    const bool hand_over = final <= kHandOverBlocks;
    hipLaunchKernelGGL(balance_final_kernel, dim3(static_cast<unsigned>(final)), dim3(1024), 0, st, T, E, k, seq_offsets,
                       S, chunk, alpha, w, hand_over, loss, counts, coef);
    if (!hand_over) {
        if ((e = hipGetLastError()) != hipSuccess) return e;
        hipLaunchKernelGGL(balance_loss_kernel, dim3(1), dim3(1024), 0, st, w.part_loss, static_cast<int>(final), loss);
    }
    return hipGetLastError();
}

hipError_t launch_balance_loss_bwd(const float *logits, int64_t T, int E, const BalanceArgs &b, float *dlogits,
                                   hipStream_t st) {
    if (T <= 0) return hipSuccess;
#define XMOE_BALANCE_BWD(LT, QQ)                                                                                     \
    hipLaunchKernelGGL((balance_bwd_kernel<LT, QQ>),                                                                 \
                       dim3(static_cast<unsigned>((T + kWaves * (64 / (LT)) - 1) / (kWaves * (64 / (LT))))),         \
                       dim3(64 * kWaves), 0, st, logits, T, E, b, dlogits)
    const bool many = T >= kManyTokens && E > 32;
    if (many && E <= 64) XMOE_BALANCE_BWD(8, 8);
    else if (many && E <= 128) XMOE_BALANCE_BWD(8, 16);
    else if (many && E <= 192) XMOE_BALANCE_BWD(8, 24);
    else if (many && E <= 256) XMOE_BALANCE_BWD(8, 32);
    else XMOE_BALANCE_SHAPE(E, XMOE_BALANCE_BWD);
#undef XMOE_BALANCE_BWD
    return hipGetLastError();
}

}  // namespace xmoe

// Residual addition and root-mean-square norm, forward and backward.
//
//   s = x + res (rounded to the dtype: the residual stream that later layers
//   add to, so the norm and its backward see the stored values)
//   rstd = 1 / sqrt(mean(s^2) + eps);  y = s * rstd * gamma
// Backward, n = s * rstd, u = dy * gamma:
//   dx = rstd * (u - n * mean(u * n)) + dsum;   dgamma = sum over rows of dy * n
//
// Both directions are one pass over the rows, which stay in registers between
// the reduction and the output: memory-bound, each input read once and each
// output written once.  Measured against a copy's 5.07 TB/s (bf16): forward of
// 8192 x 7168 with bf16 and 8-bit outputs (530 MB) 110 us, 4.8 TB/s; of 4096 x
// 2048 (67 MB, part of it in the last-level cache) 13.2 us; backward of 32768 x
// 4096 (1.07 GB) 223 us, 4.8 TB/s, and 5 us for dgamma's sum.  One token of
// 2048: 2.6 us.
#include <algorithm>

#include "common.hpp"
#include "kernels.hpp"
#include "mx8.hpp"

namespace xmoe {

namespace {

// Sum over the WPR waves of a row (fixed order).  red: one float per wave.
template <int WPR>
__device__ __forceinline__ float row_sum(float v, float *red, int wave) {
    v = wave_sum(v);
    if constexpr (WPR > 1) {
        if ((threadIdx.x & 63) == 0) red[wave] = v;
        __syncthreads();
        const int w0 = wave / WPR * WPR;
        v = red[w0];
#pragma unroll
        for (int i = 1; i < WPR; ++i) v += red[w0 + i];
    }
    return v;
}

constexpr int fwd_threads(int wpr) { return wpr > 4 ? 64 * wpr : 256; }

// WPR waves per row, VPL 16-byte vectors per lane (vector c of a row belongs to
// lane c % 64 of wave (c / 64) % WPR).  No __restrict__: sum or y may be x or
// res (every lane reads its own vectors before it writes them).
template <typename T, int VPL, int WPR>
__global__ __launch_bounds__(fwd_threads(WPR)) void add_rmsnorm_kernel(const T *x, const T *res, const T *gamma,
                                                                       int64_t ntok, int d, float eps, T *sum, T *y,
                                                                       uint8_t *q, uint8_t *scale, float *rstd) {
    constexpr int V = Elem<T>::kVec;
    constexpr int kWaves = fwd_threads(WPR) / 64, RPB = kWaves / WPR;
    __shared__ float red[kWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * RPB + wave / WPR;
    const bool live = t < ntok;
    const int nvec = d / V;
    const int c0 = (wave % WPR) * 64 + lane;
    float f[VPL][V];
    uint4 g[VPL];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int c = c0 + i * 64 * WPR;
#pragma unroll
        for (int e = 0; e < V; ++e) f[i][e] = 0.0f;
        if (live && c < nvec) {
            const uint4 a = reinterpret_cast<const uint4 *>(x + t * d)[c];
            g[i] = reinterpret_cast<const uint4 *>(gamma)[c];
            Elem<T>::unpack(a, f[i]);
            if (res) {
                float b[V];
                Elem<T>::unpack(reinterpret_cast<const uint4 *>(res + t * d)[c], b);
#pragma unroll
                for (int e = 0; e < V; ++e) f[i][e] += b[e];
                const uint4 r = Elem<T>::pack(f[i]);  // the norm sees the stored (rounded) sum
                Elem<T>::unpack(r, f[i]);
                if (sum) reinterpret_cast<uint4 *>(sum + t * d)[c] = r;
            } else if (sum) {
                reinterpret_cast<uint4 *>(sum + t * d)[c] = a;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) ss = __builtin_fmaf(f[i][e], f[i][e], ss);
    ss = row_sum<WPR>(ss, red, wave);
    const float rs = 1.0f / sqrtf(ss / static_cast<float>(d) + eps);
    if (rstd && live && c0 == 0) rstd[t] = rs;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int c = c0 + i * 64 * WPR;
        const bool in = live && c < nvec;
        if (in) {
            float gv[V];
            Elem<T>::unpack(g[i], gv);
#pragma unroll
            for (int e = 0; e < V; ++e) f[i][e] = f[i][e] * rs * gv[e];
            if (y) reinterpret_cast<uint4 *>(y + t * d)[c] = Elem<T>::pack(f[i]);
        }
        if (q) {  // from the fp32 values: one rounding to 8 bits
            uint32_t o[V / 4];
            const uint32_t b = mx8_quant<V>(f[i], o);
            const uint32_t w = mx8_scale_dword<V>(c < nvec ? b : kMxOne, lane);
            if (in) {
                uint32_t *dst = reinterpret_cast<uint32_t *>(q + t * d + static_cast<int64_t>(c) * V);
                if constexpr (V == 8) *reinterpret_cast<uint2 *>(dst) = make_uint2(o[0], o[1]);
                else *dst = o[0];
                if (c % (128 / V) == 0)
                    *reinterpret_cast<uint32_t *>(scale + (static_cast<int64_t>(c / (128 / V)) * ntok + t) * 4) = w;
            }
        }
    }
}

// Backward: a block takes rows blockIdx.x * RPB + r, then every gridDim.x * RPB
// further, and keeps its columns' share of dgamma in registers; its partial sum
// goes to part[blockIdx.x] once all its rows are done.  dx may be dy or dsum.
template <typename T, int VPL, int WPR, int NW>
__global__ __launch_bounds__(64 * NW) void add_rmsnorm_bwd_kernel(const T *dy, const T *dsum, const T *s,
                                                                  const T *gamma, const float *rstd, int64_t ntok,
                                                                  int d, T *dx, float *part) {
    constexpr int V = Elem<T>::kVec;
    constexpr int RPB = NW / WPR;
    __shared__ float red[2][NW];
    __shared__ float dgs[RPB > 1 ? (RPB - 1) * WPR * 64 * V : 1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int nvec = d / V;
    const int c0 = (wave % WPR) * 64 + lane;
    uint4 g[VPL];
    float dg[VPL][V];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int c = c0 + i * 64 * WPR;
        g[i] = c < nvec ? reinterpret_cast<const uint4 *>(gamma)[c] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < V; ++e) dg[i][e] = 0.0f;
    }
    int turn = 0;
    // the trip count is the same for all waves of the block (the row sums meet a barrier)
    for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * RPB; t0 < ntok;
         t0 += static_cast<int64_t>(gridDim.x) * RPB, turn ^= 1) {
        const int64_t t = t0 + wave / WPR;
        const bool live = t < ntok;
        const float rs = live ? rstd[t] : 0.0f;
        uint4 a[VPL], b[VPL];
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int c = c0 + i * 64 * WPR;
            const bool in = live && c < nvec;
            a[i] = in ? reinterpret_cast<const uint4 *>(dy + t * d)[c] : make_uint4(0, 0, 0, 0);
            b[i] = in ? reinterpret_cast<const uint4 *>(s + t * d)[c] : make_uint4(0, 0, 0, 0);
        }
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            float yv[V], nv[V], gv[V];
            Elem<T>::unpack(a[i], yv);
            Elem<T>::unpack(b[i], nv);
            Elem<T>::unpack(g[i], gv);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float n = nv[e] * rs;
                dg[i][e] = __builtin_fmaf(yv[e], n, dg[i][e]);
                dot = __builtin_fmaf(yv[e] * gv[e], n, dot);
            }
        }
        const float m = row_sum<WPR>(dot, red[turn], wave) / static_cast<float>(d);
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int c = c0 + i * 64 * WPR;
            if (!(live && c < nvec)) continue;
            float yv[V], nv[V], gv[V], o[V];
            Elem<T>::unpack(a[i], yv);
            Elem<T>::unpack(b[i], nv);
            Elem<T>::unpack(g[i], gv);
#pragma unroll
            for (int e = 0; e < V; ++e) o[e] = rs * (yv[e] * gv[e] - nv[e] * rs * m);
            if (dsum) {
                float r[V];
                Elem<T>::unpack(reinterpret_cast<const uint4 *>(dsum + t * d)[c], r);
#pragma unroll
                for (int e = 0; e < V; ++e) o[e] += r[e];
            }
            reinterpret_cast<uint4 *>(dx + t * d)[c] = Elem<T>::pack(o);
        }
    }
    // the block's row slots added in slot order, one vector of each lane at a time
    const int slot = wave / WPR, col = (wave % WPR) * 64 + lane;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int c = c0 + i * 64 * WPR;
        if constexpr (RPB > 1) {
            __syncthreads();
            if (slot > 0) {
#pragma unroll
                for (int e = 0; e < V; ++e) dgs[((slot - 1) * V + e) * WPR * 64 + col] = dg[i][e];
            }
            __syncthreads();
            if (slot == 0) {
                for (int r = 0; r < RPB - 1; ++r)
#pragma unroll
                    for (int e = 0; e < V; ++e) dg[i][e] += dgs[(r * V + e) * WPR * 64 + col];
            }
        }
        if (slot == 0 && c < nvec) {
            float *p = part + static_cast<int64_t>(blockIdx.x) * d + static_cast<int64_t>(c) * V;
#pragma unroll
            for (int e = 0; e < V; e += 4)
                *reinterpret_cast<float4 *>(p + e) = make_float4(dg[i][e], dg[i][e + 1], dg[i][e + 2], dg[i][e + 3]);
        }
    }
}

// dgamma[c] = sum over the blocks' partial sums: 32 columns a block, whose 32 row
// groups take every 32nd partial and meet in LDS (fixed order).
__global__ __launch_bounds__(1024) void dgamma_kernel(const float *__restrict__ part, int nblk, int d,
                                                      float *__restrict__ dgamma) {
    __shared__ float s[32][33];
    const int col = threadIdx.x & 31, grp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + col;
    float v = 0.0f;
    if (c < d) {
#pragma unroll 8
        for (int b = grp; b < nblk; b += 32) v += part[static_cast<int64_t>(b) * d + c];
    }
    s[grp][col] = v;
    __syncthreads();
    // a wave per two columns' 32 sums
    v = s[threadIdx.x & 31][threadIdx.x >> 5];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
    const int w = blockIdx.x * 32 + (threadIdx.x >> 5);
    if ((threadIdx.x & 31) == 0 && w < d) dgamma[w] = v;
}

// Waves per row and vectors per lane: a row of nvec 16-byte vectors.  Up to 4
// vectors a lane; with few rows a row is spread over more waves instead, so
// that a row's latency is that of one vector (bf16, one wave a row against the
// spread: 1 x 2048 5.5 -> 3.0 us, 256 x 4096 6.4 -> 3.9, 1024 x 2048 7.1 -> 5.1).
// Past 4096 waves the device is full and the two are level.
struct RowShape {
    int vpl, wpr;
};
RowShape fwd_shape(int64_t T, int nvec) {
    int wpr = 1;
    while (64 * 4 * wpr < nvec) wpr *= 2;
    while (wpr < 16 && T * wpr < 4096 && 64 * wpr < nvec) wpr *= 2;
    const int need = (nvec + 64 * wpr - 1) / (64 * wpr);
    return {need <= 1 ? 1 : need <= 2 ? 2 : 4, wpr};
}

// Backward blocks of NW waves: rows are dealt to blocks in turn.  One block for
// each compute unit: twice as many double dgamma's partial sums and leave less
// of the rows in flight to each (4096 x 2048 23.7 against 19.7 us, 32768 x 4096
// 226 against 223, 20000 x 1024 31.4 against 33.0); half as many leave units idle.
constexpr int bwd_waves(int wpr) { return wpr > 8 ? wpr : 8; }
RowShape bwd_shape(int nvec) {
    int wpr = 1;
    while (64 * 4 * wpr < nvec) wpr *= 2;
    const int need = (nvec + 64 * wpr - 1) / (64 * wpr);
    return {need <= 1 ? 1 : need <= 2 ? 2 : 4, wpr};
}
int bwd_blocks(int64_t T, int nvec) {
    const RowShape r = bwd_shape(nvec);
    const int rpb = bwd_waves(r.wpr) / r.wpr;
    const int64_t n = (T + rpb - 1) / rpb;
    return static_cast<int>(std::min<int64_t>(n, 256));
}

template <typename T>
hipError_t fwd(const void *x, const void *res, const void *gamma, int64_t ntok, int d, float eps, void *sum, void *y,
               void *q, void *scale, float *rstd, hipStream_t st) {
    const RowShape r = fwd_shape(ntok, d / Elem<T>::kVec);
#define XMOE_NORM(VPL, WPR)                                                                                    \
    do {                                                                                                       \
        constexpr int rpb = fwd_threads(WPR) / 64 / WPR;                                                       \
        hipLaunchKernelGGL((add_rmsnorm_kernel<T, VPL, WPR>), dim3(static_cast<unsigned>((ntok + rpb - 1) / rpb)), \
                           dim3(fwd_threads(WPR)), 0, st, static_cast<const T *>(x), static_cast<const T *>(res), \
                           static_cast<const T *>(gamma), ntok, d, eps, static_cast<T *>(sum), static_cast<T *>(y), \
                           static_cast<uint8_t *>(q), static_cast<uint8_t *>(scale), rstd);                    \
    } while (0)
#define XMOE_NORM_VPL(WPR)                   \
    switch (r.vpl) {                         \
        case 1: XMOE_NORM(1, WPR); break;    \
        case 2: XMOE_NORM(2, WPR); break;    \
        default: XMOE_NORM(4, WPR); break;   \
    }
    switch (r.wpr) {
        case 1: XMOE_NORM_VPL(1) break;
        case 2: XMOE_NORM_VPL(2) break;
        case 4: XMOE_NORM_VPL(4) break;
        case 8: XMOE_NORM_VPL(8) break;
        default: XMOE_NORM_VPL(16) break;
    }
#undef XMOE_NORM_VPL
#undef XMOE_NORM
    return hipGetLastError();
}

template <typename T>
hipError_t bwd(const void *dy, const void *dsum, const void *s, const void *gamma, const float *rstd, int64_t ntok,
               int d, void *dx, float *part, int nblk, hipStream_t st) {
    const RowShape r = bwd_shape(d / Elem<T>::kVec);
#define XMOE_NORM_BWD(VPL, WPR)                                                                                 \
    hipLaunchKernelGGL((add_rmsnorm_bwd_kernel<T, VPL, WPR, bwd_waves(WPR)>), dim3(static_cast<unsigned>(nblk)), \
                       dim3(64 * bwd_waves(WPR)), 0, st, static_cast<const T *>(dy), static_cast<const T *>(dsum), \
                       static_cast<const T *>(s), static_cast<const T *>(gamma), rstd, ntok, d,                 \
                       static_cast<T *>(dx), part)
    switch (r.wpr) {
        case 1:
            if (r.vpl == 1) XMOE_NORM_BWD(1, 1);
            else if (r.vpl == 2) XMOE_NORM_BWD(2, 1);
            else XMOE_NORM_BWD(4, 1);
            break;
        case 2: XMOE_NORM_BWD(4, 2); break;
        case 4: XMOE_NORM_BWD(4, 4); break;
        case 8: XMOE_NORM_BWD(4, 8); break;
        default: XMOE_NORM_BWD(4, 16); break;
    }
#undef XMOE_NORM_BWD
    return hipGetLastError();
}

}  // namespace

hipError_t launch_add_rmsnorm(int dt, const void *x, const void *res, const void *gamma, int64_t T, int d, float eps,
                              void *sum, void *y, void *q, void *scale, float *rstd, hipStream_t s) {
    if (T <= 0) return hipSuccess;
    return dt == kBF16 ? fwd<bf16_t>(x, res, gamma, T, d, eps, sum, y, q, scale, rstd, s)
                       : fwd<float>(x, res, gamma, T, d, eps, sum, y, q, scale, rstd, s);
}

size_t add_rmsnorm_bwd_workspace(int64_t T, int d, int dt) {
    const int n = bwd_blocks(T, d / (dt == kBF16 ? 8 : 4));
    return static_cast<size_t>(std::max(n, 1)) * d * sizeof(float);
}

hipError_t launch_add_rmsnorm_bwd(int dt, const void *dy, const void *dsum, const void *sum, const void *gamma,
                                  const float *rstd, int64_t T, int d, void *dx, float *dgamma, void *ws,
                                  hipStream_t s) {
    float *part = static_cast<float *>(ws);
    const int n = bwd_blocks(T, d / (dt == kBF16 ? 8 : 4));
    if (n > 0) {
        const hipError_t e = dt == kBF16 ? bwd<bf16_t>(dy, dsum, sum, gamma, rstd, T, d, dx, part, n, s)
                                         : bwd<float>(dy, dsum, sum, gamma, rstd, T, d, dx, part, n, s);
        if (e != hipSuccess) return e;
    }
    // no rows: dgamma = 0
    hipLaunchKernelGGL(dgamma_kernel, dim3(static_cast<unsigned>((d + 31) / 32)), dim3(1024), 0, s, part, n, d, dgamma);
    return hipGetLastError();
}

}  // namespace xmoe

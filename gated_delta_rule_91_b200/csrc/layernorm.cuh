// layernorm.cuh -- layer norm over the last axis, with the residual stream
// (gdr_layernorm_fwd, gdr_layernorm_bwd):
//     h = x + residual (rounded to the stream's type: it is what is normalised)
//     y = (h - mean) / sqrt(var + eps) * w + b
//     dx = rstd (g - mean(g) - n mean(g n)) + dres,   g = dy w,  n = (h - mean) rstd
//     dw = sum_rows dy n,   db = sum_rows dy
// HBM-bound: every row is read once into registers (raw, as stored) and both
// statistics are taken from there, the variance from centred values.  TPR
// threads share a row and hold NV vectors of V elements each.
#pragma once
#include "common.cuh"
#include "conv.cuh"

namespace gdr {

struct NormArgs {
    long long R;
    int D;
    float eps;
    const void *x, *res;   // rows x D; res may be null
    const float *w, *b;    // b may be null
    void *y, *h;           // h null without a residual
    // backward (x is the stored stream h)
    const void *dy, *dres;
    void *dx;
    float *part;           // [blocks][2][D]
};

// Sums of NS values over the TPR threads of a row.  `buf` has two sides of (NT/32) NS floats that calls take in
// turn, so that one barrier a call is enough (a side is written again only after the next call's barrier).
template <int TPR, int NT, int NS>
__device__ __forceinline__ void norm_reduce(float (&s)[NS], float *buf, int side) {
#pragma unroll
    for (int k = 0; k < NS; ++k) s[k] = warp_sum(s[k], 32);
    if (TPR > 32) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        constexpr int W = TPR > 32 ? TPR / 32 : 1;
        float *b = buf + side * (NT / 32) * NS;
        if (lane == 0)
#pragma unroll
            for (int k = 0; k < NS; ++k) b[warp * NS + k] = s[k];
        __syncthreads();
        const int w0 = warp / W * W;
#pragma unroll
        for (int k = 0; k < NS; ++k) {
            s[k] = 0.f;
#pragma unroll
            for (int i = 0; i < W; ++i) s[k] += b[(w0 + i) * NS + k];
        }
    }
}

// V elements as they are stored, and their values.
template <typename T, int V> struct NormRaw {
    T e[V];
};
template <> struct NormRaw<__nv_bfloat16, 8> {
    uint4 e;
};
template <> struct NormRaw<float, 4> {
    float4 e;
};
template <typename T, int V>
__device__ __forceinline__ void norm_values(const NormRaw<T, V> &r, float *v) {
    ConvVec<T, V>::ld(reinterpret_cast<const T *>(&r), v);
}
template <typename T, int V>
__device__ __forceinline__ NormRaw<T, V> norm_load(const void *p, size_t at) {
    return *reinterpret_cast<const NormRaw<T, V> *>(static_cast<const T *>(p) + at);
}
template <int V>
__device__ __forceinline__ void norm_weights(const float *p, int c, float *v) {
    if (V == 8) {
        ConvVec<float, 4>::ld(p + c, v);
        ConvVec<float, 4>::ld(p + c + V / 2, v + V / 2);
    } else {
        ConvVec<float, V == 8 ? 4 : V>::ld(p + c, v);
    }
}

template <typename T, int V, int TPR, int NV, int NT>
__global__ void __launch_bounds__(NT) norm_fwd_kernel(NormArgs a) {
    __shared__ float buf[2 * (NT / 32)];
    const int rl = threadIdx.x / TPR, tr = threadIdx.x % TPR;
    const long long row = (long long)blockIdx.x * (NT / TPR) + rl;
    const bool live = row < a.R;
    const size_t base = (size_t)(live ? row : 0) * a.D;
    // every load of the row before the first store: the stream's store may not move past a load by itself
    NormRaw<T, V> rx[NV], rr[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + tr) * V;
        if (live && c < a.D) rx[i] = norm_load<T, V>(a.x, base + c);
    }
    if (a.res)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + tr) * V;
            if (live && c < a.D) rr[i] = norm_load<T, V>(a.res, base + c);
        }
    float v[NV][V];
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + tr) * V;
#pragma unroll
        for (int e = 0; e < V; ++e) v[i][e] = 0.f;
        if (!live || c >= a.D) continue;
        norm_values<T, V>(rx[i], v[i]);
        if (a.res) {
            float r[V];
            norm_values<T, V>(rr[i], r);
#pragma unroll
            for (int e = 0; e < V; ++e) v[i][e] = to_f32(from_f32<T>(v[i][e] + r[e]));
            ConvVec<T, V>::st(static_cast<T *>(a.h) + base + c, v[i]);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) s[0] += v[i][e];
    }
    norm_reduce<TPR, NT, 1>(s, buf, 0);
    const float mean = s[0] / (float)a.D;
    s[0] = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + tr) * V;
        if (c >= a.D) continue;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            v[i][e] -= mean;
            s[0] = fmaf(v[i][e], v[i][e], s[0]);
        }
    }
    norm_reduce<TPR, NT, 1>(s, buf, 1);
    if (!live) return;
    const float rstd = 1.f / sqrtf(s[0] / (float)a.D + a.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + tr) * V;
        if (c >= a.D) continue;
        float w[V], b[V];
        norm_weights<V>(a.w, c, w);
        if (a.b) norm_weights<V>(a.b, c, b);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            v[i][e] = v[i][e] * rstd * w[e];
            if (a.b) v[i][e] += b[e];
        }
        ConvVec<T, V>::st(static_cast<T *>(a.y) + base + c, v[i]);
    }
}

// One block walks rows blockIdx.x * (NT/TPR) + rl, + gridDim.x * (NT/TPR), ...; the next row is read while this one
// is reduced.  Every thread keeps its columns' dw and db, and the block's row slots are joined in order at the end.
template <typename T, int V, int TPR, int NV, int NT>
__global__ void __launch_bounds__(NT) norm_bwd_kernel(NormArgs a) {
    __shared__ float buf[2 * (NT / 32) * 3];
    extern __shared__ float join[];  // [NT/TPR][2][D] when NT > TPR
    const int rl = threadIdx.x / TPR, tr = threadIdx.x % TPR;
    float w[NV][V], aw[NV][V], ab[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + tr) * V;
#pragma unroll
        for (int e = 0; e < V; ++e) aw[i][e] = ab[i][e] = w[i][e] = 0.f;
        if (c < a.D) norm_weights<V>(a.w, c, w[i]);
    }
    const float inv = 1.f / (float)a.D;
    const long long per = (long long)gridDim.x * (NT / TPR);
    const long long trips = (a.R + per - 1) / per;  // the same for every thread: the row sums use block barriers
    NormRaw<T, V> rh[NV], rg[NV], rd[NV];
    auto fetch = [&](long long k) {
        const long long row = k * per + (long long)blockIdx.x * (NT / TPR) + rl;
        if (row >= a.R) return;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + tr) * V;
            if (c >= a.D) continue;
            rh[i] = norm_load<T, V>(a.x, (size_t)row * a.D + c);
            rg[i] = norm_load<T, V>(a.dy, (size_t)row * a.D + c);
            if (a.dres) rd[i] = norm_load<T, V>(a.dres, (size_t)row * a.D + c);
        }
    };
    fetch(0);
    for (long long k = 0; k < trips; ++k) {
        const long long row = k * per + (long long)blockIdx.x * (NT / TPR) + rl;
        const bool live = row < a.R;
        const size_t base = (size_t)(live ? row : 0) * a.D;
        float h[NV][V], g[NV][V], dx[NV][V], s1[1] = {0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + tr) * V;
#pragma unroll
            for (int e = 0; e < V; ++e) h[i][e] = g[i][e] = dx[i][e] = 0.f;
            if (!live || c >= a.D) continue;
            norm_values<T, V>(rh[i], h[i]);
            norm_values<T, V>(rg[i], g[i]);
            if (a.dres) norm_values<T, V>(rd[i], dx[i]);
#pragma unroll
            for (int e = 0; e < V; ++e) s1[0] += h[i][e];
        }
        if (k + 1 < trips) fetch(k + 1);
        norm_reduce<TPR, NT, 1>(s1, buf, 0);
        const float mean = s1[0] * inv;
        float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + tr) * V;
            if (!live || c >= a.D) continue;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                h[i][e] -= mean;
                const float gw = g[i][e] * w[i][e];
                s[0] = fmaf(h[i][e], h[i][e], s[0]);
                s[1] += gw;
                s[2] = fmaf(gw, h[i][e], s[2]);
            }
        }
        norm_reduce<TPR, NT, 3>(s, buf, 1);
        const float rstd = 1.f / sqrtf(s[0] * inv + a.eps);
        const float m1 = s[1] * inv, m2 = s[2] * inv * rstd;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + tr) * V;
            if (!live || c >= a.D) continue;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float n = h[i][e] * rstd;
                dx[i][e] = fmaf(rstd, g[i][e] * w[i][e] - m1 - n * m2, dx[i][e]);
                aw[i][e] = fmaf(g[i][e], n, aw[i][e]);
                ab[i][e] += g[i][e];
            }
            ConvVec<T, V>::st(static_cast<T *>(a.dx) + base + c, dx[i]);
        }
    }
    float *out = a.part + (size_t)blockIdx.x * 2 * a.D;
    if (NT > TPR) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + tr) * V;
            if (c >= a.D) continue;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                join[(rl * 2) * a.D + c + e] = aw[i][e];
                join[(rl * 2 + 1) * a.D + c + e] = ab[i][e];
            }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < 2 * a.D; c += NT) {
            float s = 0.f;
            for (int r = 0; r < NT / TPR; ++r) s += join[r * 2 * a.D + c];
            out[c] = s;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + tr) * V;
            if (c >= a.D) continue;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                out[c + e] = aw[i][e];
                out[a.D + c + e] = ab[i][e];
            }
        }
    }
}

// dw, db: the blocks' partial sums in order, in 64 bits.  Block: 32 columns x 32 rows at a time.
__global__ void __launch_bounds__(1024) norm_sum_kernel(int blocks, int D, const float *__restrict__ part,
                                                        float *__restrict__ dw, float *__restrict__ db) {
    __shared__ double red[32][32];
    const int lane = threadIdx.x & 31, wy = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    double s = 0.0;
    if (c < D)
#pragma unroll 4
        for (int k = wy; k < blocks; k += 32) s += (double)part[((size_t)k * 2 + blockIdx.y) * D + c];
    red[wy][lane] = s;
    __syncthreads();
    if (wy == 0 && c < D) {
        for (int y = 1; y < 32; ++y) s += red[y][lane];
        (blockIdx.y ? db : dw)[c] = (float)s;
    }
}

// ---- host side ----------------------------------------------------------------------------------
constexpr int kNormMaxD = 16384;
constexpr int kNormBwdMaxBlocks = 148 * 4;

// Calls F<V, TPR, NV, NT>: vectors of 16 bytes where D allows, else single elements.  The fewest threads per row
// that hold it in at most M elements a thread (the backward keeps five arrays of them), a warp where that is enough.
template <typename T, bool BWD, template <typename, int, int, int, int> class F, typename... A>
cudaError_t norm_pick(int D, A... args) {
    constexpr int V = sizeof(T) == 2 ? 8 : 4, M = BWD ? 8 : 16;
    if (D % V == 0) {
        if (D <= 32 * V) return F<T, V, 32, 1, 256>::go(args...);
        if (D <= 32 * M) return F<T, V, 32, M / V, 256>::go(args...);
        if (D <= 128 * M) return F<T, V, 128, M / V, 256>::go(args...);
        if (D <= 256 * M) return F<T, V, 256, M / V, 256>::go(args...);
        if (D <= 512 * M) return F<T, V, 512, M / V, 512>::go(args...);
        if (D <= 512 * 16) return F<T, V, 512, 16 / V, 512>::go(args...);
        return F<T, V, 512, kNormMaxD / (512 * V), 512>::go(args...);
    }
    if (D <= 32 * M) return F<T, 1, 32, M, 256>::go(args...);
    if (D <= 128 * M) return F<T, 1, 128, M, 256>::go(args...);
    if (D <= 512 * M) return F<T, 1, 512, M, 512>::go(args...);
    if (D <= 512 * 16) return F<T, 1, 512, 16, 512>::go(args...);
    return F<T, 1, 512, kNormMaxD / 512, 512>::go(args...);
}

template <typename T, int V, int TPR, int NV, int NT>
struct NormFwd {
    static cudaError_t go(NormArgs a, cudaStream_t s) {
        const long long grid = (a.R + NT / TPR - 1) / (NT / TPR);
        norm_fwd_kernel<T, V, TPR, NV, NT><<<(unsigned)grid, NT, 0, s>>>(a);
        g_launches.fetch_add(1, std::memory_order_relaxed);
        return cudaGetLastError();
    }
};
template <typename T, int V, int TPR, int NV, int NT>
struct NormBwd {
    static cudaError_t go(NormArgs a, float *dw, float *db, cudaStream_t s) {
        long long grid = (a.R + NT / TPR - 1) / (NT / TPR);
        if (grid > kNormBwdMaxBlocks) grid = kNormBwdMaxBlocks;
        const size_t smem = NT > TPR ? (size_t)(NT / TPR) * 2 * a.D * 4 : 0;
        cudaError_t e = cudaFuncSetAttribute(norm_bwd_kernel<T, V, TPR, NV, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)smem);
        if (e != cudaSuccess) return e;
        norm_bwd_kernel<T, V, TPR, NV, NT><<<(unsigned)grid, NT, smem, s>>>(a);
        norm_sum_kernel<<<dim3((a.D + 31) / 32, db ? 2 : 1), 1024, 0, s>>>((int)grid, a.D, a.part, dw, db);
        g_launches.fetch_add(2, std::memory_order_relaxed);
        return cudaGetLastError();
    }
};

}  // namespace gdr

// conv.cuh -- the short causal convolution (gdr_conv_fwd, gdr_conv_bwd):
// depthwise over C channels, width K <= 8, optional bias and SiLU, the last
// K-1 inputs carried between calls (a decode token is T = 1):
//     z[t,c] = bias[c] + sum_{j<K} w[c,j] x[t-K+1+j, c],   y = z sigmoid(z) or z
// HBM-bound: x is read and y written once.  A thread owns V neighbouring
// channels (16 bytes forward, 8 bytes of bf16 backward, where its windows of
// inputs, dz and tap sums have to stay in registers) and walks a run of
// tokens with the last K-1 inputs in registers, so that only the K-1 inputs
// before a run are read a second time, from L2.
#pragma once
#include "common.cuh"

namespace gdr {

constexpr int kShortConvMax = 8;

struct ConvArgs {
    int B, T, C, ldx, silu, run, runs;  // token stride of x; tokens per run, runs per sequence
    const void *x;                      // [B,T,C]
    const float *w, *bias;              // [C,K], [C] or null
    const void *state_in;               // [B,K-1,C] or null
    void *state_out;                    // may equal state_in; or null
    void *y;                            // [B,T,C]
    // backward
    const void *dy, *dstate_out;
    void *dx, *dstate_in;
    float *part;                        // [slots][K+1][C]
};

template <typename T, int V> struct ConvVec;
template <> struct ConvVec<float, 4> {
    static __device__ __forceinline__ void ld(const float *p, float *v) {
        const float4 u = *reinterpret_cast<const float4 *>(p);
        v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
    }
    static __device__ __forceinline__ void st(float *p, const float *v) {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    }
};
template <> struct ConvVec<__nv_bfloat16, 8> {
    static __device__ __forceinline__ void ld(const __nv_bfloat16 *p, float *v) { load8(p, v); }
    static __device__ __forceinline__ void st(__nv_bfloat16 *p, const float *v) {
        __nv_bfloat162 h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<uint4 *>(h);
    }
};
template <> struct ConvVec<__nv_bfloat16, 4> {
    static __device__ __forceinline__ void ld(const __nv_bfloat16 *p, float *v) {
        const float4 u = load4(p);
        v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
    }
    static __device__ __forceinline__ void st(__nv_bfloat16 *p, const float *v) {
        __nv_bfloat162 h[2] = {__floats2bfloat162_rn(v[0], v[1]), __floats2bfloat162_rn(v[2], v[3])};
        *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<uint2 *>(h);
    }
};
template <typename T> struct ConvVec<T, 1> {
    static __device__ __forceinline__ void ld(const T *p, float *v) { v[0] = to_f32(*p); }
    static __device__ __forceinline__ void st(T *p, const float *v) { *p = from_f32<T>(v[0]); }
};

// Input token t (may be negative: the carried window, zero without one).
template <typename T, int V, int K>
__device__ __forceinline__ void conv_input(const ConvArgs &a, int b, int t, int c, float *v) {
    if (t >= 0) {
        ConvVec<T, V>::ld(static_cast<const T *>(a.x) + ((size_t)b * a.T + t) * a.ldx + c, v);
    } else if (a.state_in) {
        ConvVec<T, V>::ld(static_cast<const T *>(a.state_in) + ((size_t)b * (K - 1) + (K - 1 + t)) * a.C + c, v);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = 0.f;
    }
}

// The taps of V channels, w[j][i] of tap j and channel i.  Their V K floats are contiguous (and 16-byte aligned for
// V >= 4): one by one they cost more than the tokens of a short run (151 us against 40 us at B=4 T=4096 C=2304 K=4).
template <int V, int K>
__device__ __forceinline__ void conv_taps(const float *w, int c, float (&t)[K][V]) {
    float f[V * K];
    const float *p = w + (size_t)c * K;
    if (V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V * K / 4; ++i) {
            const float4 u = *reinterpret_cast<const float4 *>(p + 4 * i);
            f[4 * i] = u.x;
            f[4 * i + 1] = u.y;
            f[4 * i + 2] = u.z;
            f[4 * i + 3] = u.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V * K; ++i) f[i] = p[i];
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < K; ++j) t[j][i] = f[i * K + j];
}

// sigmoid(z): for z < -88 the quotient is 0 (an infinite exponential), for large z it is 1.
__device__ __forceinline__ float conv_sigmoid(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

// One thread: V channels x one run.  Runs of a channel group are CG threads apart, so that a warp's
// loads of one token are contiguous.
template <typename T, int V, int K>
__global__ void __launch_bounds__(256) conv_fwd_kernel(ConvArgs a) {
    const int CG = a.C / V;
    const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
    if (id >= (long long)CG * a.runs * a.B) return;
    const int c = (int)(id % CG) * V;
    const long long br = id / CG;
    const int r = (int)(br % a.runs), b = (int)(br / a.runs);
    const int t0 = r * a.run, t1 = min(a.T, t0 + a.run);
    float w[K][V], bias[V], win[K - 1 > 0 ? K - 1 : 1][V];
    conv_taps<V, K>(a.w, c, w);
#pragma unroll
    for (int i = 0; i < V; ++i) bias[i] = a.bias ? a.bias[c + i] : 0.f;
#pragma unroll
    for (int j = 0; j < K - 1; ++j) conv_input<T, V, K>(a, b, t0 - (K - 1) + j, c, win[j]);
    const T *px = static_cast<const T *>(a.x) + ((size_t)b * a.T + t0) * a.ldx + c;
    T *py = static_cast<T *>(a.y) + ((size_t)b * a.T + t0) * a.C + c;
    for (int t = t0; t < t1; t += 4) {
        float x[4][V];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (t + u < t1) ConvVec<T, V>::ld(px + (size_t)u * a.ldx, x[u]);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (t + u < t1) {
                float z[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float s = fmaf(w[K - 1][i], x[u][i], bias[i]);
#pragma unroll
                    for (int j = 0; j < K - 1; ++j) s = fmaf(w[j][i], win[j][i], s);
                    z[i] = a.silu ? s * conv_sigmoid(s) : s;
                }
                ConvVec<T, V>::st(py + (size_t)u * a.C, z);
#pragma unroll
                for (int j = 0; j + 1 < K - 1; ++j)
#pragma unroll
                    for (int i = 0; i < V; ++i) win[j][i] = win[j + 1][i];
                if (K > 1)
#pragma unroll
                    for (int i = 0; i < V; ++i) win[K - 2 > 0 ? K - 2 : 0][i] = x[u][i];
            }
        }
        px += (size_t)4 * a.ldx;
        py += (size_t)4 * a.C;
    }
    // The window after the last token, written by the thread of run 0: no other run reads state_in
    // (a run has at least K-1 tokens), so state_out may be the same buffer.
    if (K > 1 && r == 0 && a.state_out) {
        float v[K - 1 > 0 ? K - 1 : 1][V];
#pragma unroll
        for (int j = 0; j < K - 1; ++j) conv_input<T, V, K>(a, b, a.T - (K - 1) + j, c, v[j]);
#pragma unroll
        for (int j = 0; j < K - 1; ++j)
            ConvVec<T, V>::st(static_cast<T *>(a.state_out) + ((size_t)b * (K - 1) + j) * a.C + c, v[j]);
    }
}

// Backward.  dz_t = dy_t silu'(z_t); dx_s = sum_j w_j dz_{s+K-1-j}; dw_j = sum_t dz_t x_{t-K+1+j}.
// A block is 32 channel groups x 8 runs; each of the 8 walks its runs (a slot's runs are slots*8 apart) and the
// eight tap sums are joined in shared memory in a fixed order before one partial row per slot is written.
template <typename T, int V, int K>
__global__ void __launch_bounds__(256, V == 4 && K <= 4 ? 2 : 1) conv_bwd_kernel(ConvArgs a, int slots) {
    __shared__ float red[8][K + 1][32 * V];
    const int lane = threadIdx.x & 31, wy = threadIdx.x >> 5;
    const int c = (blockIdx.x * 32 + lane) * V, slot = blockIdx.y;
    const bool on = c < a.C;
    float w[K][V], bias[V], aw[K][V], ab[V];
    if (on) conv_taps<V, K>(a.w, c, w);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        bias[i] = on && a.bias ? a.bias[c + i] : 0.f;
        ab[i] = 0.f;
#pragma unroll
        for (int j = 0; j < K; ++j) aw[j][i] = 0.f;
    }
    constexpr int U = 4;  // tokens in flight
    const long long nruns = (long long)a.runs * a.B;
    for (long long q = (long long)slot * 8 + wy; on && q < nruns; q += (long long)slots * 8) {
        const int r = (int)(q % a.runs), b = (int)(q / a.runs);
        const int t0 = r * a.run, t1 = min(a.T, t0 + a.run);
        float xw[K][V], dz[K][V];  // inputs t-K+1 .. t and dz of tokens t-K+1 .. t
#pragma unroll
        for (int j = 0; j < K; ++j) {
            if (j < K - 1) conv_input<T, V, K>(a, b, t0 - (K - 1) + j, c, xw[j + 1]);
#pragma unroll
            for (int i = 0; i < V; ++i) dz[j][i] = 0.f;
        }
        // dx of token s = t - (K-1); the run emits its own tokens, run 0 the carried window's too
        const int first = r == 0 ? -(K - 1) : t0;
        const T *px = static_cast<const T *>(a.x) + (size_t)b * a.T * a.ldx + c;
        const T *pg = static_cast<const T *>(a.dy) + (size_t)b * a.T * a.C + c;
        for (int tb = t0; tb < t1 + K - 1; tb += U) {
            float x[U][V], g[U][V];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (tb + u < min(a.T, t1 + K - 1)) {
                    ConvVec<T, V>::ld(px + (size_t)(tb + u) * a.ldx, x[u]);
                    ConvVec<T, V>::ld(pg + (size_t)(tb + u) * a.C, g[u]);
                } else {  // dz is 0 past the end
#pragma unroll
                    for (int i = 0; i < V; ++i) x[u][i] = g[u][i] = 0.f;
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int t = tb + u, s = t - (K - 1);
#pragma unroll
                for (int j = 0; j + 1 < K; ++j)
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        xw[j][i] = xw[j + 1][i];
                        dz[j][i] = dz[j + 1][i];
                    }
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    xw[K - 1][i] = x[u][i];
                    float d = g[u][i];
                    if (a.silu) {
                        float z = bias[i];
#pragma unroll
                        for (int j = 0; j < K; ++j) z = fmaf(w[j][i], xw[j][i], z);
                        const float sg = conv_sigmoid(z);
                        d *= sg * fmaf(z, 1.f - sg, 1.f);
                    }
                    dz[K - 1][i] = d;
                }
                if (t < t1) {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        ab[i] += dz[K - 1][i];
#pragma unroll
                        for (int j = 0; j < K; ++j) aw[j][i] = fmaf(dz[K - 1][i], xw[j][i], aw[j][i]);
                    }
                }
                if (s < first || s >= t1) continue;
                float dx[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    dx[i] = 0.f;
#pragma unroll
                    for (int j = 0; j < K; ++j) dx[i] = fmaf(w[j][i], dz[K - 1 - j][i], dx[i]);
                }
                if (K > 1 && a.dstate_out && s >= a.T - (K - 1)) {
                    float e[V];
                    ConvVec<T, V>::ld(static_cast<const T *>(a.dstate_out) + ((size_t)b * (K - 1) + (s - a.T + K - 1)) * a.C + c,
                                      e);
#pragma unroll
                    for (int i = 0; i < V; ++i) dx[i] += e[i];
                }
                if (s >= 0)
                    ConvVec<T, V>::st(static_cast<T *>(a.dx) + ((size_t)b * a.T + s) * a.C + c, dx);
                else if (a.dstate_in)
                    ConvVec<T, V>::st(static_cast<T *>(a.dstate_in) + ((size_t)b * (K - 1) + (K - 1 + s)) * a.C + c, dx);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < K; ++j) red[wy][j][lane * V + i] = aw[j][i];
        red[wy][K][lane * V + i] = ab[i];
    }
    __syncthreads();
    for (int k = threadIdx.x; k < (K + 1) * 32 * V; k += 256) {
        const int j = k / (32 * V), i = k % (32 * V), ch = blockIdx.x * 32 * V + i;
        if (ch >= a.C) continue;
        float s = 0.f;
        for (int y = 0; y < 8; ++y) s += red[y][j][i];
        a.part[((size_t)slot * (K + 1) + j) * a.C + ch] = s;
    }
}

// dw[c][j] and dbias[c]: the slots' partial sums in order, in 64 bits.
__global__ void __launch_bounds__(256) conv_sum_kernel(int slots, int K, int C, const float *__restrict__ part,
                                                       float *__restrict__ dw, float *__restrict__ dbias) {
    __shared__ double red[8][32];
    const int lane = threadIdx.x & 31, wy = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane, j = blockIdx.y;
    double s = 0.0;
    if (c < C)
        for (int k = wy; k < slots; k += 8) s += (double)part[((size_t)k * (K + 1) + j) * C + c];
    red[wy][lane] = s;
    __syncthreads();
    if (wy == 0 && c < C) {
        for (int y = 1; y < 8; ++y) s += red[y][lane];
        if (j < K)
            dw[(size_t)c * K + j] = (float)s;
        else if (dbias)
            dbias[c] = (float)s;
    }
}

// ---- host side ------------------------------------------------------------------------------
// Slots of the backward: the blocks (32 V channels x 8 runs) that fit the SMs at once, two each; bounded by the runs.
inline int conv_bwd_slots(int B, int T, int C, int V, int run) {
    const long long runs = (long long)((T + run - 1) / run) * B;
    const long long cols = (C + 32 * V - 1) / (32 * V);
    long long s = (148 * 2) / cols;
    const long long most = (runs + 7) / 8;
    if (s > most) s = most;
    return (int)(s < 1 ? 1 : s);
}

template <typename T, int V, int K>
cudaError_t conv_fwd_launch(ConvArgs a, cudaStream_t s) {
    a.run = 32;
    a.runs = (a.T + a.run - 1) / a.run;
    const long long threads = (long long)(a.C / V) * a.runs * a.B;
    conv_fwd_kernel<T, V, K><<<(unsigned)((threads + 255) / 256), 256, 0, s>>>(a);
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return cudaGetLastError();
}
constexpr int kConvBwdRun = 32;
template <typename T, int V, int K>
cudaError_t conv_bwd_launch(ConvArgs a, float *dw, float *dbias, cudaStream_t s) {
    a.run = kConvBwdRun;
    a.runs = (a.T + a.run - 1) / a.run;
    const int slots = conv_bwd_slots(a.B, a.T, a.C, V, a.run);
    conv_bwd_kernel<T, V, K><<<dim3((a.C + 32 * V - 1) / (32 * V), slots), 256, 0, s>>>(a, slots);
    conv_sum_kernel<<<dim3((a.C + 31) / 32, K + 1), 256, 0, s>>>(slots, K, a.C, a.part, dw, dbias);
    g_launches.fetch_add(2, std::memory_order_relaxed);
    return cudaGetLastError();
}

template <typename T, int V>
cudaError_t conv_fwd_width(int K, const ConvArgs &a, cudaStream_t s) {
    switch (K) {
        case 1: return conv_fwd_launch<T, V, 1>(a, s);
        case 2: return conv_fwd_launch<T, V, 2>(a, s);
        case 3: return conv_fwd_launch<T, V, 3>(a, s);
        case 4: return conv_fwd_launch<T, V, 4>(a, s);
        case 5: return conv_fwd_launch<T, V, 5>(a, s);
        case 6: return conv_fwd_launch<T, V, 6>(a, s);
        case 7: return conv_fwd_launch<T, V, 7>(a, s);
        default: return conv_fwd_launch<T, V, 8>(a, s);
    }
}
template <typename T, int V>
cudaError_t conv_bwd_width(int K, const ConvArgs &a, float *dw, float *dbias, cudaStream_t s) {
    switch (K) {
        case 1: return conv_bwd_launch<T, V, 1>(a, dw, dbias, s);
        case 2: return conv_bwd_launch<T, V, 2>(a, dw, dbias, s);
        case 3: return conv_bwd_launch<T, V, 3>(a, dw, dbias, s);
        case 4: return conv_bwd_launch<T, V, 4>(a, dw, dbias, s);
        case 5: return conv_bwd_launch<T, V, 5>(a, dw, dbias, s);
        case 6: return conv_bwd_launch<T, V, 6>(a, dw, dbias, s);
        case 7: return conv_bwd_launch<T, V, 7>(a, dw, dbias, s);
        default: return conv_bwd_launch<T, V, 8>(a, dw, dbias, s);
    }
}

}  // namespace gdr

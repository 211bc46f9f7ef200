// conv.cuh -- the short causal convolution (gdr_conv_fwd, gdr_conv_bwd):
// depthwise over C channels, width K <= 8, optional bias and SiLU, the last
// K-1 inputs carried between calls (a decode token is T = 1):
//     z[t,c] = bias[c] + sum_{j<K} w[c,j] x[t-K+1+j, c],   y = z sigmoid(z) or z
// HBM-bound by its bytes: x is read and y written once.  A thread owns V = 4
// neighbouring channels (8 bytes of bf16: with 8 its windows leave one block a
// SM) and walks a run of tokens with the last K-1 inputs in registers, so that
// only the K-1 inputs before a run are read a second time, from L2.  B=4 T=4096
// C=2304 K=4 bf16, calls back to back (as all times here unless they say cold):
// forward 35 us (4.3 TB/s; 14 warp instructions an element, two
// of them exponential and reciprocal: half of all issue slots and 55 % of that
// unit's at 24 warps a SM, for which 36 bytes a thread spill, 84 of fp32),
// backward 57 us (4.0 TB/s; 12 warps a SM, since its
// two windows, the taps and their sums take 165 registers: held to 128 it spilled
// and lost 4 us, held to 96 it took 151 us).
#pragma once
#include "launch.cuh"

namespace gdr {

constexpr int kShortConvMax = 8;
constexpr int kConvMax = 0x7fffffff - 1024;  // of T and C: token counters run past T by a run and the groups read ahead,
                                              // channels past C by a warp's

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

// V elements as they are stored: a read that is not converted does not wait.
template <typename T, int V> struct RowRaw {
    T e[V];
};
template <> struct RowRaw<__nv_bfloat16, 8> {
    uint4 e;
};
template <> struct RowRaw<__nv_bfloat16, 4> {
    uint2 e;
};
template <> struct RowRaw<float, 4> {
    float4 e;
};
template <typename T, int V>
__device__ __forceinline__ void raw_values(const RowRaw<T, V> &r, float *v) {
    ConvVec<T, V>::ld(reinterpret_cast<const T *>(&r), v);
}
template <typename T, int V>
__device__ __forceinline__ RowRaw<T, V> raw_load(const T *p) {
    return *reinterpret_cast<const RowRaw<T, V> *>(p);
}

// The same as pairs of fp32 (V = 1: the second of the pair is 0), for the packed arithmetic of common.cuh.
template <int V> struct Pairs {
    static constexpr int N = V > 1 ? V / 2 : 1;
    float2 p[N];
};
template <typename T, int V>
__device__ __forceinline__ Pairs<V> raw_pairs(const RowRaw<T, V> &r) {
    float v[V];
    raw_values<T, V>(r, v);
    Pairs<V> o;
#pragma unroll
    for (int i = 0; i < Pairs<V>::N; ++i) o.p[i] = make_float2(v[V > 1 ? 2 * i : 0], V > 1 ? v[V > 1 ? 2 * i + 1 : 0] : 0.f);
    return o;
}
template <typename T, int V>
__device__ __forceinline__ void pairs_store(T *p, const Pairs<V> &o) {
    float v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = (i & 1) ? o.p[i / 2].y : o.p[i / 2].x;
    ConvVec<T, V>::st(p, v);
}

// Input token t (may be negative: the carried window, zero without one).
template <typename T, int V, int K>
__device__ __forceinline__ RowRaw<T, V> conv_input(const ConvArgs &a, int b, int t, int c) {
    if (t >= 0) return raw_load<T, V>(static_cast<const T *>(a.x) + ((size_t)b * a.T + t) * a.ldx + c);
    if (a.state_in) return raw_load<T, V>(static_cast<const T *>(a.state_in) + ((size_t)b * (K - 1) + (K - 1 + t)) * a.C + c);
    return RowRaw<T, V>{};
}

// The taps of V channels, w[j] of tap j.  Their V K floats are contiguous and start on 16 bytes where V K is a
// multiple of 4; read one by one they cost more than the tokens of a short run (B=4 T=4096 C=2304 K=4, runs of 16
// tokens of 8 channels: 154 us, against 70 us as vectors with runs of 32).
template <int V, int K>
__device__ __forceinline__ void conv_taps(const float *w, int c, Pairs<V> (&t)[K]) {
    float f[V * K];
    const float *p = w + (size_t)c * K;
    if (V * K % 4 == 0 && V % 2 == 0) {
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
    for (int i = 0; i < Pairs<V>::N; ++i)
#pragma unroll
        for (int j = 0; j < K; ++j) t[j].p[i] = make_float2(f[(V > 1 ? 2 * i : 0) * K + j], V > 1 ? f[(V > 1 ? 2 * i + 1 : 0) * K + j] : 0.f);
}
template <int V>
__device__ __forceinline__ Pairs<V> conv_bias(const float *bias, int c) {
    Pairs<V> o;
#pragma unroll
    for (int i = 0; i < Pairs<V>::N; ++i)
        o.p[i] = bias ? make_float2(bias[c + (V > 1 ? 2 * i : 0)], V > 1 ? bias[c + (V > 1 ? 2 * i + 1 : 0)] : 0.f) : make_float2(0.f, 0.f);
    return o;
}

// 1 / (1 + e^-z) of a pair: 0 where the exponential overflows, 1 where it vanishes.
__device__ __forceinline__ float2 conv_sigmoid2(float2 z) {
    const float2 one = make_float2(1.f, 1.f), e = fmul2(z, make_float2(-kLog2e, -kLog2e));
    const float2 d = ffma2(make_float2(ex2_ftz(e.x), ex2_ftz(e.y)), one, one);
    return make_float2(rcp_ftz(d.x), rcp_ftz(d.y));
}

// Reading ahead.  A warp works on 32 V channels (V = 4: 256 bytes of bf16, 512 of fp32) of one run of tokens; rows come
// in groups of U tokens through a ring of GR groups in shared memory by 16-byte asynchronous copies
// (they need rows that start on 16 bytes), so that the bytes in flight do not cost registers: with the same reads
// held in registers the forward took 53 us and the backward 106 us at B=4 T=4096 C=2304.  V = 1 is the form for rows
// without that alignment: each lane reads its own channel.
// The backward takes smaller groups: their values are in registers beside two windows.
constexpr int kConvFwdU = 8, kConvFwdGroups = 3, kConvBwdU = 4, kConvBwdGroups = 4;

template <typename T, int V, int U, int GROUPS>
struct ConvRing {
    static constexpr int kRow = 32 * V * (int)sizeof(T);        // bytes of a warp's row
    static constexpr int kBytes = GROUPS * U * kRow;  // of one tensor
};

// A lane's part of the copies of one tensor: L lanes a row, so 32 / L rows at once.
template <typename T, int V, int U>
struct ConvStage {
    static constexpr int kRow = ConvRing<T, V, U, 1>::kRow, L = kRow / 16 > 0 ? kRow / 16 : 1, S = 32 / L, E = 16 / (int)sizeof(T);
    const T *src;  // this lane's next source
    size_t step;   // S rows
    uint8_t *dst;  // this lane's place in group 0
    bool on;
    // base: channel c0 of the run's first token; `cols` channels exist from there on
    __device__ __forceinline__ void start(uint8_t *ring, const T *base, size_t ld, int cols) {
        const int lane = threadIdx.x & 31, row = lane / L, col = (lane % L) * E;
        src = base + row * ld + col;
        step = S * ld;
        dst = ring + row * kRow + (lane % L) * 16;
        on = col < cols;
    }
    // the group's U tokens, `left` of which exist, into place `at`
    __device__ __forceinline__ void group(int at, int left) {
        uint8_t *d = dst + at * U * kRow;
        const int row = (threadIdx.x & 31) / L;
#pragma unroll
        for (int u = 0; u < U; u += S) {
            if (on && u + row < left) cp_async16(d + u * kRow, src);
            src += step;
        }
    }
};

// Forward: a warp is 32 V channels of one run.
template <typename T, int V, int K>
__global__ void __launch_bounds__(256, K <= 4 ? 3 : 1) conv_fwd_kernel(ConvArgs a) {
    constexpr int NP = Pairs<V>::N, U = kConvFwdU, GR = kConvFwdGroups;
    using Ring = ConvRing<T, V, U, GR>;
    constexpr bool kStaged = V == 4;
    extern __shared__ __align__(16) uint8_t conv_smem[];
    const int lane = threadIdx.x & 31;
    const int CW = (a.C + 32 * V - 1) / (32 * V);
    const long long id = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (id >= (long long)CW * a.runs * a.B) return;
    const int c0 = (int)(id % CW) * 32 * V, c = c0 + lane * V;
    const bool on = c < a.C;
    const long long br = id / CW;
    const int r = (int)(br % a.runs), b = (int)(br / a.runs);
    const int t0 = r * a.run, t1 = min(a.T, t0 + a.run);
    const T *xb = static_cast<const T *>(a.x) + (size_t)b * a.T * a.ldx + c0;
    uint8_t *ring = conv_smem + (threadIdx.x >> 5) * Ring::kBytes;
    ConvStage<T, V, U> stage;
    stage.start(ring, xb + (size_t)t0 * a.ldx, a.ldx, a.C - c0);
    RowRaw<T, V> next[U];  // V = 1: the next group in registers
    auto fetch = [&](int at, int t) {
        if (kStaged) {
            stage.group(at, t1 - t);
            cp_async_commit();
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (on && t + u < t1) next[u] = raw_load<T, V>(xb + (size_t)(t + u) * a.ldx + lane * V);
        }
    };
#pragma unroll
    for (int grp = 0; grp < (kStaged ? GR - 1 : 1); ++grp) fetch(grp, t0 + grp * U);
    Pairs<V> w[K], win[K], bias;  // inputs t-K+1 .. t
    if (on) {
        conv_taps<V, K>(a.w, c, w);
        bias = conv_bias<V>(a.bias, c);
#pragma unroll
        for (int j = 0; j < K - 1; ++j) win[j + 1] = raw_pairs<T, V>(conv_input<T, V, K>(a, b, t0 - (K - 1) + j, c));
    }
    T *py = static_cast<T *>(a.y) + ((size_t)b * a.T + t0) * a.C + c;
    const bool silu = a.silu;
    auto token = [&](const RowRaw<T, V> &x) {
#pragma unroll
        for (int j = 0; j + 1 < K; ++j) win[j] = win[j + 1];
        win[K - 1] = raw_pairs<T, V>(x);
        Pairs<V> z = bias;
#pragma unroll
        for (int j = 0; j < K; ++j)
#pragma unroll
            for (int i = 0; i < NP; ++i) z.p[i] = ffma2(w[j].p[i], win[j].p[i], z.p[i]);
        if (silu)
#pragma unroll
            for (int i = 0; i < NP; ++i) z.p[i] = fmul2(z.p[i], conv_sigmoid2(z.p[i]));
        pairs_store<T, V>(py, z);
        py += a.C;
    };
    int at = 0, to = GR - 1;
    for (int t = t0; t < t1; t += U) {
        RowRaw<T, V> now[U];
        if (kStaged) {
            cp_async_wait<GR - 2>();
            __syncwarp();
            fetch(to, t + (GR - 1) * U);  // into the place of the group before, which every lane has read
            const uint8_t *p = ring + at * U * Ring::kRow + lane * V * sizeof(T);
#pragma unroll
            for (int u = 0; u < U; ++u) now[u] = *reinterpret_cast<const RowRaw<T, V> *>(p + u * Ring::kRow);
            to = at;
            at = at + 1 == GR ? 0 : at + 1;
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) now[u] = next[u];
            fetch(0, t + U);
        }
        if (!on) continue;
        if (t + U <= t1) {
#pragma unroll
            for (int u = 0; u < U; ++u) token(now[u]);
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (t + u < t1) token(now[u]);
        }
    }
    if (kStaged) cp_async_wait<0>();
    // The window after the last token, written by the thread of run 0: no other run reads state_in
    // (a run has at least K-1 tokens), so state_out may be the same buffer.
    if (K > 1 && r == 0 && on && a.state_out) {
        RowRaw<T, V> v[K];
#pragma unroll
        for (int j = 0; j < K - 1; ++j) v[j] = conv_input<T, V, K>(a, b, a.T - (K - 1) + j, c);
#pragma unroll
        for (int j = 0; j < K - 1; ++j)
            *reinterpret_cast<RowRaw<T, V> *>(static_cast<T *>(a.state_out) + ((size_t)b * (K - 1) + j) * a.C + c) = v[j];
    }
}

// Backward.  dz_t = dy_t silu'(z_t); dx_s = sum_j w_j dz_{s+K-1-j}; dw_j = sum_t dz_t x_{t-K+1+j}.
// A block is 32 channel groups x 4 runs; each of the 4 walks its runs (a slot's runs are slots*4 apart) and the
// four tap sums are joined in shared memory in a fixed order before one partial row per slot is written.  A run's
// first K-1 tokens emit no dx of their own run, and K-1 tokens past its end only finish it; the tokens between
// take no checks (with them everywhere the kernel ran 85 instructions an element and 135 us at B=4 T=4096 C=2304).
constexpr int kConvBwdWarps = 4;
template <typename T, int V, int K>
__global__ void __launch_bounds__(kConvBwdWarps * 32, K <= 4 ? 3 : 2) conv_bwd_kernel(ConvArgs a, int slots) {
    constexpr int NP = Pairs<V>::N, U = kConvBwdU, GR = kConvBwdGroups;
    using Ring = ConvRing<T, V, U, GR>;
    constexpr bool kStaged = V == 4;
    extern __shared__ __align__(16) uint8_t conv_smem[];
    float(*red)[K + 1][32 * V] = reinterpret_cast<float(*)[K + 1][32 * V]>(conv_smem);  // over the rings, at the end
    const int lane = threadIdx.x & 31, wy = threadIdx.x >> 5;
    uint8_t *ring = conv_smem + wy * 2 * Ring::kBytes;
    const int c0 = blockIdx.x * 32 * V, c = c0 + lane * V, slot = blockIdx.y;
    const bool on = c < a.C, silu = a.silu;
    const float2 zero = make_float2(0.f, 0.f), one = make_float2(1.f, 1.f), mone = make_float2(-1.f, -1.f);
    Pairs<V> w[K], bias, aw[K], ab;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        ab.p[i] = zero;
#pragma unroll
        for (int j = 0; j < K; ++j) aw[j].p[i] = zero;
    }
    if (on) {
        conv_taps<V, K>(a.w, c, w);
        bias = conv_bias<V>(a.bias, c);
    }
    const long long nruns = (long long)a.runs * a.B;
    for (long long q = (long long)slot * kConvBwdWarps + wy; q < nruns; q += (long long)slots * kConvBwdWarps) {
        const int r = (int)(q % a.runs), b = (int)(q / a.runs);
        const int t0 = r * a.run, t1 = min(a.T, t0 + a.run), tend = t1 + K - 1;
        T *pd = static_cast<T *>(a.dx) + ((size_t)b * a.T + t0) * a.C + c;  // dx of the run's next token
        RowRaw<T, V> nx[U], ng[U];  // V = 1: the next tokens
        const int tl = min(a.T, tend);
        const T *xb = static_cast<const T *>(a.x) + (size_t)b * a.T * a.ldx + c0;
        const T *gb = static_cast<const T *>(a.dy) + (size_t)b * a.T * a.C + c0;
        ConvStage<T, V, U> stage_x, stage_g;
        stage_x.start(ring, xb + (size_t)t0 * a.ldx, a.ldx, a.C - c0);
        stage_g.start(ring + Ring::kBytes, gb + (size_t)t0 * a.C, a.C, a.C - c0);
        auto fetch = [&](int at, int tb) {
            if (kStaged) {
                stage_x.group(at, tl - tb);
                stage_g.group(at, tl - tb);
                cp_async_commit();
            } else {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    nx[u] = ng[u] = RowRaw<T, V>{};
                    if (on && tb + u < tl) {
                        nx[u] = raw_load<T, V>(xb + (size_t)(tb + u) * a.ldx + lane * V);
                        ng[u] = raw_load<T, V>(gb + (size_t)(tb + u) * a.C + lane * V);
                    }
                }
            }
        };
        __syncwarp();  // every lane has read the last run's groups
#pragma unroll
        for (int grp = 0; grp < (kStaged ? GR - 1 : 1); ++grp) fetch(grp, t0 + grp * U);
        Pairs<V> xw[K], dz[K];  // inputs t-K+1 .. t and dz of tokens t-K+1 .. t
#pragma unroll
        for (int j = 0; j < K; ++j) {
            if (on && j < K - 1) xw[j + 1] = raw_pairs<T, V>(conv_input<T, V, K>(a, b, t0 - (K - 1) + j, c));
#pragma unroll
            for (int i = 0; i < NP; ++i) dz[j].p[i] = zero;
        }
        // token t enters the windows; its tap sums if it is the run's own
        auto enter = [&](const RowRaw<T, V> &rx, const RowRaw<T, V> &rg, bool mine) {
#pragma unroll
            for (int j = 0; j + 1 < K; ++j) {
                xw[j] = xw[j + 1];
                dz[j] = dz[j + 1];
            }
            xw[K - 1] = raw_pairs<T, V>(rx);
            Pairs<V> d = raw_pairs<T, V>(rg);
            if (silu)
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    float2 z = bias.p[i];
#pragma unroll
                    for (int j = 0; j < K; ++j) z = ffma2(w[j].p[i], xw[j].p[i], z);
                    const float2 sg = conv_sigmoid2(z);
                    d.p[i] = fmul2(d.p[i], fmul2(sg, ffma2(z, ffma2(sg, mone, one), one)));
                }
            dz[K - 1] = d;
            if (mine)
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    ab.p[i] = ffma2(d.p[i], one, ab.p[i]);
#pragma unroll
                    for (int j = 0; j < K; ++j) aw[j].p[i] = ffma2(d.p[i], xw[j].p[i], aw[j].p[i]);
                }
        };
        auto gradient = [&] {  // dx of token t - (K-1)
            Pairs<V> o;
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                o.p[i] = fmul2(w[0].p[i], dz[K - 1].p[i]);
#pragma unroll
                for (int j = 1; j < K; ++j) o.p[i] = ffma2(w[j].p[i], dz[K - 1 - j].p[i], o.p[i]);
            }
            return o;
        };
        int at = 0, to = GR - 1;
        for (int tb = t0; tb < tend; tb += U) {
            RowRaw<T, V> cx[U], cg[U];
            if (kStaged) {
                cp_async_wait<GR - 2>();
                __syncwarp();
                fetch(to, tb + (GR - 1) * U);
                const uint8_t *p = ring + at * U * Ring::kRow + lane * V * sizeof(T);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    cx[u] = cg[u] = RowRaw<T, V>{};  // dz is 0 past the end
                    if (tb + u < tl) {
                        cx[u] = *reinterpret_cast<const RowRaw<T, V> *>(p + u * Ring::kRow);
                        cg[u] = *reinterpret_cast<const RowRaw<T, V> *>(p + u * Ring::kRow + Ring::kBytes);
                    }
                }
                to = at;
                at = at + 1 == GR ? 0 : at + 1;
            } else {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    cx[u] = nx[u];
                    cg[u] = ng[u];
                }
                fetch(0, tb + U);
            }
            if (!on) continue;
            if (tb >= t0 + K - 1 && tb + U <= t1) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    enter(cx[u], cg[u], true);
                    pairs_store<T, V>(pd, gradient());
                    pd += a.C;
                }
                continue;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int t = tb + u, s = t - (K - 1);
                enter(cx[u], cg[u], t < t1);
                if (s >= t1 || (s < t0 && r > 0)) continue;
                Pairs<V> o = gradient();
                if (K > 1 && a.dstate_out && s >= a.T - (K - 1)) {
                    const Pairs<V> e = raw_pairs<T, V>(raw_load<T, V>(
                        static_cast<const T *>(a.dstate_out) + ((size_t)b * (K - 1) + (s - a.T + K - 1)) * a.C + c));
#pragma unroll
                    for (int i = 0; i < NP; ++i) o.p[i] = ffma2(e.p[i], one, o.p[i]);
                }
                if (s >= t0) {
                    pairs_store<T, V>(pd, o);
                    pd += a.C;
                } else if (a.dstate_in) {  // run 0: the carried window
                    pairs_store<T, V>(static_cast<T *>(a.dstate_in) + ((size_t)b * (K - 1) + (K - 1 + s)) * a.C + c, o);
                }
            }
        }
    }
    if (kStaged) cp_async_wait<0>();
    __syncthreads();
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < K; ++j) red[wy][j][lane * V + i] = (i & 1) ? aw[j].p[i / 2].y : aw[j].p[i / 2].x;
        red[wy][K][lane * V + i] = (i & 1) ? ab.p[i / 2].y : ab.p[i / 2].x;
    }
    __syncthreads();
    for (int k = threadIdx.x; k < (K + 1) * 32 * V; k += kConvBwdWarps * 32) {
        const int j = k / (32 * V), i = k % (32 * V), ch = blockIdx.x * 32 * V + i;
        if (ch >= a.C) continue;
        float s = 0.f;
        for (int y = 0; y < kConvBwdWarps; ++y) s += red[y][j][i];
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
// Tokens per run of the forward: of 8, 16, .. 160 the one whose rounds of blocks (`fit` of them at once) come to the
// fewest tokens, 8 more a run for its taps and window.  fp32 up to K = 4 is nearer to HBM and takes at most 40.  C=2304, us
// of the chosen run (others): bf16 K=4 B=4 T=512 8.6 (16; 64: 12.7), T=4096 34.9 (88; 16: 39.2, 64: 34.7, 104: 39.0), T=4400
// 37.0 (96; 64: 39.2, 128: 44.7), T=6000 45.4 (128; 32: 49.5, 160: 53.6), T=65536 at B=1 107 (112; 32: 117, 160: 115); K=7
// T=4400 49.5 (144; 32: 78, 64: 64); fp32 K=4 T=4096 54.7 (32; 16: 57.7, 64: 58.5, 128: 62).  Over 36 such sizes the choice
// costs 1 % more than the best of all.
inline int conv_fwd_run(int B, int T, int C, int K, int V, bool f32, int fit) {
    const long long cols = (C + 32 * V - 1) / (32 * V);
    const int most = f32 && K <= 4 ? 40 : 160;
    long long best = -1;
    int at = 8;
    for (int run = 8; run <= most && run < T + 8; run += 8) {
        const long long blocks = (cols * ((T + run - 1) / run) * B + 7) / 8;
        const long long cost = (blocks + fit - 1) / fit * ((run < T ? run : T) + 8);
        if (best < 0 || cost < best) {
            best = cost;
            at = run;
        }
    }
    return at;
}
// The backward is one launch that fits (slots x columns, three blocks an SM up to K = 4); a warp's runs are as long as
// their number stays the same for every warp and no run passes 192 tokens.  C=2304 K=4 bf16: B=4 T=4096 58 us (172;
// 64, 2.7 runs a warp: 66, 192: 62), T=6000 82 us (128; 64: 86, 172: 88), T=65536 at B=1 194 us (64: 215), T=512 19 us (20; 32:
// 17, 64: 19, 128: 27).
struct ConvPlan {
    int run, slots;
};
inline ConvPlan conv_bwd_plan(int B, int T, int C, int K, int V) {
    const long long cols = (C + 32 * V - 1) / (32 * V), fit = sm_count() * (K <= 4 ? 3 : 2) / cols, room = fit < 1 ? 1 : fit;
    const long long warps = room * kConvBwdWarps, need = (T + 191) / 192;
    const long long trips = (B * need + warps - 1) / warps;
    const long long runs = warps * trips / B;  // per sequence, at least `need`
    const long long run = ((T + runs - 1) / runs + 3) / 4 * 4;
    ConvPlan p;
    p.run = run < 16 ? 16 : (int)run;
    const long long most = ((long long)((T + p.run - 1) / p.run) * B + kConvBwdWarps - 1) / kConvBwdWarps;
    p.slots = (int)(most < room ? most : room);
    return p;
}

template <typename T, int V, int K>
cudaError_t conv_fwd_launch(ConvArgs a, cudaStream_t s) {
    constexpr size_t smem = V == 4 ? (size_t)8 * ConvRing<T, V, kConvFwdU, kConvFwdGroups>::kBytes : 0;
    int fit = 0;
    cudaError_t e = prepare_kernel(reinterpret_cast<const void *>(conv_fwd_kernel<T, V, K>), smem, 256, &fit);
    if (e != cudaSuccess) return e;
    a.run = conv_fwd_run(a.B, a.T, a.C, K, V, sizeof(T) == 4, fit > 0 ? fit : 1);
    a.runs = (a.T + a.run - 1) / a.run;
    const long long warps = (long long)((a.C + 32 * V - 1) / (32 * V)) * a.runs * a.B;
    conv_fwd_kernel<T, V, K><<<(unsigned)((warps + 7) / 8), 256, smem, s>>>(a);
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return cudaGetLastError();
}
template <typename T, int V, int K>
cudaError_t conv_bwd_launch(ConvArgs a, float *dw, float *dbias, cudaStream_t s) {
    const ConvPlan plan = conv_bwd_plan(a.B, a.T, a.C, K, V);
    const int slots = plan.slots;
    a.run = plan.run;
    a.runs = (a.T + a.run - 1) / a.run;
    constexpr size_t rings = V == 4 ? (size_t)2 * kConvBwdWarps * ConvRing<T, V, kConvBwdU, kConvBwdGroups>::kBytes : 0;
    constexpr size_t red = (size_t)kConvBwdWarps * (K + 1) * 32 * V * 4, smem = rings > red ? rings : red;
    cudaError_t e = prepare_kernel(reinterpret_cast<const void *>(conv_bwd_kernel<T, V, K>), smem);
    if (e != cudaSuccess) return e;
    conv_bwd_kernel<T, V, K><<<dim3((a.C + 32 * V - 1) / (32 * V), slots), kConvBwdWarps * 32, smem, s>>>(a, slots);
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

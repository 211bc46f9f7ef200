// layernorm.cuh -- layer norm over the last axis, with the residual stream
// (gdr_layernorm_fwd, gdr_layernorm_bwd):
//     h = x + residual (rounded to the stream's type: it is what is normalised)
//     y = (h - mean) / sqrt(var + eps) * w + b
//     dx = rstd (g - mean(g) - n mean(g n)) + dres,   g = dy w,  n = (h - mean) rstd
//     dw = sum_rows dy n,   db = sum_rows dy
// HBM-bound: every row is read once into registers (raw, as stored) and both
// statistics are taken from there, the variance from centred values.  TPR
// threads share a row and hold NV vectors of V elements each.  16384 x 2048
// bf16 with the residual stream, calls back to back: forward 47 us (5.7 TB/s), backward 68 us (3.9
// TB/s: rows at 16 warps a SM, bound by their exchanges and half of all issue
// slots, and 4 us for the sum of the blocks' partial rows).
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

// Sums of NS (1, 2, 4 or 8) values over the TPR threads of a row.  A warp halves the values and the lanes that hold
// them together (NS = 8: 4 + 2 + 1 + 2 exchanges, not 40).  `buf` has two sides of (NT/32) NS floats that calls take
// in turn, so that one barrier a call is enough (a side is written again only after the next call's barrier).
template <int TPR, int NT, int NS>
__device__ __forceinline__ void norm_reduce(float (&s)[NS], float *buf) {
    constexpr int LG = NS == 1 ? 0 : NS == 2 ? 1 : NS == 4 ? 2 : 3;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int l = 0; l < LG; ++l) {
        const int half = NS >> (l + 1), off = 16 >> l;
        const bool up = lane & off;
#pragma unroll
        for (int k = 0; k < half; ++k) {
            const float send = up ? s[k] : s[k + half], keep = up ? s[k + half] : s[k];
            s[k] = keep + __shfl_xor_sync(0xffffffffu, send, off);
        }
    }
#pragma unroll
    for (int off = 16 >> LG; off; off >>= 1) s[0] += __shfl_xor_sync(0xffffffffu, s[0], off);
    if (TPR == 32) {
        const float mine = s[0];
#pragma unroll
        for (int k = 0; k < NS; ++k) s[k] = __shfl_sync(0xffffffffu, mine, k << (5 - LG));
    } else {
        const int warp = threadIdx.x >> 5;
        constexpr int W = TPR > 32 ? TPR / 32 : 1;
        if ((lane & ((32 >> LG) - 1)) == 0) buf[warp * NS + (lane >> (5 - LG))] = s[0];
        __syncthreads();
        const int w0 = warp / W * W;
        if (W <= 4) {
#pragma unroll
            for (int k = 0; k < NS; ++k) {
                s[k] = 0.f;
#pragma unroll
                for (int i = 0; i < W; ++i) s[k] += buf[(w0 + i) * NS + k];
            }
        } else {  // W NS reads and sums would cost more than the row's own arithmetic: 32 / NS lanes share a value's
            constexpr int L = 32 / NS < W ? 32 / NS : W;
            const int k = NS == 1 ? 0 : lane / L;
            float v = 0.f;
#pragma unroll
            for (int i = 0; i < W; i += L) v += buf[(w0 + i + lane % L) * NS + k];
#pragma unroll
            for (int off = L / 2; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
#pragma unroll
            for (int j = 0; j < NS; ++j) s[j] = NS == 1 ? v : __shfl_sync(0xffffffffu, v, j * L);
        }
    }
}

// The backward's row over two to four warps takes one barrier: each warp centres its values on its own mean, and the sums
// are then moved to the row's (sum (h - m)^2 = sum (h - m_w)^2 + n_w (m_w - m)^2).  At 16384 x 2048 bf16 and cold caches 77 us, 84 with a
// barrier for the mean and one for the sums; over 8 and 16 warps every thread's joining of them costs more than the
// barrier (16384 x 4096: 152 us against 135), and so does the forward's.
__device__ __forceinline__ float norm_warp_sum(float x) {
#pragma unroll
    for (int off = 16; off; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}
// Three sums over a warp, halving the values and the lanes that hold them together.  Lane l has the sum l / 8 (lanes from
// 24 on: 0).
__device__ __forceinline__ float norm_warp_sums(const float (&s)[4]) {
    const int lane = threadIdx.x & 31;
    const bool up = lane & 16, odd = lane & 8;
    const float a = (up ? s[2] : s[0]) + __shfl_xor_sync(0xffffffffu, up ? s[0] : s[2], 16);
    const float b = (up ? 0.f : s[1]) + __shfl_xor_sync(0xffffffffu, up ? s[1] : 0.f, 16);
    float v = (odd ? b : a) + __shfl_xor_sync(0xffffffffu, odd ? a : b, 8);
#pragma unroll
    for (int off = 4; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}
// Columns of the row that its warp w holds.
template <int V, int TPR, int NV>
__device__ __forceinline__ float norm_warp_count(int w, int D) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) n += min(max(D - (i * TPR + w * 32) * V, 0), 32 * V);
    return (float)n;
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
    RowRaw<T, V> rx[NV], rr[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + tr) * V;
        if (live && c < a.D) rx[i] = raw_load<T, V>(static_cast<const T *>(a.x) + base + c);
    }
    if (a.res)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPR + tr) * V;
            if (live && c < a.D) rr[i] = raw_load<T, V>(static_cast<const T *>(a.res) + base + c);
        }
    float v[NV][V];
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + tr) * V;
#pragma unroll
        for (int e = 0; e < V; ++e) v[i][e] = 0.f;
        if (!live || c >= a.D) continue;
        raw_values<T, V>(rx[i], v[i]);
        if (a.res) {
            float r[V];
            raw_values<T, V>(rr[i], r);
#pragma unroll
            for (int e = 0; e < V; ++e) v[i][e] = to_f32(from_f32<T>(v[i][e] + r[e]));
            ConvVec<T, V>::st(static_cast<T *>(a.h) + base + c, v[i]);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) s[0] += v[i][e];
    }
    norm_reduce<TPR, NT, 1>(s, buf);
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
    norm_reduce<TPR, NT, 1>(s, buf + NT / 32);
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

// The backward reads rows ahead into shared memory, every thread its own 16-byte vectors (so that no barrier is
// needed): kDepth rows of three tensors.  Without vectors (V = 1) the next row waits in registers.
template <int V, int NV, int NT>
struct NormRing {
    static constexpr int kDepth = V == 1 ? 0 : NV * NT <= 256 ? 4 : NV * NT <= 1024 ? 3 : NV * NT <= 2048 ? 2 : 1;
    static constexpr size_t kBytes = (size_t)kDepth * 3 * NV * NT * 16;
};

// One block walks rows blockIdx.x * (NT/TPR) + rl, + gridDim.x * (NT/TPR), ...  Every thread keeps its columns' dw and
// db, and the block's row slots are joined in order at the end.
// The arithmetic is on packed pairs: as scalars it took 59 instructions an element.  16384 x 2048 bf16 with dres:
// 125 us as scalars.  A row stays in registers between its passes: read again from the ring, with the weights in shared
// memory and 20 or 24 warps an SM rather than 16, it took 83 us with cold caches (77 as it is).
template <typename T, int V, int TPR, int NV, int NT>
__global__ void __launch_bounds__(NT, V > 1 && V * NV <= 16 ? 512 / NT : 1) norm_bwd_kernel(NormArgs a) {
    constexpr int NP = Pairs<V>::N;
    constexpr int W = TPR / 32;
    constexpr bool kOne = W > 1 && W <= 4;  // one barrier a row
    __shared__ float4 sums[kOne ? 2 * (NT / 32) : 1];  // rows take the two sides in turn
    __shared__ float counts[W];
    __shared__ float buf[(NT / 32) * (1 + 4)];
    extern __shared__ __align__(16) float join[];  // the ring; at the end [NT/TPR][2][D] when NT > TPR
    uint4 *ring = reinterpret_cast<uint4 *>(join) + threadIdx.x;
    using Ring = NormRing<V, NV, NT>;
    const int rl = threadIdx.x / TPR, tr = threadIdx.x % TPR;
    const float2 zero = make_float2(0.f, 0.f), one = make_float2(1.f, 1.f);
    Pairs<V> w[NV], aw[NV], ab[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + tr) * V;
        float v[V];
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = 0.f;
        if (c < a.D) norm_weights<V>(a.w, c, v);
#pragma unroll
        for (int e = 0; e < NP; ++e) {
            aw[i].p[e] = ab[i].p[e] = zero;
            w[i].p[e] = make_float2(v[V > 1 ? 2 * e : 0], V > 1 ? v[V > 1 ? 2 * e + 1 : 0] : 0.f);
        }
    }
    const float inv = 1.f / (float)a.D;
    float inv_own = inv;
    if (kOne) {
        const float n = norm_warp_count<V, TPR, NV>(tr >> 5, a.D);
        inv_own = n > 0.f ? 1.f / n : 0.f;
        if (threadIdx.x < W) counts[threadIdx.x] = norm_warp_count<V, TPR, NV>(threadIdx.x, a.D);  // read after a row's barrier
    }
    const long long per = (long long)gridDim.x * (NT / TPR);
    const long long trips = (a.R + per - 1) / per;  // the same for every thread: the row sums use block barriers
    RowRaw<T, V> rh[NV], rg[NV], rd[NV];
    long long row = (long long)blockIdx.x * (NT / TPR) + rl;
    auto fetch = [&](long long at, const void *src, RowRaw<T, V> (&dst)[NV]) {  // V = 1: the next row in registers
        if (at >= a.R) return;
        const T *p = static_cast<const T *>(src) + (size_t)at * a.D + tr * V;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if ((i * TPR + tr) * V < a.D) dst[i] = raw_load<T, V>(p + i * TPR * V);
    };
    auto stage = [&](long long at, int place) {  // a row's vectors into the thread's own places of the ring
        if (at < a.R) {
            const size_t o = (size_t)at * a.D + tr * V;
            uint4 *d = ring + place * 3 * NV * NT;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if ((i * TPR + tr) * V >= a.D) continue;
                cp_async16(d + i * NT, static_cast<const T *>(a.x) + o + i * TPR * V);
                cp_async16(d + (NV + i) * NT, static_cast<const T *>(a.dy) + o + i * TPR * V);
                if (a.dres) cp_async16(d + (2 * NV + i) * NT, static_cast<const T *>(a.dres) + o + i * TPR * V);
            }
        }
        cp_async_commit();
    };
    int place = 0;
    if (Ring::kDepth > 0) {
#pragma unroll
        for (int j = 0; j < Ring::kDepth - 1; ++j) stage(row + j * per, j);
    } else {
        fetch(row, a.x, rh);
        fetch(row, a.dy, rg);
        if (a.dres) fetch(row, a.dres, rd);
    }
    for (long long k = 0; k < trips; ++k, row += per) {
        const bool live = row < a.R;
        Pairs<V> h[NV], g[NV];
        float2 s1 = zero;
        const uint4 *at = ring + place * 3 * NV * NT;
        if (Ring::kDepth > 0) {
            int to = place + Ring::kDepth - 1;
            if (to >= Ring::kDepth) to -= Ring::kDepth;
            stage(row + (Ring::kDepth - 1) * per, to);  // this thread has read what was there
            cp_async_wait<Ring::kDepth - 1>();
            if (++place == Ring::kDepth) place = 0;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                rh[i] = *reinterpret_cast<const RowRaw<T, V> *>(at + i * NT);
                rg[i] = *reinterpret_cast<const RowRaw<T, V> *>(at + (NV + i) * NT);
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!live || (i * TPR + tr) * V >= a.D) {
#pragma unroll
                for (int e = 0; e < NP; ++e) h[i].p[e] = g[i].p[e] = zero;
                continue;
            }
            h[i] = raw_pairs<T, V>(rh[i]);
            g[i] = raw_pairs<T, V>(rg[i]);
#pragma unroll
            for (int e = 0; e < NP; ++e) s1 = ffma2(h[i].p[e], one, s1);
        }
        if (Ring::kDepth == 0 && k + 1 < trips) {
            fetch(row + per, a.x, rh);
            fetch(row + per, a.dy, rg);
        }
        float m[1] = {s1.x + s1.y};
        if (kOne)
            m[0] = norm_warp_sum(m[0]);
        else
            norm_reduce<TPR, NT, 1>(m, buf);
        const float2 mean = make_float2(-m[0] * inv_own, V > 1 ? -m[0] * inv_own : 0.f);
        float2 ss = zero, sg = zero, sh = zero;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if ((i * TPR + tr) * V >= a.D) continue;
#pragma unroll
            for (int e = 0; e < NP; ++e) {
                h[i].p[e] = ffma2(h[i].p[e], one, mean);
                const float2 gw = fmul2(g[i].p[e], w[i].p[e]);
                ss = ffma2(h[i].p[e], h[i].p[e], ss);
                sg = ffma2(gw, one, sg);
                sh = ffma2(gw, h[i].p[e], sh);
            }
        }
        float s[4] = {ss.x + ss.y, sg.x + sg.y, sh.x + sh.y, 0.f};
        float shift = 0.f;  // the mean that h is centred on, less the row's
        if (kOne) {
            const float sum = norm_warp_sums(s);
            const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w0 = warp / W * W;
            float4 *side = sums + (k & 1) * (NT / 32);
            // lanes 0, 8, 16 write the sums, lane 24 the warp's mean
            if (lane % 8 == 0) reinterpret_cast<float *>(&side[warp])[(lane / 8 + 1) & 3] = lane == 24 ? m[0] * inv_own : sum;
            __syncthreads();
            float row_mean = 0.f;
#pragma unroll
            for (int i = 0; i < W; ++i) row_mean = fmaf(side[w0 + i].x, counts[i], row_mean);
            row_mean *= inv;
            s[0] = s[1] = s[2] = 0.f;
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const float4 o = side[w0 + i];
                const float d = o.x - row_mean;
                s[0] += fmaf(d * d, counts[i], o.y);
                s[1] += o.z;
                s[2] += fmaf(d, o.z, o.w);
            }
            shift = m[0] * inv_own - row_mean;
        } else {
            norm_reduce<TPR, NT, 4>(s, buf + NT / 32);
        }
        if (live) {
            const float rstd = 1.f / sqrtf(s[0] * inv + a.eps);
            // dx = rstd g w - rstd mean(g w) - (h - mean) rstd^3 mean(g w (h - mean))
            const float b2 = -rstd * rstd * (rstd * s[2] * inv), b1 = fmaf(b2, shift, -rstd * s[1] * inv), sr = shift * rstd;
            const float2 r2 = make_float2(rstd, rstd), c1 = make_float2(b1, b1), c2 = make_float2(b2, b2), s2 = make_float2(sr, sr);
            T *p = static_cast<T *>(a.dx) + (size_t)row * a.D + tr * V;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if ((i * TPR + tr) * V >= a.D) continue;
                Pairs<V> dx;
                if (a.dres) dx = raw_pairs<T, V>(Ring::kDepth > 0 ? *reinterpret_cast<const RowRaw<T, V> *>(at + (2 * NV + i) * NT) : rd[i]);
#pragma unroll
                for (int e = 0; e < NP; ++e) {
                    float2 d = ffma2(fmul2(g[i].p[e], w[i].p[e]), r2, ffma2(h[i].p[e], c2, c1));
                    dx.p[e] = a.dres ? ffma2(d, one, dx.p[e]) : d;
                    aw[i].p[e] = ffma2(g[i].p[e], kOne ? ffma2(h[i].p[e], r2, s2) : fmul2(h[i].p[e], r2), aw[i].p[e]);
                    ab[i].p[e] = ffma2(g[i].p[e], one, ab[i].p[e]);
                }
                pairs_store<T, V>(p + i * TPR * V, dx);
            }
        }
        if (Ring::kDepth == 0 && a.dres && k + 1 < trips) fetch(row + per, a.dres, rd);
    }
    if (Ring::kDepth > 0) cp_async_wait<0>();
    if (NT > TPR) __syncthreads();  // the ring becomes the slots' sums
    float *out = a.part + (size_t)blockIdx.x * 2 * a.D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + tr) * V;
        if (c >= a.D) continue;
        float *dst = NT > TPR ? join + rl * 2 * a.D + c : out + c;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            dst[e] = (e & 1) ? aw[i].p[e / 2].y : aw[i].p[e / 2].x;
            dst[a.D + e] = (e & 1) ? ab[i].p[e / 2].y : ab[i].p[e / 2].x;
        }
    }
    if (NT > TPR) {
        __syncthreads();
        for (int c = threadIdx.x; c < 2 * a.D; c += NT) {
            float s = 0.f;
            for (int r = 0; r < NT / TPR; ++r) s += join[r * 2 * a.D + c];
            out[c] = s;
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
#pragma unroll 8
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
constexpr int kNormBwdMaxBlocks = 148 * 8;

// Calls F<V, TPR, NV, NT>: vectors of 16 bytes where D allows, else single elements.  The fewest threads per row
// that hold it in at most 16 elements a thread, a warp where that is enough: a thread's exchanges with the others are
// then spread over 16 elements, and the backward's five arrays of them still fit its registers (single elements are half
// a pair each, so 4 of them: 18304 x 1333 fp32 takes 194 us, and took 369 with 8, in blocks of 512 threads that spilled).
// Wider rows have more elements a thread than the backward's registers hold: vectors above 8192 columns spill 484 (bf16) and
// 644 bytes a thread (4096 x 16384 bf16: 199 us, 2.7 TB/s), single elements above 2048 columns 170 to 2400 (8192 x 3001 fp32:
// 235 us, 1.7 TB/s).
template <typename T, bool BWD, template <typename, int, int, int, int> class F, typename... A>
cudaError_t norm_pick(int D, A... args) {
    constexpr int V = sizeof(T) == 2 ? 8 : 4, M = 16, S = BWD ? 4 : 16;
    if (D % V == 0) {
        if (D <= 32 * V) return F<T, V, 32, 1, 256>::go(args...);
        if (D <= 32 * M) return F<T, V, 32, M / V, 256>::go(args...);
        if (D <= 128 * M) return F<T, V, 128, M / V, 128>::go(args...);
        if (D <= 256 * M) return F<T, V, 256, M / V, 256>::go(args...);
        if (D <= 512 * M) return F<T, V, 512, M / V, 512>::go(args...);
        return F<T, V, 512, kNormMaxD / (512 * V), 512>::go(args...);
    }
    if (D <= 32 * S) return F<T, 1, 32, S, 256>::go(args...);
    if (D <= 128 * S) return F<T, 1, 128, S, 128>::go(args...);
    if (D <= 256 * S) return F<T, 1, 256, S, 256>::go(args...);
    if (D <= 512 * S) return F<T, 1, 512, S, 512>::go(args...);
    if (D <= 512 * 8) return F<T, 1, 512, 8, 512>::go(args...);
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
        constexpr int per = NT / TPR;
        auto kernel = norm_bwd_kernel<T, V, TPR, NV, NT>;
        // the instance's largest D: a limit that followed this call's D could be lowered under another thread's launch
        constexpr size_t sums = NT > TPR ? (size_t)per * 2 * (TPR * NV * V) * 4 : 0, ring = NormRing<V, NV, NT>::kBytes;
        constexpr size_t smem = sums > ring ? sums : ring;
        int most = 0;  // one wave: a second one of a few blocks would cost as much as the first
        cudaError_t e = prepare_kernel(reinterpret_cast<const void *>(kernel), smem, NT, &most);
        if (e != cudaSuccess) return e;
        long long grid = (a.R + per - 1) / per;
        if (most > kNormBwdMaxBlocks) most = kNormBwdMaxBlocks;
        if (grid > most) grid = most;
        kernel<<<(unsigned)grid, NT, smem, s>>>(a);
        norm_sum_kernel<<<dim3((a.D + 31) / 32, db ? 2 : 1), 1024, 0, s>>>((int)grid, a.D, a.part, dw, db);
        g_launches.fetch_add(2, std::memory_order_relaxed);
        return cudaGetLastError();
    }
};

}  // namespace gdr

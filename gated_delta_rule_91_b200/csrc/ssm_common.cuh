// ssm_common.cuh -- the selective state space scan's arguments and per-chunk
// gates, shared by its kernels.
//
// Per (b, h), with z_t = delta_t + delta_bias_h, Delta_t = softplus(z_t) (or
// z_t itself) and a_t = exp(A_h Delta_t):
//     S_t = a_t S_{t-1} + Delta_t x_t B_t^T,   y_t = S_t C_t + D_h x_t
// (S: P x N fp32).  Over a chunk, with c_t = A sum_{s <= t} Delta_s (inclusive,
// from the chunk's first token):
//     y_i   = sum_{j <= i} e^{c_i - c_j} Delta_j (C_i . B_j) x_j + e^{c_i} S_in C_i + D x_i
//     S_out = e^{c_last} S_in + sum_j e^{c_last - c_j} Delta_j x_j B_j^T
// Only differences c_i - c_j with j <= i are exponentiated, so a decaying
// state (A < 0) never overflows; the sums c run over one chunk, in 64 bits,
// since a difference of long sums loses what is near the diagonal in 32.
#pragma once
#include "common.cuh"

namespace gdr {

struct SsmArgs {
    int B, T, H, G, P, N;
    const void *x, *Bm, *Cm;     // [B,T,H,P], [B,T,G,N]: token strides ldx, ldb, ldc
    int ldx, ldb, ldc;
    const float *delta;          // [B,T,H]
    const float *A, *D, *bias;   // [H]; D, bias may be null
    int softplus;
    const float *S0;             // [B,H,P,N] or null
    // backward
    const void *dy;              // [B,T,H,P]
    const float *dS_T;           // or null
    // outputs
    void *y;
    float *S_T;
    void *dx, *dB, *dC;
    float *ddelta, *dA, *dD, *dbias, *dS0;
};

__device__ __forceinline__ float ssm_softplus(float z) { return fmaxf(z, 0.f) + log1pf(expf(-fabsf(z))); }

// Delta_t of token t of (b, h); 0 past the end (an identity token).
__device__ __forceinline__ float ssm_step_size(const SsmArgs &a, int b, int t, int h) {
    if (t >= a.T) return 0.f;
    float z = a.delta[((size_t)b * a.T + t) * a.H + h];
    if (a.bias) z += a.bias[h];
    return a.softplus ? ssm_softplus(z) : z;
}

// One warp: Delta and the inclusive sums c of Q tokens from t0 into shared
// arrays; lane l owns tokens l*Q/32 ...
template <int Q>
__device__ __forceinline__ void ssm_gates(const SsmArgs &a, int b, int h, int t0, float *s_dt, double *s_c) {
    constexpr int E = Q / 32;
    const int lane = threadIdx.x & 31;
    const double Ah = (double)a.A[h];
    double c[E], run = 0.0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const float d = ssm_step_size(a, b, t0 + lane * E + e, h);
        s_dt[lane * E + e] = d;
        run += Ah * (double)d;
        c[e] = run;
    }
    double incl = run;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const double o = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += o;
    }
    const double before = incl - run;
#pragma unroll
    for (int e = 0; e < E; ++e) s_c[lane * E + e] = before + c[e];
}

}  // namespace gdr

// ssm_simt.cuh -- the selective scan and its gradients on CUDA cores in fp32
// (fp32 inputs; bf16 with GDR_SSM_KERNEL=simt, to cross-check the tensor-core
// kernels).  Chunks of 64 tokens, all chunks of all heads in parallel:
//   1. state  U_c = sum_j w_j x_j B_j^T per chunk, w_j = e^{c_last - c_j} Delta_j
//   2. scan   S_in(c+1) = e^{c_last} S_in(c) + U_c over the chunks, elementwise
//   3. output y from the chunk's products and S_in
// and for the gradients the same states, V_c = sum_i e^{c_i} dy_i C_i^T with
// the reverse scan G_out(c-1) = e^{c_last} G_out(c) + V_c, then every chunk's
// gradients from (S_in, G_out).  What bounds them is the fp32 FMA rate with
// operands from shared memory: a thread's 4 x 4..8 tile is read as vectors
// along both tile axes, so every product's operands are stored with the
// summed index outermost.  fp32 B=3 T=777 H=6 P=N=64: 42 us; gradients of B=2 T=333
// H=4 P=128 N=64: 72 us, 38 of them the chunks' gradients (latency: 48 to 234 blocks of one to three a SM).
#pragma once
#include "launch.cuh"
#include "ssm_common.cuh"

namespace gdr {

constexpr int kSsmQ = 64;          // tokens per chunk
constexpr int kSsmThreads = 256;   // 16 x 16
constexpr int kSsmLdQ = 68;        // row stride of [k][64] operands

// acc[r][c] += sum_k At[k][4 ty + r] * Bt[k][4 tx + (c & 3) + 64 (c >> 2)], k < K.
template <int NC>
__device__ __forceinline__ void ssm_mm(float (&acc)[4][NC], const float *At, int lda, const float *Bt, int ldb, int K,
                                       int ty, int tx) {
#pragma unroll 4
    for (int k = 0; k < K; ++k) {
        const float4 av = *reinterpret_cast<const float4 *>(At + k * lda + 4 * ty);
        const float a[4] = {av.x, av.y, av.z, av.w};
#pragma unroll
        for (int cb = 0; cb < NC / 4; ++cb) {
            const float4 bv = *reinterpret_cast<const float4 *>(Bt + k * ldb + 64 * cb + 4 * tx);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                acc[r][4 * cb] = fmaf(a[r], bv.x, acc[r][4 * cb]);
                acc[r][4 * cb + 1] = fmaf(a[r], bv.y, acc[r][4 * cb + 1]);
                acc[r][4 * cb + 2] = fmaf(a[r], bv.z, acc[r][4 * cb + 2]);
                acc[r][4 * cb + 3] = fmaf(a[r], bv.w, acc[r][4 * cb + 3]);
            }
        }
    }
}

// 64 tokens x W columns of a token-strided tensor -> dst[t][c] (row stride W + 4), rows past `valid` zero.
template <typename T, int W>
__device__ __forceinline__ void ssm_load_rows(float *dst, const T *src, size_t ld, int valid) {
    for (int i = threadIdx.x; i < kSsmQ * (W / 4); i += kSsmThreads) {
        const int t = i / (W / 4), c = (i % (W / 4)) * 4;
        const float4 v = t < valid ? load4(src + (size_t)t * ld + c) : make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4 *>(dst + t * (W + 4) + c) = v;
    }
}
// The same tile transposed: dst[c][t], row stride kSsmLdQ.
template <typename T, int W>
__device__ __forceinline__ void ssm_load_cols(float *dst, const T *src, size_t ld, int valid) {
    for (int i = threadIdx.x; i < kSsmQ * (W / 4); i += kSsmThreads) {
        const int t = i % kSsmQ, c = (i / kSsmQ) * 4;
        const float4 v = t < valid ? load4(src + (size_t)t * ld + c) : make_float4(0.f, 0.f, 0.f, 0.f);
        dst[c * kSsmLdQ + t] = v.x;
        dst[(c + 1) * kSsmLdQ + t] = v.y;
        dst[(c + 2) * kSsmLdQ + t] = v.z;
        dst[(c + 3) * kSsmLdQ + t] = v.w;
    }
}

// ---- 1. chunk states ------------------------------------------------------------------
// BWD: V_c = sum_i e^{c_i} dy_i C_i^T instead of U_c.  Writes out[b][chunk][h][p][n] and
// dec[b][chunk][h] = e^{c_last}.  Grid (chunks * P/64, H, B).
template <typename T, int P, int N, bool BWD>
__global__ void __launch_bounds__(kSsmThreads) ssm_state_simt_kernel(SsmArgs a, float *__restrict__ out,
                                                                     float *__restrict__ dec) {
    extern __shared__ float sm_f[];
    float *sx = sm_f;                    // [64 j][68]: 64 columns p
    float *sb = sx + kSsmQ * kSsmLdQ;    // [64 j][N + 4]
    __shared__ float s_dt[kSsmQ], s_w[kSsmQ];
    __shared__ double s_c[kSsmQ];
    const int nch = (a.T + kSsmQ - 1) / kSsmQ;
    const int ch = blockIdx.x / (P / 64), p0 = (blockIdx.x % (P / 64)) * 64, h = blockIdx.y, b = blockIdx.z;
    const int g = h / (a.H / a.G), t0 = ch * kSsmQ, valid = min(kSsmQ, a.T - t0);
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const size_t tok = (size_t)b * a.T + t0;
    if (tid < 32) ssm_gates<kSsmQ>(a, b, h, t0, s_dt, s_c);
    if (BWD)
        ssm_load_rows<T, 64>(sx, static_cast<const T *>(a.dy) + (tok * a.H + h) * P + p0, (size_t)a.H * P, valid);
    else
        ssm_load_rows<T, 64>(sx, static_cast<const T *>(a.x) + tok * a.ldx + (size_t)h * P + p0, a.ldx, valid);
    if (BWD)
        ssm_load_rows<T, N>(sb, static_cast<const T *>(a.Cm) + tok * a.ldc + (size_t)g * N, a.ldc, valid);
    else
        ssm_load_rows<T, N>(sb, static_cast<const T *>(a.Bm) + tok * a.ldb + (size_t)g * N, a.ldb, valid);
    __syncthreads();
    if (tid < kSsmQ)
        s_w[tid] = BWD ? expf((float)s_c[tid]) : s_dt[tid] * expf((float)(s_c[kSsmQ - 1] - s_c[tid]));
    __syncthreads();
    for (int i = tid; i < kSsmQ * 16; i += kSsmThreads) {
        float4 *v = reinterpret_cast<float4 *>(sx + (i >> 4) * kSsmLdQ + (i & 15) * 4);
        const float w = s_w[i >> 4];
        *v = make_float4(v->x * w, v->y * w, v->z * w, v->w * w);
    }
    __syncthreads();
    float acc[4][N / 16] = {};
    ssm_mm<N / 16>(acc, sx, kSsmLdQ, sb, N + 4, kSsmQ, ty, tx);
    const size_t unit = ((size_t)b * nch + ch) * a.H + h;
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int cb = 0; cb < N / 64; ++cb)
            *reinterpret_cast<float4 *>(out + (unit * P + p0 + 4 * ty + r) * N + 64 * cb + 4 * tx) =
                make_float4(acc[r][4 * cb], acc[r][4 * cb + 1], acc[r][4 * cb + 2], acc[r][4 * cb + 3]);
    if (!BWD && p0 == 0 && tid == 0) dec[unit] = expf((float)s_c[kSsmQ - 1]);
}

// ---- 2. scan over the chunks ------------------------------------------------------------
// st[b][c][h][...]: U_c in, the state entering chunk c out (REV: V_c in, the gradient of the
// state leaving chunk c out).  One thread per 4 state elements; `last` may be null.
constexpr int kScanBatch = 8;
template <bool REV>
__global__ void __launch_bounds__(256) ssm_scan_kernel(int nch, int H, int PN4, long long total, float *__restrict__ st,
                                                       const float *__restrict__ dec, const float *__restrict__ first,
                                                       float *__restrict__ last) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= total) return;
    const int e = (int)(i % PN4);
    const long long bh = i / PN4;
    const int h = (int)(bh % H);
    const long long b = bh / H;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (first) s = reinterpret_cast<const float4 *>(first)[i];
    float4 *p = reinterpret_cast<float4 *>(st) + ((b * nch * H + h) * PN4 + e);
    const float *d = dec + b * nch * H + h;
    const size_t step = (size_t)H * PN4;
    // The chain is only the FMA: a batch of chunks is read before the first of it is overwritten (13 chunks of 18 heads of
    // 64 x 64: 7 us, against 24 us with one chunk in flight).
    for (int k0 = 0; k0 < nch; k0 += kScanBatch) {
        float4 u[kScanBatch];
        float f[kScanBatch];
#pragma unroll
        for (int j = 0; j < kScanBatch; ++j) {
            const int c = REV ? nch - 1 - (k0 + j) : k0 + j;
            if (k0 + j < nch) {
                u[j] = p[c * step];
                f[j] = d[(size_t)c * H];
            }
        }
#pragma unroll
        for (int j = 0; j < kScanBatch; ++j) {
            const int c = REV ? nch - 1 - (k0 + j) : k0 + j;
            if (k0 + j < nch) {
                p[c * step] = s;
                s = make_float4(fmaf(f[j], s.x, u[j].x), fmaf(f[j], s.y, u[j].y), fmaf(f[j], s.z, u[j].z),
                                fmaf(f[j], s.w, u[j].w));
            }
        }
    }
    if (last) reinterpret_cast<float4 *>(last)[i] = s;
}

// ---- 3. outputs ----------------------------------------------------------------------------
template <int P, int N>
struct SsmYSmem {
    static constexpr int kOp = (P > N ? P : N) * kSsmLdQ;  // one operand, floats: [P or N][68] or [64][P or N + 4]
    static constexpr int kBytes = (3 * kOp + kSsmQ * kSsmLdQ) * 4;
};
template <typename T, int P, int N>
__global__ void __launch_bounds__(kSsmThreads) ssm_y_simt_kernel(SsmArgs a, const float *__restrict__ states) {
    using L = SsmYSmem<P, N>;
    extern __shared__ float sm_f[];
    float *sc = sm_f, *sb = sc + L::kOp, *sx = sb + L::kOp, *smt = sx + L::kOp;
    __shared__ float s_dt[kSsmQ];
    __shared__ double s_c[kSsmQ];
    const int nch = (a.T + kSsmQ - 1) / kSsmQ;
    const int ch = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
    const int g = h / (a.H / a.G), t0 = ch * kSsmQ, valid = min(kSsmQ, a.T - t0);
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const size_t tok = (size_t)b * a.T + t0;
    if (tid < 32) ssm_gates<kSsmQ>(a, b, h, t0, s_dt, s_c);
    ssm_load_cols<T, N>(sc, static_cast<const T *>(a.Cm) + tok * a.ldc + (size_t)g * N, a.ldc, valid);
    ssm_load_cols<T, N>(sb, static_cast<const T *>(a.Bm) + tok * a.ldb + (size_t)g * N, a.ldb, valid);
    ssm_load_rows<T, P>(sx, static_cast<const T *>(a.x) + tok * a.ldx + (size_t)h * P, a.ldx, valid);
    __syncthreads();
    {   // M^T[j][i] = e^{c_i - c_j} Delta_j C_i . B_j, i >= j
        float k4[4][4] = {};
        ssm_mm<4>(k4, sc, kSsmLdQ, sb, kSsmLdQ, N, ty, tx);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int j = 4 * tx + c;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = 4 * ty + r;
                smt[j * kSsmLdQ + i] = i >= j ? k4[r][c] * s_dt[j] * expf((float)(s_c[i] - s_c[j])) : 0.f;
            }
        }
    }
    __syncthreads();
    float acc[4][P / 16] = {};
    const size_t unit = ((size_t)b * nch + ch) * a.H + h;
#pragma unroll 1
    for (int half = 0; half < N / 64; ++half) {  // S^T of 64 state columns at a time: [n][p]
        ssm_load_cols<float, 64>(sb, states + unit * P * N + half * 64, N, 64);
        if (P == 128) ssm_load_cols<float, 64>(sb + 64 * kSsmLdQ, states + (unit * P + 64) * N + half * 64, N, 64);
        __syncthreads();
#pragma unroll
        for (int pb = 0; pb < P / 64; ++pb) {
            float part[4][4] = {};
            ssm_mm<4>(part, sc + half * 64 * kSsmLdQ, kSsmLdQ, sb + pb * 64 * kSsmLdQ, kSsmLdQ, 64, ty, tx);
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[r][4 * pb + c] += part[r][c];
        }
        __syncthreads();
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const float e = expf((float)s_c[4 * ty + r]);
#pragma unroll
        for (int c = 0; c < P / 16; ++c) acc[r][c] *= e;
    }
    ssm_mm<P / 16>(acc, smt, kSsmLdQ, sx, P + 4, kSsmQ, ty, tx);
    const float D = a.D ? a.D[h] : 0.f;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int i = 4 * ty + r;
        if (i >= valid) continue;
        T *dst = static_cast<T *>(a.y) + ((tok + i) * a.H + h) * P;
#pragma unroll
        for (int c = 0; c < P / 16; ++c) {
            const int p = 4 * tx + (c & 3) + 64 * (c >> 2);
            dst[p] = from_f32<T>(a.D ? fmaf(D, sx[i * (P + 4) + p], acc[r][c]) : acc[r][c]);
        }
    }
}

// ---- gradients of one chunk ------------------------------------------------------------------
// With K_ij = C_i.B_j, L_ij = e^{c_i - c_j} (j <= i), W_ij = dy_i.x_j, R_ij = L K W:
//     dx_j = Delta_j (sum_i L_ij K_ij dy_i + e^{c_last - c_j} G B_j) + D dy_j
//     dC_i = sum_j L_ij W_ij Delta_j B_j + e^{c_i} S_in^T dy_i          (summed over the group's heads)
//     dB_j = sum_i L_ij W_ij Delta_j C_i + Delta_j e^{c_last - c_j} G^T x_j
//     dDelta_j (as the write's weight) = sum_{i >= j} R_ij + e^{c_last - c_j} x_j.G B_j
//     d log a_t = sum_{i >= t > j} R_ij Delta_j + sum_{i >= t} e^{c_i} dy_i.S_in C_i
//                 + sum_{j < t} Delta_j e^{c_last - c_j} x_j.G B_j + e^{c_last} <G, S_in>
// The double sum of d log a_t is the difference of the prefix sums of the
// columns and rows of strict pairs, which starts at exactly 0.  Both are sums in
// 64 bits of the same R_ij (times Delta_j, exact there): in 32 bits they round
// apart, and the remainder stays in every later token's difference (dA was up to
// 5.5e-6 off, 2e-7 now).
// part[0..2][b*nch+ch][h]: this chunk's sums for dA, d(delta_bias), dD.
__device__ __forceinline__ void ssm_token_grads(const SsmArgs &a, int b, int h, int t0, int valid, int Q, const float *s_dt,
                                                const double *colU, const float *diag, const double *row, const float *gx,
                                                const float *sy, double cross, const float *dw_diag, double *part,
                                                size_t unit, size_t units) {
    // One warp; token arrays of Q (a multiple of 32): colU strict column sums of R (without Delta_j), diag R_jj,
    // row strict row sums of R Delta, gx = e^{c_last-c_j} x_j.G B_j, sy = e^{c_i} dy_i.S_in C_i, dw_diag = dy_i.x_i.
    const int lane = threadIdx.x & 31, E = Q / 32;
    const double Ah = (double)a.A[h];
    double pre = 0.0, suf = 0.0;
    for (int e = 0; e < E; ++e) {
        const int t = lane * E + e;
        pre += (double)s_dt[t] * (colU[t] + (double)gx[t]) - row[t];
        suf += (double)sy[t];
    }
    double p = pre, s = suf;
    for (int off = 1; off < 32; off <<= 1) {
        const double up = __shfl_up_sync(0xffffffffu, p, off), dn = __shfl_down_sync(0xffffffffu, s, off);
        if (lane >= off) p += up;
        if (lane + off < 32) s += dn;
    }
    double before = p - pre, after = s;  // sums of the tokens before this lane's; of this lane's tokens and on
    double sA = 0.0, sB = 0.0, sD = 0.0;
    for (int e = 0; e < E; ++e) {
        const int t = lane * E + e;
        const double dlog = before + after + cross;
        const double dd = colU[t] + (double)diag[t] + (double)gx[t] + Ah * dlog;
        before += (double)s_dt[t] * (colU[t] + (double)gx[t]) - row[t];
        after -= (double)sy[t];
        if (t < valid) {
            const size_t at = ((size_t)b * a.T + t0 + t) * a.H + h;
            double f = 1.0;
            if (a.softplus) {
                float z = a.delta[at];
                if (a.bias) z += a.bias[h];
                f = 1.0 / (1.0 + exp(-(double)z));
            }
            const double raw = dd * f;
            a.ddelta[at] = (float)raw;
            sA += (double)s_dt[t] * dlog;
            sB += raw;
            sD += (double)dw_diag[t];
        }
    }
    for (int off = 16; off; off >>= 1) {
        sA += __shfl_xor_sync(0xffffffffu, sA, off);
        sB += __shfl_xor_sync(0xffffffffu, sB, off);
        sD += __shfl_xor_sync(0xffffffffu, sD, off);
    }
    if (lane == 0) {
        part[unit] = sA;
        part[units + unit] = sB;
        part[2 * units + unit] = sD;
    }
}

template <int P, int N>
struct SsmGradSmem {
    static constexpr int kOp = (P > N ? P : N) * kSsmLdQ;
    static constexpr int kQQ = kSsmQ * kSsmLdQ;
    static constexpr int kBytes = (4 * kOp + 3 * kQQ) * 4;
};

// dBh, dCh: this head's gradients [B,T,H,N] fp32 (summed over each group by ssm_group_sum_kernel).  roles = 2: a chunk's
// dx is a block of its own beside the rest; where the chunks do not fill the SMs that is shorter (a chunk with P = 128,
// N = 64 takes 63 us as one block).
template <typename T, int P, int N>
__global__ void __launch_bounds__(kSsmThreads) ssm_grad_simt_kernel(SsmArgs a, int roles, const float *__restrict__ Sin,
                                                                    const float *__restrict__ Gout,
                                                                    float *__restrict__ dBh, float *__restrict__ dCh,
                                                                    double *__restrict__ part) {
    using L = SsmGradSmem<P, N>;
    extern __shared__ float sm_f[];
    float *s0 = sm_f, *sbt = s0 + L::kOp, *sxt = sbt + L::kOp, *syt = sxt + L::kOp;
    float *s_m = syt + L::kOp, *s_k = s_m + L::kQQ, *s_kt = s_k + L::kQQ;  // M'[i][j], dK[i][j], dK[j][i]
    __shared__ float s_dt[kSsmQ], s_diag[kSsmQ], s_gx[kSsmQ], s_sy[kSsmQ], s_wd[kSsmQ];
    __shared__ double s_part[16][kSsmQ], s_colU[kSsmQ], s_row[kSsmQ];
    __shared__ double s_c[kSsmQ], s_red[8];
    const int nch = (a.T + kSsmQ - 1) / kSsmQ;
    const int ch = blockIdx.x / roles, role = roles == 1 ? 2 : blockIdx.x % roles, h = blockIdx.y, b = blockIdx.z;
    const int g = h / (a.H / a.G), t0 = ch * kSsmQ, valid = min(kSsmQ, a.T - t0);
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const size_t tok = (size_t)b * a.T + t0;
    const size_t unit = ((size_t)b * nch + ch) * a.H + h, units = (size_t)a.B * nch * a.H;
    const T *xg = static_cast<const T *>(a.x) + tok * a.ldx + (size_t)h * P;
    const T *bg = static_cast<const T *>(a.Bm) + tok * a.ldb + (size_t)g * N;
    const T *cg = static_cast<const T *>(a.Cm) + tok * a.ldc + (size_t)g * N;
    const T *yg = static_cast<const T *>(a.dy) + (tok * a.H + h) * P;
    const size_t ldy = (size_t)a.H * P;
    const float *S = Sin + unit * P * N, *G = Gout + unit * P * N;

    if (tid < 32) ssm_gates<kSsmQ>(a, b, h, t0, s_dt, s_c);
    ssm_load_cols<T, N>(s0, cg, a.ldc, valid);
    ssm_load_cols<T, N>(sbt, bg, a.ldb, valid);
    ssm_load_cols<T, P>(sxt, xg, a.ldx, valid);
    ssm_load_cols<T, P>(syt, yg, ldy, valid);
    __syncthreads();
    {
        float k4[4][4] = {}, w4[4][4] = {};
        double col[4] = {}, row[4] = {};  // 64 bits: a pair's R Delta in its row's sum and in its column's cancels exactly
        ssm_mm<4>(k4, s0, kSsmLdQ, sbt, kSsmLdQ, N, ty, tx);
        ssm_mm<4>(w4, syt, kSsmLdQ, sxt, kSsmLdQ, P, ty, tx);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int j = 4 * tx + c;
            const float dj = s_dt[j];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = 4 * ty + r;
                const float l = i >= j ? expf((float)(s_c[i] - s_c[j])) : 0.f;
                const float m = l * k4[r][c], dk = l * w4[r][c] * dj, R = m * w4[r][c];
                s_m[i * kSsmLdQ + j] = m;
                s_k[i * kSsmLdQ + j] = dk;
                s_kt[j * kSsmLdQ + i] = dk;
                if (i > j) {
                    row[r] = fma((double)R, (double)dj, row[r]);
                    col[c] += (double)R;
                }
                if (i == j) {
                    s_diag[i] = R;
                    s_wd[i] = w4[r][c];
                }
            }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
#pragma unroll
            for (int off = 8; off; off >>= 1) row[r] += __shfl_xor_sync(0xffffffffu, row[r], off);
            if (tx == 0) s_row[4 * ty + r] = row[r];
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) s_part[ty][4 * tx + c] = col[c];
    }
    __syncthreads();
    if (tid < kSsmQ) {
        double s = 0.0;
        for (int k = 0; k < 16; ++k) s += s_part[k][tid];
        s_colU[tid] = s;
    }
    __syncthreads();  // M' and dK are read next, whichever part comes first
    const double clast = s_c[kSsmQ - 1];
    if (role != 1) {  // dC: e^{c_i} S^T dy_i, its product with C_i, then the chunk's own part
        float acc[4][N / 16] = {};
#pragma unroll 1
        for (int pb = 0; pb < P / 64; ++pb) {
            ssm_load_rows<float, N>(s0, S + (size_t)pb * 64 * N, N, 64);
            __syncthreads();
            ssm_mm<N / 16>(acc, syt + pb * 64 * kSsmLdQ, kSsmLdQ, s0, N + 4, 64, ty, tx);
            __syncthreads();
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = 4 * ty + r;
            const float e = expf((float)s_c[i]);
            float dot = 0.f;
#pragma unroll
            for (int c = 0; c < N / 16; ++c) {
                acc[r][c] *= e;
                if (i < valid) dot = fmaf(acc[r][c], to_f32(cg[(size_t)i * a.ldc + 4 * tx + (c & 3) + 64 * (c >> 2)]), dot);
            }
            dot = warp_sum(dot, 16);
            if (tx == 0) s_sy[i] = dot;
        }
        ssm_load_rows<T, N>(s0, bg, a.ldb, valid);
        __syncthreads();
        ssm_mm<N / 16>(acc, s_kt, kSsmLdQ, s0, N + 4, kSsmQ, ty, tx);
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (4 * ty + r < valid)
#pragma unroll
                for (int cb = 0; cb < N / 64; ++cb)
                    *reinterpret_cast<float4 *>(dCh + ((tok + 4 * ty + r) * a.H + h) * N + 64 * cb + 4 * tx) =
                        make_float4(acc[r][4 * cb], acc[r][4 * cb + 1], acc[r][4 * cb + 2], acc[r][4 * cb + 3]);
        __syncthreads();
    }
    if (role != 1) {  // dB
        float acc[4][N / 16] = {};
#pragma unroll 1
        for (int pb = 0; pb < P / 64; ++pb) {
            ssm_load_rows<float, N>(s0, G + (size_t)pb * 64 * N, N, 64);
            __syncthreads();
            ssm_mm<N / 16>(acc, sxt + pb * 64 * kSsmLdQ, kSsmLdQ, s0, N + 4, 64, ty, tx);
            __syncthreads();
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int j = 4 * ty + r;
            const float e = expf((float)(clast - s_c[j]));
            float dot = 0.f;
#pragma unroll
            for (int c = 0; c < N / 16; ++c) {
                acc[r][c] *= e;
                if (j < valid) dot = fmaf(acc[r][c], to_f32(bg[(size_t)j * a.ldb + 4 * tx + (c & 3) + 64 * (c >> 2)]), dot);
                acc[r][c] *= s_dt[j];
            }
            dot = warp_sum(dot, 16);
            if (tx == 0) s_gx[j] = dot;
        }
        ssm_load_rows<T, N>(s0, cg, a.ldc, valid);
        __syncthreads();
        ssm_mm<N / 16>(acc, s_k, kSsmLdQ, s0, N + 4, kSsmQ, ty, tx);
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (4 * ty + r < valid)
#pragma unroll
                for (int cb = 0; cb < N / 64; ++cb)
                    *reinterpret_cast<float4 *>(dBh + ((tok + 4 * ty + r) * a.H + h) * N + 64 * cb + 4 * tx) =
                        make_float4(acc[r][4 * cb], acc[r][4 * cb + 1], acc[r][4 * cb + 2], acc[r][4 * cb + 3]);
        __syncthreads();
    }
    if (role != 0) {  // dx
        float acc[4][P / 16] = {};
#pragma unroll 1
        for (int half = 0; half < N / 64; ++half) {
            ssm_load_cols<float, 64>(s0, G + half * 64, N, 64);
            if (P == 128) ssm_load_cols<float, 64>(s0 + 64 * kSsmLdQ, G + 64 * N + half * 64, N, 64);
            __syncthreads();
#pragma unroll
            for (int pb = 0; pb < P / 64; ++pb) {
                float q4[4][4] = {};
                ssm_mm<4>(q4, sbt + half * 64 * kSsmLdQ, kSsmLdQ, s0 + pb * 64 * kSsmLdQ, kSsmLdQ, 64, ty, tx);
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int c = 0; c < 4; ++c) acc[r][4 * pb + c] += q4[r][c];
            }
            __syncthreads();
        }
        ssm_load_rows<T, P>(s0, yg, ldy, valid);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float e = expf((float)(clast - s_c[4 * ty + r]));
#pragma unroll
            for (int c = 0; c < P / 16; ++c) acc[r][c] *= e;
        }
        __syncthreads();
        ssm_mm<P / 16>(acc, s_m, kSsmLdQ, s0, P + 4, kSsmQ, ty, tx);
        const float D = a.D ? a.D[h] : 0.f;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int j = 4 * ty + r;
            if (j >= valid) continue;
            T *dst = static_cast<T *>(a.dx) + ((tok + j) * a.H + h) * P;
#pragma unroll
            for (int c = 0; c < P / 16; ++c) {
                const int p = 4 * tx + (c & 3) + 64 * (c >> 2);
                float v = s_dt[j] * acc[r][c];
                if (a.D) v = fmaf(D, s0[j * (P + 4) + p], v);
                dst[p] = from_f32<T>(v);
            }
        }
    }
    if (role == 1) return;
    double dot = 0.0;  // e^{c_last} <G, S_in>
    for (int i = tid; i < P * N; i += kSsmThreads) dot += (double)S[i] * (double)G[i];
    for (int off = 16; off; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
    if ((tid & 31) == 0) s_red[tid >> 5] = dot;
    __syncthreads();
    if (tid < 32) {
        double cross = 0.0;
        for (int w = 0; w < 8; ++w) cross += s_red[w];
        ssm_token_grads(a, b, h, t0, valid, kSsmQ, s_dt, s_colU, s_diag, s_row, s_gx, s_sy, cross * exp(clast), s_wd, part,
                        unit, units);
    }
}

// dst[b,t,g,n] = sum over the group's heads of src[b,t,h,n], 4 columns a thread, heads in order.
template <typename T>
__global__ void __launch_bounds__(256) ssm_group_sum_kernel(long long total4, int heads, int N4, const float *__restrict__ sB,
                                                            const float *__restrict__ sC, T *__restrict__ dB,
                                                            T *__restrict__ dC) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= total4) return;
    const float *src = blockIdx.y ? sC : sB;
    T *dst = blockIdx.y ? dC : dB;
    const long long bg = i / N4;
    const int n = (int)(i % N4) * 4;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < heads; ++k) {
        const float4 v = load4(src + (bg * heads + k) * (N4 * 4LL) + n);
        s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
    }
    T *d = dst + bg * (N4 * 4LL) + n;
    d[0] = from_f32<T>(s.x);
    d[1] = from_f32<T>(s.y);
    d[2] = from_f32<T>(s.z);
    d[3] = from_f32<T>(s.w);
}

// dA, d(delta_bias), dD of head blockIdx.x: sums over (b, chunk) in 64 bits, in a fixed order.
__global__ void __launch_bounds__(256) ssm_head_sum_kernel(int n, int H, const double *__restrict__ part, float *dA,
                                                           float *dbias, float *dD) {
    __shared__ double red[3][8];
    const int h = blockIdx.x, tid = threadIdx.x;
    double s[3] = {0.0, 0.0, 0.0};
    for (int i = tid; i < n; i += 256)
        for (int k = 0; k < 3; ++k) s[k] += part[((size_t)k * n + i) * H + h];
    for (int k = 0; k < 3; ++k) {
        for (int off = 16; off; off >>= 1) s[k] += __shfl_xor_sync(0xffffffffu, s[k], off);
        if ((tid & 31) == 0) red[k][tid >> 5] = s[k];
    }
    __syncthreads();
    if (tid < 3) {
        double t = 0.0;
        for (int w = 0; w < 8; ++w) t += red[tid][w];
        float *dst = tid == 0 ? dA : tid == 1 ? dbias : dD;
        if (dst) dst[h] = (float)t;
    }
}

// ---- host side ---------------------------------------------------------------------------------
inline size_t ssm_align(size_t x) { return (x + 255) & ~(size_t)255; }

// Workspaces: chunk states and decays; the gradients' also holds V/G, the heads' dB and dC and the sums.
struct SsmSimtWs {
    size_t st, dec, g, dBh, dCh, part, fwd_total, bwd_total;
};
inline SsmSimtWs ssm_simt_ws(int B, int T, int H, int P, int N) {
    const size_t units = (size_t)B * ((T + kSsmQ - 1) / kSsmQ) * H;
    SsmSimtWs w;
    w.st = 0;
    w.dec = ssm_align(units * P * N * 4);
    w.fwd_total = w.g = w.dec + ssm_align(units * 4);
    w.dBh = w.g + ssm_align(units * P * N * 4);
    w.dCh = w.dBh + ssm_align((size_t)B * T * H * N * 4);
    w.part = w.dCh + ssm_align((size_t)B * T * H * N * 4);
    w.bwd_total = w.part + ssm_align(3 * units * 8);
    return w;
}

inline cudaError_t ssm_launch_scan(bool rev, int B, int nch, int H, int PN, float *st, const float *dec,
                                   const float *first, float *last, cudaStream_t s) {
    const long long total = (long long)B * H * (PN / 4);
    const unsigned grid = (unsigned)((total + 255) / 256);
    if (rev)
        ssm_scan_kernel<true><<<grid, 256, 0, s>>>(nch, H, PN / 4, total, st, dec, first, last);
    else
        ssm_scan_kernel<false><<<grid, 256, 0, s>>>(nch, H, PN / 4, total, st, dec, first, last);
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return cudaGetLastError();
}

template <typename K, typename... A>
cudaError_t ssm_launch(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t s, A... args) {
    cudaError_t e = prepare_kernel(reinterpret_cast<const void *>(kernel), smem);
    if (e != cudaSuccess) return e;
    kernel<<<grid, threads, smem, s>>>(args...);
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return cudaGetLastError();
}

template <typename T, int P, int N>
cudaError_t ssm_simt_fwd(const SsmArgs &a, void *ws, cudaStream_t s) {
    const SsmSimtWs w = ssm_simt_ws(a.B, a.T, a.H, P, N);
    const int nch = (a.T + kSsmQ - 1) / kSsmQ;
    float *st = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + w.st);
    float *dec = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + w.dec);
    const size_t sm = (size_t)kSsmQ * (kSsmLdQ + N + 4) * 4;
    cudaError_t e = ssm_launch(ssm_state_simt_kernel<T, P, N, false>, dim3(nch * (P / 64), a.H, a.B), kSsmThreads, sm, s, a,
                               st, dec);
    if (e == cudaSuccess) e = ssm_launch_scan(false, a.B, nch, a.H, P * N, st, dec, a.S0, a.S_T, s);
    if (e == cudaSuccess)
        e = ssm_launch(ssm_y_simt_kernel<T, P, N>, dim3(nch, a.H, a.B), kSsmThreads, (size_t)SsmYSmem<P, N>::kBytes, s, a,
                       (const float *)st);
    return e;
}

template <typename T, int P, int N>
cudaError_t ssm_simt_bwd(const SsmArgs &a, void *ws, cudaStream_t s) {
    const SsmSimtWs w = ssm_simt_ws(a.B, a.T, a.H, P, N);
    const int nch = (a.T + kSsmQ - 1) / kSsmQ;
    uint8_t *base = static_cast<uint8_t *>(ws);
    float *st = reinterpret_cast<float *>(base + w.st), *dec = reinterpret_cast<float *>(base + w.dec);
    float *g = reinterpret_cast<float *>(base + w.g);
    double *part = reinterpret_cast<double *>(base + w.part);
    float *dBh = reinterpret_cast<float *>(base + w.dBh), *dCh = reinterpret_cast<float *>(base + w.dCh);
    const size_t sm = (size_t)kSsmQ * (kSsmLdQ + N + 4) * 4;
    const dim3 grid(nch * (P / 64), a.H, a.B);
    cudaError_t e = ssm_launch(ssm_state_simt_kernel<T, P, N, false>, grid, kSsmThreads, sm, s, a, st, dec);
    if (e == cudaSuccess) e = ssm_launch(ssm_state_simt_kernel<T, P, N, true>, grid, kSsmThreads, sm, s, a, g, dec);
    if (e == cudaSuccess) e = ssm_launch_scan(false, a.B, nch, a.H, P * N, st, dec, a.S0, nullptr, s);
    if (e == cudaSuccess) e = ssm_launch_scan(true, a.B, nch, a.H, P * N, g, dec, a.dS_T, a.dS0, s);
    int dev = 0, sms = 0;
    if (e == cudaSuccess) e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int roles = 2LL * nch * a.H * a.B <= sms ? 2 : 1;
    if (e == cudaSuccess)
        e = ssm_launch(ssm_grad_simt_kernel<T, P, N>, dim3(nch * roles, a.H, a.B), kSsmThreads,
                       (size_t)SsmGradSmem<P, N>::kBytes, s, a, roles, (const float *)st, (const float *)g, dBh, dCh, part);
    if (e != cudaSuccess) return e;
    const long long total4 = (long long)a.B * a.T * a.G * (N / 4);
    ssm_group_sum_kernel<T><<<dim3((unsigned)((total4 + 255) / 256), 2), 256, 0, s>>>(
        total4, a.H / a.G, N / 4, dBh, dCh, static_cast<T *>(a.dB), static_cast<T *>(a.dC));
    ssm_head_sum_kernel<<<a.H, 256, 0, s>>>(a.B * nch, a.H, part, a.dA, a.dbias, a.dD);
    g_launches.fetch_add(2, std::memory_order_relaxed);
    return cudaGetLastError();
}

}  // namespace gdr

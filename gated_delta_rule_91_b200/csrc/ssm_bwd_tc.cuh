// ssm_bwd_tc.cuh -- the selective scan's gradients on the 5th-generation
// tensor cores, bf16 inputs, P, N in {64, 128}; formulas at the gradient kernel
// of ssm_simt.cuh.  Chunks of 128 tokens:
//   1. ssm_tc_state_kernel per chunk: U_c and V_c, every weighted row in two
//      bf16 parts
//   2. ssm_scan_kernel over the chunks, fp32: S_in(c), and in reverse G_out(c)
//   3. ssm_tc_grad_kernel: a CTA owns one chunk of one group and walks heads of
//      it, so that C B^T is formed once and dB, dC are summed over the heads in
//      TMEM.  Per head (W = dy x^T, L the decays, tokens on the TMEM lanes):
//        W   = dY X^T                              N = 128   K = P
//        dC += dK B,  dB += dK^T C                 N = N     K = 128    dK = L W Delta
//        dXi = M'^T dY                             N = P     K = 128    M' = L (C B^T)
//        T   = dY S_in  -> dC += e^{c_i} T,        dlog: e^{c_i} C_i . T_i
//        T   = X G_out  -> dB += w_j T,            dDelta: e^{c_last-c_j} B_j . T_j
//        T   = B G_out^T -> dx = Delta (dXi + e^{c_last-c_j} T) + D dy
//      (N = N, N, P and K = P, P, N).
// What leaves in fp32 (the gradients of delta, A, the bias and S0) is not
// touched by a bf16 rounding above 2^-17: the double sums of R = L K W are
// taken on CUDA cores from the fp32 accumulators, and S_in and G_out enter
// their products as two bf16 parts.  dx, dB and dC take bf16 operands.
#pragma once
#include "ssm_tc.cuh"

namespace gdr {

template <int P, int N>
struct SsmGradTc {
    static constexpr uint32_t XB = P / 64 * kTile, BB = N / 64 * kTile;
    static constexpr uint32_t kSBlock = P * 128, SB = N / 64 * kSBlock;  // a state part: P rows, blocks of 64 columns n
    static constexpr uint32_t oB = 0, oC = BB, oX = 2 * BB, oY = oX + XB, oR = oY + XB;
    static constexpr uint32_t oM = oR, oK = oR + 2 * kTile;   // M', dK
    static constexpr uint32_t oHi = oR, oLo = oR + SB;        // S_in, then G_out
    static constexpr uint32_t oGate = oR + 4 * kTile;
    // doubles c[2][128], red[2][8]; floats dt[2][128], e, row, el, hi, lo [128], col[288]; per head, two sets:
    // rowp[2][128], colp[4][128], diag, wd, gxp[2][128], syp[2][128] and four joined arrays of 128
    static constexpr uint32_t kSet = (2 + 4 + 1 + 1 + 2 + 2) * 128;
    static constexpr uint32_t kGate = (256 + 16) * 8 + (256 + 5 * 128 + 288 + 2 * kSet + 4 * 128) * 4;
    static constexpr uint32_t oBar = oGate + kGate;
    static constexpr uint32_t kAlloc = oBar + 64 + 1024;
};

// Column sums of a 32 x 32 block held as v[column] per lane (row): v[0] ends as the sum of column `lane`.
__device__ __forceinline__ void ssm_column_sums(float *v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) {
        const bool up = lane & s;
#pragma unroll
        for (int k = 0; k < s; ++k) {
            const float send = up ? v[k] : v[k + s], keep = up ? v[k + s] : v[k];
            v[k] = keep + __shfl_xor_sync(0xffffffffu, send, s);
        }
    }
}

constexpr int kGradThreads = 288;  // 8 warps of tokens, and one for the gates and the per-token sums

template <int P, int N>
__global__ void __launch_bounds__(kGradThreads, 1) ssm_tc_grad_kernel(
    const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_b,
    const __grid_constant__ CUtensorMap tm_c, const __grid_constant__ CUtensorMap tm_dy,
    const __grid_constant__ CUtensorMap tm_dx, SsmArgs a, int splits, int per, const float *__restrict__ Sin,
    const float *__restrict__ Gout, float *__restrict__ dBp, float *__restrict__ dCp, float *__restrict__ part) {
    using L = SsmGradTc<P, N>;
    using namespace sm100;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const uint32_t sb = smem_u32(sm);
    double *s_c2 = reinterpret_cast<double *>(sm + L::oGate), *s_red2 = s_c2 + 256;
    float *s_dt2 = reinterpret_cast<float *>(s_red2 + 16);
    float *s_e = s_dt2 + 256, *s_rowf = s_e + 128, *s_el = s_rowf + 128, *s_hi = s_el + 128, *s_lo = s_hi + 128;
    float *s_col = s_lo + 128, *s_set = s_col + 288, *s_join = s_set + 2 * L::kSet;
    uint64_t *bar_bc = reinterpret_cast<uint64_t *>(sm + L::oBar), *bar_x = bar_bc + 1, *bar_y = bar_bc + 2,
             *mma_bar = bar_bc + 3;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bar_bc + 4);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int q = warp & 3, half = (warp >> 2) & 1, row = q * 32 + lane;
    const bool worker = warp < 8;  // one lane of a TMEM quarter and half of the columns each
    const int nch = (a.T + kTcQ - 1) / kTcQ, HG = a.H / a.G;
    int u = blockIdx.x;
    const int sp = u % splits;
    u /= splits;
    const int g = u % a.G;
    u /= a.G;
    const int ch = u % nch, b = u / nch;
    const int h0 = g * HG + sp * per, nh = min(per, HG - sp * per);
    const int t0 = ch * kTcQ, valid = min(kTcQ, a.T - t0);

    if (tid == 0) {
        mbar_init(bar_bc, 1);
        mbar_init(bar_x, 1);
        mbar_init(bar_y, 1);
        mbar_init(mma_bar, 1);
        fence_mbar_init();
        *abort_flag = 0;
    }
    if (warp == 0) tmem_alloc(tmem_slot, 512);
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    const uint32_t tmem = *tmem_slot;
    const uint32_t tl = tmem + ((uint32_t)(q * 32) << 16);
    constexpr uint32_t tK = 0, tT = 128, tC = 256, tB = 256 + N;

    int n_x = 0, n_y = 0, d_x = 0, d_y = 0;
    bool bc_open = false, mma_open = false;
    auto issue_x = [&](int h) {
        mbar_expect_tx(bar_x, L::XB);
        for (int i = 0; i < P / 64; ++i) tma_load_4d(sm + L::oX + i * kTile, &tm_x, bar_x, i * 64, h, t0, b);
        ++n_x;
    };
    auto issue_y = [&](int h) {
        mbar_expect_tx(bar_y, L::XB);
        for (int i = 0; i < P / 64; ++i) tma_load_4d(sm + L::oY + i * kTile, &tm_dy, bar_y, i * 64, h, t0, b);
        ++n_y;
    };
    if (tid == 0) {
        mbar_expect_tx(bar_bc, 2 * L::BB);
        for (int i = 0; i < N / 64; ++i) {
            tma_load_4d(sm + L::oB + i * kTile, &tm_b, bar_bc, i * 64, g, t0, b);
            tma_load_4d(sm + L::oC + i * kTile, &tm_c, bar_bc, i * 64, g, t0, b);
        }
        bc_open = true;
        issue_x(h0);
        issue_y(h0);
    }
    if (warp == 8) ssm_tc_gates(a, b, h0, t0, s_dt2, s_c2);
    __syncthreads();

    auto worker_sync = [] { asm volatile("bar.sync 1, 256;" ::: "memory"); };
    uint32_t mma_phase = 0;
    auto mma_sync_point = [&]() {
        if (tid == 0) {
            mma_commit(mma_bar);
            mma_open = !mbar_wait(mma_bar, mma_phase);
            if (mma_open) *abort_flag = 1;
        }
        mma_phase ^= 1;
        worker_sync();
        tc_after_sync();
    };
    const size_t units = (size_t)a.B * nch * a.H;
    // 8 columns of row p = 0 .. P-1 of a state: chunk i of this thread
    constexpr int kChunks = P * N / 8 / 256;
    auto chunk_p = [&](int i) { return (i * 256 + tid) / (N / 8); };
    auto chunk_n = [&](int i) { return (i * 256 + tid) % (N / 8); };
    auto chunk_off = [&](int i) {
        const int p = chunk_p(i), n8 = chunk_n(i);
        return (uint32_t)(n8 >> 3) * L::kSBlock + sw128_offset(p, n8 & 7);
    };
    auto load_state = [&](const float *src, float (&v)[kChunks][8]) {
#pragma unroll
        for (int i = 0; i < kChunks; ++i) load8(src + (size_t)(i * 256 + tid) * 8, v[i]);
    };

    // Warps 0-7 walk the heads (barrier 1 among themselves); warp 8 prepares the next head's gates and finishes the
    // last head's per-token sums beside them.  All meet once a head, at barrier 0.
    auto token_sums = [&](int hh) {
        const int set = hh & 1;
        const float *s_rowp = s_set + set * L::kSet, *s_colp = s_rowp + 256, *s_diag = s_colp + 512, *s_wd = s_diag + 128,
                    *s_gxp = s_wd + 128, *s_syp = s_gxp + 256;
        for (int t = lane; t < 128; t += 32) {
            s_join[t] = s_colp[t] + s_colp[128 + t] + s_colp[256 + t] + s_colp[384 + t];
            s_join[128 + t] = s_rowp[t] + s_rowp[128 + t];
            s_join[256 + t] = s_gxp[t] + s_gxp[128 + t];
            s_join[384 + t] = s_syp[t] + s_syp[128 + t];
        }
        __syncwarp();
        double cross = 0.0;
        for (int w = 0; w < 8; ++w) cross += s_red2[set * 8 + w];
        ssm_token_grads(a, b, h0 + hh, t0, valid, kTcQ, s_dt2 + set * 128, s_join, s_diag, s_join + 128, s_join + 256,
                        s_join + 384, cross * exp2(s_c2[set * 128 + 127]), s_wd, part,
                        ((size_t)b * nch + ch) * a.H + h0 + hh, units);
        __syncwarp();
    };
    if (!worker) {
#pragma unroll 1
        for (int hh = 0; hh <= nh; ++hh) {
            __syncthreads();
            if (*abort_flag) break;
            if (hh > 0) token_sums(hh - 1);
            if (hh + 1 < nh) ssm_tc_gates(a, b, h0 + hh + 1, t0, s_dt2 + ((hh + 1) & 1) * 128, s_c2 + ((hh + 1) & 1) * 128);
        }
    }
    int hh = 0;
#pragma unroll 1
    for (; worker && hh < nh; ++hh) {
        __syncthreads();
        const int h = h0 + hh, set = hh & 1;
        const size_t unit = ((size_t)b * nch + ch) * a.H + h;  // of the states
        const double *s_c = s_c2 + set * 128;
        const float *s_dt = s_dt2 + set * 128;
        float *s_rowp = s_set + set * L::kSet, *s_colp = s_rowp + 256, *s_diag = s_colp + 512, *s_wd = s_diag + 128,
              *s_gxp = s_wd + 128, *s_syp = s_gxp + 256;
        double *s_red = s_red2 + set * 8;
        {   // tables
            const double last = s_c[127];
            if (tid < 128) {
                const double c = s_c[tid], r = tid >= 32 ? s_c[(tid & ~31) - 1] : 0.0;
                s_e[tid] = exp2f((float)c);
                s_rowf[tid] = exp2f((float)(c - r));
                s_el[tid] = exp2f((float)(last - c));
                const float hi = (float)c;
                s_hi[tid] = hi;
                s_lo[tid] = (float)(c - (double)hi);
            } else {
                for (int i = tid - 128; i < 192; i += 128) {
                    const int I = i < 32 ? 1 : i < 96 ? 2 : 3, j = i < 32 ? i : i < 96 ? i - 32 : i - 96;
                    s_col[(I - 1) * 96 + j] = exp2f((float)(s_c[32 * I - 1] - s_c[j]));
                }
            }
        }
        if (tid == 0) {
            if (bc_open) {
                if (!mbar_wait(bar_bc, 0)) *abort_flag = 1;
                else bc_open = false;
            }
            if (!mbar_wait(bar_x, (uint32_t)(hh & 1))) *abort_flag = 1;
            else ++d_x;
            if (!mbar_wait(bar_y, (uint32_t)(hh & 1))) *abort_flag = 1;
            else ++d_y;
        }
        worker_sync();
        if (*abort_flag) break;
        // ---- W = dY X^T (and once K = C B^T) ----
        if (tid == 0) {
            tc_after_sync();
            if (hh == 0)
#pragma unroll
                for (int kk = 0; kk < N / 16; ++kk)
                    mma_bf16(tmem + tK, desc_k(sb + L::oC, kk), desc_k(sb + L::oB, kk), idesc_bf16(128, 128, false, false), kk > 0);
#pragma unroll
            for (int kk = 0; kk < P / 16; ++kk)
                mma_bf16(tmem + tT, desc_k(sb + L::oY, kk), desc_k(sb + L::oX, kk), idesc_bf16(128, 128, false, false), kk > 0);
        }
        mma_sync_point();
        if (*abort_flag) break;
        // ---- M' = L K, dK = L W Delta, and the sums of R = M' W ----
        {
            const float rf = s_rowf[row], ci = s_hi[row], cl = s_lo[row];
            float rsum = 0.f;
#pragma unroll 1
            for (int jb = 0; jb < 2; ++jb) {
                const int J = half * 2 + jb;
                uint8_t *dm = sm + L::oM + half * kTile, *dk = sm + L::oK + half * kTile;
                if (J > q) {
                    const uint4 z = make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        *reinterpret_cast<uint4 *>(dm + sw128_offset(row, jb * 4 + i)) = z;
                        *reinterpret_cast<uint4 *>(dk + sw128_offset(row, jb * 4 + i)) = z;
                    }
                    s_colp[q * 128 + J * 32 + lane] = 0.f;
                    continue;
                }
                float kv[32], wv[32], rr[32];
                tmem_ld32(tl + tK + J * 32, kv);
                tmem_ld32(tl + tT + J * 32, wv);
                if (J < q) {
                    const float *col = s_col + (q - 1) * 96 + J * 32;
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const float l = rf * col[i], d = s_dt[J * 32 + i];
                        kv[i] *= l;
                        rr[i] = kv[i] * wv[i];
                        rsum = fmaf(rr[i], d, rsum);
                        wv[i] *= l * d;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const int j = J * 32 + i;
                        const float e = exp2f((ci - s_hi[j]) + (cl - s_lo[j])), l = i <= lane ? e : 0.f, d = s_dt[j];
                        const float w = wv[i];
                        kv[i] = i <= lane ? kv[i] * l : 0.f;
                        rr[i] = kv[i] * w;
                        wv[i] = i <= lane ? w * (l * d) : 0.f;
                        if (i == lane) {
                            s_diag[row] = rr[i];
                            s_wd[row] = w;
                            rr[i] = 0.f;
                        }
                        if (i > lane) rr[i] = 0.f;
                        rsum = fmaf(rr[i], d, rsum);
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    st_bf16x8(dm + sw128_offset(row, jb * 4 + i), kv + 8 * i);
                    st_bf16x8(dk + sw128_offset(row, jb * 4 + i), wv + 8 * i);
                }
                ssm_column_sums(rr);
                s_colp[q * 128 + J * 32 + lane] = rr[0];
            }
            s_rowp[half * 128 + row] = rsum;
        }
        fence_async_smem();
        tc_before_sync();
        worker_sync();
        // ---- the chunk's own products ----
        if (tid == 0) {
            tc_after_sync();
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
                mma_bf16(tmem + tT, desc_mn(sb + L::oM, kk), desc_mn(sb + L::oY, kk), idesc_bf16(128, P, true, true), kk > 0);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
                mma_bf16(tmem + tC, desc_k(sb + L::oK, kk), desc_mn(sb + L::oB, kk), idesc_bf16(128, N, false, true),
                         hh > 0 || kk > 0);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
                mma_bf16(tmem + tB, desc_mn(sb + L::oK, kk), desc_mn(sb + L::oC, kk), idesc_bf16(128, N, true, true),
                         hh > 0 || kk > 0);
        }
        float st[kChunks][8], dxi[P / 2];
        load_state(Sin + unit * P * N, st);
        mma_sync_point();
        if (*abort_flag) break;
        {
#pragma unroll
            for (int c = 0; c < P / 2; c += 32) tmem_ld32(tl + tT + half * (P / 2) + c, dxi + c);
#pragma unroll
            for (int i = 0; i < kChunks; ++i) st_split8(sm + L::oHi + chunk_off(i), sm + L::oLo + chunk_off(i), st[i]);
        }
        fence_async_smem();
        tc_before_sync();
        worker_sync();
        // ---- T = dY S_in ----
        if (tid == 0) {
            tc_after_sync();
#pragma unroll
            for (int pt = 0; pt < 2; ++pt)
#pragma unroll
                for (int kk = 0; kk < P / 16; ++kk)
                    mma_bf16(tmem + tT, desc_k(sb + L::oY, kk), desc_mn(sb + (pt ? L::oLo : L::oHi), kk, L::kSBlock),
                             idesc_bf16(128, N, false, true), pt > 0 || kk > 0);
        }
        {
            load_state(Gout + unit * P * N, st);
            float dot = 0.f;  // <G, S_in>, S_in from its two parts
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {
                float x[8], y[8];
                ld8s(sm + L::oHi + chunk_off(i), x);
                ld8s(sm + L::oLo + chunk_off(i), y);
#pragma unroll
                for (int e = 0; e < 8; ++e) dot = fmaf(x[e] + y[e], st[i][e], dot);
            }
            double dd = dot;
#pragma unroll
            for (int off = 16; off; off >>= 1) dd += __shfl_xor_sync(0xffffffffu, dd, off);
            if (lane == 0) s_red[warp] = dd;
        }
        mma_sync_point();
        if (*abort_flag) break;
        {
            const float e = s_e[row];
            float dot = 0.f;
#pragma unroll 1
            for (int c = half * (N / 2); c < (half + 1) * (N / 2); c += 32) {
                float t[32], acc[32];
                tmem_ld32(tl + tT + c, t);
                tmem_ld32(tl + tC + c, acc);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float v[8];
                    ld8s(sm + L::oC + (uint32_t)(c >> 6) * kTile + sw128_offset(row, ((c & 63) >> 3) + i), v);
#pragma unroll
                    for (int k = 0; k < 8; ++k) dot = fmaf(v[k], t[8 * i + k], dot);
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) acc[i] = fmaf(e, t[i], acc[i]);
                tmem_st32(tl + tC + c, acc);
            }
            tmem_wait_st();
            s_syp[half * 128 + row] = e * dot;
#pragma unroll
            for (int i = 0; i < kChunks; ++i) st_split8(sm + L::oHi + chunk_off(i), sm + L::oLo + chunk_off(i), st[i]);
        }
        fence_async_smem();
        tc_before_sync();
        worker_sync();
        // ---- T = X G_out ----
        if (tid == 0) {
            tc_after_sync();
#pragma unroll
            for (int pt = 0; pt < 2; ++pt)
#pragma unroll
                for (int kk = 0; kk < P / 16; ++kk)
                    mma_bf16(tmem + tT, desc_k(sb + L::oX, kk), desc_mn(sb + (pt ? L::oLo : L::oHi), kk, L::kSBlock),
                             idesc_bf16(128, N, false, true), pt > 0 || kk > 0);
        }
        mma_sync_point();
        if (*abort_flag) break;
        if (tid == 0 && hh + 1 < nh) issue_x(h + 1);
        {
            const float el = s_el[row], w = el * s_dt[row];
            float dot = 0.f;
#pragma unroll 1
            for (int c = half * (N / 2); c < (half + 1) * (N / 2); c += 32) {
                float t[32], acc[32];
                tmem_ld32(tl + tT + c, t);
                tmem_ld32(tl + tB + c, acc);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float v[8];
                    ld8s(sm + L::oB + (uint32_t)(c >> 6) * kTile + sw128_offset(row, ((c & 63) >> 3) + i), v);
#pragma unroll
                    for (int k = 0; k < 8; ++k) dot = fmaf(v[k], t[8 * i + k], dot);
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) acc[i] = fmaf(w, t[i], acc[i]);
                tmem_st32(tl + tB + c, acc);
            }
            tmem_wait_st();
            s_gxp[half * 128 + row] = el * dot;
        }
        tc_before_sync();
        worker_sync();
        // ---- T = B G_out^T ----
        if (tid == 0) {
            tc_after_sync();
#pragma unroll
            for (int kk = 0; kk < N / 16; ++kk)
                mma_bf16(tmem + tT, desc_k(sb + L::oB, kk), desc_k(sb + L::oHi, kk, L::kSBlock), idesc_bf16(128, P, false, false),
                         kk > 0);
        }
        mma_sync_point();
        if (*abort_flag) break;
        // ---- dx over dY ----
        {
            const float el = s_el[row], dt = s_dt[row], D = a.D ? a.D[h] : 0.f;
#pragma unroll
            for (int cc = 0; cc < P / 2; cc += 32) {
                const int c = half * (P / 2) + cc;
                float t[32];
                tmem_ld32(tl + tT + c, t);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint8_t *p = sm + L::oY + (uint32_t)(c >> 6) * kTile + sw128_offset(row, ((c & 63) >> 3) + i);
                    float y[8];
                    ld8s(p, y);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float v = dt * fmaf(el, t[8 * i + k], dxi[cc + 8 * i + k]);
                        y[k] = a.D ? fmaf(D, y[k], v) : v;
                    }
                    st_bf16x8(p, y);
                }
            }
        }
        fence_async_smem();
        tc_before_sync();
        worker_sync();
        if (tid == 0) {
            for (int i = 0; i < P / 64; ++i) tma_store_4d(&tm_dx, sm + L::oY + i * kTile, i * 64, h, t0, b);
            bulk_commit();
            bulk_wait_read_all();
            if (hh + 1 < nh) issue_y(h + 1);
        }
    }
    if (worker) __syncthreads();  // the last head's sums (or, given up, the meeting that warp 8 still waits at)
    if (*abort_flag) {
        if (tid == 0) {
            record_status(GDR_ERR_TIMEOUT);
            if (bc_open) mbar_wait(bar_bc, 0);
            if (d_x < n_x) mbar_wait(bar_x, (uint32_t)(d_x & 1));
            if (d_y < n_y) mbar_wait(bar_y, (uint32_t)(d_y & 1));
            if (mma_open) mbar_wait(mma_bar, mma_phase ^ 1);
            bulk_wait_all();
        }
    } else {
        tc_after_sync();
        if (worker) {
            const bool on = row < valid;
            const size_t at = (((size_t)b * a.T + t0 + row) * a.G + g);
#pragma unroll 1
            for (int which = 0; which < 2; ++which) {
#pragma unroll 1
                for (int c = half * (N / 2); c < (half + 1) * (N / 2); c += 32) {
                    float v[32];
                    tmem_ld32(tl + (which ? tB : tC) + c, v);
                    if (!on) continue;
                    if (splits == 1) {
                        uint8_t *dst = reinterpret_cast<uint8_t *>(static_cast<__nv_bfloat16 *>(which ? a.dB : a.dC) + at * N + c);
#pragma unroll
                        for (int i = 0; i < 4; ++i) st_bf16x8(dst + 16 * i, v + 8 * i);
                    } else {
                        float4 *dst = reinterpret_cast<float4 *>((which ? dBp : dCp) + (at * splits + sp) * N + c);
#pragma unroll
                        for (int i = 0; i < 8; ++i) dst[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                    }
                }
            }
        }
        if (tid == 0) bulk_wait_all();
    }
    tc_before_sync();
    __syncthreads();
    if (warp == 0) {
        tc_after_sync();
        tmem_dealloc(tmem, 512);
    }
}

// ---- host side ------------------------------------------------------------------------------
// CTAs per group of heads: the fewest heads in a row for the SMs, one CTA where that is as good.
inline int ssm_grad_splits(int B, int T, int H, int G) {
    const int nch = (T + kTcQ - 1) / kTcQ, HG = H / G, sms = ssm_sm_count();
    int best = 1;
    long long cost = -1;
    for (int s = 1; s <= HG; ++s) {
        const int per = (HG + s - 1) / s;
        if ((HG + per - 1) / per != s) continue;
        const long long c = (((long long)B * nch * G * s + sms - 1) / sms) * per;
        if (cost < 0 || c < cost) {
            cost = c;
            best = s;
        }
    }
    return best;
}

struct SsmTcBwdWs {
    size_t st, g, dec, part, dBp, dCp, total;
    int splits;
};
inline SsmTcBwdWs ssm_tc_bwd_ws(int B, int T, int H, int G, int P, int N) {
    const size_t units = (size_t)B * ((T + kTcQ - 1) / kTcQ) * H;
    SsmTcBwdWs w;
    w.splits = ssm_grad_splits(B, T, H, G);
    w.st = 0;
    w.g = ssm_align(units * P * N * 4);
    w.dec = 2 * w.g;
    w.part = w.dec + ssm_align(units * 4);
    w.dBp = w.part + ssm_align(3 * units * 4);
    const size_t p = w.splits > 1 ? ssm_align((size_t)B * T * G * w.splits * N * 4) : 0;
    w.dCp = w.dBp + p;
    w.total = w.dCp + p;
    return w;
}

template <int P, int N>
cudaError_t ssm_tc_bwd(const SsmArgs &a, void *ws, cudaStream_t s) {
    CUtensorMap mx, mb, mc, my, mdx;
    if (!ssm_token_map(&mx, a.x, a.B, a.T, a.H, P, a.ldx) || !ssm_token_map(&mb, a.Bm, a.B, a.T, a.G, N, a.ldb) ||
        !ssm_token_map(&mc, a.Cm, a.B, a.T, a.G, N, a.ldc) || !ssm_token_map(&my, a.dy, a.B, a.T, a.H, P, a.H * P) ||
        !ssm_token_map(&mdx, a.dx, a.B, a.T, a.H, P, a.H * P))
        return cudaErrorInvalidValue;
    const SsmTcBwdWs w = ssm_tc_bwd_ws(a.B, a.T, a.H, a.G, P, N);
    const int nch = (a.T + kTcQ - 1) / kTcQ, HG = a.H / a.G, per = (HG + w.splits - 1) / w.splits;
    uint8_t *base = static_cast<uint8_t *>(ws);
    float *st = reinterpret_cast<float *>(base + w.st), *g = reinterpret_cast<float *>(base + w.g);
    float *dec = reinterpret_cast<float *>(base + w.dec), *part = reinterpret_cast<float *>(base + w.part);
    float *dBp = reinterpret_cast<float *>(base + w.dBp), *dCp = reinterpret_cast<float *>(base + w.dCp);
    const dim3 grid((unsigned)(a.B * a.H) * (unsigned)nch);
    cudaError_t e = ssm_launch(ssm_tc_state_kernel<P, N, false>, grid, 256, (size_t)SsmStateTc<P, N, false>::kAlloc, s, mx, mb,
                               a, 1, st, dec);
    if (e == cudaSuccess)
        e = ssm_launch(ssm_tc_state_kernel<P, N, true>, grid, 256, (size_t)SsmStateTc<P, N, true>::kAlloc, s, my, mc, a, 1, g,
                       dec);
    if (e == cudaSuccess) e = ssm_launch_scan(false, a.B, nch, a.H, P * N, st, dec, a.S0, nullptr, s);
    if (e == cudaSuccess) e = ssm_launch_scan(true, a.B, nch, a.H, P * N, g, dec, a.dS_T, a.dS0, s);
    if (e == cudaSuccess)
        e = ssm_launch(ssm_tc_grad_kernel<P, N>, dim3((unsigned)((size_t)a.B * nch * a.G * w.splits)), kGradThreads,
                       (size_t)SsmGradTc<P, N>::kAlloc, s, mx, mb, mc, my, mdx, a, w.splits, per, (const float *)st,
                       (const float *)g, dBp, dCp, part);
    if (e != cudaSuccess) return e;
    if (w.splits > 1) {
        const long long total4 = (long long)a.B * a.T * a.G * (N / 4);
        ssm_group_sum_kernel<__nv_bfloat16><<<dim3((unsigned)((total4 + 255) / 256), 2), 256, 0, s>>>(
            total4, w.splits, N / 4, dBp, dCp, static_cast<__nv_bfloat16 *>(a.dB), static_cast<__nv_bfloat16 *>(a.dC));
        g_launches.fetch_add(1, std::memory_order_relaxed);
    }
    ssm_head_sum_kernel<<<a.H, 256, 0, s>>>(a.B * nch, a.H, part, a.dA, a.dbias, a.dD);
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return cudaGetLastError();
}

}  // namespace gdr

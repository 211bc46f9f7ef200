// ssm_bwd_tc.cuh -- the selective scan's gradients on the 5th-generation
// tensor cores, bf16 inputs, P, N in {64, 128}; formulas at the gradient kernel
// of ssm_simt.cuh.  Chunks of 128 tokens:
//   1. ssm_tc_walk_kernel   S_in(c) of every chunk, walking forwards, and G_out(c),
//      walking backwards, in one launch (segments from the same walk and
//      ssm_scan_kernel first where heads are few), each state in fp32
//   2. ssm_tc_grad_kernel   a CTA owns one chunk of one group and walks heads of
//      it, so that B and C are read once and dB, dC are summed over the heads in
//      TMEM.  Per head (W = dy x^T, L the decays, tokens on the TMEM lanes):
//        K   = C B^T,  W = dY X^T                  N = 128   K = N, P
//        dC += dK B,  dB += dK^T C                 N = N     K = 128    dK = L W Delta
//        dXi = M'^T dY                             N = P     K = 128    M' = L (C B^T)
//        T   = dY S_in  -> dC += e^{c_i} T,        dlog: e^{c_i} C_i . T_i
//        T   = X G_out  -> dB += w_j T,            dDelta: e^{c_last-c_j} B_j . T_j
//        T   = B G_out^T -> dx = Delta (dXi + e^{c_last-c_j} T) + D dy
//      (N = N, N, P and K = P, P, N).
// Operands that are not bf16 themselves enter as bf16 parts, as in the forward: M' and dK as two, S_in and G_out as three
// where fp32 results follow from the product and G_out as two for dx.  The double sums of R = L K W are taken on CUDA
// cores from the fp32 accumulators.  With one part for M', dK and dx's G_out, and the states kept as two, dx, dB and dC
// were 2.3e-3 off 64 bits (one rounding: 1.7e-3), dS0 2.5e-6 and dA and the bias's gradient up to 1e-5; now 1e-7 to 4e-7.
// B=4 T=4096 H=16 P=N=128: 440 us (walk 129, gradients 301), 308 with the fewer parts.
#pragma once
#include "ssm_tc.cuh"

namespace gdr {

// ---- 2. the gradients of every chunk -------------------------------------------------------
template <int P, int N>
struct SsmGradTc {
    static constexpr uint32_t XB = P / 64 * kTile, BB = N / 64 * kTile;
    static constexpr uint32_t kSBlock = N * 128, SB = P / 64 * kSBlock;  // a state part: N rows, blocks of 64 columns p
    static constexpr uint32_t oB = 0, oC = BB, oX = 2 * BB, oY = oX + XB, oR = oY + XB;
    static constexpr uint32_t oM = oR, oK = oR + 2 * kTile;   // M', dK: the first parts, then the second
    static constexpr uint32_t oHi = oR, oLo = oR + SB;        // S_in, then G_out: two parts; the third
    static constexpr uint32_t oThirdS = oX, oThirdG = oY;     // in the tiles of X (read again behind it) and of dY
    // A state arrives in fp32: S_in's first bytes in X's tile, from the moment W is formed, the rest over M' and dK; G_out
    // whole over S_in's parts.
    static constexpr uint32_t kRaw = P * N * 4, kRawX = kRaw < XB ? kRaw : XB;
    static constexpr uint32_t oGate = oR + 4 * kTile;
    // two tables; doubles: warp sums of the token sums [4][2], totals [4][3], <G, S> [16], rowp[4][128], colp[4][128];
    // floats: diag, wd, gxp[4][128], syp[4][128]
    static constexpr uint32_t oSum = oGate + 2 * SsmGate::kBytes;
    static constexpr uint32_t oBar = oSum + (8 + 12 + 16 + 8 * 128) * 8 + 10 * 128 * 4;
    static constexpr uint32_t kAlloc = oBar + 64 + 1024;
};

// Column sums of a 32 x 8 block held as v[column] per lane (row): v[0] ends as the sum of column lane & 7.
__device__ __forceinline__ void ssm_column_sums(double *v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int s = 4; s > 0; s >>= 1) {
        const bool up = lane & s;
#pragma unroll
        for (int k = 0; k < s; ++k) {
            const double send = up ? v[k] : v[k + s], keep = up ? v[k + s] : v[k];
            v[k] = keep + __shfl_xor_sync(0xffffffffu, send, s);
        }
    }
    v[0] += __shfl_xor_sync(0xffffffffu, v[0], 8);
    v[0] += __shfl_xor_sync(0xffffffffu, v[0], 16);
}
__device__ __forceinline__ double ssm_warp_scan(double x) {  // inclusive
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const double o = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += o;
    }
    return x;
}
constexpr int kGradThreads = 512;  // a TMEM quarter and a quarter of the columns per warp

template <int P, int N>
__global__ void __launch_bounds__(kGradThreads, 1) ssm_tc_grad_kernel(
    const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_b,
    const __grid_constant__ CUtensorMap tm_c, const __grid_constant__ CUtensorMap tm_dy,
    const __grid_constant__ CUtensorMap tm_dx, SsmArgs a, int splits, int per, const float *__restrict__ gates,
    const float4 *__restrict__ Sin, const float4 *__restrict__ Gout, float *__restrict__ dBp, float *__restrict__ dCp,
    double *__restrict__ part) {
    using L = SsmGradTc<P, N>;
    using namespace sm100;
    constexpr int NW = N / 4, PW = P / 4;  // columns of a warp
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const uint32_t sb = smem_u32(sm);
    double *s_tw = reinterpret_cast<double *>(sm + L::oSum);
    double *s_tot = s_tw + 8, *s_red = s_tot + 12, *s_rowp = s_red + 16, *s_colp = s_rowp + 512;
    float *s_diag = reinterpret_cast<float *>(s_colp + 512), *s_wd = s_diag + 128,
          *s_gxp = s_wd + 128, *s_syp = s_gxp + 512;
    uint64_t *bar_bc = reinterpret_cast<uint64_t *>(sm + L::oBar), *bar_x = bar_bc + 1, *bar_y = bar_bc + 2,
             *bar_g = bar_bc + 3, *mma_bar = bar_bc + 4, *bar_s = bar_bc + 5, *bar_r = bar_bc + 6;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bar_bc + 7);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int q = warp & 3, prt = warp >> 2, row = q * 32 + lane;  // TMEM lane, column quarter
    const int nch = (a.T + kTcQ - 1) / kTcQ, HG = a.H / a.G;
    int u = blockIdx.x;
    const int sp = u % splits;
    u /= splits;
    const int g = u % a.G;
    u /= a.G;
    const int ch = u % nch, b = u / nch;
    const int h0 = g * HG + sp * per, nh = min(per, HG - sp * per);
    const int t0 = ch * kTcQ, valid = min(kTcQ, a.T - t0);
    const size_t unit0 = ((size_t)b * nch + ch) * a.H, units = (size_t)a.B * nch * a.H;

    if (tid == 0) {
        mbar_init(bar_bc, 1);
        mbar_init(bar_x, 1);
        mbar_init(bar_y, 1);
        mbar_init(bar_g, 1);
        mbar_init(mma_bar, 1);
        mbar_init(bar_s, 1);
        mbar_init(bar_r, 1);
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

    constexpr int kIo = 384;              // issues copies (a warp above the diagonal); thread 0 issues products
    int n_x = 0, n_y = 0, n_g = 0, n_s = 0, n_r = 0;  // issued, by that thread
    uint32_t r_phase = 0;                             // everyone's
    bool mma_open = false;
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
    auto issue_g = [&](int hh) {
        mbar_expect_tx(bar_g, SsmGate::kBytes);
        bulk_load_g2s(sm + L::oGate + (hh & 1) * SsmGate::kBytes, gates + (unit0 + h0 + hh) * SsmGate::stride, SsmGate::kBytes,
                      bar_g);
        ++n_g;
    };
    if (tid == kIo) {
        mbar_expect_tx(bar_bc, 2 * L::BB);
        for (int i = 0; i < N / 64; ++i) {
            tma_load_4d(sm + L::oB + i * kTile, &tm_b, bar_bc, i * 64, g, t0, b);
            tma_load_4d(sm + L::oC + i * kTile, &tm_c, bar_bc, i * 64, g, t0, b);
        }
        issue_x(h0);
        issue_y(h0);
        issue_g(0);
    }
    uint32_t mma_phase = 0;
    auto mma_sync_point = [&]() {  // thread 0 has committed its products
        if (tid == 0) {
            mma_open = !mbar_wait(mma_bar, mma_phase);
            if (mma_open) *abort_flag = 1;
        }
        mma_phase ^= 1;
        __syncthreads();
        tc_after_sync();
    };
    // A state, 8 columns p of a row n at a time: chunk i of this thread.  Every thread reads its chunks before any writes
    // its parts over them.
    constexpr int kChunks = P * N / 8 / kGradThreads;
    auto issue_raw = [&](uint64_t *bar, uint32_t to, const float4 *src, size_t unit, uint32_t from, uint32_t bytes) {
        mbar_expect_tx(bar, bytes);
        bulk_load_g2s(sm + to, reinterpret_cast<const uint8_t *>(src + unit * (P * N / 4)) + from, bytes, bar);
    };
    auto wait_raw = [&] {
        if (!mbar_wait(bar_r, r_phase)) *abort_flag = 1;
        r_phase ^= 1;
    };
    auto read_raw = [&](int i, bool in_x, float (&x)[8]) {
        const int n = (i * kGradThreads + tid) % N, p8 = (i * kGradThreads + tid) / N;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const uint32_t at = (uint32_t)((2 * p8 + u) * N + n) * 16;
            const float4 v = *reinterpret_cast<const float4 *>(
                sm + (!in_x ? L::oR + at : at < L::kRawX ? L::oX + at : L::oR + at - L::kRawX));
            x[4 * u] = v.x;
            x[4 * u + 1] = v.y;
            x[4 * u + 2] = v.z;
            x[4 * u + 3] = v.w;
        }
    };
    auto write_parts = [&](int i, uint32_t third, const float (&x)[8]) {
        const int n = (i * kGradThreads + tid) % N, p8 = (i * kGradThreads + tid) / N;
        const uint32_t off = (uint32_t)(p8 >> 3) * L::kSBlock + sw128_offset(n, p8 & 7);
        float r[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) r[e] = x[e];
        *reinterpret_cast<uint4 *>(sm + L::oHi + off) = take_bf16x8(r);
        *reinterpret_cast<uint4 *>(sm + L::oLo + off) = take_bf16x8(r);
        *reinterpret_cast<uint4 *>(sm + third + off) = take_bf16x8(r);
    };
    // the three parts of a state, the smallest first (the tensor core truncates what it adds to a larger sum)
    auto part_at = [&](int part, uint32_t third) { return sb + (part == 0 ? third : part == 1 ? L::oLo : L::oHi); };
#pragma unroll 1
    for (int hh = 0; hh < nh; ++hh) {
        const int h = h0 + hh;
        const size_t unit = unit0 + h;
        const float *s_g = reinterpret_cast<const float *>(sm + L::oGate + (hh & 1) * SsmGate::kBytes);
        const float *s_dt = s_g + SsmGate::dt;
        if (tid < 2 * P * N * 2 / 128) {  // this head's states on their way into L2: a line of each a thread
            prefetch_l2(Sin + unit * (P * N / 4) + tid * 8);
            prefetch_l2(Gout + unit * (P * N / 4) + tid * 8);
        }
        if (tid == 0) {
            if (hh == 0 && !mbar_wait(bar_bc, 0)) *abort_flag = 1;
            if (!mbar_wait(bar_g, (uint32_t)(hh & 1)) || !mbar_wait(bar_x, 0) ||
                !mbar_wait(bar_y, (uint32_t)(hh & 1)))
                *abort_flag = 1;
        }
        if (tid == kIo) bulk_wait_read_all();  // the last head's dx leaves through the buffer of M' and dK
        __syncthreads();
        if (*abort_flag) break;
        if (tid == kIo && hh + 1 < nh) issue_g(hh + 1);  // the other table was last read a head ago
        __syncwarp();
        // ---- K = C B^T, W = dY X^T ----
        if (tid == 0) {
            tc_after_sync();
#pragma unroll
            for (int kk = 0; kk < N / 16; ++kk)
                mma_bf16(tmem + tK, desc_k(sb + L::oC, kk), desc_k(sb + L::oB, kk), idesc_bf16(128, 128, false, false), kk > 0);
#pragma unroll
            for (int kk = 0; kk < P / 16; ++kk)
                mma_bf16(tmem + tT, desc_k(sb + L::oY, kk), desc_k(sb + L::oX, kk), idesc_bf16(128, 128, false, false), kk > 0);
            mma_commit(mma_bar);
        }
        mma_sync_point();
        if (*abort_flag) break;
        if (tid == kIo) {
            issue_raw(bar_s, L::oX, Sin, unit, 0, L::kRawX);
            ++n_s;
        }
        __syncwarp();
        // ---- M' = L K, dK = L W Delta, and the sums of R = M' W: rows i, 32 columns j, 16 at a time (with all 32 the
        // kernel spilled, and beside its shared memory there is next to no L1 for that).  The first bf16 parts go to shared
        // memory, the second wait in TMEM over the K they come from: 8 columns of M', 8 of dK. ----
        {
            uint8_t *dm = sm + L::oM + (prt >> 1) * kTile, *dk = sm + L::oK + (prt >> 1) * kTile;
            double rsum = 0.0;
            if (prt > q) {
                const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    *reinterpret_cast<uint4 *>(dm + sw128_offset(row, (prt & 1) * 4 + i)) = zero;
                    *reinterpret_cast<uint4 *>(dk + sw128_offset(row, (prt & 1) * 4 + i)) = zero;
                }
                s_colp[q * 128 + prt * 32 + lane] = 0.0;
            } else {
                const float rf = s_g[SsmGate::rowf + row], ci = s_g[SsmGate::hi + row], cl = s_g[SsmGate::lo + row];
                float dg = 0.f, wd = 0.f;
#pragma unroll 1
                for (int hb = 0; hb < 2; ++hb) {
                    const int j0 = prt * 32 + hb * 16;
                    float kv[16], wv[16], rr[16];
                    const float4 *dt4 = reinterpret_cast<const float4 *>(s_dt + j0);
                    tmem_ld16x2(tl + tK + j0, kv, tl + tT + j0, wv);
                    if (prt < q) {
                        const float2 rf2 = make_float2(rf, rf);
                        const float4 *col4 = reinterpret_cast<const float4 *>(s_g + SsmGate::col + (q - 1) * 96 + j0);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float4 c4 = col4[i], d4 = dt4[i];
                            const float2 c2[2] = {make_float2(c4.x, c4.y), make_float2(c4.z, c4.w)};
                            const float2 d2[2] = {make_float2(d4.x, d4.y), make_float2(d4.z, d4.w)};
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                const int n = 4 * i + 2 * u;
                                const float2 l = fmul2(rf2, c2[u]), w = make_float2(wv[n], wv[n + 1]);
                                const float2 kk = fmul2(make_float2(kv[n], kv[n + 1]), l), r = fmul2(kk, w);
                                const float2 dk2 = fmul2(w, fmul2(l, d2[u]));
                                kv[n] = kk.x;
                                kv[n + 1] = kk.y;
                                rr[n] = r.x;
                                rr[n + 1] = r.y;
                                wv[n] = dk2.x;
                                wv[n + 1] = dk2.y;
                            }
                        }
                    } else {
                        const float4 *hi4 = reinterpret_cast<const float4 *>(s_g + SsmGate::hi + j0);
                        const float4 *lo4 = reinterpret_cast<const float4 *>(s_g + SsmGate::lo + j0);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float4 h4 = hi4[i], l4 = lo4[i], d4 = dt4[i];
                            const float l[4] = {exp2f((ci - h4.x) + (cl - l4.x)), exp2f((ci - h4.y) + (cl - l4.y)),
                                                exp2f((ci - h4.z) + (cl - l4.z)), exp2f((ci - h4.w) + (cl - l4.w))};
                            const float d[4] = {d4.x, d4.y, d4.z, d4.w};
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                const int n = 4 * i + u, at = hb * 16 + n;  // column of the block; the row's is lane
                                const float w = wv[n], r = kv[n] * l[u] * w;
                                if (at == lane) {
                                    dg = r;
                                    wd = w;
                                }
                                kv[n] = at <= lane ? kv[n] * l[u] : 0.f;
                                wv[n] = at <= lane ? w * (l[u] * d[u]) : 0.f;
                                rr[n] = at < lane ? r : 0.f;
                            }
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        *reinterpret_cast<uint4 *>(dm + sw128_offset(row, (prt & 1) * 4 + hb * 2 + i)) = take_bf16x8(kv + 8 * i);
                        *reinterpret_cast<uint4 *>(dk + sw128_offset(row, (prt & 1) * 4 + hb * 2 + i)) = take_bf16x8(wv + 8 * i);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        kv[i] = __uint_as_float(take_bf16x2(kv[2 * i], kv[2 * i + 1]));
                        wv[i] = __uint_as_float(take_bf16x2(wv[2 * i], wv[2 * i + 1]));
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) kv[8 + i] = wv[i];
                    tmem_st16(tl + tK + j0, kv);
                    // 64 bits: a pair's R Delta in its row's sum and in its column's cancels exactly behind both
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        double r[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            r[e] = (double)rr[8 * half + e];
                            rsum = fma(r[e], (double)s_dt[j0 + 8 * half + e], rsum);
                        }
                        ssm_column_sums(r);
                        if (lane < 8) s_colp[q * 128 + j0 + 8 * half + lane] = r[0];
                    }
                }
                tmem_wait_st();
                if (prt == q) {
                    s_diag[row] = dg;
                    s_wd[row] = wd;
                }
            }
            s_rowp[prt * 128 + row] = rsum;
        }
        fence_async_smem();
        tc_before_sync();
        __syncthreads();
        // ---- the chunk's own products, of the first parts and then of the second ----
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
            if (part == 1) {
                if (prt <= q) {  // above the diagonal the zeros stay
                    uint8_t *dm = sm + L::oM + (prt >> 1) * kTile, *dk = sm + L::oK + (prt >> 1) * kTile;
#pragma unroll
                    for (int hb = 0; hb < 2; ++hb) {
                        float v[16];
                        tmem_ld16(tl + tK + prt * 32 + hb * 16, v);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            *reinterpret_cast<float4 *>(dm + sw128_offset(row, (prt & 1) * 4 + hb * 2 + i)) =
                                make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                            *reinterpret_cast<float4 *>(dk + sw128_offset(row, (prt & 1) * 4 + hb * 2 + i)) =
                                make_float4(v[8 + 4 * i], v[9 + 4 * i], v[10 + 4 * i], v[11 + 4 * i]);
                        }
                    }
                }
                fence_async_smem();
                tc_before_sync();
                __syncthreads();
            }
            if (tid == 0) {
                tc_after_sync();
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    mma_bf16(tmem + tT, desc_mn(sb + L::oM, kk), desc_mn(sb + L::oY, kk), idesc_bf16(128, P, true, true),
                             part > 0 || kk > 0);
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    mma_bf16(tmem + tC, desc_k(sb + L::oK, kk), desc_mn(sb + L::oB, kk), idesc_bf16(128, N, false, true),
                             hh > 0 || part > 0 || kk > 0);
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    mma_bf16(tmem + tB, desc_mn(sb + L::oK, kk), desc_mn(sb + L::oC, kk), idesc_bf16(128, N, true, true),
                             hh > 0 || part > 0 || kk > 0);
                mma_commit(mma_bar);
            }
            __syncwarp();
            mma_sync_point();
            if (*abort_flag) break;
        }
        if (*abort_flag) break;
        if (L::kRaw > L::kRawX && tid == kIo) {
            issue_raw(bar_r, L::oR, Sin, unit, L::kRawX, L::kRaw - L::kRawX);
            ++n_r;
        }
        __syncwarp();
        float dxi[PW];  // Delta dXi + D dy
        tmem_ldw<PW>(tl + tT + prt * PW, dxi);
        {
            const float dt = s_dt[row], D = s_g[SsmGate::D];
            const int c = prt * PW;
#pragma unroll
            for (int i = 0; i < PW / 8; ++i) {
                float y[8];
                if (a.D) ld8s(sm + L::oY + (uint32_t)(c >> 6) * kTile + sw128_offset(row, ((c & 63) >> 3) + i), y);
#pragma unroll
                for (int k = 0; k < 8; ++k) dxi[8 * i + k] = a.D ? fmaf(dt, dxi[8 * i + k], D * y[k]) : dt * dxi[8 * i + k];
            }
        }
        float st[kChunks][8];  // this thread's part of S_in, for <G, S_in>
        if (!mbar_wait(bar_s, (uint32_t)(hh & 1))) *abort_flag = 1;
        if (L::kRaw > L::kRawX) wait_raw();
#pragma unroll
        for (int i = 0; i < kChunks; ++i) read_raw(i, true, st[i]);
        __syncthreads();
        if (*abort_flag) break;
#pragma unroll
        for (int i = 0; i < kChunks; ++i) write_parts(i, L::oThirdS, st[i]);
        fence_async_smem();
        tc_before_sync();
        __syncthreads();
        // ---- T = dY S_in ----
        if (tid == 0) {
            tc_after_sync();
#pragma unroll
            for (int pt = 0; pt < 3; ++pt)
#pragma unroll
                for (int kk = 0; kk < P / 16; ++kk)
                    mma_bf16(tmem + tT, desc_k(sb + L::oY, kk), desc_k(part_at(pt, L::oThirdS), kk, L::kSBlock),
                             idesc_bf16(128, N, false, false), pt > 0 || kk > 0);
            mma_commit(mma_bar);
        }
        __syncwarp();
        mma_sync_point();
        if (*abort_flag) break;
        if (tid == kIo) {
            issue_raw(bar_r, L::oR, Gout, unit, 0, L::kRaw);
            ++n_r;
            issue_x(h);  // the third part was over it
        }
        __syncwarp();
        {
            const float e = s_g[SsmGate::e + row];
            float dot = 0.f;
#pragma unroll 1
            for (int c = prt * NW; c < (prt + 1) * NW; c += 16) {
                float t[16], acc[16];
                tmem_ld16x2(tl + tT + c, t, tl + tC + c, acc);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float v[8];
                    ld8s(sm + L::oC + (uint32_t)(c >> 6) * kTile + sw128_offset(row, ((c & 63) >> 3) + i), v);
#pragma unroll
                    for (int k = 0; k < 8; ++k) dot = fmaf(v[k], t[8 * i + k], dot);
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[i] = fmaf(e, t[i], acc[i]);
                tmem_st16(tl + tC + c, acc);
            }
            tmem_wait_st();
            s_syp[prt * 128 + row] = e * dot;
        }
        wait_raw();
        {
            float dot = 0.f;  // <G, S_in>
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {
                float x[8];
                read_raw(i, false, x);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    dot = fmaf(x[e], st[i][e], dot);
                    st[i][e] = x[e];
                }
            }
            __syncthreads();
            if (*abort_flag) break;
#pragma unroll
            for (int i = 0; i < kChunks; ++i) write_parts(i, L::oThirdG, st[i]);
            double sum = (double)dot;
#pragma unroll
            for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            if (lane == 0) s_red[warp] = sum;
        }
        if (tid == 0 && !mbar_wait(bar_x, 1)) *abort_flag = 1;
        fence_async_smem();
        tc_before_sync();
        __syncthreads();
        if (*abort_flag) break;
        // ---- T = X G_out ----
        if (tid == 0) {
            tc_after_sync();
#pragma unroll
            for (int pt = 0; pt < 3; ++pt)
#pragma unroll
                for (int kk = 0; kk < P / 16; ++kk)
                    mma_bf16(tmem + tT, desc_k(sb + L::oX, kk), desc_k(part_at(pt, L::oThirdG), kk, L::kSBlock),
                             idesc_bf16(128, N, false, false), pt > 0 || kk > 0);
            mma_commit(mma_bar);
        }
        __syncwarp();
        mma_sync_point();
        if (*abort_flag) break;
        if (tid == kIo && hh + 1 < nh) {
            issue_x(h + 1);
            issue_y(h + 1);
        }
        __syncwarp();
        {
            const float el = s_g[SsmGate::el + row], w = el * s_dt[row];
            float dot = 0.f;
#pragma unroll 1
            for (int c = prt * NW; c < (prt + 1) * NW; c += 16) {
                float t[16], acc[16];
                tmem_ld16x2(tl + tT + c, t, tl + tB + c, acc);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float v[8];
                    ld8s(sm + L::oB + (uint32_t)(c >> 6) * kTile + sw128_offset(row, ((c & 63) >> 3) + i), v);
#pragma unroll
                    for (int k = 0; k < 8; ++k) dot = fmaf(v[k], t[8 * i + k], dot);
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[i] = fmaf(w, t[i], acc[i]);
                tmem_st16(tl + tB + c, acc);
            }
            tmem_wait_st();
            s_gxp[prt * 128 + row] = el * dot;
        }
        tc_before_sync();
        __syncthreads();
        // ---- T = B G_out^T; beside it the per-token sums of this head, a token a thread of warps 4-7 ----
        if (tid == 0) {
            tc_after_sync();
#pragma unroll
            for (int pt = 1; pt < 3; ++pt)
#pragma unroll
                for (int kk = 0; kk < N / 16; ++kk)
                    mma_bf16(tmem + tT, desc_k(sb + L::oB, kk), desc_mn(part_at(pt, 0), kk, L::kSBlock),
                             idesc_bf16(128, P, false, true), pt > 1 || kk > 0);
            mma_commit(mma_bar);
        }
        __syncwarp();
        if (warp >= 4 && warp < 8) {
            const int t = tid - 128, w4 = warp - 4;
            const double cg = (s_colp[t] + s_colp[128 + t] + s_colp[256 + t] + s_colp[384 + t]) +
                              (double)(s_gxp[t] + s_gxp[128 + t] + s_gxp[256 + t] + s_gxp[384 + t]);
            const double rw = s_rowp[t] + s_rowp[128 + t] + s_rowp[256 + t] + s_rowp[384 + t], dt = (double)s_dt[t];
            const double suf = (double)(s_syp[t] + s_syp[128 + t] + s_syp[256 + t] + s_syp[384 + t]);
            const double pre = fma(dt, cg, -rw);
            const double pre_in = ssm_warp_scan(pre), suf_in = ssm_warp_scan(suf);
            if (lane == 31) {
                s_tw[w4] = pre_in;
                s_tw[4 + w4] = suf_in;
            }
            asm volatile("bar.sync 1, 128;" ::: "memory");
            double before = pre_in - pre, after = suf - suf_in;
            double cross = 0.0;
#pragma unroll
            for (int w = 0; w < 16; ++w) cross += s_red[w];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                if (w < w4) before += s_tw[w];
                if (w >= w4) after += s_tw[4 + w];
            }
            const double dlog = before + after + cross * (double)s_g[SsmGate::elast];
            double raw = ((double)s_g[SsmGate::A] * dlog + cg + (double)s_diag[t]) * (double)s_g[SsmGate::sig + t], sA = 0.0, sD = 0.0;
            if (t < valid) {
                a.ddelta[((size_t)b * a.T + t0 + t) * a.H + h] = (float)raw;
                sA = dt * dlog;
                sD = (double)s_wd[t];
            } else {
                raw = 0.0;
            }
#pragma unroll
            for (int off = 16; off; off >>= 1) {
                sA += __shfl_xor_sync(0xffffffffu, sA, off);
                raw += __shfl_xor_sync(0xffffffffu, raw, off);
                sD += __shfl_xor_sync(0xffffffffu, sD, off);
            }
            if (lane == 0) {
                s_tot[w4 * 3] = sA;
                s_tot[w4 * 3 + 1] = raw;
                s_tot[w4 * 3 + 2] = sD;
            }
        }
        mma_sync_point();
        if (*abort_flag) break;
        // ---- dx, over G_out ----
        {
            const float w = s_g[SsmGate::el + row] * s_dt[row];
            const int c = prt * PW;
            float t[PW];
            tmem_ldw<PW>(tl + tT + c, t);
#pragma unroll
            for (int i = 0; i < PW; ++i) t[i] = fmaf(w, t[i], dxi[i]);
#pragma unroll
            for (int i = 0; i < PW / 8; ++i)
                st_bf16x8(sm + L::oR + (uint32_t)(c >> 6) * kTile + sw128_offset(row, ((c & 63) >> 3) + i), t + 8 * i);
        }
        fence_async_smem();
        tc_before_sync();
        __syncthreads();
        if (tid == kIo) {
            for (int i = 0; i < P / 64; ++i) tma_store_4d(&tm_dx, sm + L::oR + i * kTile, i * 64, h, t0, b);
            bulk_commit();
        }
        __syncwarp();
        if (tid < 3) part[tid * units + unit] = s_tot[tid] + s_tot[3 + tid] + s_tot[6 + tid] + s_tot[9 + tid];
    }
    if (*abort_flag) {
        if (tid == 0 && mma_open) mbar_wait(mma_bar, mma_phase ^ 1);
        if (tid == kIo) {
            record_status(GDR_ERR_TIMEOUT);
            mbar_wait(bar_bc, 0);
            mbar_wait(bar_x, (uint32_t)((n_x - 1) & 1));
            mbar_wait(bar_y, (uint32_t)((n_y - 1) & 1));
            mbar_wait(bar_g, (uint32_t)((n_g - 1) & 1));
            if (n_s > 0) mbar_wait(bar_s, (uint32_t)((n_s - 1) & 1));
            if (n_r > 0) mbar_wait(bar_r, (uint32_t)((n_r - 1) & 1));
            bulk_wait_all();
        }
    } else {
        tc_after_sync();
        const bool on = row < valid;
        const size_t at = (((size_t)b * a.T + t0 + row) * a.G + g);
        const int c = prt * NW;
#pragma unroll 1
        for (int which = 0; which < 2; ++which) {
            float v[NW];
            tmem_ldw<NW>(tl + (which ? tB : tC) + c, v);
            if (!on) continue;
            if (splits == 1) {
                uint8_t *dst = reinterpret_cast<uint8_t *>(static_cast<__nv_bfloat16 *>(which ? a.dB : a.dC) + at * N + c);
#pragma unroll
                for (int i = 0; i < NW / 8; ++i) st_bf16x8(dst + 16 * i, v + 8 * i);
            } else {
                float4 *dst = reinterpret_cast<float4 *>((which ? dBp : dCp) + (at * splits + sp) * N + c);
#pragma unroll
                for (int i = 0; i < NW / 4; ++i) dst[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            }
        }
    }
    if (tid == kIo) bulk_wait_all();
    tc_before_sync();
    __syncthreads();
    if (warp == 0) {
        tc_after_sync();
        tmem_dealloc(tmem, 512);
    }
}

// ---- host side ------------------------------------------------------------------------------
// CTAs per group of heads: a CTA costs about half a head's time beside its heads (the first loads, dB and dC), and with
// several of them partial sums in fp32 and a launch that adds them.  Measured: B=4 T=4096 H=16 P=N=128, one CTA 440 us (two:
// 466); B=1 T=4096, four 174 us (eight: 188, two: 241); B=2 T=1024 H=4 G=2 P=64, two 62 us (one: 70).
inline int ssm_grad_splits(int B, int T, int H, int G) {
    const int nch = (T + kTcQ - 1) / kTcQ, HG = H / G, sms = sm_count();
    int best = 1;
    double cost = -1;
    for (int s = 1; s <= HG; ++s) {
        const int per = (HG + s - 1) / s;
        if ((HG + per - 1) / per != s) continue;
        const double c = (double)(((long long)B * nch * G * s + sms - 1) / sms) * (per + (s > 1 ? 0.7 : 0.5)) + (s > 1 ? 0.3 : 0.0);
        if (cost < 0 || c < cost) {
            cost = c;
            best = s;
        }
    }
    return best;
}

// Chunks per segment of the walk: rounds of chunks over the SMs (one CTA each, both directions); a cut costs the
// segments' own sums first (a chunk there about 0.8 of one with its states written) and one to three launches.  Measured:
// B=4 T=4096 H=16 P=N=128, uncut 440 us (2 segments: 545); B=1 T=4096, 4 segments 173 us (1: 231, 8: 189); B=1 T=2048 H=8 P=64,
// 8 segments 66 us (1: 85, 4: 72, 16: 78).
inline int ssm_walk_chunks(int B, int T, int H) {
    const int nch = (T + kTcQ - 1) / kTcQ, sms = sm_count();
    double best = 1e30;
    int at = nch;
    for (int m = nch; m >= 1; m = m > 64 ? m * 3 / 4 : m - 1) {
        const int R = (nch + m - 1) / m;
        const double rounds = (double)((2LL * B * H * R + sms - 1) / sms);
        const double cost = R == 1 ? rounds * (m + 2.0) : rounds * (1.8 * m + 4.0) + (R > kJoinMost ? 4.0 : 1.0);
        if (cost < best * 0.999) {
            best = cost;
            at = m;
        }
    }
    return at;
}

struct SsmTcBwdWs {
    size_t gates, st, g, segS, segG, dec, part, dBp, dCp, total;
    int splits, m, R;
};
inline SsmTcBwdWs ssm_tc_bwd_ws(int B, int T, int H, int G, int P, int N) {
    const int nch = (T + kTcQ - 1) / kTcQ;
    const size_t units = (size_t)B * nch * H;
    SsmTcBwdWs w;
    w.splits = ssm_grad_splits(B, T, H, G);
    w.m = ssm_walk_chunks(B, T, H);
    w.R = (nch + w.m - 1) / w.m;
    const size_t segs = w.R > 1 ? (size_t)B * w.R * H : 0;
    w.gates = 0;
    w.st = ssm_gate_bytes(B, T, H);
    w.g = w.st + ssm_align(units * P * N * 4);
    w.segS = w.g + ssm_align(units * P * N * 4);
    w.segG = w.segS + ssm_align(segs * P * N * 4);
    w.dec = w.segG + ssm_align(segs * P * N * 4);
    w.part = w.dec + ssm_align(segs * 4);
    w.dBp = w.part + ssm_align(3 * units * 8);
    const size_t p = w.splits > 1 ? ssm_align((size_t)B * T * G * w.splits * N * 4) : 0;
    w.dCp = w.dBp + p;
    w.total = w.dCp + p;
    return w;
}

template <int P, int N>
cudaError_t ssm_tc_bwd(const SsmArgs &a, void *ws, cudaStream_t s) {
    const int nch = (a.T + kTcQ - 1) / kTcQ;
    const SsmTcBwdWs w = ssm_tc_bwd_ws(a.B, a.T, a.H, a.G, P, N);
    uint8_t *base = static_cast<uint8_t *>(ws);
    float4 *st = reinterpret_cast<float4 *>(base + w.st), *g = reinterpret_cast<float4 *>(base + w.g);
    float *segS = reinterpret_cast<float *>(base + w.segS), *segG = reinterpret_cast<float *>(base + w.segG);
    float *dec = reinterpret_cast<float *>(base + w.dec);
    double *part = reinterpret_cast<double *>(base + w.part);
    float *dBp = reinterpret_cast<float *>(base + w.dBp), *dCp = reinterpret_cast<float *>(base + w.dCp);
    float *gates = reinterpret_cast<float *>(base + w.gates);
    CUtensorMap mx, mb, mc, my, mdx;
    if (!ssm_token_map(&mx, a.x, a.B, a.T, a.H, P, a.ldx) || !ssm_token_map(&mb, a.Bm, a.B, a.T, a.G, N, a.ldb) ||
        !ssm_token_map(&mc, a.Cm, a.B, a.T, a.G, N, a.ldc) || !ssm_token_map(&my, a.dy, a.B, a.T, a.H, P, a.H * P) ||
        !ssm_token_map(&mdx, a.dx, a.B, a.T, a.H, P, a.H * P))
        return cudaErrorInvalidValue;
    cudaError_t e = ssm_launch_gates(a, gates, s);
    const dim3 grid(2u * (unsigned)(a.B * a.H) * (unsigned)w.R);
    const size_t smem = SsmWalkTc<P, N>::kAlloc;
    if (e == cudaSuccess && w.R > 1) {
        e = ssm_launch(ssm_tc_walk_kernel<P, N, false>, grid, SsmWalkTc<P, N>::kThreads, smem, s, mx, mb, my, mc, a, w.m, 2,
                       (const float *)gates, st, g, segS, segG, dec);
        if (e == cudaSuccess && w.R > kJoinMost) {
            e = ssm_launch_scan(false, a.B, w.R, a.H, P * N, segS, dec, a.S0, nullptr, s);
            if (e == cudaSuccess) e = ssm_launch_scan(true, a.B, w.R, a.H, P * N, segG, dec, a.dS_T, nullptr, s);
        }
    }
    if (e == cudaSuccess)
        e = ssm_launch(ssm_tc_walk_kernel<P, N, true>, grid, SsmWalkTc<P, N>::kThreads, smem, s, mx, mb, my, mc, a, w.m, 2,
                       (const float *)gates, st, g, segS, segG, dec);
    const int per = (a.H / a.G + w.splits - 1) / w.splits;
    if (e == cudaSuccess)
        e = ssm_launch(ssm_tc_grad_kernel<P, N>, dim3((unsigned)((size_t)a.B * nch * a.G * w.splits)), kGradThreads,
                       (size_t)SsmGradTc<P, N>::kAlloc, s, mx, mb, mc, my, mdx, a, w.splits, per,
                       (const float *)gates, (const float4 *)st, (const float4 *)g, dBp, dCp, part);
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

// ssm_tc.cuh -- the selective scan's forward on the 5th-generation tensor
// cores (tcgen05 + TMEM + TMA), bf16 inputs, P, N in {64, 128}, fp32 state.
//
// Chunks of Q = 128 tokens (ssm_common.cuh has the formulas).  Products of one
// chunk and head, tokens or state rows on the 128 TMEM lanes:
//     K  = C B^T                      M = 128 (i)   N = 128 (j)  K = N
//     Y2 = C S_in^T                   M = 128 (i)   N = P        K = N
//     Y1 = (K * L Delta) X            M = 128 (i)   N = P        K = 128 (j)
//     S  = e^{c_last} S + (w B)^T X   M = 128 (n)   N = P        K = 128 (j)
//     y  = Y1 + e^{c_i} Y2 + D x,     w_j = e^{c_last - c_j} Delta_j
// Roundings to bf16: the decayed scores (K * L Delta), the entering state as
// the operand of Y2, and w B.  The state itself stays fp32 in TMEM, and where
// it is an output w B is split into two bf16 parts (its rounding is then below
// 2^-17), so that S_T is exact to fp32 sums.
//
// The decay e^{c_i - c_j} of a pair in different 32-token blocks is the product
// of a row and a column factor around the later block's start (both <= 1 for a
// decaying state, so a product underflows only where the decay does); only the
// four diagonal blocks take an exponential per pair.
//
// A long sequence over few heads is cut into segments of whole chunks:
//   1. ssm_tc_state_kernel  sum_j w_j x_j B_j^T of a segment (one product over
//      its tokens: the weights reach to the segment's end)
//   2. ssm_scan_kernel      the states between the segments, elementwise, fp32
//   3. ssm_tc_y_kernel      walks its segment from that state
// One segment alone is a single launch (3 with the state written at its end).
#pragma once
#include <cuda.h>

#include "sm100.cuh"
#include "ssm_common.cuh"
#include "ssm_simt.cuh"

namespace gdr {

constexpr int kTcQ = 128;
constexpr uint32_t kTile = 128 * 128;  // 128 rows x 64 bf16, 128B swizzle

// ---- tensor maps ----------------------------------------------------------------------
typedef CUresult (*SsmEncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline SsmEncodeFn ssm_encode_fn() {
    static SsmEncodeFn fn = nullptr;
    if (!fn) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<SsmEncodeFn>(p);
    }
    return fn;
}
// [B, T, heads, d] bf16 with token stride ld: boxes of 64 channels x 1 head x 128 tokens; tokens past T read as
// zero and are not written.
inline bool ssm_token_map(CUtensorMap *map, const void *base, int B, int T, int heads, int d, int ld) {
    SsmEncodeFn enc = ssm_encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)T, (cuuint64_t)B};
    const cuuint64_t strides[3] = {(cuuint64_t)d * 2, (cuuint64_t)ld * 2, (cuuint64_t)T * ld * 2};
    const cuuint32_t box[4] = {64, 1, kTcQ, 1}, estr[4] = {1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ---- operands -------------------------------------------------------------------------
// Step kk (16 of the summed index) of a K-major tile (rows: M or N; blocks of 64 columns `block` bytes apart).
__device__ __forceinline__ uint64_t desc_k(uint32_t base, int kk, uint32_t block = kTile) {
    return sm100::smem_desc_sw128(base + (uint32_t)(kk >> 2) * block + (uint32_t)(kk & 3) * 32, 16, 1024);
}
// The same of an MN-major tile (rows: the summed index).
__device__ __forceinline__ uint64_t desc_mn(uint32_t base, int kk, uint32_t block = kTile) {
    return sm100::smem_desc_sw128(base + (uint32_t)kk * 2048, block, 1024);
}

// 8 bf16 of a 16-byte chunk times w.
__device__ __forceinline__ void ld8s(const uint8_t *p, float *v) {
    load8(reinterpret_cast<const __nv_bfloat16 *>(p), v);
}
// v as two bf16 parts: v = hi + lo up to 2^-17 |v|.
__device__ __forceinline__ void st_split8(uint8_t *hi, uint8_t *lo, float *v) {
    float r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = v[i] - __bfloat162float(__float2bfloat16_rn(v[i]));
    sm100::st_bf16x8(hi, v);
    sm100::st_bf16x8(lo, r);
}

// One warp: Delta and c (log2 units, 64 bits) of 128 tokens from t0.
__device__ __forceinline__ void ssm_tc_gates(const SsmArgs &a, int b, int h, int t0, float *s_dt, double *s_c) {
    ssm_gates<kTcQ>(a, b, h, t0, s_dt, s_c);
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int e = 0; e < 4; ++e) s_c[lane * 4 + e] *= 1.4426950408889634074;
}

// ---- 1. segment states ------------------------------------------------------------------
// BWD: sum_i e^{c_i} dy_i C_i^T with c from the segment's start.  out[b][seg][h][P][N], dec[b][seg][h].
template <int P, int N, bool BWD>
struct SsmStateTc {
    static constexpr uint32_t XB = P / 64 * kTile, BB = N / 64 * kTile;
    static constexpr uint32_t oX = 0, oB = XB, oHi = oB + BB, oLo = oHi + BB, oZero = oLo + BB;
    static constexpr uint32_t kHiBlock = N == 64 ? 2 * kTile : kTile;  // distance of the second 64 lanes
    static constexpr uint32_t oCtl = oZero + (N == 64 ? kTile : 0);
    static constexpr uint32_t kAlloc = oCtl + 128 * 4 + 128 * 8 + 128 + 1024;
};

template <int P, int N, bool BWD>
__global__ void __launch_bounds__(256) ssm_tc_state_kernel(const __grid_constant__ CUtensorMap tm_x,
                                                           const __grid_constant__ CUtensorMap tm_b, SsmArgs a, int m,
                                                           float *__restrict__ out, float *__restrict__ dec) {
    using L = SsmStateTc<P, N, BWD>;
    using namespace sm100;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const uint32_t sb = smem_u32(sm);
    double *s_c = reinterpret_cast<double *>(sm + L::oCtl);
    float *s_dt = reinterpret_cast<float *>(s_c + 128);
    uint64_t *tma_bar = reinterpret_cast<uint64_t *>(s_dt + 128), *mma_bar = tma_bar + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(tma_bar + 2);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int tid = threadIdx.x, warp = tid >> 5;
    const int nch = (a.T + kTcQ - 1) / kTcQ, R = (nch + m - 1) / m;
    const int seg = blockIdx.x % R, bh = blockIdx.x / R, h = bh % a.H, b = bh / a.H, g = h / (a.H / a.G);
    const int c0 = seg * m, cn = min(m, nch - c0);

    if (tid == 0) {
        mbar_init(tma_bar, 1);
        mbar_init(mma_bar, 1);
        fence_mbar_init();
        *abort_flag = 0;
    }
    if (warp == 0) tmem_alloc(tmem_slot, P);
    if (N == 64)
        for (int i = tid; i < (int)kTile / 16; i += 256) reinterpret_cast<uint4 *>(sm + L::oZero)[i] = make_uint4(0, 0, 0, 0);
    fence_async_smem();
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    const uint32_t tmem = *tmem_slot;

    // forward: chunks from the last, so that the decay to the segment's end is known; backward: from the first
    auto chunk = [&](int k) { return BWD ? c0 + k : c0 + cn - 1 - k; };
    auto issue = [&](int k) {
        mbar_expect_tx(tma_bar, L::XB + L::BB);
        for (int i = 0; i < P / 64; ++i) tma_load_4d(sm + L::oX + i * kTile, &tm_x, tma_bar, i * 64, h, chunk(k) * kTcQ, b);
        for (int i = 0; i < N / 64; ++i) tma_load_4d(sm + L::oB + i * kTile, &tm_b, tma_bar, i * 64, g, chunk(k) * kTcQ, b);
    };
    if (tid == 0) issue(0);
    double edge = 0.0;  // log2 decay between this chunk and the segment's end (start for BWD)
    bool pending = false;
    int k = 0;
#pragma unroll 1
    for (; k < cn; ++k) {
        if (warp == 1) ssm_tc_gates(a, b, h, chunk(k) * kTcQ, s_dt, s_c);
        if (tid == 0 && !mbar_wait(tma_bar, (uint32_t)(k & 1))) *abort_flag = 1;
        __syncthreads();
        if (*abort_flag) break;
        {   // the weighted rows in two bf16 parts: row tid & 127, half of the columns
            const int r = tid & 127, half = tid >> 7;
            const double last = s_c[127];
            const float w = BWD ? exp2f((float)(s_c[r] + edge)) : s_dt[r] * exp2f((float)(last - s_c[r] + edge));
            edge += last;
            constexpr int CH = N / 16;  // 16-byte chunks of a half row
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int c = half * CH + i;
                const uint32_t off = (uint32_t)(c >> 3) * kTile + sw128_offset(r, c & 7);
                float v[8];
                ld8s(sm + L::oB + off, v);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] *= w;
                st_split8(sm + L::oHi + off, sm + L::oLo + off, v);
            }
        }
        fence_async_smem();
        __syncthreads();
        if (tid == 0) {
            tc_after_sync();
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    mma_bf16(tmem, desc_mn(sb + (part ? L::oLo : L::oHi), kk, part ? kTile : L::kHiBlock),
                             desc_mn(sb + L::oX, kk), idesc_bf16(128, P, true, true), k > 0 || part > 0 || kk > 0);
            mma_commit(mma_bar);
            if (!mbar_wait(mma_bar, (uint32_t)(k & 1))) {
                *abort_flag = 1;
                pending = true;
            } else if (k + 1 < cn) {
                issue(k + 1);
            }
        }
        __syncthreads();
        if (*abort_flag) break;
    }
    if (*abort_flag) {
        if (tid == 0) {
            record_status(GDR_ERR_TIMEOUT);
            // one wait more for what is still in flight: the chunk's copies, or its products
            mbar_wait(pending ? mma_bar : tma_bar, (uint32_t)(k & 1));
        }
    } else {
        tc_after_sync();
        const int n = (warp & 3) * 32 + (tid & 31), half = warp >> 2;
        const size_t unit = ((size_t)b * R + seg) * a.H + h;
        if ((warp & 3) * 32 < N) {
#pragma unroll 1
            for (int c = half * (P / 2); c < (half + 1) * (P / 2); c += 32) {
                float v[32];
                tmem_ld32(tmem + ((uint32_t)((warp & 3) * 32) << 16) + c, v);
#pragma unroll
                for (int i = 0; i < 32; ++i) out[(unit * P + c + i) * N + n] = v[i];
            }
        }
        if (!BWD && tid == 0) dec[unit] = exp2f((float)edge);
    }
    tc_before_sync();
    __syncthreads();
    if (warp == 0) {
        tc_after_sync();
        tmem_dealloc(tmem, P);
    }
}

// ---- 3. outputs ------------------------------------------------------------------------------
// LO: the state's own product takes both parts of w B, and S_T is written at the end (one segment).
template <int P, int N, bool LO>
struct SsmYTc {
    static constexpr uint32_t XB = P / 64 * kTile, BB = N / 64 * kTile;
    static constexpr uint32_t oX = 0, oB = XB, oLo = oB + BB, oZero = oLo + (LO ? BB : 0);
    static constexpr uint32_t kHiBlock = N == 64 ? (LO ? 2 : 1) * kTile : kTile;
    static constexpr uint32_t oC = oZero + (N == 64 ? kTile : 0);  // C, then the decayed scores
    static constexpr uint32_t kSBlock = N * 128;                   // S^T: N rows of 64 columns p
    static constexpr uint32_t oS = oC + 2 * kTile;
    static constexpr uint32_t oGate = oS + P / 64 * kSBlock;
    // doubles c[2][128]; floats dt[2][128], e[128], row[128], w[128], col[3][96], hi[128], lo[128]
    static constexpr uint32_t kGate = 2 * 128 * 8 + (2 * 128 + 3 * 128 + 3 * 96 + 2 * 128) * 4;
    static constexpr uint32_t oBar = oGate + kGate;
    static constexpr uint32_t kAlloc = oBar + 64 + 1024;
    static constexpr uint32_t kTmemCols = P == 64 ? 256 : 512;
};

// The tables of one chunk from its Delta and c (log2): e_i = 2^{c_i}, row factor 2^{c_i - r} (r: c at the end of
// the block of 32 before i's), w_j, column factors Delta_j 2^{r_I - c_j} of the blocks I = 1..3, and c in two parts
// (differences of nearby tokens are then exact to fp32 however far the sum has run).
__device__ __forceinline__ void ssm_tc_tables(const float *s_dt, const double *s_c, float *s_e, float *s_row, float *s_w,
                                              float *s_col, float *s_hi, float *s_lo) {
    const int tid = threadIdx.x;
    const double last = s_c[127];
    if (tid < 128) {
        const double c = s_c[tid];
        const double r = tid >= 32 ? s_c[(tid & ~31) - 1] : 0.0;
        s_e[tid] = exp2f((float)c);
        s_row[tid] = exp2f((float)(c - r));
        s_w[tid] = s_dt[tid] * exp2f((float)(last - c));
        const float hi = (float)c;
        s_hi[tid] = hi;
        s_lo[tid] = (float)(c - (double)hi);
    } else {
        for (int i = tid - 128; i < 192; i += 128) {  // 32 + 64 + 96 pairs (I, j < 32 I)
            const int I = i < 32 ? 1 : i < 96 ? 2 : 3, j = i < 32 ? i : i < 96 ? i - 32 : i - 96;
            s_col[(I - 1) * 96 + j] = s_dt[j] * exp2f((float)(s_c[32 * I - 1] - s_c[j]));
        }
    }
}

template <int P, int N, bool LO>
__global__ void __launch_bounds__(256, P == 64 && !LO ? 2 : 1) ssm_tc_y_kernel(const __grid_constant__ CUtensorMap tm_x,
                                                       const __grid_constant__ CUtensorMap tm_b,
                                                       const __grid_constant__ CUtensorMap tm_c,
                                                       const __grid_constant__ CUtensorMap tm_y, SsmArgs a, int m,
                                                       const float *__restrict__ states) {
    using L = SsmYTc<P, N, LO>;
    using namespace sm100;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const uint32_t sb = smem_u32(sm);
    double *s_c2 = reinterpret_cast<double *>(sm + L::oGate);
    float *s_dt2 = reinterpret_cast<float *>(s_c2 + 256);
    float *s_e = s_dt2 + 256, *s_row = s_e + 128, *s_w = s_row + 128, *s_col = s_w + 128, *s_hi = s_col + 288,
          *s_lo = s_hi + 128;
    uint64_t *bar_x = reinterpret_cast<uint64_t *>(sm + L::oBar), *bar_bc = bar_x + 1, *mma_bar = bar_x + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bar_x + 3);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int q = warp & 3, half = warp >> 2, row = q * 32 + lane;  // TMEM lane (token i or state row n), column half
    const int nch = (a.T + kTcQ - 1) / kTcQ, R = (nch + m - 1) / m;
    const int seg = blockIdx.x % R, bh = blockIdx.x / R, h = bh % a.H, b = bh / a.H, g = h / (a.H / a.G);
    const int c0 = seg * m, cn = min(m, nch - c0);

    if (tid == 0) {
        mbar_init(bar_x, 1);
        mbar_init(bar_bc, 1);
        mbar_init(mma_bar, 1);
        fence_mbar_init();
        *abort_flag = 0;
    }
    if (warp == 0) tmem_alloc(tmem_slot, L::kTmemCols);
    if (N == 64)
        for (int i = tid; i < (int)kTile / 16; i += 256) reinterpret_cast<uint4 *>(sm + L::oZero)[i] = make_uint4(0, 0, 0, 0);
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    const uint32_t tmem = *tmem_slot;
    const uint32_t tl = tmem + ((uint32_t)(q * 32) << 16);
    constexpr uint32_t tK = 0, tY2 = 128, tS = 128 + P;  // Y1 takes K's columns once K is read

    auto issue_bc = [&](int k) {
        mbar_expect_tx(bar_bc, 2 * L::BB);
        for (int i = 0; i < N / 64; ++i) {
            tma_load_4d(sm + L::oB + i * kTile, &tm_b, bar_bc, i * 64, g, (c0 + k) * kTcQ, b);
            tma_load_4d(sm + L::oC + i * kTile, &tm_c, bar_bc, i * 64, g, (c0 + k) * kTcQ, b);
        }
    };
    auto issue_x = [&](int k) {
        mbar_expect_tx(bar_x, L::XB);
        for (int i = 0; i < P / 64; ++i) tma_load_4d(sm + L::oX + i * kTile, &tm_x, bar_x, i * 64, h, (c0 + k) * kTcQ, b);
    };
    int n_bc = 0, n_x = 0, d_bc = 0, d_x = 0;  // issued and awaited, by thread 0
    if (tid == 0) {
        issue_bc(0);
        issue_x(0);
        n_bc = n_x = 1;
    }
    if (warp == 1) ssm_tc_gates(a, b, h, c0 * kTcQ, s_dt2, s_c2);
    {   // the entering state: lane n, columns p
        const float *src = states ? states + (((size_t)b * R + seg) * a.H + h) * P * N : a.S0 ? a.S0 + (size_t)bh * P * N : nullptr;
#pragma unroll 1
        for (int c = half * (P / 2); c < (half + 1) * (P / 2); c += 32) {
            float v[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = src && row < N ? src[(size_t)(c + i) * N + row] : 0.f;
            tmem_st32(tl + tS + c, v);
        }
        tmem_wait_st();
    }
    uint32_t mma_phase = 0;
    bool mma_open = false;
    auto mma_sync_point = [&]() {
        if (tid == 0) {
            mma_commit(mma_bar);
            mma_open = !mbar_wait(mma_bar, mma_phase);
            if (mma_open) *abort_flag = 1;
        }
        mma_phase ^= 1;
        __syncthreads();
        tc_after_sync();
    };
    const float D = a.D ? a.D[h] : 0.f;
    __syncthreads();

#pragma unroll 1
    for (int k = 0; k < cn; ++k) {
        const double *s_c = s_c2 + (k & 1) * 128;
        const float *s_dt = s_dt2 + (k & 1) * 128;
        ssm_tc_tables(s_dt, s_c, s_e, s_row, s_w, s_col, s_hi, s_lo);
        if (row < N) {  // S^T as the bf16 operand [n][p]; the fp32 state decays to the chunk's end
            const float el = exp2f((float)s_c[127]);
#pragma unroll 1
            for (int c = half * (P / 2); c < (half + 1) * (P / 2); c += 32) {
                float v[32];
                tmem_ld32(tl + tS + c, v);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    st_bf16x8(sm + L::oS + (c >> 6) * L::kSBlock + sw128_offset(row, ((c & 63) >> 3) + i), v + 8 * i);
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] *= el;
                tmem_st32(tl + tS + c, v);
            }
            tmem_wait_st();
        }
        if (tid == 0) {
            if (!mbar_wait(bar_bc, (uint32_t)(k & 1))) *abort_flag = 1;
            else ++d_bc;
        }
        fence_async_smem();
        tc_before_sync();
        __syncthreads();
        if (*abort_flag) break;
        if (tid == 0) {
            tc_after_sync();
#pragma unroll
            for (int kk = 0; kk < N / 16; ++kk)
                mma_bf16(tmem + tK, desc_k(sb + L::oC, kk), desc_k(sb + L::oB, kk), idesc_bf16(128, 128, false, false), kk > 0);
#pragma unroll
            for (int kk = 0; kk < N / 16; ++kk)
                mma_bf16(tmem + tY2, desc_k(sb + L::oC, kk), desc_mn(sb + L::oS, kk, L::kSBlock),
                         idesc_bf16(128, P, false, true), kk > 0);
        }
        if (warp == 1 && k + 1 < cn)
            ssm_tc_gates(a, b, h, (c0 + k + 1) * kTcQ, s_dt2 + ((k + 1) & 1) * 128, s_c2 + ((k + 1) & 1) * 128);
        mma_sync_point();
        if (*abort_flag) break;

        // decayed scores -> bf16 [i][j] over C (C's products are done)
        const float rf = s_row[row], ci = s_hi[row], cl = s_lo[row];
#pragma unroll
        for (int jb = 0; jb < 2; ++jb) {
            const int J = half * 2 + jb;  // 32-column block
            uint8_t *dst = sm + L::oC + half * kTile;
            float v[32];
            if (J > q) {
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = 0.f;
            } else {
                tmem_ld32(tl + tK + J * 32, v);
                if (J < q) {
                    const float *col = s_col + (q - 1) * 96 + J * 32;
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] *= rf * col[i];
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const int j = J * 32 + i;
                        const float e = exp2f((ci - s_hi[j]) + (cl - s_lo[j])) * s_dt[j];
                        v[i] = i <= lane ? v[i] * e : 0.f;
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) st_bf16x8(dst + sw128_offset(row, jb * 4 + i), v + 8 * i);
        }
        if (LO || k + 1 < cn) {  // w B in place (B's product is done), its second part beside it
            const int r = tid & 127;
            const float w = s_w[r];
            constexpr int CH = N / 16;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int c = (tid >> 7) * CH + i;
                uint8_t *p = sm + L::oB + (uint32_t)(c >> 3) * kTile + sw128_offset(r, c & 7);
                float v[8];
                ld8s(p, v);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] *= w;
                if (LO) st_split8(p, p + L::BB, v);
                else st_bf16x8(p, v);
            }
        }
        if (tid == 0) {
            if (!mbar_wait(bar_x, (uint32_t)(k & 1))) *abort_flag = 1;
            else ++d_x;
        }
        fence_async_smem();
        tc_before_sync();
        __syncthreads();
        if (*abort_flag) break;
        if (tid == 0) {
            tc_after_sync();
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
                mma_bf16(tmem + tK, desc_k(sb + L::oC, kk), desc_mn(sb + L::oX, kk), idesc_bf16(128, P, false, true), kk > 0);
            if (LO || k + 1 < cn) {
#pragma unroll
                for (int part = 0; part < (LO ? 2 : 1); ++part)
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        mma_bf16(tmem + tS, desc_mn(sb + (part ? L::oLo : L::oB), kk, part ? kTile : L::kHiBlock),
                                 desc_mn(sb + L::oX, kk), idesc_bf16(128, P, true, true), 1);
            }
        }
        mma_sync_point();
        if (*abort_flag) break;
        if (tid == 0 && k + 1 < cn) {
            issue_bc(k + 1);
            ++n_bc;
        }
        {   // y = Y1 + e^{c_i} Y2 + D x over the x tile
            const float e = s_e[row];
#pragma unroll 1
            for (int c = half * (P / 2); c < (half + 1) * (P / 2); c += 32) {
                float y1[32], y2[32];
                tmem_ld32(tl + tK + c, y1);
                tmem_ld32(tl + tY2 + c, y2);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint8_t *p = sm + L::oX + (uint32_t)(c >> 6) * kTile + sw128_offset(row, ((c & 63) >> 3) + i);
                    float x[8];
                    ld8s(p, x);
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        const float y = fmaf(e, y2[8 * i + u], y1[8 * i + u]);
                        x[u] = a.D ? fmaf(D, x[u], y) : y;
                    }
                    st_bf16x8(p, x);
                }
            }
        }
        fence_async_smem();
        tc_before_sync();
        __syncthreads();
        if (tid == 0) {
            for (int i = 0; i < P / 64; ++i) tma_store_4d(&tm_y, sm + L::oX + i * kTile, i * 64, h, (c0 + k) * kTcQ, b);
            bulk_commit();
            bulk_wait_read_all();
            if (k + 1 < cn) {
                issue_x(k + 1);
                ++n_x;
            }
        }
    }
    if (*abort_flag) {
        if (tid == 0) {  // wait, bounded, for what is still in flight
            record_status(GDR_ERR_TIMEOUT);
            if (d_bc < n_bc) mbar_wait(bar_bc, (uint32_t)(d_bc & 1));
            if (d_x < n_x) mbar_wait(bar_x, (uint32_t)(d_x & 1));
            if (mma_open) mbar_wait(mma_bar, mma_phase ^ 1);
            bulk_wait_all();
        }
    } else {
        if (LO && a.S_T && row < N) {
            float *dst = a.S_T + (size_t)bh * P * N;
#pragma unroll 1
            for (int c = half * (P / 2); c < (half + 1) * (P / 2); c += 32) {
                float v[32];
                tmem_ld32(tl + tS + c, v);
#pragma unroll
                for (int i = 0; i < 32; ++i) dst[(size_t)(c + i) * N + row] = v[i];
            }
        }
        if (tid == 0) bulk_wait_all();
    }
    tc_before_sync();
    __syncthreads();
    if (warp == 0) {
        tc_after_sync();
        tmem_dealloc(tmem, L::kTmemCols);
    }
}

// ---- host side ------------------------------------------------------------------------------
inline int ssm_sm_count() {
    static int n = 0;
    if (n == 0) {
        int dev = 0, v = 0;
        if (cudaGetDevice(&dev) == cudaSuccess &&
            cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess)
            n = v;
        else
            return 148;
    }
    return n;
}

// Chunks per segment: the fewest rounds of chunks over the SMs' places, where an extra segment costs its state's
// traffic (about a fifth of a chunk's time in each of the launches).
inline int ssm_tc_chunks(int B, int T, int H, int P) {
    const int nch = (T + kTcQ - 1) / kTcQ, places = ssm_sm_count() * (P == 64 ? 2 : 1);
    double best = 1e30;
    int at = nch;
    for (int m = nch; m >= 1; m = m > 64 ? m * 3 / 4 : m - 1) {
        const int R = (nch + m - 1) / m;
        const double rounds = (double)(((long long)B * H * R + places - 1) / places);
        const double cost = R == 1 ? rounds * m : rounds * (1.4 * m + 1.0) + 2.0;
        if (cost < best * 0.999) {
            best = cost;
            at = m;
        }
    }
    return at;
}

struct SsmTcFwdWs {
    size_t st, dec, total;
};
inline SsmTcFwdWs ssm_tc_fwd_ws(int B, int T, int H, int P, int N) {
    const int m = ssm_tc_chunks(B, T, H, P), nch = (T + kTcQ - 1) / kTcQ, R = (nch + m - 1) / m;
    SsmTcFwdWs w{};
    if (R == 1) return w;
    const size_t units = (size_t)B * R * H;
    w.dec = ssm_align(units * P * N * 4);
    w.total = w.dec + ssm_align(units * 4);
    return w;
}

template <int P, int N>
cudaError_t ssm_tc_fwd(const SsmArgs &a, void *ws, cudaStream_t s) {
    CUtensorMap mx, mb, mc, my;
    if (!ssm_token_map(&mx, a.x, a.B, a.T, a.H, P, a.ldx) || !ssm_token_map(&mb, a.Bm, a.B, a.T, a.G, N, a.ldb) ||
        !ssm_token_map(&mc, a.Cm, a.B, a.T, a.G, N, a.ldc) || !ssm_token_map(&my, a.y, a.B, a.T, a.H, P, a.H * P))
        return cudaErrorInvalidValue;
    const int m = ssm_tc_chunks(a.B, a.T, a.H, P), nch = (a.T + kTcQ - 1) / kTcQ, R = (nch + m - 1) / m;
    const dim3 grid((unsigned)(a.B * a.H) * (unsigned)R);
    if (R == 1)
        return ssm_launch(ssm_tc_y_kernel<P, N, true>, grid, 256, (size_t)SsmYTc<P, N, true>::kAlloc, s, mx, mb, mc, my, a, m,
                          (const float *)nullptr);
    const SsmTcFwdWs w = ssm_tc_fwd_ws(a.B, a.T, a.H, P, N);
    float *st = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + w.st);
    float *dec = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + w.dec);
    cudaError_t e = ssm_launch(ssm_tc_state_kernel<P, N, false>, grid, 256, (size_t)SsmStateTc<P, N, false>::kAlloc, s, mx, mb,
                               a, m, st, dec);
    if (e == cudaSuccess) e = ssm_launch_scan(false, a.B, R, a.H, P * N, st, dec, a.S0, a.S_T, s);
    if (e == cudaSuccess)
        e = ssm_launch(ssm_tc_y_kernel<P, N, false>, grid, 256, (size_t)SsmYTc<P, N, false>::kAlloc, s, mx, mb, mc, my, a, m,
                       (const float *)st);
    return e;
}

}  // namespace gdr

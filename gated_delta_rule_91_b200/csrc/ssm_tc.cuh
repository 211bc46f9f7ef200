// ssm_tc.cuh -- the selective scan's forward on the 5th-generation tensor
// cores (tcgen05 + TMEM + TMA), bf16 inputs, P, N in {64, 128}, fp32 state.
//
// Chunks of Q = 128 tokens (ssm_common.cuh has the formulas).  Products of one
// chunk and head, tokens or state rows on the 128 TMEM lanes:
//     K  = C B^T                      M = 128 (i)   N = 128 (j)  K = N
//     Y2 = C S_in^T                   M = 128 (i)   N = P        K = N
//     Y1 = (K * L Delta) X            M = 128 (i)   N = P        K = 128 (j)
//     U  = B^T (w X)                  M = 128 (n)   N = P        K = 128 (j)
//     y  = Y1 + e^{c_i} Y2 + D x,     S = e^{c_last} S + U,      w_j = e^{c_last - c_j} Delta_j
// x, B and C are bf16 themselves; an operand that is not enters as bf16 parts, each the rounding of what the ones before
// it left: two (2^-17 of a term, below the rounding of y) for the decayed scores, the entering state and, where only y
// reads the state, w X; three (2^-26) for w X where the state leaves in fp32.  S_T is then 1.3e-7 off 64 bits at B=4
// T=4096 H=16 P=N=128 and y one rounding (1.7e-3).  With one part for y and two for S_T (2.5e-6 and 1.7e-3, y 1.4e-3
// from its fp32 value) the call takes 136 us, not 173.  A chunk's U has an accumulator of its own, its small parts
// first: summed onto a long memory's state, whose every accumulation the tensor core truncates, S_T was 2.5e-6 off.
//
// The decay e^{c_i - c_j} of a pair in different 32-token blocks is the product
// of a row and a column factor around the later block's start (both <= 1 for a
// decaying state, so a product underflows only where the decay does); only the
// four diagonal blocks take an exponential per pair.
//
//   0. ssm_gate_kernel      the decays of every chunk and head as tables
// A long sequence over few heads is cut into segments of whole chunks:
//   1. ssm_tc_walk_kernel   a segment's own sum of w_j x_j B_j^T, decayed to its end
//   2. ssm_scan_kernel      the states between many segments, elementwise, fp32
//   3. ssm_tc_y_kernel      walks its segment from that state
// One segment alone is 0 and 3, with the state written at its end.
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
    static std::atomic<SsmEncodeFn> known{nullptr};  // several threads may ask first
    SsmEncodeFn fn = known.load(std::memory_order_relaxed);
    if (!fn) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<SsmEncodeFn>(p);
        known.store(fn, std::memory_order_relaxed);
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
    return encode_map(enc, map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
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
// ---- 0. gates ---------------------------------------------------------------------------
// One table per unit = (b, chunk, head), read by the other kernels as one bulk copy: computed in place by a warp of
// each of them, the softplus and the 64-bit sums took 4600 of a chunk's 9100 cycles.  Floats at:
struct SsmGate {
    static constexpr int dt = 0, e = 128, rowf = 256, el = 384, hi = 512, lo = 640;  // per token, see below
    static constexpr int col = 768;                       // [I-1][96]: 2^{r_I - c_j} of the blocks I = 1..3, j < 32 I
    static constexpr int last = 1056, elast = 1058;       // c_last (a double) and 2^{c_last}
    static constexpr int A = 1059, D = 1060;              // the head's (D: 0 without one)
    static constexpr int misc = 1056, sig = 1072;         // (the last five: one copy of 64 bytes); d softplus / dz
    static constexpr int w = 1200, stride = 1328;         // dt el
    static constexpr uint32_t kFwdBytes = sig * 4, kBytes = w * 4;
};
// With c the sums in log2 units: e = 2^c, rowf = 2^{c - r} (r: c at the end of the block of 32 before the token's), el =
// 2^{c_last - c}, and c in two parts (differences of nearby tokens are then exact to fp32 however far the sum has run).
__global__ void __launch_bounds__(128) ssm_gate_kernel(SsmArgs a, float *__restrict__ gates) {
    __shared__ double s_w[4];
    const int nch = (a.T + kTcQ - 1) / kTcQ, t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int h = blockIdx.x % a.H, bc = blockIdx.x / a.H, ch = bc % nch, b = bc / nch, tok = ch * kTcQ + t;
    float *out = gates + (size_t)blockIdx.x * SsmGate::stride;
    float z = 0.f, d = 0.f;
    if (tok < a.T) {
        z = a.delta[((size_t)b * a.T + tok) * a.H + h];
        if (a.bias) z += a.bias[h];
        d = a.softplus ? ssm_softplus(z) : z;
    }
    // 2^-1e6 is 0 and 2^1e6 infinite in any case; without the bound a sum past the float range has no first part (a NaN stays)
    double c_in = (double)a.A[h] * (double)d * 1.4426950408889634074;
    if (c_in < -1e6) c_in = -1e6;
    if (c_in > 1e6) c_in = 1e6;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const double o = __shfl_up_sync(0xffffffffu, c_in, off);
        if (lane >= off) c_in += o;
    }
    if (lane == 31) s_w[warp] = c_in;
    __syncthreads();
    double r = 0.0;
    for (int w = 0; w < warp; ++w) r += s_w[w];
    const double c = r + c_in, last = s_w[0] + s_w[1] + s_w[2] + s_w[3];
    const float hi = (float)c;
    out[SsmGate::dt + t] = d;
    out[SsmGate::e + t] = exp2f(hi);
    out[SsmGate::rowf + t] = exp2f((float)c_in);
    out[SsmGate::el + t] = exp2f((float)(last - c));
    out[SsmGate::hi + t] = hi;
    out[SsmGate::lo + t] = (float)(c - (double)hi);
    out[SsmGate::w + t] = d * exp2f((float)(last - c));
    out[SsmGate::sig + t] = a.softplus ? 1.f / (1.f + expf(-z)) : 1.f;
    for (int I = warp + 1; I < 4; ++I) {
        r += s_w[I - 1];
        out[SsmGate::col + (I - 1) * 96 + t] = exp2f((float)(r - c));
    }
    if (t == 0) {
        *reinterpret_cast<double *>(out + SsmGate::last) = last;
        out[SsmGate::elast] = exp2f((float)last);
        out[SsmGate::A] = a.A[h];
        out[SsmGate::D] = a.D ? a.D[h] : 0.f;
    }
}

// ---- 1. walks over the chunks ------------------------------------------------------------
// Up to this many segments are joined by every reader itself (it reads the sums of the segments before its own);
// ssm_scan_kernel joins more.  B=4 T=4096 H=16 P=N=128, 2 segments: 173 us, with the scan's launch 182 us; B=1, 8
// segments: 58 us and 60 us.
constexpr int kJoinMost = 8;

// The state entering segment seg (leaving it, rev), columns cp .. cp + W - 1 of row n: from the scanned segments, or
// joined here from the segments' own sums and decays.
template <int W, int P, int N>
__device__ __forceinline__ void ssm_enter_segment(float (&v)[W], const float *segs, const float *dec, const float *first,
                                                  int R, int seg, int b, int h, int H, int cp, int n, bool rev) {
    const bool on = n < N;
    auto load = [&](const float *src, float (&x)[W]) {
#pragma unroll
        for (int i = 0; i < W; ++i) x[i] = src && on ? src[(size_t)(cp + i) * N + n] : 0.f;
    };
    if (R > kJoinMost) {
        load(segs + (((size_t)b * R + seg) * H + h) * P * N, v);
        return;
    }
    load(first ? first + ((size_t)b * H + h) * P * N : nullptr, v);
    const int before = rev ? R - 1 - seg : seg;
#pragma unroll 1
    for (int k = 0; k < before; ++k) {
        const size_t unit = ((size_t)b * R + (rev ? R - 1 - k : k)) * H + h;
        float x[W];
        load(segs + unit * P * N, x);
        const float d = dec[unit];
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = fmaf(d, v[i], x[i]);
    }
}

// A CTA walks the chunks of one (b, h, segment), forwards (S <- e^{c_last} S + B^T (w X)) or, rev, backwards (G <-
// e^{c_last} G + C^T (e^c dY)), the state in registers and a chunk's own sum in TMEM (lanes n, columns p, fp32), the
// weighted rows in three bf16 parts.
// OUT: from the state that enters the segment, every chunk's entering state is written to out_S or out_G (fp32,
// [unit][P / 4][N][4], unit = (b, chunk, head): a warp writes 512 bytes at once), and dS0 at the end.  Otherwise: from
// zero, the segment's own sum goes to seg_S or seg_G [b][seg][h][P][N], and its decay to dec.
// Two or three stages of operands: while a chunk's products run, the next chunk's rows are weighted.  At P = N = 128 the
// segments' sums of 16 chunks take 50 us (B=4 T=4096 H=16: 41 with two parts) and the states of 32 chunks 129 us (109 with
// two parts, whose states left as bf16 through shared memory; states stored row by row took 9400 cycles a chunk against 5600
// then).  What bounds it is the operands' way from L2, 64 KB a chunk and SM, and the states' to memory.
template <int P, int N>
struct SsmWalkTc {
    static constexpr int kThreads = 512, PW = P / 4;
    static constexpr int ST = P == 64 ? 3 : 2;                           // stages
    static constexpr uint32_t XB = P / 64 * kTile, BB = N / 64 * kTile, kStage = 2 * XB + BB;
    static constexpr uint32_t oX = 0, oLo = XB, oB = 2 * XB, oZero = ST * kStage;  // X, weighted in place; its second part
    static constexpr uint32_t oThird = oZero + (N == 64 ? kTile : 0);    // the third part: of one chunk at a time
    static constexpr uint32_t kGate = 128 * 4 + 64;                      // the rows' weights and the decay
    static constexpr uint32_t oGate = oThird + XB, oCtl = oGate + 2 * kGate;
    static constexpr uint32_t kAlloc = oCtl + 96 + 1024;
};

template <int P, int N, bool OUT>
__global__ void __launch_bounds__(512, 1) ssm_tc_walk_kernel(
    const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_b,
    const __grid_constant__ CUtensorMap tm_dy, const __grid_constant__ CUtensorMap tm_c, SsmArgs a, int m, int dirs,
    const float *__restrict__ gates, float4 *__restrict__ out_S, float4 *__restrict__ out_G, float *__restrict__ seg_S, float *__restrict__ seg_G, float *__restrict__ dec) {
    using L = SsmWalkTc<P, N>;
    using namespace sm100;
    constexpr int PW = L::PW;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const uint32_t sb = smem_u32(sm);
    constexpr int ST = L::ST;
    uint64_t *tma_bar = reinterpret_cast<uint64_t *>(sm + L::oCtl), *bar_g = tma_bar + ST, *mma_bar = bar_g + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(mma_bar + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int q = warp & 3, prt = warp >> 2, row = q * 32 + lane, cp = prt * PW;  // state row n, first column p
    const int nch = (a.T + kTcQ - 1) / kTcQ, R = (nch + m - 1) / m;
    int u = blockIdx.x;
    const bool rev = dirs == 2 && (u & 1);
    if (dirs == 2) u >>= 1;
    const int seg = u % R, bh = u / R, h = bh % a.H, b = bh / a.H, g = h / (a.H / a.G);
    const int c0 = seg * m, cn = min(m, nch - c0);
    auto chunk = [&](int k) { return rev ? c0 + cn - 1 - k : c0 + k; };

    if (tid == 0) {
        for (int i = 0; i < ST + 3; ++i) mbar_init(tma_bar + i, 1);
        fence_mbar_init();
        *abort_flag = 0;
    }
    if (warp == 0) tmem_alloc(tmem_slot, P);
    if (N == 64)
        for (int i = tid; i < (int)kTile / 16; i += 512) reinterpret_cast<uint4 *>(sm + L::oZero)[i] = make_uint4(0, 0, 0, 0);
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    const uint32_t tmem = *tmem_slot;
    const uint32_t tl = tmem + ((uint32_t)(q * 32) << 16) + cp;
    constexpr int kIo = 384;  // the thread that issues copies; thread 0 issues products
    auto issue = [&](int k) {
        uint8_t *st = sm + (k % ST) * L::kStage;
        uint64_t *bar = tma_bar + k % ST;
        mbar_expect_tx(bar, L::XB + L::BB);
        for (int i = 0; i < P / 64; ++i)
            tma_load_4d(st + L::oX + i * kTile, rev ? &tm_dy : &tm_x, bar, i * 64, h, chunk(k) * kTcQ, b);
        for (int i = 0; i < N / 64; ++i)
            tma_load_4d(st + L::oB + i * kTile, rev ? &tm_c : &tm_b, bar, i * 64, g, chunk(k) * kTcQ, b);
    };
    auto issue_g = [&](int k) {
        const float *src = gates + (((size_t)b * nch + chunk(k)) * a.H + h) * SsmGate::stride;
        uint8_t *dst = sm + L::oGate + (k & 1) * L::kGate;
        mbar_expect_tx(bar_g + (k & 1), L::kGate);
        bulk_load_g2s(dst, src + (rev ? SsmGate::e : SsmGate::w), 512, bar_g + (k & 1));
        bulk_load_g2s(dst + 512, src + SsmGate::misc, 64, bar_g + (k & 1));
    };
    auto prefetch = [&](int k) {  // two stages leave less than a load's latency from memory
        if (k >= cn) return;
        for (int i = 0; i < P / 64; ++i) tma_prefetch_4d(rev ? &tm_dy : &tm_x, i * 64, h, chunk(k) * kTcQ, b);
        for (int i = 0; i < N / 64; ++i) tma_prefetch_4d(rev ? &tm_c : &tm_b, i * 64, g, chunk(k) * kTcQ, b);
    };
    int n_t = 0, n_g = 0;  // issued, by that thread
    if (tid == kIo)
        for (int k = 0; k < ST && k < cn; ++k) {
            if (k < 2) {
                issue_g(k);
                n_g = k + 1;
            }
            issue(k);
            n_t = k + 1;
            if (ST == 2) prefetch(k + 2);
        }
    __syncwarp();
    // every thread: the chunk's rows weighted in place, the second part in registers until its buffer is free
    constexpr int CH = P / 32;
    uint4 second[CH], third[CH];
    auto convert = [&](int k) {
        if (!mbar_wait(bar_g + (k & 1), (uint32_t)(k >> 1) & 1) || !mbar_wait(tma_bar + k % ST, (uint32_t)(k / ST) & 1)) {
            *abort_flag = 1;
            return;
        }
        uint8_t *st = sm + (k % ST) * L::kStage + L::oX;
        const int r = tid & 127;
        const float w = reinterpret_cast<const float *>(sm + L::oGate + (k & 1) * L::kGate)[r];
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = (tid >> 7) * CH + i;
            uint8_t *p = st + (uint32_t)(c >> 3) * kTile + sw128_offset(r, c & 7);
            float x[8];
            ld8s(p, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= w;
            *reinterpret_cast<uint4 *>(p) = take_bf16x8(x);
            second[i] = take_bf16x8(x);
            third[i] = take_bf16x8(x);
        }
    };
    auto convert_third = [&] {  // the products of the chunk before are done
        const int r = tid & 127;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = (tid >> 7) * CH + i;
            *reinterpret_cast<uint4 *>(sm + L::oThird + (uint32_t)(c >> 3) * kTile + sw128_offset(r, c & 7)) = third[i];
        }
    };
    auto convert_second = [&](int k) {
        uint8_t *st = sm + (k % ST) * L::kStage + L::oLo;
        const int r = tid & 127;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = (tid >> 7) * CH + i;
            *reinterpret_cast<uint4 *>(st + (uint32_t)(c >> 3) * kTile + sw128_offset(r, c & 7)) = second[i];
        }
    };
    float v[PW];
    {
        if (OUT)
            ssm_enter_segment<PW, P, N>(v, rev ? seg_G : seg_S, dec, rev ? a.dS_T : a.S0, R, seg, b, h, a.H, cp, row, rev);
        else
#pragma unroll
            for (int i = 0; i < PW; ++i) v[i] = 0.f;
    }
    convert(0);
    convert_second(0);
    fence_async_smem();
    tc_before_sync();
    __syncthreads();
    double edge = 0.0;
    const bool keep = !OUT || (rev && seg == 0 && a.dS0);  // the state behind the last chunk is an output
    bool mma_open = false;
    int k = 0;
#pragma unroll 1
    for (; k < cn && !*abort_flag; ++k) {
        const float *s_g = reinterpret_cast<const float *>(sm + L::oGate + (k & 1) * L::kGate) + 128 - SsmGate::misc;
        const float el = s_g[SsmGate::elast];
        const bool update = keep || k + 1 < cn;
        edge += *reinterpret_cast<const double *>(s_g + SsmGate::last);
        if (tid == kIo && k > 0 && k - 1 + ST < cn) {  // into the stage of the chunk before
            issue(k - 1 + ST);
            n_t = k + ST;
            if (ST == 2) prefetch(k + 3);
        }
        __syncwarp();
        convert_third();
        if (OUT && row < N) {
            float4 *dst = (rev ? out_G : out_S) + ((((size_t)b * nch + chunk(k)) * a.H + h) * (P / 4) + cp / 4) * N + row;
#pragma unroll
            for (int i = 0; i < PW / 4; ++i) dst[(size_t)i * N] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        }
        fence_async_smem();
        tc_before_sync();
        __syncthreads();
        if (tid == 0 && update) {
            tc_after_sync();
            const uint32_t st = sb + (k % ST) * L::kStage, at = st + L::oB;
            const uint32_t block = N == 64 ? sb + L::oZero - at : kTile;  // the second 64 lanes
#pragma unroll
            for (int part = 2; part >= 0; --part)
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    mma_bf16(tmem, desc_mn(at, kk, block), desc_mn(part == 2 ? sb + L::oThird : st + (part ? L::oLo : L::oX), kk),
                             idesc_bf16(128, P, true, true), part < 2 || kk > 0);
            mma_commit(mma_bar);
        }
        __syncwarp();
        if (k + 1 < cn) {
            convert(k + 1);
            convert_second(k + 1);
        }
        fence_async_smem();
        if (tid == 0 && update) {
            mma_open = !mbar_wait(mma_bar, (uint32_t)(k & 1));
            if (mma_open) *abort_flag = 1;
        }
        tc_before_sync();
        __syncthreads();
        tc_after_sync();
        if (tid == kIo && k + 2 < cn) {  // this chunk's table is done with
            issue_g(k + 2);
            n_g = k + 3;
        }
        __syncwarp();
        if (update && row < N) {
            float u[PW];
            tmem_ldw<PW>(tl, u);
#pragma unroll
            for (int i = 0; i < PW; ++i) v[i] = fmaf(el, v[i], u[i]);
        }
    }
    if (*abort_flag) {
        if (tid == kIo) {
            record_status(GDR_ERR_TIMEOUT);
            for (int i = n_t > ST ? n_t - ST : 0; i < n_t; ++i) mbar_wait(tma_bar + i % ST, (uint32_t)(i / ST) & 1);
            for (int i = n_g > 1 ? n_g - 2 : 0; i < n_g; ++i) mbar_wait(bar_g + (i & 1), (uint32_t)(i >> 1) & 1);
        }
        if (tid == 0 && mma_open) mbar_wait(mma_bar, (uint32_t)((k - 1) & 1));
    } else {
        if (keep && row < N) {
            float *dst = OUT ? a.dS0 + (size_t)bh * P * N : (rev ? seg_G : seg_S) + (((size_t)b * R + seg) * a.H + h) * P * N;
#pragma unroll
            for (int i = 0; i < PW; ++i) dst[(size_t)(cp + i) * N + row] = v[i];
        }
        if (!OUT && !rev && tid == 0) dec[((size_t)b * R + seg) * a.H + h] = exp2f((float)edge);
    }
    tc_before_sync();
    __syncthreads();
    if (warp == 0) {
        tc_after_sync();
        tmem_dealloc(tmem, P);
    }
}

// ---- 3. outputs ------------------------------------------------------------------------------
// LO: S_T is written at the end (one segment).  With P = 64 two CTAs of 8 warps share an SM; with P = 128 a CTA has 16
// warps, which take the registers of an SM.  Each of a chunk's two rounds of products waits for register conversions and
// block barriers.  The scores stay in TMEM, as the A operand of their product.
template <int P, int N, bool LO>
struct SsmYTc {
    static constexpr int NT = P == 128 ? 512 : 256, kParts = NT / 128;  // warps of one TMEM quarter: column parts
    // P = 64, N = 128: two CTAs share an SM only if the state's second part takes the first one's place
    static constexpr bool kTurns = P == 64 && N == 128 && !LO;
    static constexpr uint32_t XB = P / 64 * kTile, BB = N / 64 * kTile;
    static constexpr uint32_t oX = 0, oB = XB, oZero = oB + BB;
    static constexpr uint32_t oC = oZero + (N == 64 ? kTile : 0);  // C, then w X's third part (LO) or its second (kTurns)
    static constexpr uint32_t oS = oC + (LO && XB > BB ? XB : BB); // S^T: N rows of 64 columns p; then w X, then y
    static constexpr uint32_t kSBlock = kTile;
    static constexpr uint32_t oLo = kTurns ? oC : oS + XB;         // the second part of S^T, then of w X
    static constexpr uint32_t oGate = oS + (kTurns ? 1 : 2) * XB;  // two tables
    static constexpr uint32_t oBar = oGate + 2 * SsmGate::kFwdBytes;
    static constexpr uint32_t kAlloc = oBar + 64 + 1024;
    static constexpr uint32_t kTmemCols = P == 64 && !LO ? 256 : 512;
};

template <int P, int N, bool LO>
__global__ void __launch_bounds__(SsmYTc<P, N, LO>::NT, P == 64 && !LO ? 2 : 1) ssm_tc_y_kernel(
    const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_b,
    const __grid_constant__ CUtensorMap tm_c, const __grid_constant__ CUtensorMap tm_y, SsmArgs a, int m,
    const float *__restrict__ gates, const float *__restrict__ states, const float *__restrict__ dec) {
    using L = SsmYTc<P, N, LO>;
    using namespace sm100;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const uint32_t sb = smem_u32(sm);
    uint64_t *bar_x = reinterpret_cast<uint64_t *>(sm + L::oBar), *bar_bc = bar_x + 1, *bar_g = bar_x + 2, *mma_bar = bar_x + 3;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bar_x + 4);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int q = warp & 3, prt = warp >> 2, row = q * 32 + lane;  // TMEM lane (token i or state row n), column part
    const int nch = (a.T + kTcQ - 1) / kTcQ, R = (nch + m - 1) / m;
    const int seg = blockIdx.x % R, bh = blockIdx.x / R, h = bh % a.H, b = bh / a.H, g = h / (a.H / a.G);
    const int c0 = seg * m, cn = min(m, nch - c0);

    if (tid == 0) {
        mbar_init(bar_x, 1);
        mbar_init(bar_bc, 1);
        mbar_init(bar_g, 1);
        mbar_init(mma_bar, 1);
        fence_mbar_init();
        *abort_flag = 0;
    }
    if (warp == 0) tmem_alloc(tmem_slot, L::kTmemCols);
    if (N == 64)
        for (int i = tid; i < (int)kTile / 16; i += L::NT) reinterpret_cast<uint4 *>(sm + L::oZero)[i] = make_uint4(0, 0, 0, 0);
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    const uint32_t tmem = *tmem_slot;
    const uint32_t tl = tmem + ((uint32_t)(q * 32) << 16);
    constexpr uint32_t tK = 0, tY = 128, tS = 128 + P;   // the scores' two bf16 parts take K's columns
    constexpr uint32_t tU = LO ? tS + P : tS;            // the chunk's own sum
    const int cp = prt * 32;                             // this warp's 32 columns p

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
    auto issue_g = [&](int k) {
        mbar_expect_tx(bar_g, SsmGate::kFwdBytes);
        bulk_load_g2s(sm + L::oGate + (k & 1) * SsmGate::kFwdBytes,
                      gates + (((size_t)b * nch + c0 + k) * a.H + h) * SsmGate::stride, SsmGate::kFwdBytes, bar_g);
    };
    auto prefetch = [&](int k) {
        if (k >= cn) return;
        for (int i = 0; i < P / 64; ++i) tma_prefetch_4d(&tm_x, i * 64, h, (c0 + k) * kTcQ, b);
        for (int i = 0; i < N / 64; ++i) {
            tma_prefetch_4d(&tm_b, i * 64, g, (c0 + k) * kTcQ, b);
            tma_prefetch_4d(&tm_c, i * 64, g, (c0 + k) * kTcQ, b);
        }
    };
    // Copies are issued by a warp whose scores are mostly above the diagonal, products by thread 0.
    constexpr int kIo = L::NT - 128;
    int n_bc = 0, n_x = 0, n_g = 0;  // issued, by that thread
    if (tid == kIo) {
        issue_g(0);
        issue_bc(0);
        issue_x(0);
        n_bc = n_x = n_g = 1;
        prefetch(1);
    }
    __syncwarp();
    {   // the entering state: lane n, columns p
        float v[32];
        ssm_enter_segment<32, P, N>(v, states, dec, a.S0, R, seg, b, h, a.H, cp, row, false);
        if (!LO && R <= kJoinMost && seg == R - 1 && a.S_T && row < N) {  // the last segment's end, in fp32
            const size_t unit = ((size_t)b * R + seg) * a.H + h;
            const float d = dec[unit];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const size_t at = (size_t)(cp + i) * N + row;
                a.S_T[(size_t)bh * P * N + at] = fmaf(d, v[i], states[unit * P * N + at]);
            }
        }
        tmem_st32(tl + tS + cp, v);
        tmem_wait_st();
    }
    uint32_t mma_phase = 0;
    bool mma_open = false;
    auto mma_sync_point = [&]() {  // thread 0 has committed its products
        if (tid == 0) {
            mma_open = !mbar_wait(mma_bar, mma_phase);
            if (mma_open) *abort_flag = 1;
        }
        mma_phase ^= 1;
        __syncthreads();
        tc_after_sync();
    };
    const float D = a.D ? a.D[h] : 0.f;

#pragma unroll 1
    for (int k = 0; k < cn; ++k) {
        const float *s_g = reinterpret_cast<const float *>(sm + L::oGate + (k & 1) * SsmGate::kFwdBytes);
        if (tid == 0 && !mbar_wait(bar_g, (uint32_t)(k & 1))) *abort_flag = 1;
        if (tid == kIo) bulk_wait_read_all();  // y of the chunk before leaves through S's tile
        __syncthreads();
        if (*abort_flag) break;
        if (tid == kIo && k + 1 < cn) {  // the other table was last read a chunk ago
            issue_g(k + 1);
            ++n_g;
        }
        __syncwarp();
        uint4 turn[4];  // kTurns: the state's second part until its place is free
        if (row < N) {  // S^T as two bf16 operands [n][p]; the fp32 state decays to the chunk's end
            const float el = s_g[SsmGate::elast];
            float v[32];
            tmem_ld32(tl + tS + cp, v);
            if (LO && k > 0) {
                float u[32];
                tmem_ld32(tl + tU + cp, u);
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] += u[i];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t off = (cp >> 6) * L::kSBlock + sw128_offset(row, ((cp & 63) >> 3) + i);
                float r[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    r[e] = v[8 * i + e];
                    v[8 * i + e] *= el;
                }
                *reinterpret_cast<uint4 *>(sm + L::oS + off) = take_bf16x8(r);
                turn[i] = take_bf16x8(r);
                if (!L::kTurns) *reinterpret_cast<uint4 *>(sm + L::oLo + off) = turn[i];
            }
            tmem_st32(tl + tS + cp, v);
            tmem_wait_st();
        }
        if (tid == 0 && (!mbar_wait(bar_bc, (uint32_t)(k & 1)) || !mbar_wait(bar_x, (uint32_t)(k & 1)))) *abort_flag = 1;
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
            for (int part = 0; part < (L::kTurns ? 1 : 2); ++part)
#pragma unroll
                for (int kk = 0; kk < N / 16; ++kk)
                    mma_bf16(tmem + tY, desc_k(sb + L::oC, kk), desc_mn(sb + (part ? L::oLo : L::oS), kk, L::kSBlock),
                             idesc_bf16(128, P, false, true), part > 0 || kk > 0);
            mma_commit(mma_bar);
        }
        mma_sync_point();
        if (*abort_flag) break;
        if (L::kTurns) {
            if (row < N)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<uint4 *>(sm + L::oS + (cp >> 6) * L::kSBlock + sw128_offset(row, ((cp & 63) >> 3) + i)) = turn[i];
            fence_async_smem();
            tc_before_sync();
            __syncthreads();
            if (tid == 0) {
                tc_after_sync();
#pragma unroll
                for (int kk = 0; kk < N / 16; ++kk)
                    mma_bf16(tmem + tY, desc_k(sb + L::oC, kk), desc_mn(sb + L::oS, kk, L::kSBlock),
                             idesc_bf16(128, P, false, true), 1);
                mma_commit(mma_bar);  // waited for behind the scores
            }
            __syncwarp();
        }

        // decayed scores -> two bf16 parts in TMEM, over K: the 32 tokens j of a block are 16 columns of the first
        // part and 16 of the second, so that a warp writes only columns that it has read
        const float rf = s_g[SsmGate::rowf + row], ci = s_g[SsmGate::hi + row], cl = s_g[SsmGate::lo + row];
#pragma unroll
        for (int jb = 0; jb < 4 / L::kParts; ++jb) {
            const int J = prt * (4 / L::kParts) + jb;  // 32-column block
            float v[32];
            if (J > q) {
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = 0.f;
            } else {
                const float4 *dt4 = reinterpret_cast<const float4 *>(s_g + SsmGate::dt + J * 32);
                tmem_ld32(tl + tK + J * 32, v);
                if (J < q) {
                    const float2 rf2 = make_float2(rf, rf);
                    const float4 *col4 = reinterpret_cast<const float4 *>(s_g + SsmGate::col + (q - 1) * 96 + J * 32);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 cc = col4[i], d = dt4[i];
                        const float2 lo = fmul2(make_float2(v[4 * i], v[4 * i + 1]),
                                                fmul2(fmul2(rf2, make_float2(cc.x, cc.y)), make_float2(d.x, d.y)));
                        const float2 hi = fmul2(make_float2(v[4 * i + 2], v[4 * i + 3]),
                                                fmul2(fmul2(rf2, make_float2(cc.z, cc.w)), make_float2(d.z, d.w)));
                        v[4 * i] = lo.x;
                        v[4 * i + 1] = lo.y;
                        v[4 * i + 2] = hi.x;
                        v[4 * i + 3] = hi.y;
                    }
                } else {
                    const float4 *hi4 = reinterpret_cast<const float4 *>(s_g + SsmGate::hi + J * 32);
                    const float4 *lo4 = reinterpret_cast<const float4 *>(s_g + SsmGate::lo + J * 32);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 hj = hi4[i], lj = lo4[i], d = dt4[i];
                        const float e[4] = {ex2_ftz((ci - hj.x) + (cl - lj.x)) * d.x, ex2_ftz((ci - hj.y) + (cl - lj.y)) * d.y,
                                            ex2_ftz((ci - hj.z) + (cl - lj.z)) * d.z, ex2_ftz((ci - hj.w) + (cl - lj.w)) * d.w};
#pragma unroll
                        for (int u = 0; u < 4; ++u) v[4 * i + u] = 4 * i + u <= lane ? v[4 * i + u] * e[u] : 0.f;
                    }
                }
            }
            float parts[32];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                parts[i] = __uint_as_float(take_bf16x2(v[2 * i], v[2 * i + 1]));
                parts[16 + i] = __uint_as_float(take_bf16x2(v[2 * i], v[2 * i + 1]));
            }
            tmem_st32(tl + tK + J * 32, parts);
        }
        if (L::kTurns) {
            mma_sync_point();
            if (*abort_flag) break;
        }
        {   // e^{c_i} C S_in^T, onto which the scores' product is summed
            const float e = s_g[SsmGate::e + row];
            float v[32];
            tmem_ld32(tl + tY + cp, v);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] *= e;
            tmem_st32(tl + tY + cp, v);
            tmem_wait_st();
        }
        if (LO || k + 1 < cn) {  // the state's own product: w X as bf16 parts (C's and S's products are done)
            const int r = tid & 127;
            const float w = s_g[SsmGate::dt + r] * s_g[SsmGate::el + r];
            constexpr int CH = P / 8 / L::kParts;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int c = (tid >> 7) * CH + i;
                const uint32_t off = (uint32_t)(c >> 3) * kTile + sw128_offset(r, c & 7);
                float v[8];
                ld8s(sm + L::oX + off, v);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] *= w;
                *reinterpret_cast<uint4 *>(sm + L::oS + off) = take_bf16x8(v);
                *reinterpret_cast<uint4 *>(sm + L::oLo + off) = take_bf16x8(v);
                if (LO) *reinterpret_cast<uint4 *>(sm + L::oC + off) = take_bf16x8(v);
            }
        }
        fence_async_smem();
        tc_before_sync();
        __syncthreads();
        if (tid == 0) {
            tc_after_sync();
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    mma_bf16_ts(tmem + tY, tmem + tK + (kk >> 1) * 32 + part * 16 + (kk & 1) * 8, desc_mn(sb + L::oX, kk),
                                idesc_bf16(128, P, false, true), 1);
            if (LO || k + 1 < cn) {
#pragma unroll
                for (int part = LO ? 2 : 1; part >= 0; --part)
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        mma_bf16(tmem + tU, desc_mn(sb + L::oB, kk, N == 64 ? L::oZero - L::oB : kTile),
                                 desc_mn(sb + (part == 0 ? L::oS : part == 1 ? L::oLo : L::oC), kk), idesc_bf16(128, P, true, true),
                                 !LO || part < 2 || kk > 0);
            }
            mma_commit(mma_bar);
        }
        uint4 xr[4];  // this thread's x, before its tile is filled again
        if (a.D)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                xr[i] = *reinterpret_cast<const uint4 *>(sm + L::oX + (uint32_t)(cp >> 6) * kTile +
                                                         sw128_offset(row, ((cp & 63) >> 3) + i));
        mma_sync_point();
        if (*abort_flag) break;
        if (tid == kIo && k + 1 < cn) {
            issue_bc(k + 1);
            issue_x(k + 1);
            ++n_bc;
            ++n_x;
            prefetch(k + 2);
        }
        __syncwarp();
        {   // + D x, over S's tile (straight from registers, 64 bytes of 32 rows a warp, the stores alone took 2000 of a
            // chunk's 9500 cycles)
            float y[32];
            tmem_ld32(tl + tY + cp, y);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float x[8];
                if (a.D) ld8s(reinterpret_cast<const uint8_t *>(&xr[i]), x);
#pragma unroll
                for (int u = 0; u < 8; ++u) x[u] = a.D ? fmaf(D, x[u], y[8 * i + u]) : y[8 * i + u];
                st_bf16x8(sm + L::oS + (uint32_t)(cp >> 6) * kTile + sw128_offset(row, ((cp & 63) >> 3) + i), x);
            }
        }
        fence_async_smem();
        tc_before_sync();
        __syncthreads();
        if (tid == kIo) {
            for (int i = 0; i < P / 64; ++i) tma_store_4d(&tm_y, sm + L::oS + i * kTile, i * 64, h, (c0 + k) * kTcQ, b);
            bulk_commit();
        }
        __syncwarp();
    }
    if (*abort_flag) {
        if (tid == 0 && mma_open) mbar_wait(mma_bar, mma_phase ^ 1);
        if (tid == kIo) {  // wait, bounded, for the last of each copy (and, above, for the products)
            record_status(GDR_ERR_TIMEOUT);
            mbar_wait(bar_g, (uint32_t)((n_g - 1) & 1));
            mbar_wait(bar_bc, (uint32_t)((n_bc - 1) & 1));
            mbar_wait(bar_x, (uint32_t)((n_x - 1) & 1));
            bulk_wait_all();
        }
    } else if (LO && a.S_T && row < N) {
        float *dst = a.S_T + (size_t)bh * P * N;
        float v[32], u[32];
        tmem_ld32(tl + tS + cp, v);
        tmem_ld32(tl + tU + cp, u);
#pragma unroll
        for (int i = 0; i < 32; ++i) dst[(size_t)(cp + i) * N + row] = v[i] + u[i];
    }
    if (tid == kIo) bulk_wait_all();
    tc_before_sync();
    __syncthreads();
    if (warp == 0) {
        tc_after_sync();
        tmem_dealloc(tmem, L::kTmemCols);
    }
}

// ---- host side ------------------------------------------------------------------------------
// Chunks per segment.  In units of a chunk of the output kernel: whole rounds of CTAs over the SMs, where two CTAs of P =
// 64 on an SM take 1.5 of one's time; a cut costs the walk over the segments first (about half of that) and two
// launches.  Measured: B=4 T=4096 H=16 P=N=128, 2 segments 173 us (1: 249, 3: 228); B=1 T=4096, 8 segments 58 us (6: 73, 16:
// 65); B=8 T=2048 H=16 P=64, uncut 107 us (2 segments: 117); B=1 T=65536 P=64, 37 segments 376 us (16: 404, 32: 411); B=2
// T=2048 H=24 P=64, 6 segments 55 us (3: 64, 8: 69).
inline int ssm_tc_chunks(int B, int T, int H, int P) {
    const int nch = (T + kTcQ - 1) / kTcQ, sms = sm_count();
    double best = 1e30;
    int at = nch;
    for (int m = nch; m >= 1; m = m > 64 ? m * 3 / 4 : m - 1) {
        const int R = (nch + m - 1) / m;
        const long long n = (long long)B * H * R, rounds = (n + sms - 1) / sms;
        const double y = P == 64 && R > 1 && n > sms ? (double)((n + 2 * sms - 1) / (2 * sms)) * 1.5 : (double)rounds;
        const double cost = R == 1 ? y * 1.1 * m : y * m + (double)rounds * (0.5 * m + 1.0) + 2.0;
        if (cost < best * 0.999) {
            best = cost;
            at = m;
        }
    }
    return at;
}

struct SsmTcFwdWs {
    size_t gates, st, dec, total;
};
inline size_t ssm_gate_bytes(int B, int T, int H) {
    return ssm_align((size_t)B * ((T + kTcQ - 1) / kTcQ) * H * SsmGate::stride * sizeof(float));
}
inline SsmTcFwdWs ssm_tc_fwd_ws(int B, int T, int H, int P, int N) {
    const int m = ssm_tc_chunks(B, T, H, P), nch = (T + kTcQ - 1) / kTcQ, R = (nch + m - 1) / m;
    SsmTcFwdWs w{};
    w.st = w.dec = w.total = ssm_gate_bytes(B, T, H);
    if (R == 1) return w;
    const size_t units = (size_t)B * R * H;
    w.dec = w.st + ssm_align(units * P * N * 4);
    w.total = w.dec + ssm_align(units * 4);
    return w;
}

inline cudaError_t ssm_launch_gates(const SsmArgs &a, float *gates, cudaStream_t s) {
    const unsigned units = (unsigned)((size_t)a.B * ((a.T + kTcQ - 1) / kTcQ) * a.H);
    ssm_gate_kernel<<<units, 128, 0, s>>>(a, gates);
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return cudaGetLastError();
}

template <int P, int N>
cudaError_t ssm_tc_fwd(const SsmArgs &a, void *ws, cudaStream_t s) {
    CUtensorMap mx, mb, mc, my;
    if (!ssm_token_map(&mx, a.x, a.B, a.T, a.H, P, a.ldx) || !ssm_token_map(&mb, a.Bm, a.B, a.T, a.G, N, a.ldb) ||
        !ssm_token_map(&mc, a.Cm, a.B, a.T, a.G, N, a.ldc) || !ssm_token_map(&my, a.y, a.B, a.T, a.H, P, a.H * P))
        return cudaErrorInvalidValue;
    const int m = ssm_tc_chunks(a.B, a.T, a.H, P), nch = (a.T + kTcQ - 1) / kTcQ, R = (nch + m - 1) / m;
    const dim3 grid((unsigned)(a.B * a.H) * (unsigned)R);
    const SsmTcFwdWs w = ssm_tc_fwd_ws(a.B, a.T, a.H, P, N);
    float *gates = static_cast<float *>(ws);
    cudaError_t e = ssm_launch_gates(a, gates, s);
    if (e != cudaSuccess) return e;
    if (R == 1)
        return ssm_launch(ssm_tc_y_kernel<P, N, true>, grid, SsmYTc<P, N, true>::NT, (size_t)SsmYTc<P, N, true>::kAlloc, s, mx,
                          mb, mc, my, a, m, (const float *)gates, (const float *)nullptr, (const float *)nullptr);
    float *st = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + w.st);
    float *dec = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + w.dec);
    e = ssm_launch(ssm_tc_walk_kernel<P, N, false>, grid, SsmWalkTc<P, N>::kThreads, (size_t)SsmWalkTc<P, N>::kAlloc, s, mx, mb,
                   mx, mb, a, m, 1, (const float *)gates, (float4 *)nullptr, (float4 *)nullptr, st, (float *)nullptr, dec);
    if (e == cudaSuccess && R > kJoinMost) e = ssm_launch_scan(false, a.B, R, a.H, P * N, st, dec, a.S0, a.S_T, s);
    if (e == cudaSuccess)
        e = ssm_launch(ssm_tc_y_kernel<P, N, false>, grid, SsmYTc<P, N, false>::NT, (size_t)SsmYTc<P, N, false>::kAlloc, s, mx,
                       mb, mc, my, a, m, (const float *)gates, (const float *)st, (const float *)dec);
    return e;
}

}  // namespace gdr

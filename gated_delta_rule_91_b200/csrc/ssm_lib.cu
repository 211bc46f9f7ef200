// ssm_lib.cu -- the C ABI (include/gdr.h) of the selective state space scan,
// the short causal convolution and the layer norm: argument validation,
// workspace sizing and kernel selection.
#include <stdlib.h>
#include <string.h>

#include <initializer_list>

#include "abi_common.cuh"
#include "conv.cuh"
#include "layernorm.cuh"
#include "ssm_simt.cuh"
#include "ssm_step.cuh"
#include "ssm_tc.cuh"
#include "ssm_bwd_tc.cuh"

namespace gdr {

cudaError_t ssm_take_status(int *status) {
    int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(status, g_status, sizeof(int));
    if (e == cudaSuccess && *status != 0) e = cudaMemcpyToSymbol(g_status, &zero, sizeof(int));
    return e;
}

}  // namespace gdr

using namespace gdr;

namespace {

gdr_status check_ssm(const char *fn, int B, int T, int H, int G, int P, int N, gdr_dtype dt) {
    if (B < 1 || T < 1 || H < 1 || G < 1 || P < 1 || N < 1)
        return fail(GDR_ERR_INVALID_ARGUMENT, "%s: sizes must be positive (B=%d T=%d H=%d G=%d P=%d N=%d)", fn, B, T, H, G,
                    P, N);
    if (dt != GDR_F32 && dt != GDR_BF16) return fail(GDR_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, (int)dt);
    if ((P != 64 && P != 128) || (N != 64 && N != 128))
        return fail(GDR_ERR_UNSUPPORTED, "%s: P=%d N=%d (supported: 64 or 128 each)", fn, P, N);
    if (H % G != 0) return fail(GDR_ERR_INVALID_ARGUMENT, "%s: H=%d is not a multiple of G=%d", fn, H, G);
    if ((long long)B * T * H * (P > N ? P : N) >= (1LL << 31))
        return fail(GDR_ERR_UNSUPPORTED, "%s: B*T*H*max(P,N) exceeds 2^31-1", fn);
    if ((long long)B * H * (P / 32) >= (1LL << 31))
        return fail(GDR_ERR_UNSUPPORTED, "%s: too many batches or heads (B=%d H=%d)", fn, B, H);
    return GDR_OK;
}
// The prompt's and the gradients' kernels take heads and batches as grid axes.
gdr_status check_ssm_grid(const char *fn, int B, int T, int H, int G, int P, int N, gdr_dtype dt) {
    gdr_status st = check_ssm(fn, B, T, H, G, P, N, dt);
    if (st == GDR_OK && (B > 65535 || H > 65535))
        return fail(GDR_ERR_UNSUPPORTED, "%s: B=%d H=%d (at most 65535 each)", fn, B, H);
    return st;
}

// An output at an input's own address (the kernels read inputs again after the first outputs are written).
bool in_place(std::initializer_list<const void *> outs, std::initializer_list<const void *> ins) {
    for (const void *o : outs)
        for (const void *i : ins)
            if (o != nullptr && o == i) return true;
    return false;
}

// Token stride `ld` of `width` elements: 0 means dense; rows start on 16-byte boundaries.
gdr_status check_stride(const char *fn, const char *name, int *ld, int width, gdr_dtype dt) {
    const int per16 = dt == GDR_F32 ? 4 : 8;
    if (*ld == 0) *ld = width;
    if (*ld < width || *ld % per16 != 0)
        return fail(GDR_ERR_INVALID_ARGUMENT, "%s: token stride %s=%d (at least %d and a multiple of %d)", fn, name, *ld,
                    width, per16);
    return GDR_OK;
}

// bf16 runs on the tensor cores; GDR_SSM_KERNEL=simt selects the CUDA-core
// kernels (used to cross-check them).  The workspace follows the same choice.
bool ssm_uses_tc(gdr_dtype dt) {
    const char *sel = getenv("GDR_SSM_KERNEL");
    return dt == GDR_BF16 && !(sel != nullptr && strcmp(sel, "simt") == 0);
}

#define SSM_SHAPES(fn, T, a, ...)                                                  \
    ((a).P == 128 ? ((a).N == 128 ? fn<T, 128, 128>(__VA_ARGS__) : fn<T, 128, 64>(__VA_ARGS__)) \
                  : ((a).N == 128 ? fn<T, 64, 128>(__VA_ARGS__) : fn<T, 64, 64>(__VA_ARGS__)))
#define SSM_TC_SHAPES(fn, a, ...)                                            \
    ((a).P == 128 ? ((a).N == 128 ? fn<128, 128>(__VA_ARGS__) : fn<128, 64>(__VA_ARGS__)) \
                  : ((a).N == 128 ? fn<64, 128>(__VA_ARGS__) : fn<64, 64>(__VA_ARGS__)))

gdr_status check_conv(const char *fn, int B, int T, int C, int K, gdr_dtype dt, int *ldx) {
    if (B < 1 || T < 1 || C < 1)
        return fail(GDR_ERR_INVALID_ARGUMENT, "%s: sizes must be positive (B=%d T=%d C=%d)", fn, B, T, C);
    if (dt != GDR_F32 && dt != GDR_BF16) return fail(GDR_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, (int)dt);
    if (K < 1 || K > kShortConvMax)
        return fail(GDR_ERR_UNSUPPORTED, "%s: conv width K=%d (supported: 1..%d)", fn, K, kShortConvMax);
    if ((long long)B * T * C >= (1LL << 31)) return fail(GDR_ERR_UNSUPPORTED, "%s: B*T*C exceeds 2^31-1", fn);
    if (T > kConvMax || C > kConvMax) return fail(GDR_ERR_UNSUPPORTED, "%s: T=%d C=%d (at most %d)", fn, T, C, kConvMax);
    if (*ldx == 0) *ldx = C;
    if (*ldx < C) return fail(GDR_ERR_INVALID_ARGUMENT, "%s: token stride ldx=%d is less than C=%d", fn, *ldx, C);
    return GDR_OK;
}

// The vector form copies 16 bytes at a time: every row of every tensor has to start on 16 bytes.
bool conv_vectors(const ConvArgs &a, gdr_dtype dt) {
    const int v = dt == GDR_F32 ? 4 : 8;
    return a.C % v == 0 && a.ldx % v == 0;
}

gdr_status check_norm(const char *fn, long long R, int D, gdr_dtype dt, float eps) {
    if (R < 1 || D < 1) return fail(GDR_ERR_INVALID_ARGUMENT, "%s: sizes must be positive (rows=%lld D=%d)", fn, R, D);
    if (dt != GDR_F32 && dt != GDR_BF16) return fail(GDR_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, (int)dt);
    if (D > kNormMaxD) return fail(GDR_ERR_UNSUPPORTED, "%s: D=%d (at most %d)", fn, D, kNormMaxD);
    if (R >= (1LL << 31)) return fail(GDR_ERR_UNSUPPORTED, "%s: rows=%lld exceeds 2^31-1", fn, R);
    if (!(eps >= 0.f) || eps > 1e30f) return fail(GDR_ERR_INVALID_ARGUMENT, "%s: eps=%g", fn, (double)eps);
    return GDR_OK;
}

}  // namespace

extern "C" {

size_t gdr_ssm_fwd_workspace_bytes(int B, int T, int H, int G, int P, int N, gdr_dtype dt) {
    if (check_ssm_grid("gdr_ssm_fwd_workspace_bytes", B, T, H, G, P, N, dt) != GDR_OK) return 0;
    return ssm_uses_tc(dt) ? ssm_tc_fwd_ws(B, T, H, P, N).total : ssm_simt_ws(B, T, H, P, N).fwd_total;
}

gdr_status gdr_ssm_fwd(int B, int T, int H, int G, int P, int N, gdr_dtype dt, int softplus, const void *x, int ldx,
                       const float *delta, const float *A, const void *Bm, int ldb, const void *Cm, int ldc,
                       const float *D, const float *delta_bias, const float *S0, void *y, float *S_T, void *workspace,
                       size_t workspace_bytes, gdr_stream_t stream) {
    const char *fn = "gdr_ssm_fwd";
    gdr_status st = check_ssm_grid(fn, B, T, H, G, P, N, dt);
    if (st == GDR_OK) st = check_stride(fn, "ldx", &ldx, H * P, dt);
    if (st == GDR_OK) st = check_stride(fn, "ldb", &ldb, G * N, dt);
    if (st == GDR_OK) st = check_stride(fn, "ldc", &ldc, G * N, dt);
    if (st != GDR_OK) return st;
    GDR_REQUIRE_PTR(x);
    GDR_REQUIRE_PTR(delta);
    GDR_REQUIRE_PTR(A);
    GDR_REQUIRE_PTR(Bm);
    GDR_REQUIRE_PTR(Cm);
    GDR_OPTIONAL_PTR(D);
    GDR_OPTIONAL_PTR(delta_bias);
    GDR_OPTIONAL_PTR(S0);
    GDR_REQUIRE_PTR(y);
    GDR_OPTIONAL_PTR(S_T);
    const size_t need = gdr_ssm_fwd_workspace_bytes(B, T, H, G, P, N, dt);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need))
        return fail(GDR_ERR_WORKSPACE, "%s: workspace %zu bytes, need %zu", fn, workspace_bytes, need);
    GDR_OPTIONAL_PTR(workspace);
    if (in_place({y, S_T}, {x, delta, A, Bm, Cm, D, delta_bias, S0}))
        return fail(GDR_ERR_INVALID_ARGUMENT, "%s: an output is an input", fn);
    SsmArgs a{};
    a.B = B; a.T = T; a.H = H; a.G = G; a.P = P; a.N = N;
    a.x = x; a.Bm = Bm; a.Cm = Cm; a.ldx = ldx; a.ldb = ldb; a.ldc = ldc;
    a.delta = delta; a.A = A; a.D = D; a.bias = delta_bias; a.softplus = softplus; a.S0 = S0;
    a.y = y; a.S_T = S_T;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = ssm_uses_tc(dt)   ? SSM_TC_SHAPES(ssm_tc_fwd, a, a, workspace, s)
                    : dt == GDR_F32 ? SSM_SHAPES(ssm_simt_fwd, float, a, a, workspace, s)
                                    : SSM_SHAPES(ssm_simt_fwd, __nv_bfloat16, a, a, workspace, s);
    if (e != cudaSuccess) return cuda_fail(e, fn);
    return GDR_OK;
}

size_t gdr_ssm_bwd_workspace_bytes(int B, int T, int H, int G, int P, int N, gdr_dtype dt) {
    if (check_ssm_grid("gdr_ssm_bwd_workspace_bytes", B, T, H, G, P, N, dt) != GDR_OK) return 0;
    return ssm_uses_tc(dt) ? ssm_tc_bwd_ws(B, T, H, G, P, N).total : ssm_simt_ws(B, T, H, P, N).bwd_total;
}

gdr_status gdr_ssm_bwd(int B, int T, int H, int G, int P, int N, gdr_dtype dt, int softplus, const void *x, int ldx,
                       const float *delta, const float *A, const void *Bm, int ldb, const void *Cm, int ldc,
                       const float *D, const float *delta_bias, const float *S0, const void *dy, const float *dS_T,
                       void *dx, float *ddelta, float *dA, void *dB, void *dC, float *dD, float *ddelta_bias, float *dS0,
                       void *workspace, size_t workspace_bytes, gdr_stream_t stream) {
    const char *fn = "gdr_ssm_bwd";
    gdr_status st = check_ssm_grid(fn, B, T, H, G, P, N, dt);
    if (st == GDR_OK) st = check_stride(fn, "ldx", &ldx, H * P, dt);
    if (st == GDR_OK) st = check_stride(fn, "ldb", &ldb, G * N, dt);
    if (st == GDR_OK) st = check_stride(fn, "ldc", &ldc, G * N, dt);
    if (st != GDR_OK) return st;
    GDR_REQUIRE_PTR(x);
    GDR_REQUIRE_PTR(delta);
    GDR_REQUIRE_PTR(A);
    GDR_REQUIRE_PTR(Bm);
    GDR_REQUIRE_PTR(Cm);
    GDR_OPTIONAL_PTR(D);
    GDR_OPTIONAL_PTR(delta_bias);
    GDR_OPTIONAL_PTR(S0);
    GDR_REQUIRE_PTR(dy);
    GDR_OPTIONAL_PTR(dS_T);
    GDR_REQUIRE_PTR(dx);
    GDR_REQUIRE_PTR(ddelta);
    GDR_REQUIRE_PTR(dA);
    GDR_REQUIRE_PTR(dB);
    GDR_REQUIRE_PTR(dC);
    GDR_OPTIONAL_PTR(dD);
    GDR_OPTIONAL_PTR(ddelta_bias);
    GDR_OPTIONAL_PTR(dS0);
    const size_t need = gdr_ssm_bwd_workspace_bytes(B, T, H, G, P, N, dt);
    if (workspace == nullptr || workspace_bytes < need)
        return fail(GDR_ERR_WORKSPACE, "%s: workspace %zu bytes, need %zu", fn, workspace_bytes, need);
    if (!aligned16(workspace)) return fail(GDR_ERR_INVALID_ARGUMENT, "%s: workspace is not 16-byte aligned", fn);
    if (in_place({dx, ddelta, dA, dB, dC, dD, ddelta_bias, dS0}, {x, delta, A, Bm, Cm, D, delta_bias, S0, dy, dS_T}))
        return fail(GDR_ERR_INVALID_ARGUMENT, "%s: an output is an input", fn);
    SsmArgs a{};
    a.B = B; a.T = T; a.H = H; a.G = G; a.P = P; a.N = N;
    a.x = x; a.Bm = Bm; a.Cm = Cm; a.ldx = ldx; a.ldb = ldb; a.ldc = ldc;
    a.delta = delta; a.A = A; a.D = D; a.bias = delta_bias; a.softplus = softplus; a.S0 = S0;
    a.dy = dy; a.dS_T = dS_T;
    a.dx = dx; a.dB = dB; a.dC = dC; a.ddelta = ddelta; a.dA = dA; a.dD = dD; a.dbias = ddelta_bias; a.dS0 = dS0;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = ssm_uses_tc(dt)   ? SSM_TC_SHAPES(ssm_tc_bwd, a, a, workspace, s)
                    : dt == GDR_F32 ? SSM_SHAPES(ssm_simt_bwd, float, a, a, workspace, s)
                                    : SSM_SHAPES(ssm_simt_bwd, __nv_bfloat16, a, a, workspace, s);
    if (e != cudaSuccess) return cuda_fail(e, fn);
    return GDR_OK;
}

gdr_status gdr_debug_ssm_plan(int B, int T, int H, int G, int P, int N, int *plan) {
    const char *fn = "gdr_debug_ssm_plan";
    gdr_status st = check_ssm_grid(fn, B, T, H, G, P, N, GDR_BF16);
    if (st != GDR_OK) return st;
    if (plan == nullptr) return fail(GDR_ERR_INVALID_ARGUMENT, "%s: plan is NULL", fn);
    const int nch = (T + kTcQ - 1) / kTcQ;
    const SsmTcBwdWs w = ssm_tc_bwd_ws(B, T, H, G, P, N);
    plan[0] = ssm_tc_chunks(B, T, H, P);
    plan[1] = (nch + plan[0] - 1) / plan[0];
    plan[2] = w.m;
    plan[3] = w.R;
    plan[4] = w.splits;
    plan[5] = (H / G + w.splits - 1) / w.splits;
    return GDR_OK;
}

gdr_status gdr_ssm_step(int B, int H, int G, int P, int N, gdr_dtype dt, int softplus, const void *x, int ldx,
                        const float *delta, const float *A, const void *Bm, int ldb, const void *Cm, int ldc,
                        const float *D, const float *delta_bias, float *S, void *y, gdr_stream_t stream) {
    const char *fn = "gdr_ssm_step";
    gdr_status st = check_ssm(fn, B, 1, H, G, P, N, dt);
    if (st == GDR_OK) st = check_stride(fn, "ldx", &ldx, H * P, dt);
    if (st == GDR_OK) st = check_stride(fn, "ldb", &ldb, G * N, dt);
    if (st == GDR_OK) st = check_stride(fn, "ldc", &ldc, G * N, dt);
    if (st != GDR_OK) return st;
    GDR_REQUIRE_PTR(x);
    GDR_REQUIRE_PTR(delta);
    GDR_REQUIRE_PTR(A);
    GDR_REQUIRE_PTR(Bm);
    GDR_REQUIRE_PTR(Cm);
    GDR_OPTIONAL_PTR(D);
    GDR_OPTIONAL_PTR(delta_bias);
    GDR_REQUIRE_PTR(S);
    GDR_REQUIRE_PTR(y);
    if (in_place({S, y}, {x, delta, A, Bm, Cm, D, delta_bias}))
        return fail(GDR_ERR_INVALID_ARGUMENT, "%s: an output is an input", fn);
    SsmArgs a{};
    a.B = B; a.T = 1; a.H = H; a.G = G; a.P = P; a.N = N;
    a.x = x; a.Bm = Bm; a.Cm = Cm; a.ldx = ldx; a.ldb = ldb; a.ldc = ldc;
    a.delta = delta; a.A = A; a.D = D; a.bias = delta_bias; a.softplus = softplus;
    a.S_T = S; a.y = y;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = dt == GDR_F32 ? (N == 128 ? ssm_step_launch<float, 128>(a, s) : ssm_step_launch<float, 64>(a, s))
                                  : (N == 128 ? ssm_step_launch<__nv_bfloat16, 128>(a, s)
                                              : ssm_step_launch<__nv_bfloat16, 64>(a, s));
    if (e != cudaSuccess) return cuda_fail(e, fn);
    return GDR_OK;
}

gdr_status gdr_conv_fwd(int B, int T, int C, int K, gdr_dtype dt, int silu, const void *x, int ldx, const float *w,
                        const float *bias, const void *conv_state_in, void *conv_state_out, void *y,
                        gdr_stream_t stream) {
    const char *fn = "gdr_conv_fwd";
    gdr_status st = check_conv(fn, B, T, C, K, dt, &ldx);
    if (st != GDR_OK) return st;
    GDR_REQUIRE_PTR(x);
    GDR_REQUIRE_PTR(w);
    GDR_OPTIONAL_PTR(bias);
    GDR_OPTIONAL_PTR(conv_state_in);
    GDR_OPTIONAL_PTR(conv_state_out);
    GDR_REQUIRE_PTR(y);
    if (in_place({y}, {x, w, bias, conv_state_in}) || in_place({conv_state_out}, {x, w, bias}))
        return fail(GDR_ERR_INVALID_ARGUMENT, "%s: an output is an input", fn);
    ConvArgs a{};
    a.B = B; a.T = T; a.C = C; a.ldx = ldx; a.silu = silu;
    a.x = x; a.w = w; a.bias = bias; a.y = y;
    a.state_in = K > 1 ? conv_state_in : nullptr;
    a.state_out = K > 1 ? conv_state_out : nullptr;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (dt == GDR_F32)
        e = conv_vectors(a, dt) ? conv_fwd_width<float, 4>(K, a, s) : conv_fwd_width<float, 1>(K, a, s);
    else
        e = conv_vectors(a, dt) ? conv_fwd_width<__nv_bfloat16, 4>(K, a, s) : conv_fwd_width<__nv_bfloat16, 1>(K, a, s);
    if (e != cudaSuccess) return cuda_fail(e, fn);
    return GDR_OK;
}

size_t gdr_conv_bwd_workspace_bytes(int B, int T, int C, int K) {
    int ld = 0;
    if (check_conv("gdr_conv_bwd_workspace_bytes", B, T, C, K, GDR_F32, &ld) != GDR_OK) return 0;
    // one bound for the vector and the scalar form
    const int slots = conv_bwd_plan(B, T, C, K, 4).slots, scalar = conv_bwd_plan(B, T, C, K, 1).slots;
    return (size_t)(slots > scalar ? slots : scalar) * (K + 1) * C * sizeof(float);
}

gdr_status gdr_conv_bwd(int B, int T, int C, int K, gdr_dtype dt, int silu, const void *x, int ldx, const float *w,
                        const float *bias, const void *conv_state_in, const void *dy, const void *dconv_state_out,
                        void *dx, float *dw, float *dbias, void *dconv_state_in, void *workspace, size_t workspace_bytes,
                        gdr_stream_t stream) {
    const char *fn = "gdr_conv_bwd";
    gdr_status st = check_conv(fn, B, T, C, K, dt, &ldx);
    if (st != GDR_OK) return st;
    GDR_REQUIRE_PTR(x);
    GDR_REQUIRE_PTR(w);
    GDR_OPTIONAL_PTR(bias);
    GDR_OPTIONAL_PTR(conv_state_in);
    GDR_REQUIRE_PTR(dy);
    GDR_OPTIONAL_PTR(dconv_state_out);
    GDR_REQUIRE_PTR(dx);
    GDR_REQUIRE_PTR(dw);
    GDR_OPTIONAL_PTR(dbias);
    GDR_OPTIONAL_PTR(dconv_state_in);
    const size_t need = gdr_conv_bwd_workspace_bytes(B, T, C, K);
    if (workspace == nullptr || workspace_bytes < need)
        return fail(GDR_ERR_WORKSPACE, "%s: workspace %zu bytes, need %zu", fn, workspace_bytes, need);
    if (!aligned16(workspace)) return fail(GDR_ERR_INVALID_ARGUMENT, "%s: workspace is not 16-byte aligned", fn);
    if (in_place({dx, dw, dbias, dconv_state_in}, {x, w, bias, conv_state_in, dy, dconv_state_out}))
        return fail(GDR_ERR_INVALID_ARGUMENT, "%s: an output is an input", fn);
    ConvArgs a{};
    a.B = B; a.T = T; a.C = C; a.ldx = ldx; a.silu = silu;
    a.x = x; a.w = w; a.bias = bias; a.dy = dy; a.dx = dx;
    a.state_in = K > 1 ? conv_state_in : nullptr;
    a.dstate_out = K > 1 ? dconv_state_out : nullptr;
    a.dstate_in = K > 1 ? dconv_state_in : nullptr;
    a.part = static_cast<float *>(workspace);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (dt == GDR_F32)
        e = conv_vectors(a, dt) ? conv_bwd_width<float, 4>(K, a, dw, dbias, s) : conv_bwd_width<float, 1>(K, a, dw, dbias, s);
    else
        e = conv_vectors(a, dt) ? conv_bwd_width<__nv_bfloat16, 4>(K, a, dw, dbias, s)
                               : conv_bwd_width<__nv_bfloat16, 1>(K, a, dw, dbias, s);
    if (e != cudaSuccess) return cuda_fail(e, fn);
    return GDR_OK;
}

gdr_status gdr_layernorm_fwd(int64_t R, int D, gdr_dtype dt, const void *x, const void *residual, const float *weight,
                             const float *bias, float eps, void *y, void *h, gdr_stream_t stream) {
    const char *fn = "gdr_layernorm_fwd";
    gdr_status st = check_norm(fn, R, D, dt, eps);
    if (st != GDR_OK) return st;
    GDR_REQUIRE_PTR(x);
    GDR_OPTIONAL_PTR(residual);
    GDR_REQUIRE_PTR(weight);
    GDR_OPTIONAL_PTR(bias);
    GDR_REQUIRE_PTR(y);
    if ((residual == nullptr) != (h == nullptr))
        return fail(GDR_ERR_INVALID_ARGUMENT, "%s: residual and h must both be given or both NULL", fn);
    GDR_OPTIONAL_PTR(h);
    NormArgs a{};
    a.R = R; a.D = D; a.eps = eps;
    a.x = x; a.res = residual; a.w = weight; a.b = bias; a.y = y; a.h = h;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = dt == GDR_F32 ? norm_pick<float, false, NormFwd>(D, a, s)
                                  : norm_pick<__nv_bfloat16, false, NormFwd>(D, a, s);
    if (e != cudaSuccess) return cuda_fail(e, fn);
    return GDR_OK;
}

size_t gdr_layernorm_bwd_workspace_bytes(int D) {
    return D >= 1 && D <= kNormMaxD ? (size_t)kNormBwdMaxBlocks * 2 * D * sizeof(float) : 0;
}

gdr_status gdr_layernorm_bwd(int64_t R, int D, gdr_dtype dt, const void *h, const float *weight, float eps,
                             const void *dy, const void *dres, void *dx, float *dweight, float *dbias, void *workspace,
                             size_t workspace_bytes, gdr_stream_t stream) {
    const char *fn = "gdr_layernorm_bwd";
    gdr_status st = check_norm(fn, R, D, dt, eps);
    if (st != GDR_OK) return st;
    GDR_REQUIRE_PTR(h);
    GDR_REQUIRE_PTR(weight);
    GDR_REQUIRE_PTR(dy);
    GDR_OPTIONAL_PTR(dres);
    GDR_REQUIRE_PTR(dx);
    GDR_REQUIRE_PTR(dweight);
    GDR_OPTIONAL_PTR(dbias);
    const size_t need = gdr_layernorm_bwd_workspace_bytes(D);
    if (workspace == nullptr || workspace_bytes < need)
        return fail(GDR_ERR_WORKSPACE, "%s: workspace %zu bytes, need %zu", fn, workspace_bytes, need);
    if (!aligned16(workspace)) return fail(GDR_ERR_INVALID_ARGUMENT, "%s: workspace is not 16-byte aligned", fn);
    NormArgs a{};
    a.R = R; a.D = D; a.eps = eps;
    a.x = h; a.w = weight; a.dy = dy; a.dres = dres; a.dx = dx;
    a.part = static_cast<float *>(workspace);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = dt == GDR_F32 ? norm_pick<float, true, NormBwd>(D, a, dweight, dbias, s)
                                  : norm_pick<__nv_bfloat16, true, NormBwd>(D, a, dweight, dbias, s);
    if (e != cudaSuccess) return cuda_fail(e, fn);
    return GDR_OK;
}

}  // extern "C"

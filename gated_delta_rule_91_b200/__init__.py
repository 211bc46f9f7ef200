"""Python binding of libgdr.so, the B200 (sm_100a) gated delta rule library.

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI declared in include/gdr.h.  PyTorch supplies device
memory (outputs, workspace) and the current CUDA stream.  There is no CPU
path: if libgdr.so is missing or no GPU is present the calls raise.

Functions (same names as the C entry points):
    gdr_fwd(q, k, v, log_alpha, beta, S0=None)          -> (o, S_T)
    gdr_step(q, k, v, log_alpha, beta, S)                -> o  (S advanced in place)
    gdr_bwd(q, k, v, log_alpha, beta, S0, dO, dS_T=None) -> dict of gradients
    gdr2_fwd(q, k, v, log_alpha, b, w, S0=None)          -> (o, S_T)
    gdr2_bwd(q, k, v, log_alpha, b, w, S0, dO, dS_T=None) -> dict of gradients
    gdr2_step(q, k, v, log_alpha, b, w, S)               -> o  (S advanced in place)
    gdr_block_prologue(xq, xk, xv, wq, wk, wv, ...)       -> (q, k, v)
    gdr_block_prologue_bwd(xq, xk, xv, wq, wk, wv, dq, dk, dv, ...) -> dict of gradients
    gdr_block_epilogue(o, g, weight, eps)                 -> y
    gdr_block_epilogue_bwd(o, g, weight, dy, eps)         -> (do, dg, dweight)
    gdr_seg_fwd / gdr_seg_combine / gdr_seg_fixup         (sequence split; see seq_split)
    gdr_ssm_fwd(x, delta, A, Bm, Cm, D, delta_bias, S0)   -> (y, S_T)   (selective state space scan)
    gdr_ssm_bwd(x, delta, A, Bm, Cm, D, delta_bias, S0, dy, dS_T) -> dict of gradients
    gdr_ssm_step(x, delta, A, Bm, Cm, S, D, delta_bias)   -> y  (S advanced in place)
    gdr_conv_fwd(x, w, bias, ...)                         -> y  (short causal convolution)
    gdr_conv_bwd(x, w, dy, bias, ...)                     -> dict of gradients
    gdr_layernorm_fwd(x, weight, bias, residual, eps)     -> (y, h)
    gdr_layernorm_bwd(h, weight, dy, dres, eps)           -> (dx, dweight, dbias)

The calls take the current CUDA stream and allocate nothing inside the
library, so they can be captured in CUDA graphs.  `autograd` wraps the
forward/backward pairs as torch.autograd Functions.
"""
import ctypes
import os

import torch

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG_DIR, "libgdr.so")

GDR_OK, GDR_ERR_INVALID_ARGUMENT, GDR_ERR_UNSUPPORTED, GDR_ERR_WORKSPACE, GDR_ERR_CUDA, \
    GDR_ERR_TIMEOUT = range(6)
GDR_F32, GDR_BF16 = 0, 1
STATUS_NAMES = {0: "GDR_OK", 1: "GDR_ERR_INVALID_ARGUMENT", 2: "GDR_ERR_UNSUPPORTED",
                3: "GDR_ERR_WORKSPACE", 4: "GDR_ERR_CUDA", 5: "GDR_ERR_TIMEOUT"}

# name -> (restype, argtypes); mirrors include/gdr.h
_I, _SZ, _P = ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p
SIGNATURES = {
    "gdr_fwd": (_I, [_I] * 6 + [_P] * 8 + [_P, _SZ, _P]),
    "gdr_fwd_workspace_bytes": (_SZ, [_I] * 6),
    "gdr_step": (_I, [_I] * 5 + [_P] * 7 + [_P]),
    "gdr_bwd": (_I, [_I] * 6 + [_P] * 14 + [_P, _SZ, _P]),
    "gdr_bwd_workspace_bytes": (_SZ, [_I] * 6),
    "gdr_bwd_noalloc": (_I, [_I] * 6 + [_P] * 14 + [_P]),
    "gdr2_fwd": (_I, [_I] * 6 + [_P] * 9 + [_P, _SZ, _P]),
    "gdr2_fwd_workspace_bytes": (_SZ, [_I] * 6),
    "gdr2_bwd": (_I, [_I] * 6 + [_P] * 16 + [_P, _SZ, _P]),
    "gdr2_bwd_workspace_bytes": (_SZ, [_I] * 6),
    "gdr2_step": (_I, [_I] * 5 + [_P] * 8 + [_P]),
    "gdr_block_prologue": (_I, [_I] * 7 + [_P] * 11 + [ctypes.c_float] + [_P] * 3 + [_P]),
    "gdr_block_prologue_bwd": (_I, [_I] * 7 + [_P] * 10 + [ctypes.c_float] + [_P] * 14 + [_P, _SZ, _P]),
    "gdr_block_prologue_bwd_workspace_bytes": (_SZ, [_I] * 4),
    "gdr_block_epilogue": (_I, [_I] * 5 + [_P] * 3 + [ctypes.c_float, _P, _P]),
    "gdr_block_epilogue_bwd": (_I, [_I] * 5 + [_P] * 3 + [ctypes.c_float] + [_P] * 5 + [_SZ, _P]),
    "gdr_block_epilogue_bwd_workspace_bytes": (_SZ, [_I]),
    "gdr_seg_fwd": (_I, [_I] * 6 + [_P] * 9 + [_P, _SZ, _P]),
    "gdr_seg_fwd_workspace_bytes": (_SZ, [_I] * 6),
    "gdr_seg_combine": (_I, [_I] * 6 + [_P] * 5 + [_P]),
    "gdr_seg_fixup": (_I, [_I] * 6 + [_P] * 3 + [_P]),
    "gdr_ssm_fwd": (_I, [_I] * 8 + [_P, _I, _P, _P, _P, _I, _P, _I] + [_P] * 5 + [_P, _SZ, _P]),
    "gdr_ssm_fwd_workspace_bytes": (_SZ, [_I] * 7),
    "gdr_ssm_bwd": (_I, [_I] * 8 + [_P, _I, _P, _P, _P, _I, _P, _I] + [_P] * 13 + [_P, _SZ, _P]),
    "gdr_ssm_bwd_workspace_bytes": (_SZ, [_I] * 7),
    "gdr_debug_ssm_plan": (_I, [_I] * 6 + [_P]),
    "gdr_ssm_step": (_I, [_I] * 7 + [_P, _I, _P, _P, _P, _I, _P, _I] + [_P] * 4 + [_P]),
    "gdr_conv_fwd": (_I, [_I] * 6 + [_P, _I] + [_P] * 5 + [_P]),
    "gdr_conv_bwd": (_I, [_I] * 6 + [_P, _I] + [_P] * 9 + [_P, _SZ, _P]),
    "gdr_conv_bwd_workspace_bytes": (_SZ, [_I] * 4),
    "gdr_layernorm_fwd": (_I, [ctypes.c_int64, _I, _I] + [_P] * 4 + [ctypes.c_float] + [_P] * 2 + [_P]),
    "gdr_layernorm_bwd": (_I, [ctypes.c_int64, _I, _I] + [_P] * 2 + [ctypes.c_float] + [_P] * 5 + [_P, _SZ, _P]),
    "gdr_layernorm_bwd_workspace_bytes": (_SZ, [_I]),
    "gdr_check_status": (_I, [_P]),
    "gdr_debug_wait_timeout": (_I, [_I, _P]),
    "gdr_last_error_string": (ctypes.c_char_p, []),
    "gdr_launch_count": (ctypes.c_uint64, []),
    "gdr_version": (_I, []),
}


class GdrError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__("%s: %s" % (STATUS_NAMES.get(status, status), msg))
        self.status = status


_lib = None


def lib():
    """The loaded libgdr.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libgdr.so not found at %s; build it with "
                               "`python -m gated_delta_rule_91_b200._build`" % LIB_PATH)
        h = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(h, name)
            fn.restype = res
            fn.argtypes = args
        _lib = h
    return _lib


def check(status):
    if status != GDR_OK:
        raise GdrError(status, lib().gdr_last_error_string().decode())


def launch_count() -> int:
    return int(lib().gdr_launch_count())


def check_status(stream=None):
    """Synchronise the stream and raise if a kernel recorded a timeout."""
    s = torch.cuda.current_stream() if stream is None else stream
    check(lib().gdr_check_status(ctypes.c_void_p(s.cuda_stream)))


def _dt(x: torch.Tensor) -> int:
    if x.dtype == torch.float32:
        return GDR_F32
    if x.dtype == torch.bfloat16:
        return GDR_BF16
    raise TypeError("q/k/v must be float32 or bfloat16, got %s" % x.dtype)


def _ptr(x):
    if x is None:
        return None
    if not x.is_cuda:
        raise ValueError("tensors must be on a CUDA device")
    if not x.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(x.data_ptr())


def _f32(x, name):
    if x is not None and x.dtype != torch.float32:
        raise TypeError("%s must be float32" % name)
    return x


def _stream(x):
    return ctypes.c_void_p(torch.cuda.current_stream(x.device).cuda_stream)


def _workspace(nbytes, device, workspace):
    if nbytes == 0:
        return None, 0
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return workspace, workspace.numel() * workspace.element_size()


def gdr_fwd(q, k, v, log_alpha, beta, S0=None, *, o=None, S_T=None, return_state=True,
            workspace=None):
    """Chunkwise forward on the current stream.  Returns (o, S_T or None)."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = _dt(q)
    _f32(log_alpha, "log_alpha"), _f32(beta, "beta"), _f32(S0, "S0")
    if o is None:
        o = torch.empty(B, T, H, dv, dtype=q.dtype, device=q.device)
    if S_T is None and return_state:
        S_T = torch.empty(B, H, dv, dk, dtype=torch.float32, device=q.device)
    L = lib()
    ws, ws_bytes = _workspace(L.gdr_fwd_workspace_bytes(B, T, H, dk, dv, dt), q.device, workspace)
    check(L.gdr_fwd(B, T, H, dk, dv, dt, _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta),
                    _ptr(S0), _ptr(o), _ptr(S_T), _ptr(ws), ws_bytes, _stream(q)))
    return o, S_T


def gdr_step(q, k, v, log_alpha, beta, S, *, o=None):
    """One decode token; S [B,H,dv,dk] fp32 is advanced in place.  Returns o."""
    B, H, dk = q.shape
    dv = v.shape[-1]
    dt = _dt(q)
    _f32(S, "S")
    if o is None:
        o = torch.empty(B, H, dv, dtype=q.dtype, device=q.device)
    check(lib().gdr_step(B, H, dk, dv, dt, _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha),
                         _ptr(beta), _ptr(S), _ptr(o), _stream(q)))
    return o


def gdr_bwd(q, k, v, log_alpha, beta, S0, dO, dS_T=None, *, want_dS0=True, workspace=None):
    """Backward of gdr_fwd.  Returns dict(dq, dk, dv, dlog_alpha, dbeta, dS0)."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = _dt(q)
    out = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
               dlog_alpha=torch.empty_like(log_alpha), dbeta=torch.empty_like(beta),
               dS0=torch.empty(B, H, dv, dk, dtype=torch.float32, device=q.device)
               if want_dS0 else None)
    L = lib()
    ws, ws_bytes = _workspace(L.gdr_bwd_workspace_bytes(B, T, H, dk, dv, dt), q.device, workspace)
    check(L.gdr_bwd(B, T, H, dk, dv, dt, _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta),
                    _ptr(S0), _ptr(dO), _ptr(dS_T), _ptr(out["dq"]), _ptr(out["dk"]),
                    _ptr(out["dv"]), _ptr(out["dlog_alpha"]), _ptr(out["dbeta"]),
                    _ptr(out["dS0"]), _ptr(ws), ws_bytes, _stream(q)))
    return out


def gdr2_fwd(q, k, v, log_alpha, b, w, S0=None, *, o=None, S_T=None, return_state=True,
             workspace=None):
    """Gated DeltaNet-2 forward.  Returns (o, S_T or None)."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = _dt(q)
    if o is None:
        o = torch.empty(B, T, H, dv, dtype=q.dtype, device=q.device)
    if S_T is None and return_state:
        S_T = torch.empty(B, H, dv, dk, dtype=torch.float32, device=q.device)
    L = lib()
    ws, ws_bytes = _workspace(L.gdr2_fwd_workspace_bytes(B, T, H, dk, dv, dt), q.device, workspace)
    check(L.gdr2_fwd(B, T, H, dk, dv, dt, _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b),
                     _ptr(w), _ptr(S0), _ptr(o), _ptr(S_T), _ptr(ws), ws_bytes, _stream(q)))
    return o, S_T


def gdr2_step(q, k, v, log_alpha, b, w, S, *, o=None):
    """One Gated DeltaNet-2 decode token.  q, k [B,H,dk]; v [B,H,dv];
    log_alpha, b [B,H,dk] fp32; w [B,H,dv] fp32; S [B,H,dv,dk] fp32 updated in
    place.  Returns o [B,H,dv]."""
    B, H, dk = q.shape
    dv = v.shape[-1]
    _f32(log_alpha, "log_alpha"), _f32(b, "b"), _f32(w, "w"), _f32(S, "S")
    if o is None:
        o = torch.empty(B, H, dv, dtype=q.dtype, device=q.device)
    check(lib().gdr2_step(B, H, dk, dv, _dt(q), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w),
                          _ptr(S), _ptr(o), _stream(q)))
    return o


def gdr2_bwd(q, k, v, log_alpha, b, w, S0, dO, dS_T=None, *, want_dS0=True, workspace=None):
    """Backward of gdr2_fwd.  Returns dict(dq, dk, dv, dlog_alpha, db, dw, dS0)."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = _dt(q)
    out = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
               dlog_alpha=torch.empty_like(log_alpha), db=torch.empty_like(b), dw=torch.empty_like(w),
               dS0=torch.empty(B, H, dv, dk, dtype=torch.float32, device=q.device) if want_dS0 else None)
    L = lib()
    ws, ws_bytes = _workspace(L.gdr2_bwd_workspace_bytes(B, T, H, dk, dv, dt), q.device, workspace)
    check(L.gdr2_bwd(B, T, H, dk, dv, dt, _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w),
                     _ptr(S0), _ptr(dO), _ptr(dS_T), _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]),
                     _ptr(out["dlog_alpha"]), _ptr(out["db"]), _ptr(out["dw"]), _ptr(out["dS0"]),
                     _ptr(ws), ws_bytes, _stream(q)))
    return out


def gdr_block_prologue(xq, xk, xv, wq, wk, wv, bq=None, bk=None, bv=None, *, conv_state=None,
                       conv_state_out=None, eps=1e-6, q=None, k=None, v=None):
    """The block's q/k/v paths after the input projections: depthwise causal
    ShortConv (taps w* [H*d, K] fp32, biases b* [H*d] or None), SiLU, and L2
    normalisation of q and k per (token, head).  xq, xk [B,T,H,dk]; xv
    [B,T,H,dv].  conv_state [B, K-1, H*(2dk+dv)] (dtype of x, channels q, k,
    v) carries the inputs before token 0; conv_state_out receives the last
    K-1 inputs and may be conv_state itself.  Returns (q, k, v)."""
    B, T, H, dk = xq.shape
    dv = xv.shape[-1]
    K = wq.shape[-1]
    dt = _dt(xq)
    for name, t in (("wq", wq), ("wk", wk), ("wv", wv), ("bq", bq), ("bk", bk), ("bv", bv)):
        _f32(t, name)
    q = torch.empty_like(xq) if q is None else q
    k = torch.empty_like(xk) if k is None else k
    v = torch.empty_like(xv) if v is None else v
    check(lib().gdr_block_prologue(B, T, H, dk, dv, K, dt, _ptr(xq), _ptr(xk), _ptr(xv), _ptr(wq),
                                   _ptr(wk), _ptr(wv), _ptr(bq), _ptr(bk), _ptr(bv),
                                   _ptr(conv_state), _ptr(conv_state_out), float(eps), _ptr(q),
                                   _ptr(k), _ptr(v), _stream(xq)))
    return q, k, v


def gdr_block_prologue_bwd(xq, xk, xv, wq, wk, wv, dyq, dyk, dyv, bq=None, bk=None, bv=None, *,
                           conv_state=None, dconv_state_out=None, eps=1e-6, want_dbias=None,
                           want_dconv_state=None, workspace=None):
    """Backward of gdr_block_prologue for incoming gradients dyq, dyk, dyv of
    (q, k, v) and optionally of the returned conv state.  Returns dict(dxq,
    dxk, dxv, dwq, dwk, dwv, dbq, dbk, dbv (None unless a bias was given or
    want_dbias), dconv_state (None unless conv_state was given or
    want_dconv_state))."""
    B, T, H, dk = xq.shape
    dv = xv.shape[-1]
    K = wq.shape[-1]
    for n, t in (("wq", wq), ("wk", wk), ("wv", wv), ("bq", bq), ("bk", bk), ("bv", bv)):
        _f32(t, n)
    want_db = (bq is not None) if want_dbias is None else want_dbias
    want_ds = (conv_state is not None) if want_dconv_state is None else want_dconv_state
    out = dict(dxq=torch.empty_like(xq), dxk=torch.empty_like(xk), dxv=torch.empty_like(xv))
    for n, t in (("dwq", wq), ("dwk", wk), ("dwv", wv)):
        out[n] = torch.empty_like(t)
    for n, d in (("dbq", dk), ("dbk", dk), ("dbv", dv)):
        out[n] = torch.empty(H * d, dtype=torch.float32, device=xq.device) if want_db else None
    out["dconv_state"] = (torch.empty(B, max(K - 1, 0), H * (2 * dk + dv), dtype=xq.dtype, device=xq.device)
                          if want_ds and K > 1 else None)
    L = lib()
    ws, ws_bytes = _workspace(L.gdr_block_prologue_bwd_workspace_bytes(H, dk, dv, K), xq.device, workspace)
    check(L.gdr_block_prologue_bwd(
        B, T, H, dk, dv, K, _dt(xq), _ptr(xq), _ptr(xk), _ptr(xv), _ptr(wq), _ptr(wk), _ptr(wv), _ptr(bq),
        _ptr(bk), _ptr(bv), _ptr(conv_state), float(eps), _ptr(dyq), _ptr(dyk), _ptr(dyv), _ptr(dconv_state_out),
        _ptr(out["dxq"]), _ptr(out["dxk"]), _ptr(out["dxv"]), _ptr(out["dwq"]), _ptr(out["dwk"]),
        _ptr(out["dwv"]), _ptr(out["dbq"]), _ptr(out["dbk"]), _ptr(out["dbv"]), _ptr(out["dconv_state"]),
        _ptr(ws), ws_bytes, _stream(xq)))
    return out


def gdr_block_epilogue(o, g, weight, eps=1e-6, *, y=None):
    """RMSNorm of the recurrent output over dv per (token, head), times the
    per-channel weight [dv] fp32 and SiLU(g) (g None: no gate).  o, g
    [B,T,H,dv].  Returns y."""
    B, T, H, dv = o.shape
    _f32(weight, "weight")
    y = torch.empty_like(o) if y is None else y
    check(lib().gdr_block_epilogue(B, T, H, dv, _dt(o), _ptr(o), _ptr(g), _ptr(weight), float(eps),
                                   _ptr(y), _stream(o)))
    return y


def gdr_block_epilogue_bwd(o, g, weight, dy, eps=1e-6, *, workspace=None):
    """Backward of gdr_block_epilogue for an incoming dy [B,T,H,dv]: returns
    (do, dg or None without a gate, dweight [dv] fp32)."""
    B, T, H, dv = o.shape
    _f32(weight, "weight")
    do = torch.empty_like(o)
    dg = None if g is None else torch.empty_like(g)
    dweight = torch.empty(dv, dtype=torch.float32, device=o.device)
    L = lib()
    ws, ws_bytes = _workspace(L.gdr_block_epilogue_bwd_workspace_bytes(dv), o.device, workspace)
    check(L.gdr_block_epilogue_bwd(B, T, H, dv, _dt(o), _ptr(o), _ptr(g), _ptr(weight), float(eps), _ptr(dy),
                                   _ptr(do), _ptr(dg), _ptr(dweight), _ptr(ws), ws_bytes, _stream(o)))
    return do, dg, dweight


def gdr_seg_fwd(q, k, v, log_alpha, beta, *, workspace=None):
    """Both forward passes of one segment of a split sequence: returns
    (o0 [B,T,H,dv] from S_in = 0, qt [B,T,H,dk] = M_<=t q_t,
     N [B,H,dv,dk], M [B,H,dk,dk])."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = _dt(q)
    o0 = torch.empty(B, T, H, dv, dtype=q.dtype, device=q.device)
    qt = torch.empty(B, T, H, dk, dtype=q.dtype, device=q.device)
    N = torch.empty(B, H, dv, dk, dtype=torch.float32, device=q.device)
    M = torch.empty(B, H, dk, dk, dtype=torch.float32, device=q.device)
    L = lib()
    ws, ws_bytes = _workspace(L.gdr_seg_fwd_workspace_bytes(B, T, H, dk, dv, dt), q.device, workspace)
    check(L.gdr_seg_fwd(B, T, H, dk, dv, dt, _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta),
                        _ptr(o0), _ptr(qt), _ptr(N), _ptr(M), _ptr(ws), ws_bytes, _stream(q)))
    return o0, qt, N, M


def gdr_seg_combine(M_all, N_all, r, S0=None, *, want_final=True):
    """Sequential combine of the segment maps: M_all [R,B,H,dk,dk], N_all
    [R,B,H,dv,dk] in segment order.  Returns (S_in of segment r, state after
    the last segment or None)."""
    R, B, H, dk, _ = M_all.shape
    dv = N_all.shape[3]
    _f32(M_all, "M_all"), _f32(N_all, "N_all"), _f32(S0, "S0")
    S_in = torch.empty(B, H, dv, dk, dtype=torch.float32, device=M_all.device)
    S_T = torch.empty_like(S_in) if want_final else None
    check(lib().gdr_seg_combine(R, r, B, H, dk, dv, _ptr(M_all), _ptr(N_all), _ptr(S0), _ptr(S_in),
                                _ptr(S_T), _stream(M_all)))
    return S_in, S_T


def gdr_seg_fixup(qt, S_in, o):
    """o += S_in q~ per token (in place); returns o."""
    B, T, H, dk = qt.shape
    dv = o.shape[-1]
    _f32(S_in, "S_in")
    check(lib().gdr_seg_fixup(B, T, H, dk, dv, _dt(qt), _ptr(qt), _ptr(S_in), _ptr(o), _stream(qt)))
    return o


def _mismatch(name, t, shape, dtype, device):
    """Raises what is wrong with an operand."""
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    raise ValueError("%s must be on the CUDA device of the other tensors (%s), got %s" % (name, device, t.device))


def _like(name, t, shape, dtype, device, keep=None):
    """`t` (None passes) as a dense operand of this shape, type and (CUDA) device; returns its address.  The library takes
    operands that start on 16 bytes: an input (`keep`: a list that outlives the launch) that does not is copied."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dtype or t.device != device:
        _mismatch(name, t, shape, dtype, device)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    at = t.data_ptr()
    if at & 15 and keep is not None:
        keep.append(t.clone())
        at = keep[-1].data_ptr()
    return at


def _ints(*sizes):
    """Sizes and strides are C ints: a larger one would wrap on its way into the library."""
    if max(sizes) >= 1 << 31:
        raise ValueError("sizes and strides must be below 2^31, got %s" % (sizes,))


def _rows(name, t, shape, lead, dtype, device, keep):
    """`t` as rows of a wider buffer: the axes from `lead` on are a dense row, and the rows of the leading axes are
    one stride apart.  Returns (address, stride in elements; 0: dense), of a dense copy in `keep` where `t` does not start
    on 16 bytes."""
    if t.shape != shape or t.dtype is not dtype or t.device != device:
        _mismatch(name, t, shape, dtype, device)
    if t.is_contiguous():
        return _like(name, t, shape, dtype, device, keep), 0
    strides = t.stride()
    width = 1
    for i in range(len(shape) - 1, lead - 1, -1):
        if shape[i] > 1 and strides[i] != width:
            raise ValueError("%s: the axes of a row must be contiguous" % name)
        width *= shape[i]
    ld, rows = 0, 1
    for i in range(lead - 1, -1, -1):
        if shape[i] > 1:
            if rows == 1:
                ld = strides[i]
                if ld < width:
                    raise ValueError("%s: rows must not overlap (stride %d, width %d)" % (name, ld, width))
            elif strides[i] != rows * ld:
                raise ValueError("%s: the rows of all batches must be one stride apart" % name)
            rows *= shape[i]
    _ints(ld)
    if t.data_ptr() & 15:
        keep.append(t.contiguous())
        return keep[-1].data_ptr(), 0
    return t.data_ptr(), ld


def _launch(device, fn, *args):
    """fn(*args, stream) on the device's current stream, with the device made current (launches go to that one)."""
    index = device.index
    if index == torch.cuda.current_device():
        check(fn(*args, torch._C._cuda_getCurrentRawStream(index)))
    else:
        with torch.cuda.device(index):
            check(fn(*args, torch._C._cuda_getCurrentRawStream(index)))


def _cuda(x, name):
    if not x.is_cuda:
        raise ValueError("%s must be on a CUDA device" % name)
    return x.device


def _scratch(nbytes, device, workspace):
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and on the tensors' device")
    return workspace, workspace.numel() * workspace.element_size()


def _ssm_operands(x, delta, A, Bm, Cm, D, delta_bias, lead, keep):
    """Sizes, type and addresses of the scan's inputs; lead = 2: [B,T,...], 1: [B,...]."""
    dev, dt = _cuda(x, "x"), _dt(x)
    if x.dim() != lead + 2 or Bm.dim() != lead + 2:
        raise ValueError("x and Bm must have %d axes, got %s and %s" % (lead + 2, tuple(x.shape), tuple(Bm.shape)))
    H, P = x.shape[-2:]
    G, N = Bm.shape[-2:]
    rows = x.shape[:lead]
    px, ldx = _rows("x", x, x.shape, lead, x.dtype, dev, keep)
    pb, ldb = _rows("Bm", Bm, rows + (G, N), lead, x.dtype, dev, keep)
    pc, ldc = _rows("Cm", Cm, rows + (G, N), lead, x.dtype, dev, keep)
    f = torch.float32
    pd = _like("delta", delta, rows + (H,), f, dev, keep)
    pA = _like("A", A, (H,), f, dev, keep)
    pD = _like("D", D, (H,), f, dev, keep)
    pbias = _like("delta_bias", delta_bias, (H,), f, dev, keep)
    return rows, H, G, P, N, dt, dev, (px, ldx, pd, pA, pb, ldb, pc, ldc, pD, pbias)


def gdr_ssm_fwd(x, delta, A, Bm, Cm, D=None, delta_bias=None, S0=None, *, softplus=False, y=None, S_T=None,
                return_state=True, workspace=None):
    """Selective state space scan: S_t = exp(A Delta_t) S_{t-1} + Delta_t x_t B_t^T, y_t = S_t C_t + D x_t, with
    Delta = softplus(delta + delta_bias) or delta + delta_bias.  x [B,T,H,P]; Bm, Cm [B,T,G,N] (H/G heads share a
    group); all three may be slices of one [B,T,channels] buffer.  delta [B,T,H], A, D, delta_bias [H] fp32; S0
    [B,H,P,N] fp32.  Returns (y, S_T or None)."""
    keep = []
    (B, T), H, G, P, N, dt, dev, ptrs = _ssm_operands(x, delta, A, Bm, Cm, D, delta_bias, 2, keep)
    y = x.new_empty((B, T, H, P)) if y is None else y
    if S_T is None and return_state:
        S_T = delta.new_empty((B, H, P, N))
    f = torch.float32
    L = lib()
    ws, ws_bytes = _scratch(L.gdr_ssm_fwd_workspace_bytes(B, T, H, G, P, N, dt), dev, workspace)
    _launch(dev, L.gdr_ssm_fwd, B, T, H, G, P, N, dt, int(softplus), *ptrs, _like("S0", S0, (B, H, P, N), f, dev, keep),
            _like("y", y, (B, T, H, P), x.dtype, dev), _like("S_T", S_T, (B, H, P, N), f, dev),
            ws.data_ptr(), ws_bytes)
    return y, S_T


def gdr_ssm_bwd(x, delta, A, Bm, Cm, D, delta_bias, S0, dy, dS_T=None, *, softplus=False, want_dS0=True,
                workspace=None):
    """Backward of gdr_ssm_fwd.  Returns dict(dx, ddelta, dA, dB, dC, dD, ddelta_bias, dS0); dD and ddelta_bias are
    None without D and delta_bias."""
    keep = []
    (B, T), H, G, P, N, dt, dev, ptrs = _ssm_operands(x, delta, A, Bm, Cm, D, delta_bias, 2, keep)
    f = torch.float32
    like = torch.empty_like  # the dense ones
    out = dict(dx=x.new_empty((B, T, H, P)), ddelta=like(delta), dA=like(A), dB=x.new_empty((B, T, G, N)),
               dC=x.new_empty((B, T, G, N)), dD=None if D is None else like(D),
               ddelta_bias=None if delta_bias is None else like(delta_bias),
               dS0=delta.new_empty((B, H, P, N)) if want_dS0 else None)
    L = lib()
    ws, ws_bytes = _scratch(L.gdr_ssm_bwd_workspace_bytes(B, T, H, G, P, N, dt), dev, workspace)
    _launch(dev, L.gdr_ssm_bwd, B, T, H, G, P, N, dt, int(softplus), *ptrs, _like("S0", S0, (B, H, P, N), f, dev, keep),
            _like("dy", dy, (B, T, H, P), x.dtype, dev, keep), _like("dS_T", dS_T, (B, H, P, N), f, dev, keep),
            *(None if t is None else t.data_ptr() for t in out.values()), ws.data_ptr(), ws_bytes)
    return out


def gdr_ssm_step(x, delta, A, Bm, Cm, S, D=None, delta_bias=None, *, softplus=False, y=None):
    """One token of gdr_ssm_fwd: x [B,H,P]; Bm, Cm [B,G,N]; delta [B,H]; S [B,H,P,N] fp32 advanced in place.
    Returns y [B,H,P]."""
    keep = []
    (B,), H, G, P, N, dt, dev, ptrs = _ssm_operands(x, delta, A, Bm, Cm, D, delta_bias, 1, keep)
    y = x.new_empty((B, H, P)) if y is None else y
    if S is None:
        raise ValueError("S is required")
    _launch(dev, lib().gdr_ssm_step, B, H, G, P, N, dt, int(softplus), *ptrs,
            _like("S", S, (B, H, P, N), torch.float32, dev),
            _like("y", y, (B, H, P), x.dtype, dev))
    return y


def _conv_operands(x, w, bias, conv_state, keep):
    dev, dt = _cuda(x, "x"), _dt(x)
    if x.dim() != 3 or w.dim() != 2:
        raise ValueError("x must be [B,T,C] and w [C,K], got %s and %s" % (tuple(x.shape), tuple(w.shape)))
    B, T, C = x.shape
    K = w.shape[1]
    _ints(B, T, C, K)
    px, ldx = _rows("x", x, x.shape, 2, x.dtype, dev, keep)
    return (B, T, C, K, dt, dev, (px, ldx, _like("w", w, (C, K), torch.float32, dev, keep),
                                  _like("bias", bias, (C,), torch.float32, dev, keep),
                                  _like("conv_state", conv_state, (B, max(K - 1, 0), C), x.dtype, dev, keep)))


def gdr_conv_fwd(x, w, bias=None, *, conv_state=None, conv_state_out=None, silu=True, y=None):
    """Depthwise causal convolution of width K with SiLU: x [B,T,C] (rows of a wider buffer are read in place), w
    [C,K] and bias [C] fp32.  conv_state [B,K-1,C] (dtype of x) carries the inputs before token 0; conv_state_out
    receives the last K-1 inputs and may be conv_state itself.  A decode token is T = 1.  Returns y [B,T,C]."""
    keep = []
    B, T, C, K, dt, dev, ptrs = _conv_operands(x, w, bias, conv_state, keep)
    y = x.new_empty((B, T, C)) if y is None else y
    _launch(dev, lib().gdr_conv_fwd, B, T, C, K, dt, int(silu), *ptrs,
            _like("conv_state_out", conv_state_out, (B, max(K - 1, 0), C), x.dtype, dev),
            _like("y", y, (B, T, C), x.dtype, dev))
    return y


def gdr_conv_bwd(x, w, dy, bias=None, *, conv_state=None, dconv_state_out=None, silu=True, want_dbias=None,
                 want_dconv_state=None, workspace=None):
    """Backward of gdr_conv_fwd.  Returns dict(dx, dw, dbias (None unless a bias was given or want_dbias),
    dconv_state (None unless conv_state was given or want_dconv_state))."""
    keep = []
    B, T, C, K, dt, dev, ptrs = _conv_operands(x, w, bias, conv_state, keep)
    f = torch.float32
    want_db = (bias is not None) if want_dbias is None else want_dbias
    want_ds = (conv_state is not None) if want_dconv_state is None else want_dconv_state
    out = dict(dx=torch.empty(B, T, C, dtype=x.dtype, device=dev), dw=torch.empty(C, K, dtype=f, device=dev),
               dbias=torch.empty(C, dtype=f, device=dev) if want_db else None,
               dconv_state=torch.empty(B, max(K - 1, 0), C, dtype=x.dtype, device=dev) if want_ds else None)
    L = lib()
    ws, ws_bytes = _scratch(L.gdr_conv_bwd_workspace_bytes(B, T, C, K), dev, workspace)
    _launch(dev, L.gdr_conv_bwd, B, T, C, K, dt, int(silu), *ptrs, _like("dy", dy, (B, T, C), x.dtype, dev, keep),
            _like("dconv_state_out", dconv_state_out, (B, max(K - 1, 0), C), x.dtype, dev, keep),
            *(None if t is None else t.data_ptr() for t in out.values()), ws.data_ptr(), ws_bytes)
    return out


def gdr_layernorm_fwd(x, weight, bias=None, *, residual=None, eps=1e-5, y=None, h=None):
    """Layer norm of h = x + residual over the last axis (x [...,D]; weight, bias [D] fp32).  Returns (y, h); h is
    None without a residual."""
    dev, dt, D = _cuda(x, "x"), _dt(x), x.shape[-1]
    _ints(D)
    y = x.new_empty(x.shape) if y is None else y
    if residual is not None and h is None:
        h = torch.empty(x.shape, dtype=x.dtype, device=dev)
    f, keep = torch.float32, []
    _launch(dev, lib().gdr_layernorm_fwd, x.numel() // max(D, 1), D, dt, _like("x", x, x.shape, x.dtype, dev, keep),
            _like("residual", residual, x.shape, x.dtype, dev, keep),
            _like("weight", weight, (D,), f, dev, keep), _like("bias", bias, (D,), f, dev, keep),
            float(eps), _like("y", y, x.shape, x.dtype, dev),
            _like("h", h, x.shape, x.dtype, dev))
    return y, h


def gdr_layernorm_bwd(h, weight, dy, *, dres=None, eps=1e-5, want_dbias=True, workspace=None):
    """Backward of gdr_layernorm_fwd from the stored stream h (x without a residual) and the gradient dres that
    reaches h along the residual stream.  Returns (dx, dweight, dbias or None)."""
    dev, dt, D = _cuda(h, "h"), _dt(h), h.shape[-1]
    _ints(D)
    f, keep = torch.float32, []
    dx = torch.empty(h.shape, dtype=h.dtype, device=dev)
    dweight = torch.empty(D, dtype=f, device=dev)
    dbias = torch.empty(D, dtype=f, device=dev) if want_dbias else None
    L = lib()
    ws, ws_bytes = _scratch(L.gdr_layernorm_bwd_workspace_bytes(D), dev, workspace)
    _launch(dev, L.gdr_layernorm_bwd, h.numel() // max(D, 1), D, dt, _like("h", h, h.shape, h.dtype, dev, keep),
            _like("weight", weight, (D,), f, dev, keep), float(eps),
            _like("dy", dy, h.shape, h.dtype, dev, keep), _like("dres", dres, h.shape, h.dtype, dev, keep),
            dx.data_ptr(), dweight.data_ptr(), None if dbias is None else dbias.data_ptr(),
            ws.data_ptr(), ws_bytes)
    return dx, dweight, dbias

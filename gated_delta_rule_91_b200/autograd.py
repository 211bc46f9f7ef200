"""torch.autograd bindings of the library's forward/backward pairs.

`gated_delta_rule(q, k, v, log_alpha, beta, S0=None)` returns (o, S_T) and
differentiates through gdr_bwd; `gated_delta_rule2(q, k, v, log_alpha, b, w,
S0=None)` does the same for Gated DeltaNet-2 through gdr2_bwd.  The forward
and the backward are the library's CUDA calls: these classes only save the
inputs and hand the incoming gradients over (the backward recomputes the
forward's states itself, so nothing else is kept).  Unused outputs arrive as
zero gradients (to the scan, the convolution and the layer norm as none).  `block_prologue(...)` (ShortConv, SiLU, q/k L2) and
`block_epilogue(o, g, weight, eps)` (RMSNorm, weight, SiLU gate) are the
block's steps around the recurrence, differentiated through
gdr_block_prologue_bwd and gdr_block_epilogue_bwd.  `selective_scan(x, delta, A,
Bm, Cm, ...)`, `short_conv(x, w, ...)` and `layer_norm(x, weight, ...)` wrap
gdr_ssm_fwd, gdr_conv_fwd and gdr_layernorm_fwd with their backwards, which
have no gradients of their own (a second derivative is an error).

A step may be captured in a CUDA graph.  torch ties the node that accumulates a
leaf's gradient to the stream on which the first live graph of that leaf was
built, so nothing of an eager step on the same leaves (its outputs, its loss)
may be alive when a backward is captured.
"""
import torch
from torch.autograd.function import once_differentiable

from . import (gdr2_bwd, gdr2_fwd, gdr_block_epilogue, gdr_block_epilogue_bwd, gdr_block_prologue,
               gdr_block_prologue_bwd, gdr_bwd, gdr_conv_bwd, gdr_conv_fwd, gdr_fwd, gdr_layernorm_bwd,
               gdr_layernorm_fwd, gdr_ssm_bwd, gdr_ssm_fwd)


def _c(x):
    return None if x is None else x.contiguous()


class GatedDeltaRule(torch.autograd.Function):
    """o_t = S_t q_t with S_t = S_{t-1} alpha_t (I - beta_t k_t k_t^T) + beta_t v_t k_t^T."""

    @staticmethod
    def forward(ctx, q, k, v, log_alpha, beta, S0):
        q, k, v, log_alpha, beta, S0 = map(_c, (q, k, v, log_alpha, beta, S0))
        o, S_T = gdr_fwd(q, k, v, log_alpha, beta, S0)
        ctx.save_for_backward(q, k, v, log_alpha, beta, S0)
        return o, S_T

    @staticmethod
    def backward(ctx, dO, dS_T):
        q, k, v, log_alpha, beta, S0 = ctx.saved_tensors
        g = gdr_bwd(q, k, v, log_alpha, beta, S0, _c(dO), _c(dS_T), want_dS0=S0 is not None)
        return g["dq"], g["dk"], g["dv"], g["dlog_alpha"], g["dbeta"], g["dS0"]


class GatedDeltaRule2(torch.autograd.Function):
    """Gated Delta Rule-2: per-channel decay alpha, erase gate b, write gate w."""

    @staticmethod
    def forward(ctx, q, k, v, log_alpha, b, w, S0):
        q, k, v, log_alpha, b, w, S0 = map(_c, (q, k, v, log_alpha, b, w, S0))
        o, S_T = gdr2_fwd(q, k, v, log_alpha, b, w, S0)
        ctx.save_for_backward(q, k, v, log_alpha, b, w, S0)
        return o, S_T

    @staticmethod
    def backward(ctx, dO, dS_T):
        q, k, v, log_alpha, b, w, S0 = ctx.saved_tensors
        g = gdr2_bwd(q, k, v, log_alpha, b, w, S0, _c(dO), _c(dS_T), want_dS0=S0 is not None)
        return g["dq"], g["dk"], g["dv"], g["dlog_alpha"], g["db"], g["dw"], g["dS0"]


def gated_delta_rule(q, k, v, log_alpha, beta, S0=None):
    """Differentiable gdr_fwd: returns (o, S_T)."""
    return GatedDeltaRule.apply(q, k, v, log_alpha, beta, S0)


def gated_delta_rule2(q, k, v, log_alpha, b, w, S0=None):
    """Differentiable gdr2_fwd: returns (o, S_T)."""
    return GatedDeltaRule2.apply(q, k, v, log_alpha, b, w, S0)


class BlockEpilogue(torch.autograd.Function):
    """y = RMSNorm(o) * weight * SiLU(g) over dv per (token, head)."""

    @staticmethod
    def forward(ctx, o, g, weight, eps):
        o, g = _c(o), _c(g)
        ctx.eps = eps
        ctx.save_for_backward(o, g, weight)
        return gdr_block_epilogue(o, g, weight, eps)

    @staticmethod
    def backward(ctx, dy):
        o, g, weight = ctx.saved_tensors
        do, dg, dweight = gdr_block_epilogue_bwd(o, g, weight, _c(dy), ctx.eps)
        return do, dg, dweight, None


def block_epilogue(o, g, weight, eps=1e-6):
    """Differentiable gdr_block_epilogue: returns y."""
    return BlockEpilogue.apply(o, g, weight, eps)


class BlockPrologue(torch.autograd.Function):
    """q = L2(SiLU(conv(xq))), k = L2(SiLU(conv(xk))), v = SiLU(conv(xv)),
    the convolution reading the carried conv state before token 0."""

    @staticmethod
    def forward(ctx, xq, xk, xv, wq, wk, wv, bq, bk, bv, conv_state, eps):
        xq, xk, xv, conv_state = map(_c, (xq, xk, xv, conv_state))
        ctx.eps = eps
        ctx.has_bias = bq is not None
        ctx.save_for_backward(xq, xk, xv, wq, wk, wv, bq, bk, bv, conv_state)
        return gdr_block_prologue(xq, xk, xv, wq, wk, wv, bq, bk, bv, conv_state=conv_state, eps=eps)

    @staticmethod
    def backward(ctx, dq, dk, dv):
        xq, xk, xv, wq, wk, wv, bq, bk, bv, conv_state = ctx.saved_tensors
        g = gdr_block_prologue_bwd(xq, xk, xv, wq, wk, wv, _c(dq), _c(dk), _c(dv), bq, bk, bv,
                                   conv_state=conv_state, eps=ctx.eps, want_dbias=ctx.has_bias,
                                   want_dconv_state=conv_state is not None)
        return (g["dxq"], g["dxk"], g["dxv"], g["dwq"], g["dwk"], g["dwv"], g["dbq"], g["dbk"], g["dbv"],
                g["dconv_state"], None)


def block_prologue(xq, xk, xv, wq, wk, wv, bq=None, bk=None, bv=None, conv_state=None, eps=1e-6):
    """Differentiable gdr_block_prologue: returns (q, k, v)."""
    return BlockPrologue.apply(xq, xk, xv, wq, wk, wv, bq, bk, bv, conv_state, eps)


def _dense_rows(x, lead):
    """x itself where the library reads it in place (rows of a wider buffer), a dense copy otherwise."""
    if x.is_contiguous():
        return x if x.data_ptr() % 16 == 0 else x.clone()
    shape, strides, width = x.shape, x.stride(), 1
    for i in range(len(shape) - 1, lead - 1, -1):
        if shape[i] > 1 and strides[i] != width:
            return x.contiguous()
        width *= shape[i]
    ld, rows = 0, 1
    for i in range(lead - 1, -1, -1):
        if shape[i] > 1:
            if (rows == 1 and strides[i] < width) or (rows > 1 and strides[i] != rows * ld):
                return x.contiguous()
            ld = strides[i] if rows == 1 else ld
            rows *= shape[i]
    per16 = 16 // x.element_size()
    return x if ld % per16 == 0 and x.data_ptr() % 16 == 0 else x.contiguous()


class SelectiveScan(torch.autograd.Function):
    """S_t = exp(A Delta_t) S_{t-1} + Delta_t x_t B_t^T, y_t = S_t C_t + D x_t."""

    @staticmethod
    def forward(ctx, x, delta, A, Bm, Cm, D, delta_bias, S0, softplus):
        x, Bm, Cm = (_dense_rows(t, 2) for t in (x, Bm, Cm))
        delta, S0 = _c(delta), _c(S0)
        ctx.softplus = softplus
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x, delta, A, Bm, Cm, D, delta_bias, S0)
        return gdr_ssm_fwd(x, delta, A, Bm, Cm, D, delta_bias, S0, softplus=softplus)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dS_T):
        x, delta, A, Bm, Cm, D, delta_bias, S0 = ctx.saved_tensors
        dy = torch.zeros_like(x, memory_format=torch.contiguous_format) if dy is None else _c(dy)
        g = gdr_ssm_bwd(x, delta, A, Bm, Cm, D, delta_bias, S0, dy, _c(dS_T), softplus=ctx.softplus,
                        want_dS0=S0 is not None and ctx.needs_input_grad[7])
        return g["dx"], g["ddelta"], g["dA"], g["dB"], g["dC"], g["dD"], g["ddelta_bias"], g["dS0"], None


def selective_scan(x, delta, A, Bm, Cm, D=None, delta_bias=None, S0=None, softplus=False):
    """Differentiable gdr_ssm_fwd: returns (y, S_T)."""
    return SelectiveScan.apply(x, delta, A, Bm, Cm, D, delta_bias, S0, softplus)


class ShortConv(torch.autograd.Function):
    """y = SiLU(bias + causal depthwise convolution of x), the window before token 0 from conv_state."""

    @staticmethod
    def forward(ctx, x, w, bias, conv_state, silu):
        x, conv_state = _dense_rows(x, 2), _c(conv_state)
        ctx.silu = silu
        ctx.save_for_backward(x, w, bias, conv_state)
        return gdr_conv_fwd(x, w, bias, conv_state=conv_state, silu=silu)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, w, bias, conv_state = ctx.saved_tensors
        g = gdr_conv_bwd(x, w, _c(dy), bias, conv_state=conv_state, silu=ctx.silu, want_dbias=ctx.needs_input_grad[2],
                         want_dconv_state=ctx.needs_input_grad[3])
        return g["dx"], g["dw"], g["dbias"], g["dconv_state"], None


def short_conv(x, w, bias=None, conv_state=None, silu=True):
    """Differentiable gdr_conv_fwd: returns y."""
    return ShortConv.apply(x, w, bias, conv_state, silu)


class LayerNorm(torch.autograd.Function):
    """y = LN(h) weight + bias with h = x + residual; h is returned for the next block's residual."""

    @staticmethod
    def forward(ctx, x, weight, bias, residual, eps):
        x, residual = _c(x), _c(residual)
        y, h = gdr_layernorm_fwd(x, weight, bias, residual=residual, eps=eps)
        ctx.eps, ctx.has_residual = eps, residual is not None
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x if h is None else h, weight)
        return y, h

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh):
        h, weight = ctx.saved_tensors
        dy = torch.zeros_like(h) if dy is None else _c(dy)
        dx, dweight, dbias = gdr_layernorm_bwd(h, weight, dy, dres=_c(dh), eps=ctx.eps, want_dbias=ctx.needs_input_grad[2])
        return dx, dweight, dbias, dx if ctx.has_residual else None, None


def layer_norm(x, weight, bias=None, residual=None, eps=1e-5):
    """Differentiable gdr_layernorm_fwd: returns y, or (y, h) with a residual."""
    y, h = LayerNorm.apply(x, weight, bias, residual, eps)
    return y if residual is None else (y, h)

"""The selective scan in blocks of 64 tokens in plain torch operations, in 64 or 32 bits and on any device, for lengths
where the token-by-token form of ssm_common takes too long; and how the library cuts a call."""
import ctypes
import math

import torch

import gated_delta_rule_91_b200 as gdr

Q = 64


def plan(B, T, H, G, P, N):
    out = (ctypes.c_int * 6)()
    gdr.check(gdr.lib().gdr_debug_ssm_plan(B, T, H, G, P, N, out))
    return dict(zip(("m", "R", "walk_m", "walk_R", "splits", "per"), out))


def _blocks(x, step, la, Bm, Cm, S0):
    """y without the skip, S_T.  la: the logarithms of the decays."""
    B, T, H, P = x.shape
    G, N = Bm.shape[2:]
    n = -(-T // Q)
    pad = lambda u: torch.cat([u, u.new_zeros(B, n * Q - T, *u.shape[2:])], 1).unflatten(1, (n, Q)).transpose(2, 3)  # noqa: E731
    of = torch.arange(H, device=x.device) // (H // G)
    xc, dc, b, c = pad(x), pad(step), pad(Bm[:, :, of]), pad(Cm[:, :, of])  # [B,n,H,Q,..], steps [B,n,H,Q]
    # the exponents are differences of sums: 64 bits in either form, as a caller of torch would
    cum = pad(la).double().cumsum(-1)
    low = torch.ones(Q, Q, dtype=torch.bool, device=x.device).tril()
    decay = (cum[..., :, None] - cum[..., None, :]).masked_fill(~low, -math.inf).exp().to(x.dtype)
    end = (cum[..., -1:] - cum).exp().to(x.dtype)
    y = ((c @ b.transpose(-1, -2)) * decay * dc[..., None, :]) @ xc
    u = (xc * (dc * end)[..., None]).transpose(-1, -2) @ b
    S = x.new_zeros(B, H, P, N) if S0 is None else S0
    ins = []
    for k in range(n):
        ins.append(S)
        S = cum[:, k, :, -1].exp().to(x.dtype)[..., None, None] * S + u[:, k]
    y = y + (c @ torch.stack(ins, 1).transpose(-1, -2)) * cum.exp().to(x.dtype)[..., None]
    return y.transpose(2, 3).flatten(1, 2)[:, :T], S


def scan_blocks(d, softplus=True, grads=False, absolute=False, dtype=torch.float64):
    """d: x, delta, A, Bm, Cm, D, bias, S0, dy, dS_T.  As ssm_common.scan64, with `absolute` the magnitudes."""
    f = lambda u: None if u is None else u.detach().to(dtype)  # noqa: E731
    x, delta, A, Bm, Cm, D, bias, S0, dy, dS_T = (f(d[k]) for k in ("x", "delta", "A", "Bm", "Cm", "D", "bias", "S0", "dy", "dS_T"))
    z = delta if bias is None else delta + bias
    step = z.clamp(min=0) + torch.log1p(torch.exp(-z.abs())) if softplus else z
    sig = torch.sigmoid(z) if softplus else torch.ones_like(z)
    la = step * A
    if absolute:
        x, Bm, Cm, step, A = x.abs(), Bm.abs(), Cm.abs(), step.abs(), A.abs()
        D, S0, dy, dS_T = (None if u is None else u.abs() for u in (D, S0, dy, dS_T))
    first = torch.zeros(x.shape[0], x.shape[2], x.shape[3], Bm.shape[3], dtype=dtype, device=x.device) if S0 is None else S0
    leaves = [u.clone().requires_grad_(grads) for u in (x, step, la, Bm, Cm, first)]
    y, S_T = _blocks(*leaves)
    out = dict(y=(y + (0 if D is None else D[:, None] * x)).detach(), S_T=S_T.detach())
    if not grads:
        return out
    dx, dw, dlog, dB, dC, dS0 = torch.autograd.grad((y, S_T), leaves, (dy, torch.zeros_like(S_T) if dS_T is None else dS_T))
    raw = (dw + A * dlog) * sig
    out.update(dx=dx + (0 if D is None else D[:, None] * dy), ddelta=raw, dA=(step * dlog).sum((0, 1)), dB=dB, dC=dC,
               dD=(dy * x).sum((0, 1, 3)), ddelta_bias=raw.sum((0, 1)), dS0=dS0)
    return out

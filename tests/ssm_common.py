"""Plain 64-bit forms of the selective scan, the short convolution and the layer norm for the tests, and the error
bounds that follow from the roundings the kernels make.

Bounds: `absolute=True` runs the same formulas on absolute values, which gives each output's sum of term
magnitudes M.  An output of type t is rounded once (eps(t)/2 of its value); bf16 tensor-core operands that are
rounded contribute eps(bf16)/2 = 2^-8 of M each; sums of n fp32 terms contribute n 2^-24 of M.
"""
import torch

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def scan64(x, delta, A, Bm, Cm, D=None, bias=None, S0=None, softplus=True, dy=None, dS_T=None, absolute=False):
    """Token by token.  Returns dict(y, S_T) and, with dy, the gradients."""
    f = lambda u: None if u is None else u.detach().cpu().double()  # noqa: E731
    x, delta, A, Bm, Cm, D, bias, S0, dy, dS_T = map(f, (x, delta, A, Bm, Cm, D, bias, S0, dy, dS_T))
    B, T, H, P = x.shape
    G, N = Bm.shape[2:]
    z = delta if bias is None else delta + bias
    step = torch.logaddexp(z, torch.zeros_like(z)) if softplus else z
    sig = torch.sigmoid(z) if softplus else torch.ones_like(z)
    a = torch.exp(step * A)
    if absolute:
        x, Bm, Cm, step, A = x.abs(), Bm.abs(), Cm.abs(), step.abs(), A.abs()
        D, S0, dy, dS_T = (None if u is None else u.abs() for u in (D, S0, dy, dS_T))
    of = torch.arange(H) // (H // G)
    b, c = Bm[:, :, of], Cm[:, :, of]
    S = torch.zeros(B, H, P, N, dtype=torch.float64) if S0 is None else S0.clone()
    states, ys = [S], []
    for t in range(T):
        S = a[:, t, :, None, None] * S + (step[:, t, :, None] * x[:, t])[..., None] * b[:, t, :, None, :]
        states.append(S)
        ys.append(torch.einsum("bhpn,bhn->bhp", S, c[:, t]))
    y = torch.stack(ys, 1) + (0 if D is None else D[:, None] * x)
    out = dict(y=y, S_T=S)
    if dy is None:
        return out
    g = torch.zeros_like(S) if dS_T is None else dS_T.clone()
    dx, db, dc = torch.zeros_like(x), torch.zeros_like(b), torch.zeros_like(c)
    dw, dlog = torch.zeros_like(step), torch.zeros_like(step)
    for t in reversed(range(T)):
        g = g + dy[:, t, :, :, None] * c[:, t, :, None, :]
        dc[:, t] = torch.einsum("bhp,bhpn->bhn", dy[:, t], states[t + 1])
        gb = torch.einsum("bhpn,bhn->bhp", g, b[:, t])
        dx[:, t] = step[:, t, :, None] * gb
        db[:, t] = step[:, t, :, None] * torch.einsum("bhpn,bhp->bhn", g, x[:, t])
        dw[:, t] = (gb * x[:, t]).sum(-1)
        g = a[:, t, :, None, None] * g
        dlog[:, t] = (g * states[t]).sum((-1, -2))
    group = lambda u: u.unflatten(2, (G, H // G)).sum(3)  # noqa: E731
    raw = (dw + A * dlog) * sig
    out.update(dx=dx + (0 if D is None else D[:, None] * dy), ddelta=raw, dA=(step * dlog).sum((0, 1)), dB=group(db),
               dC=group(dc), dD=(dy * x).sum((0, 1, 3)), ddelta_bias=raw.sum((0, 1)), dS0=g)
    return out


def conv64(x, w, bias=None, state=None, silu=True, dy=None, dstate_out=None, absolute=False):
    f = lambda u: None if u is None else u.detach().cpu().double()  # noqa: E731
    x, w, bias, state, dy, dstate_out = map(f, (x, w, bias, state, dy, dstate_out))
    B, T, C = x.shape
    K = w.shape[1]
    full = torch.cat([x.new_zeros(B, K - 1, C) if state is None else state, x], 1)
    z = sum(full[:, j:j + T] * w[:, j] for j in range(K)) + (0 if bias is None else bias)
    zabs = sum(full[:, j:j + T].abs() * w[:, j].abs() for j in range(K)) + (0 if bias is None else bias.abs())
    sg = torch.sigmoid(z) if silu else torch.ones_like(z)
    out = dict(y=z * sg, state=full[:, T:], zabs=zabs)
    if dy is None:
        return out
    if absolute:  # |silu'| <= 1.1 and |silu''| <= 0.5: a change of z by e changes dz by at most e |dy| / 2
        full, w, dy = full.abs(), w.abs(), dy.abs()
        dz = 1.1 * dy + zabs * dy
        dstate_out = None if dstate_out is None else dstate_out.abs()
    else:
        dz = dy * sg * (1 + z * (1 - sg)) if silu else dy
    dfull = torch.zeros_like(full)
    for j in range(K):
        dfull[:, j:j + T] += dz * w[:, j]
    if dstate_out is not None:
        dfull[:, T:] += dstate_out
    out.update(dx=dfull[:, K - 1:], dw=torch.stack([(dz * full[:, j:j + T]).sum((0, 1)) for j in range(K)], 1),
               dbias=dz.sum((0, 1)), dconv_state=dfull[:, :K - 1])
    return out


def norm64(h, w, b=None, eps=1e-5, dy=None, dres=None):
    """Also returns the magnitudes for the bounds: my for y, mx for dx, mw for dw."""
    f = lambda u: None if u is None else u.detach().cpu().double()  # noqa: E731
    h, w, b, dy, dres = map(f, (h, w, b, dy, dres))
    var, mean = torch.var_mean(h, -1, correction=0, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    n = (h - mean) * rstd
    # relative to fp32's half step: the mean's own error is that of |h|'s mean, scaled by rstd
    nerr = n.abs() + (h.abs() + h.abs().mean(-1, keepdim=True)) * rstd
    out = dict(y=n * w + (0 if b is None else b), my=nerr * w.abs() + (0 if b is None else b.abs()))
    if dy is None:
        return out
    g = dy * w
    mg, mgn = g.abs().mean(-1, keepdim=True), (g.abs() * nerr).mean(-1, keepdim=True)
    out.update(dx=rstd * (g - g.mean(-1, keepdim=True) - n * (g * n).mean(-1, keepdim=True)) + (0 if dres is None else dres),
               dw=(dy * n).sum(0), db=dy.sum(0), mw=(dy.abs() * nerr).sum(0), mb=dy.abs().sum(0),
               mx=rstd * (g.abs() + mg + nerr * mgn * 3) + (0 if dres is None else dres.abs()))
    return out


def within(got, want, bound, what=""):
    """Every element within its bound; a non-finite result fails."""
    got = got.detach().cpu().double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.isfinite(got).all(), what
    err = (got - want).abs()
    worst = (err / (bound + 1e-300)).max().item() if err.numel() else 0.0
    assert worst <= 1.0, "%s: error is %.3g of its bound" % (what, worst)

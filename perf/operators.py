"""What is measured of the selective-scan block's operators: the state space scan (prompt, gradients, single
token), the short causal convolution in front of it, and the layer norm with its residual.

`run` takes the framework's calls where `own` is true and plain torch operations elsewhere.  Notation: per batch
and head, with the step Delta_t = softplus(delta_t + delta_bias) and the decay a_t = exp(A Delta_t),
    S_t = a_t S_{t-1} + Delta_t x_t B_t^T,    y_t = S_t C_t + D x_t        (S: P x N, H/G heads share B and C)
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
CHUNK = 64  # tokens per block of the plain scan


# ---- the cases --------------------------------------------------------------------------------------------------

def listed():
    return [
        # one mixer layer of a training or prefill batch, at this repository's layer workload B=4 T=4096 H=16 d=128
        dict(name="scan_fwd_layer", op="scan_fwd", B=4, T=4096, H=16, G=1, P=128, N=128, dtype="bf16", s0=True),
        # a long document over few heads: the largest prompt
        dict(name="scan_fwd_long", op="scan_fwd", B=1, T=65536, H=16, G=2, P=64, N=128, dtype="bf16", s0=False),
        # an fp32 evaluation of a ragged prompt that goes on from a carried state, every head with its own B and C
        dict(name="scan_fwd_odd_f32", op="scan_fwd", B=3, T=777, H=6, G=6, P=64, N=64, dtype="f32", s0=True),
        # the gradients of the layer workload
        dict(name="scan_bwd_layer", op="scan_bwd", B=4, T=4096, H=16, G=1, P=128, N=128, dtype="bf16", s0=True),
        # a gradient check in fp32 at an odd length, groups of two heads, unequal P and N
        dict(name="scan_bwd_odd_f32", op="scan_bwd", B=2, T=333, H=4, G=2, P=128, N=64, dtype="f32", s0=True),
        # decoding a large batch, at this repository's decode workload B=256 H=16 d=128
        dict(name="scan_step_batch", op="scan_step", B=256, T=1, H=16, G=1, P=128, N=128, dtype="bf16", s0=True),
        # decoding one sequence: latency only
        dict(name="scan_step_one", op="scan_step", B=1, T=1, H=16, G=1, P=64, N=128, dtype="f32", s0=True),
        # the convolution over x, B and C (16 x 128 + 2 x 128 channels) of the layer workload
        dict(name="conv_fwd_layer", op="conv_fwd", B=4, T=4096, C=2304, K=4, dtype="bf16", bias=True, state=False),
        # the same channels for one token of the decode batch, with its carried window
        dict(name="conv_token_batch", op="conv_fwd", B=256, T=1, C=2304, K=4, dtype="bf16", bias=True, state=True),
        # the convolution's gradients at the layer workload
        dict(name="conv_bwd_layer", op="conv_bwd", B=4, T=4096, C=2304, K=4, dtype="bf16", bias=True, state=False),
        # the block's norm with the residual stream, B*T rows of H*d = 2048 channels
        dict(name="norm_fwd_layer", op="norm_fwd", R=16384, D=2048, dtype="bf16", bias=True, residual=True),
        # its gradients
        dict(name="norm_bwd_layer", op="norm_bwd", R=16384, D=2048, dtype="bf16", bias=True, residual=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan_fwd", "scan_fwd", "scan_bwd", "scan_bwd", "scan_step", "conv_fwd", "conv_bwd", "norm_fwd",
                     "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("scan"):
        G = rng.choice([1, 1, 2, 4])
        H = G * rng.randint(1, 16 // G)
        c = dict(op=op, H=H, G=G, P=rng.choice([64, 128]), N=rng.choice([64, 128]), dtype=dtype, s0=rng.random() < 0.5)
        if op == "scan_step":
            return dict(c, B=_log(rng, 1, 256), T=1, s0=True)
        B = _log(rng, 1, 8)
        # fp32 work is for checks and small models: up to a sixteenth of the largest bf16 length
        return dict(c, B=B, T=_log(rng, 1, (16384 if dtype == "bf16" else 2048) // B))
    if op.startswith("conv"):
        B = _log(rng, 1, 64)
        C = _log(rng, 64, 4096)
        C = C if rng.random() < 0.25 else -(-C // 64) * 64
        return dict(op=op, B=B, T=_log(rng, 1, max(1, min(8192, (1 << 25) // (B * C)))), C=C, K=rng.choice([2, 3, 4, 4, 7]),
                    dtype=dtype, bias=rng.random() < 0.7, state=rng.random() < 0.5)
    D = _log(rng, 64, 8192)
    D = D if rng.random() < 0.3 else -(-D // 64) * 64
    return dict(op=op, R=_log(rng, 1, max(1, min(32768, (1 << 25) // D))), D=D, dtype=dtype, bias=rng.random() < 0.7,
                residual=rng.random() < 0.6)


# ---- inputs -----------------------------------------------------------------------------------------------------

def prepare(case, seed):
    """Inputs on the GPU.  Activations follow the path's own distributions: the scan reads SiLU outputs, the step
    sizes lie between 0.001 and 0.1 around their bias, A in [-16, -1], taps are of the fan-in bound's size."""
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 1_000_003 + 17)
    t = TYPES[case["dtype"]]
    rand = lambda *s: torch.rand(*s, generator=g, device="cuda")  # noqa: E731
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    op, st = case["op"], dict(case)
    if op.startswith("scan"):
        B, T, H, G, P, N = (case[k] for k in "BTHGPN")
        xbc = randn(B, T, H * P + 2 * G * N)
        st["xbc"] = (xbc * torch.sigmoid(xbc)).to(t)  # one buffer: the convolution's output, sliced by the caller
        st["delta"] = 0.5 * randn(B, T, H)
        step = torch.exp(rand(H) * math.log(100.0) + math.log(0.001))
        st["delta_bias"] = step + torch.log(-torch.expm1(-step))  # softplus(delta_bias) = step
        st["A"] = -(1 + 15 * rand(H))
        st["D"] = 1 + 0.1 * randn(H)
        st["S0"] = 0.1 * randn(B, H, P, N) if case["s0"] else None
        if op == "scan_bwd":
            st["dy"] = randn(B, T, H, P).to(t)
            st["dS_T"] = 0.1 * randn(B, H, P, N) if case["s0"] else None
        if op == "scan_step":
            st["S"] = st.pop("S0")
    elif op.startswith("conv"):
        B, T, C, K = (case[k] for k in "BTCK")
        st["x"] = randn(B, T, C).to(t)
        st["w"] = (2 * rand(C, K) - 1) / math.sqrt(K)
        st["b"] = (2 * rand(C) - 1) / math.sqrt(K) if case["bias"] else None
        st["window"] = randn(B, K - 1, C).to(t) if case["state"] else None
        if op == "conv_bwd":
            st["dy"] = randn(B, T, C).to(t)
    else:
        R, D = case["R"], case["D"]
        st["x"] = (randn(R, D) + 0.3).to(t)
        st["res"] = randn(R, D).to(t) if case["residual"] else None
        st["w"] = 1 + 0.1 * randn(D)
        st["b"] = 0.1 * randn(D) if case["bias"] else None
        if op == "norm_bwd":
            st["dy"] = randn(R, D).to(t)
            st["dres"] = randn(R, D).to(t) if case["residual"] else None
    return st


def _slices(s):
    """x, B and C as views of the convolution's output."""
    H, G, P, N = (s[k] for k in "HGPN")
    x, Bm, Cm = s["xbc"].split([H * P, G * N, G * N], dim=-1)
    return x.unflatten(-1, (H, P)), Bm.unflatten(-1, (G, N)), Cm.unflatten(-1, (G, N))


# ---- one pass ---------------------------------------------------------------------------------------------------

EPS = 1e-5


def run(s):
    return {"scan_fwd": _scan_fwd, "scan_bwd": _scan_bwd, "scan_step": _scan_step, "conv_fwd": _conv_fwd,
            "conv_bwd": _conv_bwd, "norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd}[s["op"]](s)


def _softplus(z):
    return z.clamp(min=0) + torch.log1p(torch.exp(-z.abs()))


def _plain_scan(x, delta, A, Bm, Cm, D, bias, S0):
    """The scan in blocks of CHUNK tokens, fp32, block states by one product over the blocks; decay exponents are
    summed in 64 bits, since they are differences of long sums."""
    B, T, H, P = x.shape
    G, N = Bm.shape[2:]
    Q = CHUNK
    n = -(-T // Q)
    step = _softplus(delta + bias)
    pad = lambda u: torch.cat([u, u.new_zeros(B, n * Q - T, *u.shape[2:])], 1).unflatten(1, (n, Q))  # noqa: E731
    heads = lambda u: u.unsqueeze(4).expand(B, n, Q, G, H // G, N).reshape(B, n, Q, H, N).transpose(2, 3)  # noqa: E731
    xc, dc = pad(x).transpose(2, 3), pad(step).transpose(2, 3)  # [B, n, H, Q, P], [B, n, H, Q]
    bc, cc = heads(pad(Bm)), heads(pad(Cm))
    cum = (dc.double() * A.double()[:, None]).cumsum(-1)  # inside a block, inclusive
    ends = cum[..., -1].cumsum(1)  # over the blocks
    low = torch.ones(Q, Q, dtype=torch.bool, device=x.device).tril()
    decay = (cum[..., :, None] - cum[..., None, :]).masked_fill(~low, -math.inf).exp().float()
    y = ((cc @ bc.transpose(-1, -2)) * decay * dc[..., None, :]) @ xc
    u = (xc * (dc * (cum[..., -1:] - cum).exp().float())[..., None]).transpose(-1, -2) @ bc  # [B, n, H, P, N]
    first = torch.zeros_like(u[:, :1]) if S0 is None else S0[:, None]
    states = torch.cat([first, u], 1)  # the block states as one lower-triangular product over the blocks
    e = torch.cat([torch.zeros_like(ends[:, :1]), ends], 1).transpose(1, 2)  # [B, H, n + 1]
    low = torch.ones(n + 1, n + 1, dtype=torch.bool, device=x.device).tril()
    between = (e[..., :, None] - e[..., None, :]).masked_fill(~low, -math.inf).exp().float()
    states = (between @ states.transpose(1, 2).flatten(3)).unflatten(3, (P, N)).transpose(1, 2)
    y = y + (cc @ states[:, :-1].transpose(-1, -2)) * cum.exp().float()[..., None]
    y = y.transpose(2, 3).flatten(1, 2)[:, :T] + D[:, None] * x
    return y, states[:, -1]


def _scan_fwd(s):
    x, Bm, Cm = _slices(s)
    if own:
        import gated_delta_rule_91_b200 as gdr
        return gdr.gdr_ssm_fwd(x, s["delta"], s["A"], Bm, Cm, s["D"], s["delta_bias"], s["S0"], softplus=True)
    y, S_T = _plain_scan(x.float(), s["delta"], s["A"], Bm.float(), Cm.float(), s["D"], s["delta_bias"], s["S0"])
    return y.to(x.dtype), S_T


def _scan_bwd(s):
    x, Bm, Cm = _slices(s)
    if own:
        import gated_delta_rule_91_b200 as gdr
        g = gdr.gdr_ssm_bwd(x, s["delta"], s["A"], Bm, Cm, s["D"], s["delta_bias"], s["S0"], s["dy"], s["dS_T"],
                            softplus=True, want_dS0=s["S0"] is not None)
        return [g[k] for k in ("dx", "ddelta", "dA", "dB", "dC", "dD", "ddelta_bias")] + [g["dS0"]] * s["s0"]
    leaves = [u.detach().float().clone().requires_grad_() for u in (x, s["delta"], s["A"], Bm, Cm, s["D"], s["delta_bias"])]
    leaves += [s["S0"].clone().requires_grad_()] if s["s0"] else []
    y, S_T = _plain_scan(*leaves[:7], leaves[7] if s["s0"] else None)
    outs = (y, S_T) if s["s0"] else (y,)
    g = torch.autograd.grad(outs, leaves, (s["dy"].float(), s["dS_T"])[:len(outs)])
    return [u.to(v.dtype) for u, v in zip(g, (x, s["delta"], s["A"], Bm, Cm, s["D"], s["delta_bias"], s["S0"]))]


def _scan_step(s):
    x, Bm, Cm = (u[:, 0] for u in _slices(s))
    if own:
        import gated_delta_rule_91_b200 as gdr
        y = gdr.gdr_ssm_step(x, s["delta"][:, 0], s["A"], Bm, Cm, s["S"], s["D"], s["delta_bias"], softplus=True)
        return y, s["S"]
    step = _softplus(s["delta"][:, 0] + s["delta_bias"])
    b, c = (u.float().repeat_interleave(s["H"] // s["G"], 1) for u in (Bm, Cm))
    xf = x.float()
    s["S"].mul_(torch.exp(step * s["A"])[..., None, None]).add_((step[..., None] * xf)[..., None] * b[:, :, None])
    y = (s["S"] * c[:, :, None]).sum(-1) + s["D"][:, None] * xf
    return y.to(x.dtype), s["S"]


def _plain_conv(x, w, b, window):
    K = w.shape[1]
    before = x.new_zeros(x.shape[0], K - 1, x.shape[2]) if window is None else window
    z = (torch.cat([before, x], 1).unfold(1, K, 1) * w).sum(-1)
    z = z if b is None else z + b
    return z * torch.sigmoid(z)


def _conv_fwd(s):
    x, window = s["x"], s["window"]
    if own:
        import gated_delta_rule_91_b200 as gdr
        y = gdr.gdr_conv_fwd(x, s["w"], s["b"], conv_state=window, conv_state_out=window)
        return (y,) if window is None else (y, window)
    y = _plain_conv(x.float(), s["w"], s["b"], None if window is None else window.float()).to(x.dtype)
    if window is None:
        return (y,)
    window.copy_(torch.cat([window, x], 1)[:, x.shape[1]:])
    return y, window


def _conv_bwd(s):
    x, b, window = s["x"], s["b"], s["window"]
    if own:
        import gated_delta_rule_91_b200 as gdr
        g = gdr.gdr_conv_bwd(x, s["w"], s["dy"], b, conv_state=window)
        return [u for u in (g["dx"], g["dw"], g["dbias"], g["dconv_state"]) if u is not None]
    given = [u for u in (x, s["w"], b, window) if u is not None]
    leaves = [u.float().clone().requires_grad_() for u in given]
    rest = iter(leaves[2:])
    y = _plain_conv(leaves[0], leaves[1], next(rest) if b is not None else None, next(rest) if window is not None else None)
    g = torch.autograd.grad(y, leaves, s["dy"].float())
    return [u.to(v.dtype) for u, v in zip(g, given)]


def _plain_norm(h, w, b):
    c = h - h.mean(-1, keepdim=True)
    y = c * torch.rsqrt((c * c).mean(-1, keepdim=True) + EPS) * w
    return y if b is None else y + b


def _norm_fwd(s):
    x, res = s["x"], s["res"]
    if own:
        import gated_delta_rule_91_b200 as gdr
        y, h = gdr.gdr_layernorm_fwd(x, s["w"], s["b"], residual=res, eps=EPS)
        return (y,) if res is None else (y, h)
    h = x if res is None else (x.float() + res.float()).to(x.dtype)  # the stream as it is stored is what is normalised
    y = _plain_norm(h.float(), s["w"], s["b"]).to(x.dtype)
    return (y,) if res is None else (y, h)


def _norm_bwd(s):
    h = s["x"]  # the stored stream
    if own:
        import gated_delta_rule_91_b200 as gdr
        dx, dw, db = gdr.gdr_layernorm_bwd(h, s["w"], s["dy"], dres=s["dres"], eps=EPS, want_dbias=s["b"] is not None)
        return (dx, dw) if db is None else (dx, dw, db)
    leaves = [u.float().clone().requires_grad_() for u in (h, s["w"], s["b"]) if u is not None]
    y = _plain_norm(leaves[0], leaves[1], leaves[2] if s["b"] is not None else None)
    g = list(torch.autograd.grad(y, leaves, s["dy"].float()))
    if s["dres"] is not None:
        g[0] = g[0] + s["dres"].float()
    return [g[0].to(h.dtype)] + g[1:]


# ---- what a pass cannot do without ------------------------------------------------------------------------------

def work(case):
    op = case["op"]
    e = 4 if case["dtype"] == "f32" else 2
    if op.startswith("scan"):
        B, T, H, G, P, N = (case[k] for k in "BTHGPN")
        x, bc, d, st, par = B * T * H * P * e, 2 * B * T * G * N * e, B * T * H * 4, B * H * P * N * 4, 3 * H * 4
        pn = B * T * H * P * N
        if op == "scan_step":  # the state in and out
            return {"bytes": 2 * x + bc + d + par + 2 * st, "flops": 5 * pn}
        if op == "scan_fwd":  # per token: decay and update of the state, and its readout
            return {"bytes": 2 * x + bc + d + par + st * (2 if case["s0"] else 1), "flops": 5 * pn}
        # the state and its gradient, and the three products dx, dB and dC
        return {"bytes": 3 * x + 2 * bc + 2 * d + 2 * par + st * (3 if case["s0"] else 0), "flops": 12 * pn}
    if op.startswith("conv"):
        B, T, C, K = (case[k] for k in "BTCK")
        x, par, win = B * T * C * e, C * (K + case["bias"]) * 4, B * (K - 1) * C * e * case["state"]
        if op == "conv_fwd":
            return {"bytes": 2 * x + par + 2 * win, "flops": B * T * C * (2 * K + 4)}
        return {"bytes": 3 * x + 2 * par + 2 * win, "flops": B * T * C * (6 * K + 12)}
    R, D = case["R"], case["D"]
    x, par = R * D * e, D * 4 * (1 + case["bias"])
    if op == "norm_fwd":
        return {"bytes": x * (4 if case["residual"] else 2) + par, "flops": 8 * R * D}
    return {"bytes": x * (4 if case["residual"] else 3) + D * 4 + par, "flops": 14 * R * D}


# ---- the definition in 64 bits ----------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f = {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    if op.startswith("scan"):
        return _exact_scan(case, f)
    if op.startswith("conv"):
        return _exact_conv(case, f)
    return _exact_norm(case, s, f)


def _exact_scan(case, f):
    """Token by token.  Gradients: G_t = dL/dS_t runs backwards; the decay's gradient follows from
    <G_t, S_t> = dy_t . S_t C_t + (gradient of log a_{t+1}), so that no state has to be kept."""
    H, G, P, N, T = (case[k] for k in "HGPNT")
    x, Bm, Cm = f["xbc"].split([H * P, G * N, G * N], dim=-1)
    x = x.unflatten(-1, (H, P))
    of = torch.arange(H, device=x.device) // (H // G)
    Bm, Cm = (u.unflatten(-1, (G, N))[:, :, of] for u in (Bm, Cm))
    raw = f["delta"] + f["delta_bias"]
    step = torch.logaddexp(raw, torch.zeros_like(raw))
    a = torch.exp(step * f["A"])
    S = f.get("S0") if case["op"] != "scan_step" else f["S"]
    S = x.new_zeros(x.shape[0], H, P, N) if S is None else S.clone()
    bwd = case["op"] == "scan_bwd"
    ys, dCs = [], []
    for t in range(T):
        S.mul_(a[:, t, :, None, None]).addcmul_((step[:, t, :, None] * x[:, t])[..., None], Bm[:, t, :, None, :])
        ys.append((S @ Cm[:, t, :, :, None])[..., 0])
        if bwd:
            dCs.append((f["dy"][:, t, :, None, :] @ S)[:, :, 0])
    y = torch.stack(ys, 1)
    if not bwd:
        out = y + f["D"][:, None] * x
        return (out[:, 0], S) if case["op"] == "scan_step" else (out, S)
    dy = f["dy"]
    g = torch.zeros_like(S) if f["dS_T"] is None else f["dS_T"].clone()
    dlog = (g * S).sum((-1, -2))
    dot = (dy * y).sum(-1)
    dxs, dBs, dws, dls = [], [], [], []
    for t in reversed(range(T)):
        g.addcmul_(dy[:, t, :, :, None], Cm[:, t, :, None, :])
        gb = (g @ Bm[:, t, :, :, None])[..., 0]
        dw = (gb * x[:, t]).sum(-1)
        dlog = dlog + dot[:, t] - step[:, t] * dw
        dxs.append(step[:, t, :, None] * gb)
        dBs.append(((step[:, t, :, None] * x[:, t])[:, :, None, :] @ g)[:, :, 0])
        dws.append(dw)
        dls.append(dlog)
        g.mul_(a[:, t, :, None, None])
    back = lambda u: torch.stack(u[::-1], 1)  # noqa: E731
    dlog, dw = back(dls), back(dws)
    if f["S0"] is None:
        dlog[:, 0] = 0  # the first decay multiplies the zero state: no rounding of the sums above may stay there
    shared = lambda u: u.unflatten(2, (G, H // G)).sum(3)  # noqa: E731
    draw_ = (dw + dlog * f["A"]) * torch.sigmoid(raw)
    return [back(dxs) + f["D"][:, None] * dy, draw_, (dlog * step).sum((0, 1)), shared(back(dBs)),
            shared(torch.stack(dCs, 1)), (dy * x).sum((0, 1, 3)), draw_.sum((0, 1))] + [g] * case["s0"]


def _exact_conv(case, f):
    B, T, C, K = (case[k] for k in "BTCK")
    x, w = f["x"], f["w"]
    win = x.new_zeros(B, K - 1, C) if f["window"] is None else f["window"]
    full = torch.cat([win, x], 1)
    z = sum(full[:, j:j + T] * w[:, j] for j in range(K))
    z = z if f["b"] is None else z + f["b"]
    sig = 1 / (1 + torch.exp(-z))
    if case["op"] == "conv_fwd":
        return (z * sig,) + ((full[:, T:],) if case["state"] else ())
    dz = f["dy"] * sig * (1 + z * (1 - sig))
    dfull = torch.zeros_like(full)
    for j in range(K):
        dfull[:, j:j + T] += dz * w[:, j]
    dw = torch.stack([(dz * full[:, j:j + T]).sum((0, 1)) for j in range(K)], 1)
    return [dfull[:, K - 1:], dw] + [dz.sum((0, 1))] * case["bias"] + [dfull[:, :K - 1]] * case["state"]


def _exact_norm(case, s, f):
    h = f["x"]
    fwd = case["op"] == "norm_fwd"
    stored = None
    if fwd and case["residual"]:
        stored = (s["x"].double() + s["res"].double()).to(s["x"].dtype)  # the stored stream defines the norm's input
        h = stored.double()
    var, mean = torch.var_mean(h, -1, correction=0, keepdim=True)
    n = (h - mean) / torch.sqrt(var + EPS)
    if fwd:
        y = n * f["w"] + (0 if f["b"] is None else f["b"])
        return (y,) if stored is None else (y, stored)
    dn = f["dy"] * f["w"]
    dx = (dn - dn.mean(-1, keepdim=True) - n * (dn * n).mean(-1, keepdim=True)) / torch.sqrt(var + EPS)
    if f["dres"] is not None:
        dx = dx + f["dres"]
    return [dx, (f["dy"] * n).sum(0)] + [f["dy"].sum(0)] * case["bias"]

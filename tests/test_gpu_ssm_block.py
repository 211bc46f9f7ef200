"""The operators of a selective-scan block together, as a model uses them: layer norm with the residual stream, input
projection, short convolution over x, B and C, scan, gated output norm (gdr_block_epilogue), output projection.

Forward and gradients in fp32 against the same block in 64 bits (torch, differentiated by autograd); a prompt followed
by single tokens against the whole prompt; and the bf16 tensor-core kernels against the CUDA-core ones.
Bound of the fp32 block: seven steps, each within 512 * 2^-24 of its magnitudes (sums of up to 400 terms), whose errors
reach the output through two norms and two projections of gain below 4: 7 * 512 * 2^-24 * 16 = 3.5e-3 of the largest value.
"""
import os

import pytest
import torch

import gated_delta_rule_91_b200 as gdr
from gated_delta_rule_91_b200 import autograd as ag

pytestmark = pytest.mark.gpu
BOUND = 7 * 512 * 2.0 ** -24 * 16


class Block:
    """W: model width, H heads of P channels, G groups of N state columns."""

    def __init__(self, W=96, H=2, G=1, P=64, N=64, K=4, seed=0, dtype=torch.float32):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.W, self.H, self.G, self.P, self.N, self.K = W, H, G, P, N, K
        self.C = H * P + 2 * G * N
        p = dict(nw=1 + 0.1 * r(W), nb=0.1 * r(W), win=r(W, H * P + self.C + H) / W ** 0.5, cw=r(self.C, K) / K ** 0.5,
                 cb=0.1 * r(self.C), A=-(1 + 3 * torch.rand(H, generator=g)), D=1 + 0.1 * r(H), bias=-2 + 0.3 * r(H),
                 ew=1 + 0.1 * r(P), wout=r(H * P, W) / (H * P) ** 0.5)
        self.p = {k: v.cuda() for k, v in p.items()}
        self.dtype = dtype

    def parts(self, z):
        gate, xbc, delta = z.split([self.H * self.P, self.C, self.H], -1)
        return gate, xbc, delta

    def split(self, xbc):
        x, b, c = xbc.split([self.H * self.P, self.G * self.N, self.G * self.N], -1)
        return x.unflatten(-1, (self.H, self.P)), b.unflatten(-1, (self.G, self.N)), c.unflatten(-1, (self.G, self.N))

    def fused(self, u, res, p, S0=None):
        y, h = ag.layer_norm(u, p["nw"], p["nb"], residual=res)
        gate, xbc, delta = self.parts(y @ p["win"])
        x, b, c = self.split(ag.short_conv(xbc, p["cw"], p["cb"]))
        o, S = ag.selective_scan(x, delta.contiguous(), p["A"], b, c, p["D"], p["bias"], S0, softplus=True)
        e = ag.block_epilogue(o, gate.unflatten(-1, (self.H, self.P)), p["ew"], 1e-6)
        return e.flatten(2) @ p["wout"], h, S

    def plain(self, u, res, p):
        h = u + res
        y = torch.nn.functional.layer_norm(h, (self.W,), p["nw"], p["nb"], 1e-5)
        gate, xbc, delta = self.parts(y @ p["win"])
        B, T, C = xbc.shape
        full = torch.cat([xbc.new_zeros(B, self.K - 1, C), xbc], 1)
        z = (full.unfold(1, self.K, 1) * p["cw"]).sum(-1) + p["cb"]
        x, b, c = self.split(z * torch.sigmoid(z))
        step = torch.nn.functional.softplus(delta + p["bias"])
        of = torch.arange(self.H, device=u.device) // (self.H // self.G)
        S, ys = x.new_zeros(B, self.H, self.P, self.N), []
        for t in range(T):
            S = torch.exp(step[:, t] * p["A"])[..., None, None] * S + (step[:, t, :, None] * x[:, t])[..., None] * b[:, t, of, None, :]
            ys.append((S * c[:, t, of, None, :]).sum(-1) + p["D"][:, None] * x[:, t])
        o = torch.stack(ys, 1)
        g = gate.unflatten(-1, (self.H, self.P))
        e = o * torch.rsqrt((o * o).mean(-1, keepdim=True) + 1e-6) * p["ew"] * g * torch.sigmoid(g)
        return e.flatten(2) @ p["wout"], h, S


def test_block_forward_and_gradients():
    m = Block()
    g = torch.Generator().manual_seed(1)
    u, res, d1, d2 = (torch.randn(2, 150, m.W, generator=g).cuda() for _ in range(4))

    def run(fn, cast):
        leaves = {k: cast(v).detach().clone().requires_grad_() for k, v in {**m.p, "u": u, "res": res}.items()}
        out, h, S = fn(leaves["u"], leaves["res"], leaves)
        torch.autograd.backward((out, h), (cast(d1), cast(d2)))
        return [out, h, S] + [leaves[k].grad for k in sorted(leaves)], ["out", "h", "S"] + sorted(leaves)

    got, names = run(m.fused, lambda t: t.float())
    want, _ = run(m.plain, lambda t: t.double())
    for n, a, b in zip(names, got, want):
        assert (a.double() - b).abs().max() <= BOUND * b.abs().max(), n


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_prompt_then_tokens(dtype):
    """The windows and states that a prompt leaves carry on token by token as the whole prompt does."""
    H, G, P, N, K, B, T0, T = 4, 2, 64, 128, 4, 3, 140, 150
    g = torch.Generator().manual_seed(2)
    C = H * P + 2 * G * N
    r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    xbc, delta, w, b = r(B, T, C).to(dtype), r(B, T, H), r(C, K) / 2, 0.1 * r(C)
    A, D = -1 - 3 * torch.rand(H, generator=g).cuda(), 1 + 0.1 * r(H)

    def cut(y):
        x, bm, cm = y.split([H * P, G * N, G * N], -1)
        return x.unflatten(-1, (H, P)), bm.unflatten(-1, (G, N)), cm.unflatten(-1, (G, N))

    def prompt(xbc, delta):
        window = torch.zeros(B, K - 1, C, dtype=dtype, device="cuda")
        x, bm, cm = cut(gdr.gdr_conv_fwd(xbc, w, b, conv_state=window, conv_state_out=window))
        y, S = gdr.gdr_ssm_fwd(x, delta, A, bm, cm, D, softplus=True)
        return y, S, window

    y, S, window = prompt(xbc, delta)
    _, S1, win1 = prompt(xbc[:, :T0].contiguous(), delta[:, :T0].contiguous())
    for t in range(T0, T):
        x, bm, cm = (v[:, 0] for v in cut(gdr.gdr_conv_fwd(xbc[:, t:t + 1].contiguous(), w, b, conv_state=win1, conv_state_out=win1)))
        yt = gdr.gdr_ssm_step(x, delta[:, t].contiguous(), A, bm, cm, S1, D, softplus=True)
        # the token's output is rounded from fp32; the prompt's went through bf16 operands (2 * 2^-8 of the magnitudes)
        tol = 2.0 ** -6 if dtype == torch.bfloat16 else 2.0 ** -13
        assert (yt.float() - y[:, t].float()).abs().max() <= tol * y.float().abs().max()
    assert torch.equal(win1, window)
    assert (S1 - S).abs().max() <= 2.0 ** -13 * S.abs().max()


@pytest.mark.parametrize("P,N,H,G", [(64, 128, 4, 1), (128, 64, 2, 2), (64, 64, 3, 1), (128, 128, 2, 1)])
def test_tensor_core_kernels_against_cuda_cores(P, N, H, G, monkeypatch):
    """The same bf16 call through both sets of kernels: one rounding of the output, and 3 * 2^-8 of its magnitude for
    bf16 operands, on either side."""
    g = torch.Generator().manual_seed(P + N)
    r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    B, T = 2, 1100
    x, bm, cm, dy = r(B, T, H, P).bfloat16(), r(B, T, G, N).bfloat16(), r(B, T, G, N).bfloat16(), r(B, T, H, P).bfloat16()
    delta, A, D, bias = r(B, T, H), -1 - 3 * torch.rand(H, generator=g).cuda(), r(H), -2 + 0.3 * r(H)
    S0, dS = r(B, H, P, N), r(B, H, P, N)

    def both():
        y, S = gdr.gdr_ssm_fwd(x, delta, A, bm, cm, D, bias, S0, softplus=True)
        gr = gdr.gdr_ssm_bwd(x, delta, A, bm, cm, D, bias, S0, dy, dS, softplus=True)
        return [y, S] + list(gr.values())

    monkeypatch.delenv("GDR_SSM_KERNEL", raising=False)
    tc = both()
    monkeypatch.setitem(os.environ, "GDR_SSM_KERNEL", "simt")
    simt = both()
    for i, (a, b) in enumerate(zip(tc, simt)):
        a, b = a.double(), b.double()
        assert (a - b).norm() <= (4 * 2.0 ** -8 if tc[i].dtype == torch.bfloat16 else 2.0 ** -14) * b.norm(), i


def test_two_captured_graphs_with_workspaces_of_their_own():
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    H, P, N, T = 2, 64, 128, 2000
    call = []
    for _ in range(2):
        x, bm, cm = r(1, T, H, P).bfloat16(), r(1, T, 1, N).bfloat16(), r(1, T, 1, N).bfloat16()
        delta, A = r(1, T, H), -1 - torch.rand(H, generator=g).cuda()
        call.append(lambda x=x, bm=bm, cm=cm, delta=delta, A=A: gdr.gdr_ssm_fwd(x, delta, A, bm, cm, softplus=True))
    want = [f() for f in call]
    graphs, got = [], []
    for f in call:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(f())
    streams = [torch.cuda.Stream() for _ in call]
    for _ in range(3):
        for s, gr in zip(streams, graphs):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                gr.replay()
        torch.cuda.synchronize()
        for (y, S), (y2, S2) in zip(want, got):
            assert torch.equal(y, y2) and torch.equal(S, S2)


def test_captured_training_step_replays_like_eager():
    """Norm, convolution, scan and their gradients as one captured step over static buffers."""
    g = torch.Generator().manual_seed(21)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    B, T, H, P, G, N, K = 2, 200, 2, 64, 1, 64, 4
    C = H * P + 2 * G * N
    leaves = [(0.5 * r(B, T, C)).bfloat16(), 1 + 0.1 * r(C), 0.1 * r(C), 0.5 * r(C, K), 0.1 * r(C), r(B, T, H),
              -1 - torch.rand(H, generator=g), r(H)]
    leaves = [v.cuda().requires_grad_() for v in leaves]
    res, dy = r(B, T, C).bfloat16().cuda(), r(B, T, H, P).bfloat16().cuda()

    def step():
        x, nw, nb, w, b, delta, A, D = leaves
        h, stream = ag.layer_norm(x, nw, nb, res)
        c = ag.short_conv(h, w, b)
        xs, bm, cm = c.split([H * P, G * N, G * N], -1)
        y, _ = ag.selective_scan(xs.unflatten(-1, (H, P)), delta, A, bm.unflatten(-1, (G, N)), cm.unflatten(-1, (G, N)), D,
                                 softplus=True)
        torch.autograd.backward((y, stream), (dy, res))
        return y.detach()

    want = step().clone()
    grads = [v.grad.clone() for v in leaves]
    for v in leaves:
        v.grad = None
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    for v in leaves:
        v.grad = None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(2):
        got.zero_()
        for v in leaves:
            v.grad.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        for i, (v, e) in enumerate(zip(leaves, grads)):
            assert torch.equal(v.grad, e), i


def test_a_second_derivative_is_an_error():
    x = torch.randn(2, 8, 16, device="cuda", requires_grad=True)
    w = torch.randn(16, 4, device="cuda", requires_grad=True)
    dx, = torch.autograd.grad(ag.short_conv(x, w).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        dx.sum().backward()
    n, = torch.autograd.grad(ag.layer_norm(x, torch.ones(16, device="cuda")).square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        n.sum().backward()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_offsets_past_32_bits(dtype):
    """Rows 2^16 elements apart: the last tokens start more than 2^31 elements behind the first.  The same as dense rows."""
    g = torch.Generator().manual_seed(4)
    B, T, H, P, G, N, ld, K = 1, 33000, 1, 64, 1, 64, 1 << 16, 4
    C = H * P + 2 * G * N
    wide = torch.empty(B, T, ld, dtype=dtype, device="cuda")
    src = torch.randn(B, T, C, generator=g).to(dtype).cuda()
    wide[..., :C] = src
    w = torch.randn(C, K, generator=g).cuda()
    assert torch.equal(gdr.gdr_conv_fwd(wide[..., :C], w), gdr.gdr_conv_fwd(src, w))
    a, b = gdr.gdr_conv_bwd(wide[..., :C], w, src), gdr.gdr_conv_bwd(src, w, src)
    assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dw"], b["dw"])
    delta, A = torch.randn(B, T, H, generator=g).cuda(), torch.tensor([-1.5], device="cuda")

    def cut(v):
        x, bm, cm = v.split([H * P, G * N, G * N], -1)
        return x.unflatten(-1, (H, P)), delta, A, bm.unflatten(-1, (G, N)), cm.unflatten(-1, (G, N))

    dense = tuple(v.contiguous() for v in cut(src))
    for p, q in zip(gdr.gdr_ssm_fwd(*cut(wide[..., :C]), softplus=True), gdr.gdr_ssm_fwd(*dense, softplus=True)):
        assert torch.equal(p, q)
    dy = dense[0].flip(1).contiguous()
    a = gdr.gdr_ssm_bwd(*cut(wide[..., :C]), None, None, None, dy, softplus=True)
    b = gdr.gdr_ssm_bwd(*dense, None, None, None, dy, softplus=True)
    assert all(a[k] is None and b[k] is None or torch.equal(a[k], b[k]) for k in a)


def test_states_past_32_bits():
    """2^31 + 2^20 state elements in one step: the last batch advances as it does alone."""
    g = torch.Generator().manual_seed(6)
    H, P, N = 64, 128, 128
    B = (1 << 31) // (H * P * N) + 1
    r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    x, bm, cm = r(B, H, P).bfloat16(), r(B, 1, N).bfloat16(), r(B, 1, N).bfloat16()
    delta, A = r(B, H), -1 - torch.rand(H, generator=g).cuda()
    S = torch.empty(B, H, P, N, device="cuda")
    S[0], S[-1] = 1.0, 0.5
    S[1:-1] = 0
    y = gdr.gdr_ssm_step(x, delta, A, bm, cm, S, softplus=True)
    for i, v in ((0, 1.0), (B - 1, 0.5)):
        one = torch.full((1, H, P, N), v, device="cuda")
        yi = gdr.gdr_ssm_step(x[i:i + 1], delta[i:i + 1], A, bm[i:i + 1], cm[i:i + 1], one, softplus=True)
        assert torch.equal(yi, y[i:i + 1]) and torch.equal(one[0], S[i])

"""gdr_layernorm_fwd and gdr_layernorm_bwd against the layer norm in 64 bits.  Bounds: sums over a row in fp32 (a
thread's elements, then a tree: fewer than 80 additions deep), the root and quotient a few units; one rounding of the output."""
import pytest
import torch

import gated_delta_rule_91_b200 as gdr
from gated_delta_rule_91_b200 import autograd as ag
from ssm_common import HALF, norm64, within

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
U = 2.0 ** -24


def inputs(R, D, dtype="bf16", seed=0, mean=0.3):
    g = torch.Generator().manual_seed(seed)
    t = TYPES[dtype]
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return dict(x=(r(R, D) + mean).to(t).cuda(), res=r(R, D).to(t).cuda(), w=(1 + 0.1 * r(D)).cuda(), b=(0.1 * r(D)).cuda(),
                dy=r(R, D).to(t).cuda(), dres=r(R, D).to(t).cuda())


def check(d, residual=True, bias=True, eps=1e-5):
    t = d["x"].dtype
    b = d["b"] if bias else None
    y, h = gdr.gdr_layernorm_fwd(d["x"], d["w"], b, residual=d["res"] if residual else None, eps=eps)
    if residual:
        assert torch.equal(h, (d["x"].float() + d["res"].float()).to(t))
    else:
        assert h is None
        h = d["x"]
    dres = d["dres"] if residual else None
    dx, dw, db = gdr.gdr_layernorm_bwd(h, d["w"], d["dy"], dres=dres, eps=eps, want_dbias=bias)
    r = norm64(h, d["w"], b, eps, d["dy"], dres)
    k = 100 * U
    within(y, r["y"], HALF[t] * r["y"].abs() + k * r["my"], "y")
    within(dx, r["dx"], HALF[t] * r["dx"].abs() + k * r["mx"], "dx")
    rows = (100 + d["x"].shape[0]) * U
    within(dw, r["dw"], rows * r["mw"], "dw")
    if bias:
        within(db, r["db"], rows * r["mb"], "db")
    else:
        assert db is None


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [1, 2, 7, 8, 33, 64, 100, 128, 256, 257, 511, 512, 513, 1024, 1025, 2047, 2048, 2056, 4096,
                               4104, 5001, 8192, 8200, 16383, 16384])
def test_widths(D, dtype):
    check(inputs(5, D, dtype, seed=D))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("R", [1, 2, 7, 8, 9, 600, 5001])
def test_rows(R, dtype):
    check(inputs(R, 128, dtype, seed=R))
    check(inputs(R, 576, dtype, seed=R + 1), residual=False)


@pytest.mark.parametrize("residual,bias,eps", [(False, False, 1e-5), (True, False, 1e-6), (False, True, 0.1)])
def test_options(residual, bias, eps):
    check(inputs(40, 320, "bf16"), residual, bias, eps)
    check(inputs(40, 320, "f32"), residual, bias, eps)


def test_large_mean_and_constant_rows():
    """A mean a hundred times the spread, and rows whose variance is 0 (eps alone)."""
    check(inputs(20, 768, "f32", seed=1, mean=100.0), residual=False)
    d = inputs(6, 256, "f32", seed=2)
    d["x"][:3] = 2.0
    check(d, residual=False, eps=1e-3)


def test_leading_axes_autograd_and_graph():
    d = inputs(24, 192, "bf16", seed=3)
    v = {k: (u.reshape(4, 6, 192) if u.dim() == 2 else u) for k, u in d.items()}
    x, res, w, b = (v[k].detach().clone().requires_grad_() for k in ("x", "res", "w", "b"))
    y, h = ag.layer_norm(x, w, b, residual=res)
    torch.autograd.backward((y, h), (v["dy"], v["dres"]))
    call = lambda: gdr.gdr_layernorm_bwd(h.detach(), v["w"], v["dy"], dres=v["dres"])  # noqa: E731
    dx, dw, db = call()
    assert torch.equal(x.grad, dx) and torch.equal(res.grad, dx) and torch.equal(w.grad, dw) and torch.equal(b.grad, db)
    x.grad = None
    ag.layer_norm(x, w.detach()).float().sum().backward()
    assert x.grad is not None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(out, (dx, dw, db)))


def test_refusals():
    d = inputs(4, 64, "bf16")
    for bad in (dict(x=d["x"].half()), dict(x=d["x"].t()), dict(weight=d["w"][:32]), dict(weight=d["w"].bfloat16()),
                dict(bias=d["b"].cpu()), dict(residual=d["res"].float()), dict(eps=-1.0), dict(eps=float("nan")),
                dict(h=torch.empty_like(d["x"]))):
        with pytest.raises((TypeError, ValueError, gdr.GdrError)):
            gdr.gdr_layernorm_fwd(**{**dict(x=d["x"], weight=d["w"], bias=d["b"]), **bad})
    with pytest.raises(gdr.GdrError):
        gdr.gdr_layernorm_fwd(torch.zeros(1, 16385, device="cuda"), torch.zeros(16385, device="cuda"))
    with pytest.raises(gdr.GdrError):
        gdr.gdr_layernorm_bwd(d["x"], d["w"], d["dy"], workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("R,D,dtype", [(3, 513, "bf16"), (700, 520, "bf16"), (900, 1032, "bf16"), (300, 516, "f32"), (300, 2052, "f32"),
                                       (100, 4104, "bf16"), (40, 6000, "bf16"), (61, 16383, "bf16")])
def test_rows_that_leave_warps_short(R, D, dtype):
    """The last warps of a row hold fewer columns or none; the mean (5) is far from zero."""
    check(inputs(R, D, dtype, seed=2, mean=5), True, True, 1e-5)

"""What a loss does not use costs nothing: outputs without a gradient reach the library as none, and gradients that nobody
asked for are not computed."""
import pytest
import torch

from gated_delta_rule_91_b200 import autograd as ag
from test_gpu_ssm import inputs

pytestmark = pytest.mark.gpu


@pytest.fixture
def calls(monkeypatch):
    seen = []
    for name in ("gdr_ssm_bwd", "gdr_conv_bwd", "gdr_layernorm_bwd"):
        def spy(*a, _f=getattr(ag, name), **k):
            out = _f(*a, **k)
            seen.append((a, k, out))
            return out
        monkeypatch.setattr(ag, name, spy)
    return seen


def test_scan(calls):
    d = inputs(2, 60, 2, 1, 64, 64, "bf16", seed=1)
    x = d["x"].detach().clone().requires_grad_()
    args = (d["delta"], d["A"], d["Bm"], d["Cm"], d["D"], d["bias"])
    y, S_T = ag.selective_scan(x, *args, d["S0"], softplus=True)
    y.backward(d["dy"])
    a, k, out = calls[0]
    assert a[9] is None and out["dS0"] is None  # no gradient of S_T, S0 is no leaf
    x.grad = None
    S0 = d["S0"].clone().requires_grad_()
    _, S_T = ag.selective_scan(x, *args, S0, softplus=True)  # y unused
    S_T.backward(d["dS_T"])
    a, k, out = calls[1]
    assert (a[8] == 0).all() and a[9] is not None and torch.equal(S0.grad, out["dS0"]) and torch.equal(x.grad, out["dx"])


def test_convolution_and_norm(calls):
    x = torch.randn(2, 30, 64, device="cuda", requires_grad=True)
    w, b, s = torch.randn(64, 4, device="cuda"), torch.randn(64, device="cuda"), torch.randn(2, 3, 64, device="cuda")
    ag.short_conv(x, w, b, s).sum().backward()
    assert calls[0][2]["dbias"] is None and calls[0][2]["dconv_state"] is None
    res, nw = torch.randn_like(x).requires_grad_(), torch.ones(64, device="cuda", requires_grad=True)
    x.grad = None
    y, h = ag.layer_norm(x, nw, torch.zeros(64, device="cuda"), res)
    y.square().sum().backward()
    a, k, out = calls[1]
    assert k["dres"] is None and out[2] is None and torch.equal(x.grad, res.grad)
    x.grad = res.grad = None
    y, h = ag.layer_norm(x, nw, None, res)
    h.sum().backward()  # the stream alone
    assert torch.equal(x.grad, torch.ones_like(x)) and torch.equal(res.grad, x.grad)

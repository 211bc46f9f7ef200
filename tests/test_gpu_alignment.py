"""Calls on tensors that do not start on 16 bytes: views of one token, of an odd channel, of one flat parameter buffer."""
import pytest
import torch

import gated_delta_rule_91_b200 as gdr
from gated_delta_rule_91_b200 import autograd as ag
from test_gpu_ssm import inputs

pytestmark = pytest.mark.gpu


def test_tokens_of_one_sequence_with_six_heads():
    d = inputs(1, 7, 6, 1, 64, 64, "bf16", seed=1)
    S, want = d["S0"].clone(), d["S0"].clone()
    for t in range(7):
        assert d["delta"][:, t].is_contiguous()
        y = gdr.gdr_ssm_step(d["x"][:, t], d["delta"][:, t], d["A"], d["Bm"][:, t], d["Cm"][:, t], S, d["D"], d["bias"], softplus=True)
        r = gdr.gdr_ssm_step(d["x"][:, t], d["delta"][:, t].clone(), d["A"], d["Bm"][:, t], d["Cm"][:, t], want, d["D"], d["bias"],
                             softplus=True)
        assert torch.equal(y, r) and torch.equal(S, want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_tokens_of_an_odd_number_of_channels(dtype):
    g = torch.Generator().manual_seed(2)
    x, w = torch.randn(1, 9, 37, generator=g).to(dtype).cuda(), torch.randn(37, 4, generator=g).cuda()
    whole = gdr.gdr_conv_fwd(x, w)
    window = torch.zeros(1, 3, 37, dtype=dtype, device="cuda")
    parts = [gdr.gdr_conv_fwd(x[:, t:t + 1], w, conv_state=window, conv_state_out=window) for t in range(9)]
    assert torch.equal(torch.cat(parts, 1), whole)
    rows = torch.randn(9, 37, generator=g).to(dtype).cuda()
    y, _ = gdr.gdr_layernorm_fwd(rows, torch.ones(37, device="cuda"))
    for i in range(9):
        assert torch.equal(gdr.gdr_layernorm_fwd(rows[i], torch.ones(37, device="cuda"))[0], y[i])


def test_parameters_in_one_flat_buffer():
    """A, D, the bias, taps and weights as views of a buffer, the gradients through autograd, one step captured."""
    d = inputs(2, 40, 3, 1, 64, 64, "bf16", seed=3)
    flat = torch.cat([torch.zeros(1, device="cuda"), d["A"], d["D"], d["bias"]]).requires_grad_()
    y, _ = ag.selective_scan(d["x"], d["delta"], flat[1:4], d["Bm"], d["Cm"], flat[4:7], flat[7:10], softplus=True)
    y.backward(d["dy"])
    g = gdr.gdr_ssm_bwd(d["x"], d["delta"], d["A"], d["Bm"], d["Cm"], d["D"], d["bias"], None, d["dy"], softplus=True)
    assert torch.equal(flat.grad[1:], torch.cat([g["dA"], g["dD"], g["ddelta_bias"]]))
    buf = torch.randn(1 + 2 * 40 * 192, device="cuda").bfloat16()
    x = buf[1:].view(2, 40, 192)
    w = torch.randn(192, 4, device="cuda")
    leaf = x.detach().requires_grad_()
    out = ag.short_conv(leaf, w)
    out.backward(torch.ones_like(out))
    assert torch.equal(out, gdr.gdr_conv_fwd(x.clone(), w))
    assert torch.equal(leaf.grad, gdr.gdr_conv_bwd(x.clone(), w, torch.ones_like(out))["dx"])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        again = gdr.gdr_conv_fwd(x, w)
    x.copy_(torch.randn(2, 40, 192, device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(again, gdr.gdr_conv_fwd(x.clone(), w))

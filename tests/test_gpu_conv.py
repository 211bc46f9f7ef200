"""gdr_conv_fwd and gdr_conv_bwd against the convolution in 64 bits.

Bounds: z is a sum of K + 1 fp32 terms; SiLU has slope at most 1.1 and its exponential, sum, and quotient add a few
units (__expf: 2 + |z| units, so 32 covers |z| <= 16); the output is rounded once."""
import pytest
import torch

import gated_delta_rule_91_b200 as gdr
from gated_delta_rule_91_b200 import autograd as ag
from ssm_common import HALF, conv64, within

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
U = 2.0 ** -24


def inputs(B, T, C, K, dtype="bf16", bias=True, state=True, extra=0, seed=0):
    g = torch.Generator().manual_seed(seed)
    t = TYPES[dtype]
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return dict(x=r(B, T, C + extra).to(t).cuda()[..., :C], w=(r(C, K) * 0.5).cuda(), bias=r(C).cuda() if bias else None,
                state=r(B, K - 1, C).to(t).cuda() if state else None, dy=r(B, T, C).to(t).cuda(),
                dstate=r(B, K - 1, C).to(t).cuda() if state else None)


def check(d, silu=True):
    t = d["x"].dtype
    B, T, C = d["x"].shape
    so = torch.empty_like(d["state"]) if d["state"] is not None else None
    y = gdr.gdr_conv_fwd(d["x"], d["w"], d["bias"], conv_state=d["state"], conv_state_out=so, silu=silu)
    r = conv64(d["x"], d["w"], d["bias"], d["state"], silu, d["dy"], d["dstate"])
    m = conv64(d["x"], d["w"], d["bias"], d["state"], silu, d["dy"], d["dstate"], absolute=True)
    within(y, r["y"], HALF[t] * r["y"].abs() + 32 * U * m["zabs"], "y")
    if so is not None:
        assert torch.equal(so.cpu().double(), r["state"])
    g = gdr.gdr_conv_bwd(d["x"], d["w"], d["dy"], d["bias"], conv_state=d["state"], dconv_state_out=d["dstate"], silu=silu)
    within(g["dx"], r["dx"], HALF[t] * r["dx"].abs() + 32 * U * m["dx"], "dx")
    # a thread's run, eight runs a slot, then 64-bit sums: at most B*T terms in fp32
    n = 32 + B * T
    within(g["dw"], r["dw"], n * U * m["dw"], "dw")
    if d["bias"] is not None:
        within(g["dbias"], r["dbias"], n * U * m["dbias"], "dbias")
    if d["state"] is not None:
        within(g["dconv_state"], r["dconv_state"], HALF[t] * r["dconv_state"].abs() + 32 * U * m["dconv_state"], "dconv_state")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [1, 2, 3, 4, 5, 6, 7, 8])
def test_widths(K, dtype):
    check(inputs(2, 45, 72, K, dtype, seed=K))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 15, 16, 17, 31, 32, 33, 64, 100, 300])
def test_lengths(T, dtype):
    check(inputs(3, T, 64, 4, dtype, seed=T))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("C,extra", [(1, 0), (7, 0), (130, 3), (64, 8), (256, 24), (1000, 0), (12, 4), (68, 0)])
def test_channels_and_strides(C, extra, dtype):
    check(inputs(2, 37, C, 4, dtype, extra=extra, seed=C))


@pytest.mark.parametrize("bias,state,silu", [(False, True, True), (True, False, True), (False, False, False), (True, True, False)])
def test_options(bias, state, silu):
    check(inputs(2, 50, 40, 4, "bf16", bias=bias, state=state), silu)
    check(inputs(2, 50, 40, 3, "f32", bias=bias, state=state), silu)


def test_many_runs_and_extreme_inputs():
    check(inputs(9, 700, 160, 4, "bf16", seed=2))
    d = inputs(1, 40, 16, 4, "f32", seed=3)
    d["x"][0, 3] = 200.0   # exp(-z) overflows for z < -88: SiLU goes to -0, not to NaN
    d["x"][0, 9] = -200.0
    y = gdr.gdr_conv_fwd(d["x"], d["w"], d["bias"])
    r = conv64(d["x"], d["w"], d["bias"])
    # the exponential's relative error grows with |z| (up to 100 here per tap), where z sigmoid(z) is z or next to 0
    within(y, r["y"], 1000 * U * (r["y"].abs() + 1), "y")


def test_window_in_place_and_tokens_follow_a_prompt():
    d = inputs(4, 60, 96, 4, "bf16", seed=4)
    whole = gdr.gdr_conv_fwd(d["x"], d["w"], d["bias"], conv_state=d["state"])
    window = d["state"].clone()
    parts = [gdr.gdr_conv_fwd(d["x"][:, :37].contiguous(), d["w"], d["bias"], conv_state=window, conv_state_out=window)]
    for t in range(37, 60):  # tokens
        parts.append(gdr.gdr_conv_fwd(d["x"][:, t:t + 1], d["w"], d["bias"], conv_state=window, conv_state_out=window))
    assert torch.equal(torch.cat(parts, 1), whole)
    assert torch.equal(window, d["x"][:, -3:])


def test_autograd_graph_and_repeat():
    d = inputs(2, 80, 64, 4, "bf16", seed=5, extra=64)
    x, w, b, s = (d[k].detach().clone().requires_grad_() for k in ("x", "w", "bias", "state"))
    y = ag.short_conv(x, w, b, s)
    y.backward(d["dy"])
    call = lambda: gdr.gdr_conv_bwd(d["x"], d["w"], d["dy"], d["bias"], conv_state=d["state"])  # noqa: E731
    g = call()
    for leaf, n in ((x, "dx"), (w, "dw"), (b, "dbias"), (s, "dconv_state")):
        assert torch.equal(leaf.grad, g[n]), n
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g2 = call()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(g[k], g2[k]) for k in g)


def test_workspace_and_refusals():
    d = inputs(2, 50, 40, 4, "bf16")
    need = gdr.lib().gdr_conv_bwd_workspace_bytes(2, 50, 40, 4)
    buf = torch.full((need + 1024,), 77, dtype=torch.uint8, device="cuda")
    gdr.gdr_conv_bwd(d["x"], d["w"], d["dy"], d["bias"], workspace=buf[:need])
    assert (buf[need:] == 77).all()
    with pytest.raises(gdr.GdrError):
        gdr.gdr_conv_bwd(d["x"], d["w"], d["dy"], d["bias"], workspace=buf[:need - 1])
    for bad in (dict(x=d["x"].half()), dict(x=d["x"].transpose(0, 1)), dict(w=d["w"].bfloat16()), dict(w=d["w"][:8]),
                dict(bias=d["bias"][:4]), dict(conv_state=d["state"][:, :2]), dict(conv_state_out=d["state"].float()),
                dict(x=d["x"][:, :1].expand(2, 50, 40))):
        with pytest.raises((TypeError, ValueError, gdr.GdrError)):
            gdr.gdr_conv_fwd(**{**dict(x=d["x"], w=d["w"], bias=d["bias"]), **bad})
    with pytest.raises(gdr.GdrError):
        gdr.gdr_conv_fwd(d["x"], torch.zeros(40, 9, device="cuda"))


@pytest.mark.parametrize("B,T,C,K,dtype", [(5000, 3, 64, 4, "bf16"), (1, 100000, 8, 4, "bf16"), (3, 17, 50001, 2, "f32"),
                                           (97, 193, 64, 4, "bf16"), (96, 192, 64, 8, "bf16"), (2, 30000, 20, 7, "f32")])
def test_runs_of_many_sequences_long_ones_and_many_channels(B, T, C, K, dtype):
    check(inputs(B, T, C, K, dtype, bias=True, state=True, extra=8, seed=1), True)

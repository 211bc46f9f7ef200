"""gdr_ssm_fwd, gdr_ssm_bwd and gdr_ssm_step against the recurrence in 64 bits, at the sizes where chunks, groups
and strides can go wrong.  Bounds: see ssm_common."""
import math

import pytest
import torch

import gated_delta_rule_91_b200 as gdr
from gated_delta_rule_91_b200 import autograd as ag
from ssm_common import HALF, scan64, within

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def inputs(B, T, H, G, P, N, dtype="bf16", seed=0, s0=True, extra=0, scale=0.5):
    """x, B and C as slices of one buffer with `extra` more channels a row; everything on the GPU."""
    g = torch.Generator().manual_seed(seed)
    t = TYPES[dtype]
    wide = torch.randn(B, T, H * P + 2 * G * N + extra, generator=g).to(t).cuda()
    x, Bm, Cm, _ = wide.split([H * P, G * N, G * N, extra], -1)
    step = torch.exp(torch.rand(H, generator=g) * math.log(100.0) + math.log(0.001))
    return dict(x=x.unflatten(-1, (H, P)), Bm=Bm.unflatten(-1, (G, N)), Cm=Cm.unflatten(-1, (G, N)),
                delta=(scale * torch.randn(B, T, H, generator=g)).cuda(),
                A=-(1 + 15 * torch.rand(H, generator=g)).cuda(), D=(1 + 0.1 * torch.randn(H, generator=g)).cuda(),
                bias=(step + torch.log(-torch.expm1(-step))).cuda(),
                S0=0.1 * torch.randn(B, H, P, N, generator=g).cuda() if s0 else None,
                dy=torch.randn(B, T, H, P, generator=g).to(t).cuda(),
                dS_T=0.1 * torch.randn(B, H, P, N, generator=g).cuda() if s0 else None)


def fwd(d, softplus=True, **kw):
    return gdr.gdr_ssm_fwd(d["x"], d["delta"], d["A"], d["Bm"], d["Cm"], d["D"], d["bias"], d["S0"], softplus=softplus, **kw)


def bwd(d, softplus=True, **kw):
    return gdr.gdr_ssm_bwd(d["x"], d["delta"], d["A"], d["Bm"], d["Cm"], d["D"], d["bias"], d["S0"], d["dy"], d["dS_T"],
                           softplus=softplus, **kw)


def ref(d, softplus=True, grads=False, absolute=False):
    return scan64(d["x"], d["delta"], d["A"], d["Bm"], d["Cm"], d["D"], d["bias"], d["S0"], softplus,
                  d["dy"] if grads else None, d["dS_T"] if grads else None, absolute)


def sum32(T):
    """fp32 sums of T tokens and of a chunk's products, and the gates' own rounding (a few units of the exponent's
    argument, at most |c| e^-|c| <= 0.37 of a term)."""
    return (T + 400) * 2.0 ** -24


def check_fwd(d, y, S_T, softplus=True):
    T, t = d["x"].shape[1], d["x"].dtype
    r, m = ref(d, softplus), ref(d, softplus, absolute=True)
    # bf16: the chunk's decayed products and the entering state are operands rounded to bf16
    operand = 2 * HALF[t] if t == torch.bfloat16 else 0.0
    within(y, r["y"], HALF[t] * r["y"].abs() + (operand + sum32(T)) * m["y"], "y")
    # the state: fp32 sums; bf16 weights are split in two bf16 parts, the rest is below 2^-17
    within(S_T, r["S_T"], ((2.0 ** -17 if t == torch.bfloat16 else 0.0) + sum32(T)) * m["S_T"], "S_T")


def check_bwd(d, g, softplus=True):
    T, t = d["x"].shape[1], d["x"].dtype
    r, m = ref(d, softplus, grads=True), ref(d, softplus, grads=True, absolute=True)
    half = HALF[t]
    bf = t == torch.bfloat16
    # dx, dB, dC: products of at most two operands rounded to bf16 (2 * 2^-8), then the output's own rounding.
    # fp32 results: operands split in two bf16 parts (2^-17 each, two of them); sums of a chunk's double sums.
    for n in ("dx", "dB", "dC"):
        within(g[n], r[n], half * r[n].abs() + ((3 * half if bf else 0.0) + sum32(T)) * m[n], n)
    wide = (2 * 2.0 ** -17 if bf else 0.0) + 2 * sum32(T)
    for n in ("ddelta", "dA", "dD", "ddelta_bias", "dS0"):
        if g[n] is not None:
            within(g[n], r[n], wide * m[n], n)


LENGTHS = [1, 2, 63, 64, 65, 127, 128, 129, 300]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", LENGTHS)
def test_forward_lengths(T, dtype):
    d = inputs(2, T, 2, 1, 64, 128, dtype, seed=T)
    check_fwd(d, *fwd(d))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("P,N", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("H,G", [(3, 1), (4, 2), (2, 2)])
def test_forward_and_backward_shapes(P, N, H, G, dtype):
    d = inputs(2, 150, H, G, P, N, dtype, seed=P + N + H, extra=16)
    check_fwd(d, *fwd(d))
    check_bwd(d, bwd(d))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", LENGTHS)
def test_backward_lengths(T, dtype):
    d = inputs(1, T, 2, 1, 64, 128, dtype, seed=T + 50, s0=T % 2 == 0)
    check_bwd(d, bwd(d))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_chunks(dtype):
    d = inputs(1, 1500, 2, 1, 64, 64, dtype, seed=9)
    check_fwd(d, *fwd(d))
    check_bwd(d, bwd(d))


@pytest.mark.parametrize("T,P", [(500, 128), (700, 64), (1100, 64), (2300, 128)])
def test_segments_joined_by_readers_and_by_a_scan(T, P):
    """Few and many segments: 4 to 18 chunks of one sequence."""
    d = inputs(1, T, 2, 2, P, 64, "bf16", seed=T)
    check_fwd(d, *fwd(d))
    check_bwd(d, bwd(d))
    d["S0"] = d["dS_T"] = None
    check_fwd(d, *fwd(d))
    check_bwd(d, bwd(d))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_state_without_its_gradient_and_strided_leaves(dtype):
    """S0 given and S_T unused; x, B and C in an order that the library does not read in place."""
    d = inputs(2, 100, 2, 2, 64, 64, dtype, seed=21)
    d["dS_T"] = None
    check_bwd(d, bwd(d))
    odd = {k: d[k].transpose(1, 2).contiguous().transpose(1, 2) for k in ("x", "Bm", "Cm")}
    assert not odd["x"].is_contiguous()
    leaf = odd["x"].detach().requires_grad_()
    y, _ = ag.selective_scan(leaf, d["delta"], d["A"], odd["Bm"], odd["Cm"], d["D"], d["bias"], d["S0"], softplus=True)
    y.backward(d["dy"])
    assert torch.equal(y.detach(), fwd(d)[0]) and torch.equal(leaf.grad, bwd(d)["dx"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_without_bias_skip_state_and_softplus(dtype):
    d = inputs(1, 140, 2, 2, 64, 64, dtype, seed=3, s0=False)
    d["delta"] = torch.rand_like(d["delta"]) * 0.1
    d["D"] = d["bias"] = None
    y, S_T = fwd(d, softplus=False)
    check_fwd(d, y, S_T, softplus=False)
    g = bwd(d, softplus=False)
    assert g["dD"] is None and g["ddelta_bias"] is None
    check_bwd(d, g, softplus=False)
    _, none = fwd(d, softplus=False, return_state=False)
    assert none is None
    assert bwd(d, softplus=False, want_dS0=False)["dS0"] is None


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strong_decay_and_identity_tokens(dtype):
    """Decays far below the smallest float, and tokens of step 0 in between (delta = -inf under softplus)."""
    d = inputs(1, 200, 2, 1, 64, 64, dtype, seed=4)
    d["delta"][:, 50:60] = 40.0       # exp(-16 * 40) underflows
    d["delta"][:, 100:140] = -math.inf
    y, S_T = fwd(d)
    check_fwd(d, y, S_T)
    check_bwd(d, bwd(d))
    g = bwd(d)
    assert (g["ddelta"][:, 100:140] == 0).all()


def test_left_padded_batch_equals_its_prompt():
    """A batch padded on the left with identity tokens carries the same state as the prompt alone."""
    d = inputs(2, 100, 2, 1, 64, 64, "f32", seed=5, s0=False)
    d["delta"][1, :37] = -math.inf
    _, S = fwd(d)
    one = {k: (v[1:, 37:].clone() if v is not None and k in ("x", "Bm", "Cm", "delta") else v) for k, v in d.items()}
    _, S1 = fwd(one)
    m = ref(one, absolute=True)["S_T"]
    within(S[1:], S1.cpu().double(), 2 * sum32(100) * m, "state")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,G,P,N", [(1, 16, 1, 64, 128), (3, 4, 2, 128, 64), (5, 2, 2, 64, 64), (2, 3, 1, 128, 128)])
def test_step(B, H, G, P, N, dtype):
    d = inputs(B, 1, H, G, P, N, dtype, seed=B, extra=8)
    S = d["S0"].clone()
    y = gdr.gdr_ssm_step(d["x"][:, 0], d["delta"][:, 0], d["A"], d["Bm"][:, 0], d["Cm"][:, 0], S, d["D"], d["bias"],
                         softplus=True)
    r, m = ref(d), ref(d, absolute=True)
    t = TYPES[dtype]
    within(y, r["y"][:, 0], HALF[t] * r["y"][:, 0].abs() + sum32(1) * m["y"][:, 0], "y")
    within(S, r["S_T"], sum32(1) * m["S_T"], "S")


def test_steps_follow_a_prompt():
    d = inputs(2, 150, 2, 1, 64, 128, "bf16", seed=11)
    y, S_T = fwd(d)
    head = {k: (v[:, :130] if v is not None and k in ("x", "Bm", "Cm") else v) for k, v in d.items()}
    head["delta"] = d["delta"][:, :130].contiguous()
    head["x"], head["Bm"], head["Cm"] = (head[k].contiguous() for k in ("x", "Bm", "Cm"))
    _, S = fwd(head)
    ys = [gdr.gdr_ssm_step(d["x"][:, t], d["delta"][:, t].contiguous(), d["A"], d["Bm"][:, t], d["Cm"][:, t], S, d["D"],
                           d["bias"], softplus=True) for t in range(130, 150)]
    r, m = ref(d), ref(d, absolute=True)
    within(torch.stack(ys, 1), r["y"][:, 130:], HALF[torch.bfloat16] * r["y"][:, 130:].abs() + (2.0 ** -17 + sum32(150)) * m["y"][:, 130:], "y")
    within(S, r["S_T"], (2.0 ** -17 + sum32(150)) * m["S_T"], "S")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_same_bits_twice_and_slices_equal_dense(dtype):
    d = inputs(2, 333, 4, 2, 64, 128, dtype, seed=6, extra=64)
    y, S_T = fwd(d)
    g = bwd(d)
    dense = {k: v.contiguous() if v is not None else None for k, v in d.items()}
    for e in (d, dense):
        y2, S2 = fwd(e)
        assert torch.equal(y, y2) and torch.equal(S_T, S2)
        g2 = bwd(e)
        assert all(torch.equal(g[k], g2[k]) for k in g)


def test_gradient_by_differences():
    """The fp32 gradients against central differences of the 64-bit loss along random directions."""
    d = inputs(1, 70, 2, 1, 64, 64, "f32", seed=7)
    g = bwd(d)
    gen = torch.Generator().manual_seed(1)
    loss = lambda e: (lambda r: (r["y"] * d["dy"].cpu().double()).sum() + (r["S_T"] * d["dS_T"].cpu().double()).sum())(ref(e))  # noqa: E731
    for name, out in (("x", "dx"), ("delta", "ddelta"), ("A", "dA"), ("Bm", "dB"), ("Cm", "dC"), ("D", "dD"),
                      ("bias", "ddelta_bias"), ("S0", "dS0")):
        v = torch.randn(d[name].shape, generator=gen, dtype=torch.float64)
        h = 1e-4
        up, dn = ({**d, name: d[name].cpu().double() + s * h * v} for s in (1, -1))
        num = (loss(up) - loss(dn)).item() / (2 * h)
        m = ref(d, grads=True, absolute=True)[out]
        ana = (g[out].cpu().double() * v).sum().item()
        # fp32 sums, and the differences' own error: third derivatives times h^2, here below 1e-6 of the magnitudes
        assert abs(num - ana) <= (2 * sum32(70) + 1e-6) * (m * v.abs()).sum().item(), name


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_autograd(dtype):
    d = inputs(2, 90, 2, 1, 64, 64, dtype, seed=8)
    leaves = {k: d[k].detach().clone().requires_grad_() for k in ("x", "delta", "A", "Bm", "Cm", "D", "bias", "S0")}
    y, S_T = ag.selective_scan(leaves["x"], leaves["delta"], leaves["A"], leaves["Bm"], leaves["Cm"], leaves["D"],
                               leaves["bias"], leaves["S0"], softplus=True)
    torch.autograd.backward((y, S_T), (d["dy"], d["dS_T"]))
    g = bwd(d)
    for k, n in (("x", "dx"), ("delta", "ddelta"), ("A", "dA"), ("Bm", "dB"), ("Cm", "dC"), ("D", "dD"),
                 ("bias", "ddelta_bias"), ("S0", "dS0")):
        assert torch.equal(leaves[k].grad, g[n]), k
    y, _ = ag.selective_scan(d["x"], d["delta"], leaves["A"], d["Bm"], d["Cm"])
    leaves["A"].grad = None
    y.float().sum().backward()
    assert leaves["A"].grad is not None


def test_graph_replay_and_other_stream():
    d = inputs(1, 200, 2, 1, 64, 128, "bf16", seed=12)
    y0, S0 = fwd(d)
    g0 = bwd(d)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y1, S1 = fwd(d)
        g1 = bwd(d)
    s.synchronize()
    assert torch.equal(y0, y1) and torch.equal(S0, S1) and all(torch.equal(g0[k], g1[k]) for k in g0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y2, S2 = fwd(d)
        g2 = bwd(d)
    for _ in range(3):
        y2.zero_(), S2.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y0, y2) and torch.equal(S0, S2) and all(torch.equal(g0[k], g2[k]) for k in g0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_workspace_of_exact_size_is_not_overrun(dtype):
    d = inputs(1, 1500, 2, 1, 64, 64, dtype, seed=13)
    L, dt = gdr.lib(), gdr.GDR_F32 if dtype == "f32" else gdr.GDR_BF16
    for need, call in ((L.gdr_ssm_fwd_workspace_bytes(1, 1500, 2, 1, 64, 64, dt), fwd),
                       (L.gdr_ssm_bwd_workspace_bytes(1, 1500, 2, 1, 64, 64, dt), bwd)):
        assert need > 0
        buf = torch.full((need + 4096,), 77, dtype=torch.uint8, device="cuda")
        call(d, workspace=buf[:need])
        assert (buf[need:] == 77).all()
        with pytest.raises(gdr.GdrError) as e:
            call(d, workspace=buf[:need - 1])
        assert e.value.status == gdr.GDR_ERR_WORKSPACE


def test_binding_refusals():
    d = inputs(2, 8, 4, 2, 64, 64, "bf16")
    ok = dict(x=d["x"], delta=d["delta"], A=d["A"], Bm=d["Bm"], Cm=d["Cm"])
    bad = [dict(x=d["x"].half()), dict(x=d["x"].transpose(0, 1)), dict(delta=d["delta"].bfloat16()), dict(A=d["A"][:2]),
           dict(Bm=d["Bm"][:, :4]), dict(Cm=d["Cm"].float()), dict(Bm=d["Bm"][..., :32]), dict(delta=d["delta"].cpu()),
           dict(x=d["x"].contiguous().transpose(2, 3)), dict(Bm=d["Bm"][:, :1].expand(2, 8, 2, 64))]
    for b in bad:
        with pytest.raises((TypeError, ValueError, gdr.GdrError)):
            gdr.gdr_ssm_fwd(**{**ok, **b})
    with pytest.raises(gdr.GdrError):  # three heads in two groups
        gdr.gdr_ssm_fwd(d["x"][:, :, :3].contiguous(), d["delta"][..., :3].contiguous(), d["A"][:3].contiguous(), d["Bm"], d["Cm"])
    with pytest.raises(ValueError):
        gdr.gdr_ssm_fwd(**ok, S0=torch.zeros(2, 4, 64, 32, device="cuda"))
    with pytest.raises(ValueError):
        gdr.gdr_ssm_step(d["x"][:, 0], d["delta"][:, 0], d["A"], d["Bm"][:, 0], d["Cm"][:, 0], None)

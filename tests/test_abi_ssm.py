"""Refusals of the selective scan's, the short convolution's and the layer norm's C entry points, on the host before
anything is launched (CPU only)."""
import ctypes

import pytest

import gated_delta_rule_91_b200 as gdr

P = ctypes.c_void_p
FAKE = 0x10000  # aligned, never dereferenced
BAD, UNS, WS = gdr.GDR_ERR_INVALID_ARGUMENT, gdr.GDR_ERR_UNSUPPORTED, gdr.GDR_ERR_WORKSPACE

SIZES = [(dict(B=0), BAD), (dict(H=-1), BAD), (dict(G=0), BAD), (dict(H=6, G=4), BAD), (dict(P=32), UNS),
         (dict(N=96), UNS), (dict(dt=5), UNS), (dict(B=1 << 20, T=1 << 12), UNS), (dict(ldx=1), BAD), (dict(ldx=516), BAD),
         (dict(ldx=-8), BAD), (dict(ldb=64), BAD), (dict(ldc=4), BAD), (dict(x=None), BAD), (dict(x=FAKE + 2), BAD),
         (dict(delta=None), BAD), (dict(A=None), BAD), (dict(Bm=FAKE + 8), BAD), (dict(Cm=None), BAD), (dict(D=FAKE + 4), BAD),
         (dict(bias=FAKE + 4), BAD), (dict(y=None), BAD)]


def _scan(fn, **kw):
    a = dict(B=1, T=4, H=4, G=2, P=128, N=64, dt=gdr.GDR_BF16, x=FAKE, ldx=0, delta=FAKE, A=FAKE, Bm=FAKE, ldb=0, Cm=FAKE,
             ldc=0, D=None, bias=None, S0=None, y=FAKE, S_T=None, dS_T=None, dx=FAKE, ws=FAKE, nws=1 << 30, dA=FAKE, S=FAKE)
    a.update(kw)
    ins = (P(a["x"]), a["ldx"], P(a["delta"]), P(a["A"]), P(a["Bm"]), a["ldb"], P(a["Cm"]), a["ldc"], P(a["D"]), P(a["bias"]))
    L, s = gdr.lib(), (a["B"], a["T"], a["H"], a["G"], a["P"], a["N"], a["dt"], 1)
    if fn == "gdr_ssm_fwd":
        return L.gdr_ssm_fwd(*s, *ins, P(a["S0"]), P(a["y"]), P(a["S_T"]), P(a["ws"]), a["nws"], None)
    if fn == "gdr_ssm_step":
        return L.gdr_ssm_step(s[0], *s[2:], *ins, P(a["S"]), P(a["y"]), None)
    return L.gdr_ssm_bwd(*s, *ins, P(a["S0"]), P(a["y"]), P(a["dS_T"]), P(a["dx"]), P(FAKE), P(a["dA"]), P(FAKE), P(FAKE),
                         None, None, None, P(a["ws"]), a["nws"], None)


@pytest.mark.parametrize("fn", ["gdr_ssm_fwd", "gdr_ssm_bwd", "gdr_ssm_step"])
@pytest.mark.parametrize("kw,status", SIZES)
def test_scan_refusals(fn, kw, status):
    if fn == "gdr_ssm_step" and "T" in kw:
        kw = dict(B=1 << 24, H=16, G=1)
    assert _scan(fn, **kw) == status
    assert gdr.lib().gdr_last_error_string().decode().startswith(fn)


@pytest.mark.parametrize("fn,kw,status", [
    ("gdr_ssm_fwd", dict(S0=FAKE + 8), BAD), ("gdr_ssm_fwd", dict(S_T=FAKE + 8), BAD), ("gdr_ssm_fwd", dict(T=0), BAD),
    ("gdr_ssm_fwd", dict(B=70000, T=1, H=2), UNS), ("gdr_ssm_bwd", dict(B=2, T=2, H=70000), UNS), ("gdr_ssm_bwd", dict(dS_T=FAKE + 4), BAD), ("gdr_ssm_bwd", dict(dx=None), BAD),
    ("gdr_ssm_bwd", dict(dA=None), BAD), ("gdr_ssm_bwd", dict(ws=None), WS), ("gdr_ssm_bwd", dict(nws=1000), WS),
    ("gdr_ssm_bwd", dict(ws=FAKE + 8), BAD), ("gdr_ssm_step", dict(S=None), BAD), ("gdr_ssm_step", dict(S=FAKE + 4), BAD)])
def test_scan_refusals_of_its_own(fn, kw, status):
    assert _scan(fn, **kw) == status
    assert gdr.lib().gdr_last_error_string().decode().startswith(fn)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), BAD), (dict(T=-1), BAD), (dict(C=0), BAD), (dict(K=0), UNS), (dict(K=9), UNS), (dict(dt=2), UNS),
    (dict(ldx=39), BAD), (dict(B=1 << 20, T=1 << 12), UNS), (dict(x=None), BAD), (dict(w=None), BAD), (dict(bias=FAKE + 4), BAD),
    (dict(st=FAKE + 2), BAD), (dict(y=None), BAD), (dict(y=FAKE + 8), BAD), (dict(ws=None), WS), (dict(nws=16), WS)])
def test_conv_refusals(kw, status):
    a = dict(B=1, T=4, C=40, K=4, dt=gdr.GDR_BF16, x=FAKE, ldx=0, w=FAKE, bias=None, st=None, y=FAKE, ws=FAKE, nws=1 << 30)
    a.update(kw)
    L = gdr.lib()
    head = (a["B"], a["T"], a["C"], a["K"], a["dt"], 1, P(a["x"]), a["ldx"], P(a["w"]), P(a["bias"]), P(a["st"]))
    if "ws" not in kw and "nws" not in kw:
        assert L.gdr_conv_fwd(*head, None, P(a["y"]), None) == status
        assert L.gdr_last_error_string().decode().startswith("gdr_conv_fwd")
    assert L.gdr_conv_bwd(*head, P(FAKE), None, P(a["y"]), P(FAKE), None, None, P(a["ws"]), a["nws"], None) == status
    assert L.gdr_last_error_string().decode().startswith("gdr_conv_bwd")


@pytest.mark.parametrize("kw,status", [
    (dict(R=0), BAD), (dict(D=0), BAD), (dict(D=16385), UNS), (dict(dt=9), UNS), (dict(R=1 << 31), UNS), (dict(eps=-1.0), BAD),
    (dict(eps=float("inf")), BAD), (dict(x=None), BAD), (dict(w=FAKE + 4), BAD), (dict(y=None), BAD), (dict(res=FAKE), BAD),
    (dict(h=FAKE), BAD)])
def test_layernorm_refusals(kw, status):
    a = dict(R=4, D=64, dt=gdr.GDR_F32, x=FAKE, res=None, w=FAKE, b=None, eps=1e-5, y=FAKE, h=None)
    a.update(kw)
    L = gdr.lib()
    assert L.gdr_layernorm_fwd(a["R"], a["D"], a["dt"], P(a["x"]), P(a["res"]), P(a["w"]), P(a["b"]), a["eps"], P(a["y"]),
                               P(a["h"]), None) == status
    assert L.gdr_last_error_string().decode().startswith("gdr_layernorm_fwd")
    if "res" in kw or "h" in kw:
        return
    assert L.gdr_layernorm_bwd(a["R"], a["D"], a["dt"], P(a["x"]), P(a["w"]), a["eps"], P(FAKE), None, P(a["y"]), P(FAKE), None,
                               P(FAKE), 1 << 30, None) == status
    assert L.gdr_layernorm_bwd(4, 64, 0, P(FAKE), P(FAKE), 1e-5, P(FAKE), None, P(FAKE), P(FAKE), None, P(FAKE), 16, None) == WS


def test_workspace_sizes():
    L = gdr.lib()
    assert L.gdr_ssm_fwd_workspace_bytes(1, 0, 1, 1, 64, 64, 0) == 0
    assert L.gdr_ssm_bwd_workspace_bytes(1, 100, 1, 1, 48, 64, 0) == 0
    assert L.gdr_ssm_bwd_workspace_bytes(1, 100, 1, 1, 64, 64, 0) > 0
    assert L.gdr_conv_bwd_workspace_bytes(1, 10, 8, 9) == 0 and L.gdr_conv_bwd_workspace_bytes(1, 10, 8, 4) > 0
    assert L.gdr_layernorm_bwd_workspace_bytes(0) == 0 and L.gdr_layernorm_bwd_workspace_bytes(16384) > 0


def test_sizes_that_wrap_in_32_bits(monkeypatch):
    """2^32 + 1 tokens of one channel are no single token: sizes and strides past a C int are refused in the binding."""
    import torch
    monkeypatch.setattr(gdr, "_cuda", lambda x, name: x.device)
    meta = dict(dtype=torch.bfloat16, device="meta")
    w = torch.empty(1, 4, device="meta")
    for x in (torch.empty(1, (1 << 32) + 1, 1, **meta), torch.empty_strided((2, 1, 1), ((1 << 32) + 8, 8, 1), **meta)):
        with pytest.raises(ValueError, match="below 2"):
            gdr.gdr_conv_fwd(x, w)
        with pytest.raises(ValueError, match="below 2"):
            gdr.gdr_conv_bwd(x, w, x)
    with pytest.raises(ValueError, match="below 2"):
        gdr.gdr_conv_fwd(torch.empty(1, 4, 1, **meta), torch.empty(1, (1 << 32) + 4, device="meta"))
    x, v = torch.empty(1, (1 << 32) + 1, **meta), torch.empty((1 << 32) + 1, device="meta")
    with pytest.raises(ValueError, match="below 2"):
        gdr.gdr_layernorm_fwd(x, v)
    with pytest.raises(ValueError, match="below 2"):
        gdr.gdr_layernorm_bwd(x, v, x)
    rows = torch.empty_strided((2, 1, 64), ((1 << 32) + 64, 64, 1), **meta)
    small = torch.empty(2, 1, 64, **meta)
    f = dict(device="meta")
    with pytest.raises(ValueError, match="below 2"):
        gdr.gdr_ssm_step(rows, torch.empty(2, 1, **f), torch.empty(1, **f), small, small, torch.empty(2, 1, 64, 64, **f))
    L = gdr.lib()
    assert L.gdr_conv_fwd(1, (1 << 31) - 1, 1, 4, gdr.GDR_BF16, 1, P(FAKE), 0, P(FAKE), None, None, None, P(2 * FAKE), None) == UNS
    assert L.gdr_conv_bwd_workspace_bytes(1, (1 << 31) - 1, 1, 4) == 0


def test_outputs_in_place_are_refused():
    L, a = gdr.lib(), [P(FAKE + 0x1000 * i) for i in range(24)]
    s = (1, 4, 4, 2, 128, 64, gdr.GDR_BF16, 1)
    ins = lambda v: (v[0], 0, v[1], v[2], v[3], 0, v[4], 0, v[5], v[6])  # noqa: E731
    assert L.gdr_ssm_fwd(*s, *ins(a), a[7], a[8], a[7], a[9], 1 << 30, None) == BAD       # S_T = S0
    assert L.gdr_ssm_fwd(*s, *ins(a), a[7], a[0], a[9], a[10], 1 << 30, None) == BAD      # y = x
    assert L.gdr_ssm_step(s[0], *s[2:], *ins(a), a[7], a[0], None) == BAD                 # y = x
    out = a[9:17]
    for i, src in ((0, a[0]), (0, a[8]), (1, a[1]), (3, a[3]), (7, a[17])):               # dx = x, dx = dy, ..., dS0 = dS_T
        assert L.gdr_ssm_bwd(*s, *ins(a), a[7], a[8], a[17], *(src if i == j else o for j, o in enumerate(out)), a[18], 1 << 30,
                             None) == BAD
        assert L.gdr_last_error_string().decode() == "gdr_ssm_bwd: an output is an input"
    c = (1, 4, 40, 4, gdr.GDR_BF16, 1, a[0], 0, a[1], a[2], a[3])
    assert L.gdr_conv_fwd(*c, a[4], a[0], None) == BAD and L.gdr_conv_fwd(*c, a[0], a[4], None) == BAD
    assert L.gdr_conv_fwd(*c, a[4], a[3], None) == BAD                                    # y = the carried window
    assert L.gdr_conv_bwd(*c, a[4], None, a[4], a[5], None, None, a[6], 1 << 30, None) == BAD
    assert L.gdr_conv_bwd(*c, a[4], a[7], a[8], a[5], None, a[3], a[6], 1 << 30, None) == BAD

"""The binding's inputs need no alignment: one that does not start on 16 bytes is copied for the call (CPU: the launch is
taken apart instead of made).  An output that does not is refused by the library."""
import ctypes

import pytest
import torch

import gated_delta_rule_91_b200 as gdr


def off(t, by=1):
    """The same values in a contiguous view that starts `by` elements behind a 16-byte boundary."""
    flat = torch.zeros(t.numel() + by, dtype=t.dtype)
    flat[by:] = t.flatten()
    v = flat[by:].view(t.shape)
    assert v.is_contiguous() and v.data_ptr() % 16 == by * t.element_size() % 16
    return v


class Launches(list):
    """Every call's arguments; `reads` {place: values}: the four floats that an argument points to, while its copy lives."""

    def __init__(self):
        self.reads, self.want = {}, ()

    def __call__(self, device, fn, *args):
        for i in self.want:
            self.reads[i] = torch.tensor(list((ctypes.c_float * 4).from_address(args[i])))
        self.append(args)


@pytest.fixture
def launches(monkeypatch):
    seen = Launches()
    monkeypatch.setattr(gdr, "_cuda", lambda x, name: x.device)
    monkeypatch.setattr(gdr, "_launch", seen)
    return seen


X, LDX, DELTA, A_, BM, LDB = 8, 9, 10, 11, 12, 13  # places in the scan's call


def test_every_unaligned_input_is_copied(launches):
    r = torch.randn
    x, b, c = r(2, 3, 4, 64), r(2, 3, 2, 64), r(2, 3, 2, 64)
    delta, A, D, bias = r(2, 3, 4), r(4), r(4), r(4)
    S = r(2, 4, 64, 64)
    un = [off(t) for t in (x, delta, A, b, c, D, bias, S)]
    step = [off(t) for t in (x[:, 0], delta[:, 0], A, b[:, 0], c[:, 0])]
    xc, w, cb, st, nw = x.flatten(2), r(256, 4), r(256), r(2, 3, 256), r(256)
    more = [off(t) for t in (x, S, D, bias, xc, w, cb, st, xc, st, nw, xc)]
    dy, dS, D1, bias1, uxc, uw, ucb, ust, udy, udst, unw, ures = more
    launches.want = (X, DELTA)
    gdr.gdr_ssm_fwd(*un)
    assert torch.equal(launches.reads[X], x.flatten()[:4]) and torch.equal(launches.reads[DELTA], delta.flatten()[:4])
    launches.want = ()
    gdr.gdr_ssm_bwd(*un, dy, dS)
    gdr.gdr_ssm_step(*step, S, D1, bias1)
    gdr.gdr_conv_fwd(uxc, uw, ucb, conv_state=ust)
    gdr.gdr_conv_bwd(uxc, uw, udy, ucb, conv_state=ust, dconv_state_out=udst)
    gdr.gdr_layernorm_fwd(uxc, unw, ucb, residual=ures)
    gdr.gdr_layernorm_bwd(uxc, unw, udy, dres=ures)
    assert len(launches) == 7
    theirs = {t.data_ptr() for t in un + step + more}
    for args in launches:
        assert not theirs & {a for a in args if isinstance(a, int)}


def test_strided_rows_and_aligned_inputs(launches):
    wide = torch.randn(2, 3, 4 * 64 + 256 + 8)
    A, delta = torch.randn(4), torch.randn(2, 3, 4)
    x, b, c = (wide[..., i:j] for i, j in ((1, 257), (260, 388), (388, 516)))
    x, b, c = x.unflatten(-1, (4, 64)), b.unflatten(-1, (2, 64)), c.unflatten(-1, (2, 64))
    assert x.data_ptr() % 16 == 4 and b.data_ptr() % 16 == 0
    launches.want = (X,)
    gdr.gdr_ssm_fwd(x, delta, A, b, c)
    args = launches[0]
    # x: a dense copy; B, C, delta and A in place
    assert args[LDX] == 0 and args[X] % 16 == 0 and torch.equal(launches.reads[X], x.flatten()[:4])
    assert args[BM] == b.data_ptr() and args[LDB] == wide.shape[-1]
    assert args[DELTA] == delta.data_ptr() and args[A_] == A.data_ptr()


def test_unaligned_outputs_reach_the_library_as_they_are(launches):
    x = torch.randn(2, 3, 8)
    y = off(torch.zeros(2, 3, 8))
    gdr.gdr_conv_fwd(x, torch.randn(8, 4), y=y)
    assert y.data_ptr() in launches[0]  # (the alignment is checked there: test_abi_ssm)

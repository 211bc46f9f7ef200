"""The bf16 scan computes in fp32: its operands enter the tensor cores as enough bf16 parts, so that what leaves in fp32 is
as exact as fp32 torch operations, and what leaves in bf16 is one rounding away from that.

Two kinds of bounds.  Elementwise (M: the sum of term magnitudes): a bf16 output is rounded once (2^-8 of its value); operands
of its products are two bf16 parts (2^-9 * 2^-8 = 2^-17 of a term each, at most two of them a term forwards: the decayed
score or the state, and the row written to the state; three backwards), fp32 sums as in test_gpu_ssm_plans.  In the 2-norm: an fp32 output may be at most
1.5 times as far from 64 bits as the same block form in fp32 torch operations, or 1e-6 where that is more (eight units of
2^-23: a sum of about 64 terms, a carry and the decay's exponential, each an unbiased half unit or so; a missing third part
costs 2.5e-6)."""
import pytest
import torch

from ssm_common import HALF, within
from ssm_plans import scan_blocks
from test_gpu_ssm import bwd, fwd, inputs

pytestmark = pytest.mark.gpu
BF = HALF[torch.bfloat16]
SIZES = [(2, 1, 2, 1, 64, 64), (1, 100, 3, 1, 128, 128), (2, 129, 4, 2, 64, 128), (1, 1000, 6, 2, 128, 64), (2, 700, 4, 4, 64, 64),
         (8, 2040, 24, 8, 64, 128), (1, 4046, 16, 1, 128, 128), (1, 16300, 16, 2, 64, 128), (4, 900, 37, 1, 128, 128)]


def sums(d):
    return (192 + 3 * -(-d["x"].shape[1] // 128)) * 2.0 ** -24


def rel(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


def as_exact_as_fp32(got, want, plain, what):
    mine, theirs = rel(got, want), rel(plain, want)
    assert mine <= max(1e-6, 1.5 * theirs), "%s: %.3g off 64 bits, fp32 operations %.3g" % (what, mine, theirs)


def lasting(size, seed, s0):
    d = inputs(*size, "bf16", seed=seed, s0=s0)
    d["A"][::2] *= 0.02  # half of the heads remember for hundreds of tokens
    return d


@pytest.mark.parametrize("s0", [True, False])
@pytest.mark.parametrize("size", SIZES)
def test_forward(size, s0):
    d = lasting(size, sum(size), s0)
    y, S_T = fwd(d)
    r, m, p = scan_blocks(d), scan_blocks(d, absolute=True), scan_blocks(d, dtype=torch.float32)
    as_exact_as_fp32(S_T, r["S_T"], p["S_T"], "S_T")
    within(S_T, r["S_T"].cpu(), sums(d) * m["S_T"].cpu(), "S_T")
    within(y, r["y"].cpu(), (BF * r["y"].abs() + (2 * 2.0 ** -17 + sums(d)) * m["y"]).cpu(), "y")


@pytest.mark.parametrize("s0", [True, False])
@pytest.mark.parametrize("size", SIZES)
def test_gradients(size, s0):
    d = lasting(size, sum(size) + 1, s0)
    g = bwd(d, want_dS0=s0)
    r, m, p = scan_blocks(d, grads=True), scan_blocks(d, grads=True, absolute=True), scan_blocks(d, grads=True, dtype=torch.float32)
    for n in ("ddelta", "dS0"):  # (the others of fp32 are sums of few values whose terms cancel: elementwise alone)
        if g[n] is not None:
            as_exact_as_fp32(g[n], r[n], p[n], n)
    for n in ("ddelta", "dA", "dD", "ddelta_bias", "dS0"):
        if g[n] is not None:
            within(g[n], r[n].cpu(), 2 * sums(d) * m[n].cpu(), n)
    for n in ("dx", "dB", "dC"):
        within(g[n], r[n].cpu(), (BF * r[n].abs() + (3 * 2.0 ** -17 + 2 * sums(d)) * m[n]).cpu(), n)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [(3, 414, 16, 2, 64, 64), (3, 206, 16, 1, 128, 128), (2, 333, 8, 2, 128, 64), (1, 1500, 16, 1, 64, 128)])
def test_sums_over_tokens(size, dtype):
    """dA and the bias's gradient: every pair of tokens enters them once through a row's sum and once, with the other sign,
    through a column's, which have to agree to more than 32 bits for the rest to be right."""
    d = inputs(*size, dtype, seed=sum(size) + 2)
    g = bwd(d)
    r, p = scan_blocks(d, grads=True), scan_blocks(d, grads=True, dtype=torch.float32)
    for n in ("ddelta", "dA", "ddelta_bias", "dS0"):
        as_exact_as_fp32(g[n], r[n], p[n], n)

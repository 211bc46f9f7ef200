"""bf16 prompts and their gradients at sizes that reach every way in which the library cuts a call: several chunks in a
segment of the outputs and of the states, segments joined by their readers and by a scan, forwards and backwards,
several heads in a block of the gradients, several blocks of a group, and an uneven last one.  Each test asserts the plan it
is there for.

Bounds (M: the sum of term magnitudes): a term of a chunk's products takes at most 128 roundings in its sum and 64 in its
decay and weight, and at most three (decay, add, carry) a chunk that it travels: (192 + 3 chunks) 2^-24 M, twice that
where two such sums are multiplied.  Operands rounded to bf16 as in test_gpu_ssm."""
import pytest
import torch

from ssm_common import HALF, within
from ssm_plans import plan, scan_blocks
from test_gpu_ssm import bwd, fwd, inputs

pytestmark = pytest.mark.gpu
BF = HALF[torch.bfloat16]


def check(d, y, S_T, g):
    chunks = -(-d["x"].shape[1] // 128)
    r, m = scan_blocks(d, grads=True), scan_blocks(d, grads=True, absolute=True)
    r, m = ({k: v.cpu() for k, v in u.items()} for u in (r, m))
    sums = (192 + 3 * chunks) * 2.0 ** -24
    within(y, r["y"], BF * r["y"].abs() + (2 * BF + sums) * m["y"], "y")
    within(S_T, r["S_T"], (2.0 ** -17 + sums) * m["S_T"], "S_T")
    for n in ("dx", "dB", "dC"):
        within(g[n], r[n], BF * r[n].abs() + (3 * BF + 2 * sums) * m[n], n)
    for n in ("ddelta", "dA", "dD", "ddelta_bias", "dS0"):
        if g[n] is not None:
            within(g[n], r[n], (2.0 ** -16 + 2 * sums) * m[n], n)


SIZES = {  # (B, T, H, G, P, N): what the plan has to be
    "readers join segments of several chunks, four blocks of four heads":
        ((1, 4046, 16, 1, 128, 128), lambda p: 1 < p["R"] <= 8 and p["m"] > 1 and 1 < p["walk_R"] <= 8 and p["walk_m"] > 1
         and p["splits"] > 1 and p["per"] >= 3),
    "two segments of outputs, states uncut, sixteen heads a block":
        ((4, 4000, 16, 1, 128, 128), lambda p: p["R"] == 2 and p["m"] > 1 and p["walk_R"] == 1 and p["splits"] == 1 and p["per"] == 16),
    "a scan joins many segments of several chunks":
        ((1, 16300, 16, 2, 64, 128), lambda p: p["R"] > 8 and p["m"] > 1 and p["walk_R"] > 1 and p["per"] == 8),
    "a scan joins the states' segments, of several chunks":
        ((1, 8100, 4, 1, 64, 128), lambda p: p["R"] > 8 and p["m"] > 1 and p["walk_R"] > 8 and p["walk_m"] > 1),
    "twenty-four heads at P = 64, blocks of several":
        ((2, 2000, 24, 1, 64, 128), lambda p: p["R"] > 1 and p["m"] > 1 and p["splits"] > 1 and p["per"] >= 3),
    "an uneven last block, readers join reversed segments":
        ((1, 3990, 11, 1, 64, 64), lambda p: 1 < p["walk_R"] <= 8 and p["walk_m"] > 1 and p["splits"] * p["per"] > 11 and p["per"] >= 3),
    "eight groups of three heads, uncut":
        ((8, 2040, 24, 8, 64, 128), lambda p: p["R"] == 1 and p["splits"] == 1 and p["per"] == 3),
    "P = 128, N = 64, a scan, an uneven last block":
        ((1, 5000, 11, 1, 128, 64), lambda p: p["R"] > 8 and p["m"] > 1 and p["walk_R"] > 1 and p["splits"] * p["per"] > 11),
}


@pytest.mark.parametrize("s0", [True, False])
@pytest.mark.parametrize("name", list(SIZES))
def test_plan(name, s0):
    size, wanted = SIZES[name]
    p = plan(*size)
    assert wanted(p), p
    d = inputs(*size, "bf16", seed=len(name) + s0, s0=s0)
    # half of the heads remember for hundreds of tokens, so that what one segment hands to the next can be seen
    d["A"][::2] *= 0.02
    check(d, *fwd(d), bwd(d, want_dS0=s0))

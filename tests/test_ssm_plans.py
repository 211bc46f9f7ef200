"""The block form that the plan tests compare with, against the token-by-token recurrence (CPU)."""
import pytest
import torch

from ssm_common import scan64
from ssm_plans import scan_blocks


@pytest.mark.parametrize("s0,softplus", [(True, True), (False, True), (True, False)])
def test_block_form_is_the_recurrence(s0, softplus):
    g = torch.Generator().manual_seed(3)
    B, T, H, G, P, N = 2, 150, 4, 2, 5, 3
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    d = dict(x=r(B, T, H, P), delta=r(B, T, H) - 2 if softplus else torch.rand(B, T, H, generator=g), A=-1 - torch.rand(H, generator=g),
             Bm=r(B, T, G, N), Cm=r(B, T, G, N), D=r(H), bias=r(H) if softplus else None, S0=r(B, H, P, N) if s0 else None,
             dy=r(B, T, H, P), dS_T=r(B, H, P, N) if s0 else None)
    for absolute in (False, True):
        want = scan64(**{k: d[k] for k in d}, softplus=softplus, absolute=absolute)
        got = scan_blocks(d, softplus, True, absolute)
        for k in got:
            # 64 bits: sums of at most 150 terms and their gradients
            assert (got[k] - want[k]).abs().max() <= 1e-11 * (1 + want[k].abs().max()), (k, absolute)

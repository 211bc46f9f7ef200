"""The scan at the ends of the number range."""
import pytest
import torch

from test_gpu_ssm import check_bwd, check_fwd, bwd, fwd, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decays_past_the_float_range(dtype):
    """A Delta below the lowest float is a decay of 0, not a difference of infinities: finite inputs, finite outputs."""
    d = inputs(1, 300, 2, 1, 64, 64, dtype, seed=4)
    d["A"][1] = -3e38
    d["delta"][:, 100:160] = 40.0  # A Delta = -1.2e40
    y, S_T = fwd(d)
    check_fwd(d, y, S_T)
    check_bwd(d, bwd(d))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", ["A", "delta", "x", "S0"])
def test_a_nan_is_not_hidden(name, dtype):
    d = inputs(1, 300, 2, 1, 64, 64, dtype, seed=5)
    d[name] = d[name].clone()
    at = {"A": (0,), "delta": (0, 10, 0), "x": (0, 10, 0, 3), "S0": (0, 0, 3, 5)}[name]
    d[name][at] = float("nan")
    y, S_T = fwd(d)
    # the state's element (3, 5), and y of its row, from token 10 on
    assert torch.isnan(S_T[0, 0, 3, 5]) and torch.isnan(y[0, 10:, 0, 3].float()).all()
    assert torch.isfinite(y[0, :, 1].float()).all() and torch.isfinite(S_T[0, 1]).all()  # the other head
    g = bwd(d)
    assert torch.isnan(g["ddelta"][0, :, 0]).any() and torch.isfinite(g["ddelta"][0, :, 1]).all()

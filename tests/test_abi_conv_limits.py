"""The convolution's largest channel counts, on the host (CPU only): channel indices run past C by a warp's channels, and
none may wrap."""
import ctypes

import pytest

import gated_delta_rule_91_b200 as gdr

P = ctypes.c_void_p
FAKE = 0x10000


@pytest.mark.parametrize("C", [(1 << 31) - 1, (1 << 31) - 127, (1 << 31) - 1024])
def test_channels_that_would_wrap_are_refused(C):
    L = gdr.lib()
    assert L.gdr_conv_bwd_workspace_bytes(1, 1, C, 4) == 0
    assert L.gdr_conv_fwd(1, 1, C, 4, gdr.GDR_BF16, 1, P(FAKE), 0, P(FAKE), None, None, None, P(2 * FAKE), None) == gdr.GDR_ERR_UNSUPPORTED
    assert L.gdr_last_error_string().decode().startswith("gdr_conv_fwd")


def test_the_largest_plan_is_sound():
    """One slot at least, and a workspace of whole rows of partial sums."""
    C = (1 << 31) - 1025
    need = gdr.lib().gdr_conv_bwd_workspace_bytes(1, 1, C, 4)
    assert need == 5 * C * 4

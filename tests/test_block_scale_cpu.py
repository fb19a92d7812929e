"""Attention's scale at its upper end: scores are taken in powers of two, scale log2(e) has to be finite too."""
import pytest

from test_block_cpu import ATTN, P, S, SK
from test_head_cpu import lib, refused  # noqa: F401


@pytest.mark.parametrize("scale", [2.4e38, 3e38, 3.4028234e38])
def test_scale_that_is_not_finite_times_log2_e(lib, scale):  # noqa: F811
    refused(lib, lib.attn_forward, lib.OPTIM_EINVAL, S, SK, SK, S, P, P, 2, *{**ATTN, "scale": scale}.values())
    refused(lib, lib.attn_backward, lib.OPTIM_EINVAL, S, S, SK, SK, S, P, S, SK, SK, P, 2, *{**ATTN, "scale": scale}.values(), P, 1 << 30)


def test_large_scales_are_taken(lib):  # noqa: F811
    """No rows: accepted, and nothing is launched."""
    for scale in (1e-45, 1.0, 2.3e38):
        lib.attn_forward(S, SK, SK, S, P, P, 2, *{**ATTN, "rows": 0, "scale": scale}.values())

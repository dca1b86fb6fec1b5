"""Which scalars the block norms take (no GPU): the kernels compute in fp32, so what
has no value there is refused and not turned into an infinity or a zero."""
from __future__ import annotations

import pytest

import rope_rope3d_apply_gb300 as r
from tests.test_blocks_host import lib, norm_args, norm_back_args  # noqa: F401

MAX = 3.4028234663852886e38   # the largest fp32 value
TINY = 2.0 ** -149            # the smallest above zero


@pytest.mark.parametrize("name", ["eps", "residual_scale", "weight_offset"])
@pytest.mark.parametrize("value,status", [(MAX, "OK"), (MAX * 1.0001, "ERR_ARG"), (1e39, "ERR_ARG"), (1e300, "ERR_ARG")])
def test_large_values(name, value, status):
    assert r.rope3d_block_norm_check(**norm_args(**{name: value})) == status
    assert r.rope3d_block_norm_backward_check(**norm_back_args(**{name: value})) == status
    if name != "eps":
        assert r.rope3d_block_norm_check(**norm_args(**{name: -value})) == status


@pytest.mark.parametrize("eps,status", [(0.0, "OK"), (-0.0, "OK"), (TINY, "OK"), (TINY * 0.4, "ERR_ARG"), (1e-300, "ERR_ARG")])
def test_eps_that_fp32_rounds_to_zero(eps, status):
    """It would divide a row of zeros by zero, which the caller's eps is there to prevent."""
    assert r.rope3d_block_norm_check(**norm_args(eps=eps)) == status
    assert r.rope3d_block_norm_backward_check(**norm_back_args(eps=eps)) == status


def test_small_scales_round_to_zero():
    """A residual scale or offset below fp32's range is zero next to any other term."""
    assert r.rope3d_block_norm_check(**norm_args(residual_scale=1e-300, weight_offset=1e-300)) == "OK"

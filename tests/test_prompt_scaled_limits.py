"""Limits of the prompt attention and of the calls of the FP8 cache with block scales, on the host."""
import pytest

from test_prompt_scaled_abi import COPY, COPY_ORDER, _call


@pytest.mark.parametrize("n", [1 << 30, (1 << 31) - 1])
def test_more_pairs_than_a_grid_takes(n):
    """Two CTAs to a pair, fewer than 2^31 to a grid: refused as unsupported, not by the launch."""
    assert _call("pkv_copy_blocks_fp8_scaled", COPY_ORDER, COPY, n=n) == 3

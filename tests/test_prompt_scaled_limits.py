"""Limits of the prompt attention and of the calls of the FP8 cache with block scales, on the host."""
import pytest
import torch

import paged_kv_decode_attention_gb300 as pkv
from test_prompt_scaled_abi import COPY, COPY_ORDER, _call


@pytest.mark.parametrize("n", [1 << 30, (1 << 31) - 1])
def test_more_pairs_than_a_grid_takes(n):
    """Two CTAs to a pair, fewer than 2^31 to a grid: refused as unsupported, not by the launch."""
    assert _call("pkv_copy_blocks_fp8_scaled", COPY_ORDER, COPY, n=n) == 3


def _up(n):
    return -(-n // 256) * 256


@pytest.mark.parametrize("b,n,hkv,maxb", [(1, 1, 8, 520), (64, 1, 8, 1001), (128, 1, 8, 530), (1, 1, 1, 1), (3, 1, 2, 17),
                                          (37, 7, 8, 150), (2, 2, 1, 4), (5, 16, 8, 300), (4, 32, 2, 33), (1, 33, 1, 64),
                                          (1, 300, 1, 4000), (4, 2000, 8, 500)])
def test_workspace_is_what_the_partials_take(b, n, hkv, maxb):
    """For each CTA, one per share of the work that is worth one: two partials of its rows (128 FP32 values each, a
    maximum and a sum) and where its share starts (24 bytes)."""
    pos, tile, cost, least = (1, 16, 1, 3) if n == 1 else (32, 4, 8, 12) if n <= 32 else (64, 4, 8, 12)
    work = b * hkv * -(-n // pos) * (-(-maxb // tile) + cost)
    sms = torch.cuda.get_device_properties(0).multi_processor_count if torch.cuda.is_available() else 152
    ctas = min(sms, -(-work // least))
    rows = ctas * 2 * 4 * (n if n <= 32 else 64)
    assert pkv.workspace_size_fp8_scaled(b, n, 4 * hkv, maxb) == _up(rows * 512) + _up(rows * 8) + _up(ctas * 24)

"""prompt_attention with scores far from zero."""
import math

import pytest
import torch

from test_gpu_prompt_attention import SCALE, _inputs, _pkv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("e", [13, 20, 24, 27])
def test_scores_far_from_zero(e):
    """Scores of deviation 2^e, up to the largest that the call takes: their differences are far beyond the rounding of
    the scores, so a row's result is the value of its highest key, to the rounding of that one weight (2^-8) and of the
    result (2^-8)."""
    lens = [300, 17, 900]
    q, k, v, cu = _inputs(lens, 2, 4, q_scale=1.0)
    q *= 2.0 ** (e // 2)
    k *= 2.0 ** (e - e // 2)
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    _pkv().prompt_attention(out, q, k, v, cu, SCALE, out_lse=lse)
    assert bool(out.isfinite().all()) and bool(lse.isfinite().all())
    clear, at = 0, 0
    for n in lens:
        hidden = torch.ones((n, n), dtype=torch.bool, device="cuda").triu(1)
        for h in range(8):
            a, b = q[at:at + n, h].double(), k[at:at + n, h // 4].double()
            x = (a @ b.T * SCALE).masked_fill(hidden, -math.inf)
            # FP32 sums of 128 exact products, the product with the scale and the difference from the maximum
            slack = 128 * 2.0 ** -24 * SCALE * (a.abs() @ b.abs().T).masked_fill(hidden, 0).amax(-1)
            slack += 2.0 ** -21 * x.amax(-1).abs()
            one = (x > (x.amax(-1) - 4 * slack - 40)[:, None]).sum(-1) == 1
            want = v[at:at + n, h // 4].double()[x.argmax(-1)]
            err = (out[at:at + n, h].double() - want).abs()
            assert bool((err[one] <= 2.0 ** -7 * 1.01 * want[one].abs()).all())
            assert bool(((lse[at:at + n, h].double() - torch.logsumexp(x, -1)).abs() <= slack + 1e-5).all())
            clear += int(one.sum())
        at += n
    assert clear > 0.9 * 8 * sum(lens)

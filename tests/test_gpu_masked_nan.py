"""A query that is not a number stays one in its own output row -- however the
keys are split between CTAs -- and reaches no other row."""
import pytest
import torch

import verify_util as V

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import paged_kv_decode_attention_gb300 as pkv
else:  # collected on CPU-only machines, every test skipped
    pkv = None


@pytest.mark.parametrize("q_len", [1, 16, 40, 70])
@pytest.mark.parametrize("bps", [12, 1 << 20])  # 6 splits in a cluster, one pass
@pytest.mark.parametrize("mask", ["tree", "window"])
def test_nan_queries(mask, q_len, bps):
    check_nan_queries(mask, q_len, bps)


@pytest.mark.parametrize("q_len", [1, 16, 40, 70])
@pytest.mark.parametrize("mask", ["tree", "window"])
def test_nan_queries_through_the_workspace(mask, q_len):
    check_nan_queries(mask, q_len, 4)  # 18 splits


@pytest.mark.parametrize("rows", [5, 4000])  # four warps a row, one warp a row
@pytest.mark.parametrize("splits", [1, 2, 9, 33, 70])
def test_combine_of_nan_partials(rows, splits):
    """A NaN log-sum-exp anywhere makes its row NaN; empty splits, NaN partials among them, do not."""
    gen = torch.Generator(device="cuda").manual_seed(splits)
    po = torch.randn((rows, splits, 128), generator=gen, device="cuda")
    lse = torch.randn((rows, splits), generator=gen, device="cuda")
    out, out_lse = torch.empty((rows, 128), dtype=torch.bfloat16, device="cuda"), torch.empty(rows, device="cuda")
    pkv.attn_combine(out, po, lse, out_lse=out_lse)
    clean, clean_lse = out.clone(), out_lse.clone()
    lse[0] = float("nan")  # every split
    po[0] = float("nan")
    lse[1, splits - 1] = float("nan")  # one
    lse[2] = -float("inf")  # none has a key
    po[2] = float("nan")
    pkv.attn_combine(out, po, lse, out_lse=out_lse)
    assert torch.isnan(out[:2]).all() and torch.isnan(out_lse[:2]).all()
    assert not out[2].any() and out_lse[2] == -float("inf")
    assert torch.equal(out[3:], clean[3:]) and torch.equal(out_lse[3:], clean_lse[3:])


def check_nan_queries(mask, q_len, bps):
    pkv.get_device_error(reset=True)
    ctx = [1000, 1000, 130]
    d = {k: v.cuda() for k, v in V.paged_case(ctx, q_len, 2, q_len, max_blocks=70).items()}
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    words = V.masks_to_words([[list(range(i + 1)) for i in range(q_len)]] * 3, q_len).cuda()

    def run(q):
        out = torch.empty_like(q)
        args = (out, q, d["k_cache"], d["v_cache"], d["block_tables"], d["context_lens"])
        if mask == "tree":
            pkv.paged_attention_tree(*args, words, V.SCALE, kv_blocks_per_split=bps, workspace=ws)
        else:
            pkv.paged_attention_window(*args, q_len, 2000, 4, V.SCALE, kv_blocks_per_split=bps, workspace=ws)
        return out

    clean = run(d["q"])
    assert torch.isfinite(clean).all()
    q = d["q"].clone()
    rows = [(0, 0, 3), (1, q_len - 1, 5), (2, q_len // 2, 0)]
    for n, (r, i, h) in enumerate(rows):
        q[r, i, h, 127 if n else slice(None)] = float("nan")  # one value is enough
    out = run(q)
    for r, i, h in rows:
        assert torch.isnan(out[r, i, h]).all(), (r, i, h)
        out[r, i, h] = clean[r, i, h]
    assert torch.equal(out, clean)
    assert pkv.get_device_error(reset=True) == 0

"""How exact the weights of the tree and window attention are.

CTAs of 128 rows (up to 32 positions a request, or few tiles and CTAs) carry
them to P.V as two BF16 parts, so that a weight is off by at most 2^-8 of 2^-8;
CTAs of 256 rows as one, off by at most 2^-8.  The first bound is too tight for
weights of one part: short contexts, where an output is often much smaller than
its terms and half a step of it does not hide their errors.  (That it would be
noticed is tested on the host, with the mistake made in a model of the kernel.)"""
import numpy as np
import pytest
import torch

import verify_util as V

if torch.cuda.is_available():
    import paged_kv_decode_attention_gb300 as pkv
else:  # GPU tests skipped
    pkv = None

NARROW = 2.0 ** -16
CTX = [1, 2, 3, 5, 8, 13, 40, 65, 130, 300]


def _chain(width):
    return [[list(range(i + 1)) for i in range(width)] for _ in CTX]


def _modelled(d, allowed, remainder):
    """The kernels' arithmetic on the host: FP32 weights against the maximum, rounded to one or two BF16 parts, FP32
    products and sums, one rounding of the output."""
    out = torch.zeros_like(d["q"])
    b, width, hq, dim = d["q"].shape
    hkv = d["k_cache"].shape[1]
    for r in range(b):
        rows, pos, seen = allowed(r)
        if len(rows) == 0:
            continue
        rows, pos, seen = torch.as_tensor(rows), torch.as_tensor(pos), torch.as_tensor(seen)
        blk = d["block_tables"][r].long()[pos // 16]
        k, v = (d[n][blk, :, pos % 16].float() for n in ("k_cache", "v_cache"))
        x = torch.einsum("nhgd,thd->nhgt", d["q"][r, rows].float().view(len(rows), hkv, 4, dim), k)
        x = x.masked_fill(~seen[:, None, None], -float("inf")) * (V.SCALE * 1.4426950408889634)
        p = torch.exp2(x - x.amax(-1, keepdim=True))
        parts = p.bfloat16().float()
        if remainder:
            parts = parts + (p - parts).bfloat16().float()
        o = torch.einsum("nhgt,thd->nhgd", parts, v) / p.sum(-1, keepdim=True)
        out[r, rows] = o.reshape(len(rows), hq, dim).bfloat16()
    return out


@pytest.mark.parametrize("width", [1, 5, 32])
def test_the_bound_tells_one_part_from_two(width):
    d = V.paged_case(CTX, width, 2, width)
    allowed = V.window_allowed(CTX, width, 1 << 20, 0)
    ref, tol = V.attention64(d, allowed, weights=NARROW)
    V.assert_within(_modelled(d, allowed, True), ref, tol, "two parts")
    with pytest.raises(AssertionError):
        V.assert_within(_modelled(d, allowed, False), ref, tol, "one part")


@pytest.mark.gpu
@pytest.mark.parametrize("width", [1, 5, 32, 40])
@pytest.mark.parametrize("bps,table", [(0, None), (1 << 20, None), (4, 24), (4, 64)])  # (cluster, workspace)
@pytest.mark.parametrize("mask", ["tree", "window"])
def test_narrow_rows(mask, width, bps, table):
    pkv.get_device_error(reset=True)
    d = {k: v.cuda() for k, v in V.paged_case(CTX, width, 2, width, max_blocks=table).items()}
    out = torch.full_like(d["q"], float("nan"))
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    args = (out, d["q"], d["k_cache"], d["v_cache"], d["block_tables"], d["context_lens"])
    if mask == "tree":
        rows = _chain(width)
        pkv.paged_attention_tree(*args, V.masks_to_words(rows, width).cuda(), V.SCALE, kv_blocks_per_split=bps,
                                 workspace=ws)
        allowed = V.tree_allowed(CTX, [width] * len(CTX), rows)
    else:
        pkv.paged_attention_window(*args, width, 200, 3, V.SCALE, kv_blocks_per_split=bps, workspace=ws)
        allowed = V.window_allowed(CTX, width, 200, 3)
    ref, tol = V.attention64(d, allowed, weights=NARROW)
    V.assert_within(out, ref, tol, f"{mask} of {width}, split {bps}")
    assert pkv.get_device_error(reset=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("width", [1, 30])
@pytest.mark.parametrize("long", [False, True])
def test_narrow_rows_beyond_one_wave(width, long):
    """Several units per CTA (short reads), and single units, the longest first."""
    pkv.get_device_error(reset=True)
    rng = np.random.default_rng(width)
    ctx = rng.integers(width, 900 if long else 250, 90).tolist()
    d = {k: v.cuda() for k, v in V.paged_case(ctx, width, 8, 1).items()}
    out = torch.full_like(d["q"], float("nan"))
    window = 1 << 20 if long else 60
    pkv.paged_attention_window(out, d["q"], d["k_cache"], d["v_cache"], d["block_tables"], d["context_lens"], width,
                               window, 4, V.SCALE, kv_blocks_per_split=1 << 20)
    ref, tol = V.attention64(d, V.window_allowed(ctx, width, window, 4), weights=NARROW)
    V.assert_within(out, ref, tol, f"{width} queries")
    assert pkv.get_device_error(reset=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("width", [1, 32, 64, 200])
def test_a_dominating_key(width):
    """Scores that rise along the context by less than the maximum may lag, and one key that holds nearly all of the
    weight: rows of one BF16 part stay within 2^-8, the others within 2^-16."""
    pkv.get_device_error(reset=True)
    ctx = [width + 300, width + 1200]  # (more than 16 tiles: 256 rows beyond 32 positions)
    d = V.paged_case(ctx, width, 2, 3)
    q = torch.randn(128, generator=torch.Generator().manual_seed(5))
    d["q"][:] = q.to(torch.bfloat16)
    for r, c in enumerate(ctx):
        for t in range(c - width + 1):
            up = 0.3 + 6.0 * t / c + (1.5 if t == c - width else 0.0)
            d["k_cache"][int(d["block_tables"][r, t // 16]), :, t % 16] = (q * (up / 8)).to(torch.bfloat16)
    d = {k: v.cuda() for k, v in d.items()}
    out = torch.full_like(d["q"], float("nan"))
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    for bps in (0, 1 << 20):
        pkv.paged_attention_window(out, d["q"], d["k_cache"], d["v_cache"], d["block_tables"], d["context_lens"], width,
                                   1 << 20, 0, V.SCALE, kv_blocks_per_split=bps, workspace=ws)
        ref, tol = V.attention64(d, V.window_allowed(ctx, width, 1 << 20, 0),
                                 weights=NARROW if width <= 32 else 2.0 ** -8)
        V.assert_within(out, ref, tol, f"width {width}, split {bps}")
    assert pkv.get_device_error(reset=True) == 0

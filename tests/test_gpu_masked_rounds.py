"""Tree and window attention with more units (row tiles x KV heads) than fit at
once, where a CTA takes several of them, and with enough of them that the
256-row CTAs are used: against the definition in 64 bits, against the same
requests a few at a time bit for bit, and with what a kernel that runs on from
one request into the next could get wrong between them (empty requests, row
tiles without queries, unused slots full of NaN, bad table entries)."""
import numpy as np
import pytest
import torch

import verify_util as V
from test_gpu_masked_attention import _cuda, run_tree, run_window

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import paged_kv_decode_attention_gb300 as pkv
else:  # collected on CPU-only machines, every test skipped
    pkv = None


@pytest.fixture(autouse=True)
def _clear_device_error():
    if pkv is not None:
        pkv.get_device_error(reset=True)
    yield
    if pkv is not None:
        assert pkv.get_device_error(reset=True) == 0


def contexts(rng, seqs, longest):
    """Lengths from zero to the longest: ends of blocks and of tiles, empty and one-token ones."""
    ctx = rng.integers(0, longest + 1, seqs)
    for i, c in enumerate((0, 1, 16, 64, 65, longest, 0, longest - 1, 63)):
        ctx[(3 * i + 1) % seqs] = c
    return ctx.tolist()


def tree_case(width, seqs, hkv, longest, seed):
    rng = np.random.default_rng(seed)
    ctx = contexts(rng, seqs, longest)
    lens = [int(rng.integers(0, min(c, width) + 1)) for c in ctx]
    lens[5 % seqs] = min(ctx[5 % seqs], width)
    rows = [V.random_tree(rng, width) for _ in ctx]
    d = _cuda(V.paged_case(ctx, width, hkv, seed))
    return ctx, lens, rows, d


# (units: 22 x 16 = 352 of 128 rows, 12 x 16 x row tiles of 256)
@pytest.mark.parametrize("longest", [400, 1400])
@pytest.mark.parametrize("width", [1, 9, 32, 33, 64, 65, 130])
def test_trees(width, longest):
    seqs = 22 if width <= 32 else 12
    ctx, lens, rows, d = tree_case(width, seqs, 16, longest, width + longest)
    out = run_tree(d, V.masks_to_words(rows, width).cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
    ref, tol = V.attention64(d, V.tree_allowed(ctx, lens, rows))
    V.assert_within(out, ref, tol, f"trees of {width}, contexts up to {longest}")


@pytest.mark.parametrize("window,sinks", [(1, 0), (30, 5), (150, 0), (700, 40)])
@pytest.mark.parametrize("q_len", [1, 20, 32, 33, 64, 100, 300])
def test_windows(q_len, window, sinks):
    rng = np.random.default_rng(q_len + window)
    ctx = contexts(rng, 22 if q_len <= 32 else 12, 900)
    d = _cuda(V.paged_case(ctx, q_len, 16, q_len, hold=V.window_hold(ctx, q_len, window, sinks)))
    out = run_window(d, window, sinks)
    ref, tol = V.attention64(d, V.window_allowed(ctx, q_len, window, sinks))
    V.assert_within(out, ref, tol, f"window {window}, sinks {sinks}, {q_len} queries")


@pytest.mark.parametrize("q_len", [1, 6, 25, 40, 64])
def test_many_rounds_equal_a_few_requests_at_a_time(q_len):
    """100 x 16 units: up to six rounds for 128-row CTAs and eleven for 256-row ones; five requests at a time
    (more than one 128-row CTA per SM where a request has two, so that the shape is the same) fit at once."""
    rng = np.random.default_rng(q_len)
    ctx = contexts(rng, 100, 130)
    window, sinks = 60, 3
    d = _cuda(V.paged_case(ctx, q_len, 16, 1))
    rows = [V.random_tree(rng, q_len) for _ in ctx]
    lens = [int(rng.integers(0, min(c, q_len) + 1)) for c in ctx]
    mask, n = V.masks_to_words(rows, q_len).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    once = 1 << 20  # one split
    tree, win = run_tree(d, mask, n, once), run_window(d, window, sinks, once)
    ref, tol = V.attention64(d, V.tree_allowed(ctx, lens, rows))
    V.assert_within(tree, ref, tol, "trees")
    ref, tol = V.attention64(d, V.window_allowed(ctx, q_len, window, sinks))
    V.assert_within(win, ref, tol, "windows")
    for r0 in range(0, 100, 5):
        part = {k: (t[r0:r0 + 5].contiguous() if k in ("q", "block_tables", "context_lens") else t)
                for k, t in d.items()}
        assert torch.equal(run_tree(part, mask[r0:r0 + 5].contiguous(), n[r0:r0 + 5].contiguous(), once),
                           tree[r0:r0 + 5])
        assert torch.equal(run_window(part, window, sinks, once), win[r0:r0 + 5])


@pytest.mark.parametrize("q_len", [1, 40])
def test_results_in_place_of_the_queries(q_len):
    """A unit's queries are read before its results are written, and the next one's are read ahead."""
    ctx = contexts(np.random.default_rng(0), 60, 200)
    d = _cuda(V.paged_case(ctx, q_len, 16, 2))
    want = run_window(d, 50, 4)
    ws = torch.empty(max(256, pkv.workspace_size_window(60, q_len, 64, d["block_tables"].shape[1], 50, 4)),
                     dtype=torch.uint8, device="cuda")
    pkv.paged_attention_window(d["q"], d["q"], d["k_cache"], d["v_cache"], d["block_tables"], d["context_lens"],
                               q_len, 50, 4, V.SCALE, workspace=ws)
    assert torch.equal(d["q"], want)


@pytest.mark.parametrize("q_len", [1, 40])
def test_bad_entries_leave_the_other_requests_alone(q_len):
    ctx = [200] * 60
    d = _cuda(V.paged_case(ctx, q_len, 16, 3, max_blocks=13))
    good = run_window(d, 50, 4)
    d["block_tables"][30, 12] = d["k_cache"].shape[0]
    out = run_window(d, 50, 4)
    assert pkv.get_device_error(reset=True) == pkv.DEVERR_BLOCK_ID
    keep = [r for r in range(60) if r != 30]
    assert torch.equal(out[keep], good[keep])
    d["block_tables"][30, 12] = d["block_tables"][30, 11]
    d["context_lens"][7] = 1 << 30
    out = run_window(d, 50, 4)
    assert pkv.get_device_error(reset=True) == pkv.DEVERR_CONTEXT
    keep = [r for r in range(60) if r not in (7, 30)]
    assert torch.equal(out[keep], good[keep])


def test_two_streams_at_once():
    """Two calls whose grids both want every SM."""
    ctx = contexts(np.random.default_rng(4), 80, 250)
    a, b = _cuda(V.paged_case(ctx, 3, 16, 5)), _cuda(V.paged_case(ctx, 40, 16, 6))
    want_a, want_b = run_window(a, 90, 4), run_window(b, 90, 4)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(10):
        with torch.cuda.stream(s):
            got.append((run_window(a, 90, 4), want_a))
        with torch.cuda.stream(t):
            got.append((run_window(b, 90, 4), want_b))
    torch.cuda.synchronize()
    for x, want in got:
        assert torch.equal(x, want)


@pytest.mark.parametrize("q_len", [1, 40])
def test_captured_and_replayed_with_new_inputs(q_len):
    window, sinks = 60, 3
    ctx = contexts(np.random.default_rng(8), 70, 200)
    d = _cuda(V.paged_case(ctx, q_len, 16, 7))
    out = torch.empty_like(d["q"])
    ws = torch.empty(max(256, pkv.workspace_size_window(70, q_len, 64, d["block_tables"].shape[1], window, sinks)),
                     dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.paged_attention_window(out, d["q"], d["k_cache"], d["v_cache"], d["block_tables"], d["context_lens"],
                                   q_len, window, sinks, V.SCALE, workspace=ws)
    for shift in (0, 11):  # the second time every request takes another's length, tables and queries
        for k in ("q", "block_tables", "context_lens"):
            d[k].copy_(d[k].roll(shift, 0))
        ctx = ctx[-shift:] + ctx[:-shift] if shift else ctx
        g.replay()
        ref, tol = V.attention64(d, V.window_allowed(ctx, q_len, window, sinks))
        torch.cuda.synchronize()
        V.assert_within(out, ref, tol, f"replay after a shift of {shift}")

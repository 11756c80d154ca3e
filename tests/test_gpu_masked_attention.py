"""pkv_paged_attention_tree and pkv_paged_attention_window against the
definition in 64 bits, at the sizes, masks and splits where they can go wrong:
contexts of zero and one token, trees of one to several hundred drafts, tiles
cut anywhere, rows that see nothing, padded batches, NaN in every slot that is
not part of a context, and table entries that name no block."""
import numpy as np
import pytest
import torch

import verify_util as V

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


def _cuda(d):
    return {k: v.cuda() for k, v in d.items()}


def run_tree(d, mask, tree_lens, bps=0, scale=V.SCALE, stream=None):
    b, n, hq, _ = d["q"].shape
    maxb = d["block_tables"].shape[1]
    ws = torch.full((max(256, pkv.workspace_size_tree(b, n, hq, maxb, bps)),), 255, dtype=torch.uint8, device="cuda")
    out = torch.full_like(d["q"], float("nan"))
    pkv.paged_attention_tree(out, d["q"], d["k_cache"], d["v_cache"], d["block_tables"], d["context_lens"], mask,
                             scale, tree_lens, kv_blocks_per_split=bps, workspace=ws, stream=stream)
    return out


def run_window(d, window, sinks, bps=0, scale=V.SCALE):
    b, n, hq, _ = d["q"].shape
    maxb = d["block_tables"].shape[1]
    ws = torch.full((max(256, pkv.workspace_size_window(b, n, hq, maxb, window, sinks, bps)),), 255,
                    dtype=torch.uint8, device="cuda")
    out = torch.full_like(d["q"], float("nan"))
    pkv.paged_attention_window(out, d["q"], d["k_cache"], d["v_cache"], d["block_tables"], d["context_lens"], n,
                               window, sinks, scale, kv_blocks_per_split=bps, workspace=ws)
    return out


def check_tree(ctx, tree_lens, width, hkv=2, seed=0, bps=0, rows=None, pass_lens=True, max_blocks=None, q_scale=1.5):
    rng = np.random.default_rng(seed)
    if rows is None:
        rows = [V.random_tree(rng, width) for _ in ctx]
    d = _cuda(V.paged_case(ctx, width, hkv, seed, max_blocks=max_blocks, q_scale=q_scale))
    mask = V.masks_to_words(rows, width).cuda()
    lens = torch.tensor(tree_lens, dtype=torch.int32).cuda() if pass_lens else None
    out = run_tree(d, mask, lens, bps)
    ref, tol = V.attention64(d, V.tree_allowed(ctx, tree_lens, rows))
    torch.cuda.synchronize()
    V.assert_within(out, ref, tol, f"tree of {width}, contexts {ctx}, split {bps}")


@pytest.mark.parametrize("width", [1, 2, 5, 16, 31, 32, 33, 47, 64, 65, 100, 128, 129, 300])
def test_tree_sizes(width):
    ctx = [width + b for b in (0, 1, 15, 16, 63, 64, 65, 200, 517)]
    check_tree(ctx, [width] * len(ctx), width, seed=width, pass_lens=False)


@pytest.mark.parametrize("width", [7, 32, 61, 130])
@pytest.mark.parametrize("bps", [0, 1, 4, 8, 13, 1000])
def test_tree_padded_batches_and_splits(width, bps):
    """Trees of different sizes in one call (none, one, all of the width), padding rows, splits that end anywhere."""
    lens = [0, 1, width, max(1, width // 2), width, 0, 3, width - 1]
    ctx = [40, 1, width, 700, 0, 0, 130, 1111]
    check_tree(ctx, lens, width, seed=17 * width + bps, bps=bps)


@pytest.mark.parametrize("width", [26, 64])
def test_tree_every_offset_of_the_drafts_in_a_tile(width):
    ctx = [width + b for b in range(0, 130, 3)]
    check_tree(ctx, [width] * len(ctx), width, hkv=1, seed=5)


@pytest.mark.parametrize("width", [9, 40])
def test_tree_masks_of_any_kind(width):
    """No bits, all bits (later drafts too), bits past the tree, and rows that see nothing at all."""
    rng = np.random.default_rng(3)
    none = [[] for _ in range(width)]
    full = [list(range(width)) for _ in range(width)]
    some = [[j for j in range(width) if rng.random() < 0.3] for _ in range(width)]
    rows = [none, none, full, some, full, some]
    lens = [width, width, width, width, width - 4, width - 4]
    ctx = [width, width + 77, width + 5, width + 300, width, width + 64]
    check_tree(ctx, lens, width, seed=11, rows=rows)


@pytest.mark.parametrize("width", [5, 40])
def test_more_requests_than_fit_at_once(width):
    """Row tiles beyond one wave, which start in the order of their lengths: zero, equal and different ones."""
    rng = np.random.default_rng(width)
    ctx = [width + int(c) for c in rng.integers(0, 300, 75)]
    ctx[3] = ctx[4] = ctx[70] = 900
    ctx[10] = ctx[20] = 0
    lens = [min(c, int(n)) for c, n in zip(ctx, rng.integers(0, width + 1, 75))]
    check_tree(ctx, lens, width, hkv=8, seed=width)
    window, sinks = 100, 3
    d = _cuda(V.paged_case(ctx, width, 8, 5, hold=V.window_hold(ctx, width, window, sinks)))
    out = run_window(d, window, sinks)
    ref, tol = V.attention64(d, V.window_allowed(ctx, width, window, sinks))
    V.assert_within(out, ref, tol, "window")


def test_tree_longer_than_its_context():
    """Drafts whose place lies before the first token have no key."""
    width = 20
    rows = [[list(range(i + 1)) for i in range(width)] for _ in range(3)]
    check_tree([5, 19, 1], [width] * 3, width, seed=2, rows=rows)


@pytest.mark.parametrize("width", [12, 50])
@pytest.mark.parametrize("hkv", [1, 4, 8, 16])
def test_tree_head_counts(width, hkv):
    check_tree([width + 33, 500, width, 64], [width, 9, width, 1], width, hkv=hkv, seed=hkv)


@pytest.mark.parametrize("width", [16, 48])
def test_tree_sharp_weights(width):
    """Logits of tens: the running maximum moves and most weights vanish."""
    check_tree([900, 77, 2000], [width, width, width - 1], width, seed=21, q_scale=12.0)


def test_tree_chain_equals_causal_chunk():
    width, ctx = 16, [16, 40, 300, 1000]
    rows = [[list(range(i + 1)) for i in range(width)] for _ in ctx]
    d = _cuda(V.paged_case(ctx, width, 8, 9))
    out = run_tree(d, V.masks_to_words(rows, width).cuda(), None)
    chunk = torch.empty_like(out)
    pkv.paged_attention(chunk, d["q"], d["k_cache"], d["v_cache"], d["block_tables"], d["context_lens"], width,
                        V.SCALE, kv_blocks_per_split=1 << 20)
    _, tol = V.attention64(d, V.tree_allowed(ctx, [width] * 4, rows))
    assert ((out.double() - chunk.double()).abs() <= 2 * tol).all()


def test_tree_full_size_chat():
    """37 requests of 2048 + U{0..255} tokens, 8 KV heads, 16 drafts: one CTA per (request, KV head)."""
    rng = np.random.default_rng(0)
    ctx = (2048 + rng.integers(0, 256, 37) + 16).tolist()
    check_tree(ctx, [16] * 37, 16, hkv=8, seed=1)


@pytest.mark.parametrize("q_len", [1, 2, 16, 31, 32, 33, 64, 65, 200])
@pytest.mark.parametrize("window,sinks", [(1, 0), (7, 1), (16, 16), (64, 4), (100, 17), (1000, 70), (1 << 30, 3)])
def test_window_sizes(q_len, window, sinks):
    ctx = [q_len, q_len + 1, q_len + 15, 16 * 20, 777, 1500, 0, 1, max(1, q_len // 2)]
    d = _cuda(V.paged_case(ctx, q_len, 2, q_len + window % 1000, hold=V.window_hold(ctx, q_len, window, sinks)))
    out = run_window(d, window, sinks)
    ref, tol = V.attention64(d, V.window_allowed(ctx, q_len, window, sinks))
    torch.cuda.synchronize()
    V.assert_within(out, ref, tol, f"window {window}, sinks {sinks}, q_len {q_len}")


@pytest.mark.parametrize("q_len", [1, 5, 64, 150])
@pytest.mark.parametrize("bps", [1, 3, 4, 8, 20, 10000])
def test_window_splits(q_len, bps):
    ctx = [2000, 1, 333, q_len, 64, 1025]
    window, sinks = 300, 33
    d = _cuda(V.paged_case(ctx, q_len, 2, bps, hold=V.window_hold(ctx, q_len, window, sinks)))
    out = run_window(d, window, sinks, bps)
    ref, tol = V.attention64(d, V.window_allowed(ctx, q_len, window, sinks))
    torch.cuda.synchronize()
    V.assert_within(out, ref, tol, f"split {bps}, q_len {q_len}")


@pytest.mark.parametrize("q_len", [1, 8, 40])
@pytest.mark.parametrize("hkv", [1, 4, 8, 16])
def test_window_head_counts(q_len, hkv):
    ctx, window, sinks = [400, 90, q_len + 17], 128, 4
    d = _cuda(V.paged_case(ctx, q_len, hkv, hkv, hold=V.window_hold(ctx, q_len, window, sinks)))
    out = run_window(d, window, sinks)
    ref, tol = V.attention64(d, V.window_allowed(ctx, q_len, window, sinks))
    V.assert_within(out, ref, tol, f"{hkv} KV heads")


def test_window_every_alignment():
    """Window starts at every offset of a block and of a tile."""
    window, sinks = 70, 5
    for q_len in (1, 6, 36):
        ctx = [q_len + 100 + 5 * i for i in range(40)]
        d = _cuda(V.paged_case(ctx, q_len, 1, q_len, hold=V.window_hold(ctx, q_len, window, sinks)))
        out = run_window(d, window, sinks)
        ref, tol = V.attention64(d, V.window_allowed(ctx, q_len, window, sinks))
        V.assert_within(out, ref, tol, f"q_len {q_len}")


@pytest.mark.parametrize("q_len", [1, 24, 80])
def test_window_sharp_weights(q_len):
    ctx, window, sinks = [900, 77, 3000], 800, 4
    d = _cuda(V.paged_case(ctx, q_len, 2, 4, hold=V.window_hold(ctx, q_len, window, sinks), q_scale=12.0))
    out = run_window(d, window, sinks)
    ref, tol = V.attention64(d, V.window_allowed(ctx, q_len, window, sinks))
    V.assert_within(out, ref, tol, "sharp")


@pytest.mark.parametrize("q_len", [1, 16, 70])
def test_contexts_that_fill_or_exceed_the_table(q_len):
    """A context as long as the table is served whole; a longer one is cut at the table and reported."""
    ctx = [320, 320]
    d = _cuda(V.paged_case(ctx, q_len, 2, 8, max_blocks=20))
    full = run_window(d, 200, 4)
    ref, tol = V.attention64(d, V.window_allowed(ctx, q_len, 200, 4))
    V.assert_within(full, ref, tol, "full table")
    mask = V.masks_to_words([[[j for j in range(i + 1)] for i in range(q_len)]] * 2, q_len).cuda()
    whole = run_tree(d, mask, None)
    assert pkv.get_device_error(reset=True) == 0
    d["context_lens"][1] = 100000
    cut = run_window(d, 200, 4)
    assert pkv.get_device_error(reset=True) == pkv.DEVERR_CONTEXT
    assert torch.equal(cut, full)
    cut = run_tree(d, mask, None)
    assert pkv.get_device_error(reset=True) == pkv.DEVERR_CONTEXT
    assert torch.equal(cut, whole)


@pytest.mark.parametrize("q_len", [1, 16, 70])
def test_bad_block_ids_are_reported(q_len):
    ctx = [300, 300]
    d = _cuda(V.paged_case(ctx, q_len, 2, 8))
    mask = V.masks_to_words([[[j for j in range(i + 1)] for i in range(q_len)]] * 2, q_len).cuda()
    good_t, good_w = run_tree(d, mask, None), run_window(d, 100, 0)
    for bad in (-1, d["k_cache"].shape[0], 2 ** 31 - 1, -2 ** 31 + 1):
        saved = int(d["block_tables"][1, 17])
        d["block_tables"][1, 17] = bad
        t = run_tree(d, mask, None)
        assert pkv.get_device_error(reset=True) == pkv.DEVERR_BLOCK_ID
        w = run_window(d, 100, 0)
        assert pkv.get_device_error(reset=True) == pkv.DEVERR_BLOCK_ID
        assert torch.equal(t[0], good_t[0]) and torch.equal(w[0], good_w[0])
        d["block_tables"][1, 17] = saved


def test_runs_are_reproducible_and_capturable():
    """The same bits again, on another stream, and replayed from a graph with new inputs in the same buffers."""
    width, ctx = 26, [600, 77, 2000, 26]
    rng = np.random.default_rng(0)
    rows = [V.random_tree(rng, width) for _ in ctx]
    d = _cuda(V.paged_case(ctx, width, 8, 3))
    mask = V.masks_to_words(rows, width).cuda()
    lens = torch.tensor([26, 20, 26, 1], dtype=torch.int32).cuda()
    b, n, hq, _ = d["q"].shape
    maxb = d["block_tables"].shape[1]
    first = run_tree(d, mask, lens)
    first_w = run_window(d, 500, 4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = run_tree(d, mask, lens)
        again_w = run_window(d, 500, 4)
    torch.cuda.synchronize()
    assert torch.equal(first, again) and torch.equal(first_w, again_w)
    ws = torch.empty(max(256, pkv.workspace_size_tree(b, n, hq, maxb)), dtype=torch.uint8, device="cuda")
    ws2 = torch.empty(max(256, pkv.workspace_size_window(b, n, hq, maxb, 500, 4)), dtype=torch.uint8, device="cuda")
    out, out_w = torch.empty_like(d["q"]), torch.empty_like(d["q"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.paged_attention_tree(out, d["q"], d["k_cache"], d["v_cache"], d["block_tables"], d["context_lens"], mask,
                                 V.SCALE, lens, workspace=ws)
        pkv.paged_attention_window(out_w, d["q"], d["k_cache"], d["v_cache"], d["block_tables"], d["context_lens"],
                                   n, 500, 4, V.SCALE, workspace=ws2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first) and torch.equal(out_w, first_w)
    d["q"].neg_()
    lens.copy_(torch.tensor([3, 26, 0, 26], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    ref, tol = V.attention64(d, V.tree_allowed(ctx, [3, 26, 0, 26], rows))
    V.assert_within(out, ref, tol, "replayed")


def test_empty_batch():
    d = _cuda(V.paged_case([20], 4, 1, 0))
    d = {k: (t[:0] if k in ("q", "block_tables", "context_lens") else t) for k, t in d.items()}
    out = torch.empty_like(d["q"])
    pkv.paged_attention_tree(out, d["q"], d["k_cache"], d["v_cache"], d["block_tables"].contiguous(),
                             d["context_lens"], torch.empty((0, 4, 1), dtype=torch.int64, device="cuda"), V.SCALE)
    pkv.paged_attention_window(out, d["q"], d["k_cache"], d["v_cache"], d["block_tables"].contiguous(),
                               d["context_lens"], 4, 8, 0, V.SCALE)

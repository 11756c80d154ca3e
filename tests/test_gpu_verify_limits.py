"""The verification-step and sliding-window calls at the edges of what they
document: the widest tree, pools whose byte offsets pass 32 bits, first calls
inside a stream capture, calls on two streams at once, results in place of the
queries, and arguments that the binding refuses."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import verify_util as V

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import paged_kv_decode_attention_gb300 as pkv
else:  # collected on CPU-only machines, every test skipped
    pkv = None

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(autouse=True)
def _clear_device_error():
    if pkv is not None:
        pkv.get_device_error(reset=True)
    yield
    if pkv is not None:
        assert pkv.get_device_error(reset=True) == 0


def _cuda(d):
    return {k: v.cuda() for k, v in d.items()}


def _tree(d, mask, lens, stream=None, out=None, ws=None):
    b, n, hq, _ = d["q"].shape
    if ws is None:
        ws = torch.empty(max(256, pkv.workspace_size_tree(b, n, hq, d["block_tables"].shape[1])), dtype=torch.uint8,
                         device="cuda")
    out = torch.full_like(d["q"], float("nan")) if out is None else out
    pkv.paged_attention_tree(out, d["q"], d["k_cache"], d["v_cache"], d["block_tables"], d["context_lens"], mask,
                             V.SCALE, lens, workspace=ws, stream=stream)
    return out


def test_widest_tree():
    width, ctx = 1024, [1024, 1500, 1100]
    rng = np.random.default_rng(0)
    rows = [V.random_tree(rng, width) for _ in ctx]
    lens = [1024, 1024, 700]
    d = _cuda(V.paged_case(ctx, width, 1, 0))
    out = _tree(d, V.masks_to_words(rows, width).cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
    ref, tol = V.attention64(d, V.tree_allowed(ctx, lens, rows))
    V.assert_within(out, ref, tol, "1024 drafts")


def test_pools_beyond_32_bit_offsets():
    """Blocks past 4 GiB of a pool: read by both attentions, written by the append, moved by the compaction."""
    hkv, blocks = 8, 140_000  # 4.6 GB per tensor
    k = torch.empty((blocks, hkv, 16, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    ctx, width = [300, 77], 20
    d = _cuda(V.paged_case(ctx, width, hkv, 3, spare=0))
    held = d["block_tables"][d["block_tables"] >= 0].long()
    top = blocks - 1 - held  # the same blocks, at the far end
    k[top], v[top] = d["k_cache"][held], d["v_cache"][held]
    far = d["block_tables"].clone()
    far[far >= 0] = (blocks - 1 - far[far >= 0])
    rng = np.random.default_rng(1)
    rows = [V.random_tree(rng, width) for _ in ctx]
    mask = V.masks_to_words(rows, width).cuda()
    near_out = _tree(d, mask, None)
    window = lambda x, t: pkv.paged_attention_window(x, d["q"], t[0], t[1], t[2], d["context_lens"], width, 64, 4,
                                                     V.SCALE, kv_blocks_per_split=1 << 20)
    near_win, far_win = torch.empty_like(near_out), torch.empty_like(near_out)
    window(near_win, (d["k_cache"], d["v_cache"], d["block_tables"]))
    window(far_win, (k, v, far))
    e = dict(d, k_cache=k, v_cache=v, block_tables=far)
    assert torch.equal(_tree(e, mask, None), near_out) and torch.equal(far_win, near_win)
    # append and compaction
    tokens = 5
    x = torch.randn((tokens, 6 * hkv, 128), device="cuda").to(torch.bfloat16)
    slots = (torch.arange(tokens, device="cuda") + (blocks - 1) * 16).to(torch.int64)
    q_out = torch.empty((tokens, 4 * hkv, 128), dtype=torch.bfloat16, device="cuda")
    pkv.qk_norm_rope_append(q_out, k, v, slots, x[:, :4 * hkv], x[:, 4 * hkv:5 * hkv], x[:, 5 * hkv:])
    assert torch.equal(k[blocks - 1, :, :tokens].transpose(0, 1), x[:, 4 * hkv:5 * hkv])
    assert torch.equal(v[blocks - 1, :, :tokens].transpose(0, 1), x[:, 5 * hkv:])
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    pkv.kv_compact(pkv.KvPools([k], [v]), i32([[blocks - 1]]), i32([5]), i32([[0, 2, 4]]), i32([3]), 5)
    for t, src in ((k, x[:, 4 * hkv:5 * hkv]), (v, x[:, 5 * hkv:])):
        assert torch.equal(t[blocks - 1, :, :3].transpose(0, 1), src[[0, 2, 4]])


def test_two_streams_at_once():
    """Calls of every operator on two streams, each with its own buffers and workspace."""
    rng = np.random.default_rng(0)
    cases = []
    for seed, width in ((1, 26), (2, 50)):
        ctx = [2000, 31 + width, 700]
        rows = [V.random_tree(rng, width) for _ in ctx]
        d = _cuda(V.paged_case(ctx, width, 8, seed))
        cases.append((d, V.masks_to_words(rows, width).cuda()))
    want = [_tree(d, m, None) for d, m in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    spaces = [torch.empty(64 << 20, dtype=torch.uint8, device="cuda") for _ in cases]
    outs = [torch.empty_like(w) for w in want]
    torch.cuda.synchronize()
    for _ in range(20):
        for (d, m), s, o, ws in zip(cases, streams, outs, spaces):
            _tree(d, m, None, stream=s, out=o, ws=ws)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


def test_outputs_in_place_of_the_queries():
    for width in (9, 50):
        ctx = [900, 64, 2000]
        d = _cuda(V.paged_case(ctx, width, 4, 7))
        mask = V.masks_to_words([[list(range(i + 1)) for i in range(width)]] * 3, width).cuda()
        want = _tree(d, mask, None)
        e = dict(d, q=d["q"].clone())
        assert torch.equal(_tree(e, mask, None, out=e["q"]), want)


FIRST_CALL = """
import sys; sys.path[:0] = [{root!r}, {root!r} + "/tests"]
import torch, verify_util as V, paged_kv_decode_attention_gb300 as pkv
i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
res = []
for width in (6, 40):
    d = {{k: v.cuda() for k, v in V.paged_case([500, 60], width, 8, 1).items()}}
    mask = V.masks_to_words([[list(range(i + 1)) for i in range(width)]] * 2, width).cuda()
    ws = torch.empty(32 << 20, dtype=torch.uint8, device="cuda")
    out, win, q_out = (torch.zeros_like(d["q"]) for _ in range(3))
    x = torch.randn((2, 48, 128), device="cuda").to(torch.bfloat16)
    qo = torch.zeros((2, 32, 128), dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([-1, -1], device="cuda")
    pools = pkv.KvPools([d["k_cache"]], [d["v_cache"]])
    acc = i32([[0], [0]])
    num = i32([1, 1])
    def calls():
        pkv.qk_norm_rope_append(qo, d["k_cache"], d["v_cache"], slots, x[:, :32], x[:, 32:40], x[:, 40:])
        pkv.paged_attention_tree(out, d["q"], d["k_cache"], d["v_cache"], d["block_tables"], d["context_lens"], mask,
                                 V.SCALE, workspace=ws)
        pkv.paged_attention_window(win, d["q"], d["k_cache"], d["v_cache"], d["block_tables"], d["context_lens"],
                                   width, 100, 4, V.SCALE, workspace=ws)
        pkv.kv_compact(pools, d["block_tables"], d["context_lens"], acc, num, width)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        calls()
    g.replay()
    torch.cuda.synchronize()
    got = out.clone(), win.clone(), qo.clone()
    calls()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, (out, win, qo))) and out.any() and win.any() and qo.any()
assert pkv.get_device_error() == 0
print("captured first")
"""


def test_first_calls_inside_a_capture():
    r = subprocess.run([sys.executable, "-c", FIRST_CALL.format(root=ROOT)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stdout + r.stderr


def test_refused_arguments():
    d = _cuda(V.paged_case([40, 50], 6, 2, 0))
    mask = torch.zeros((2, 6, 1), dtype=torch.int64, device="cuda")
    args = [torch.empty_like(d["q"]), d["q"], d["k_cache"], d["v_cache"], d["block_tables"], d["context_lens"]]

    def tree(at=None, value=None, **kw):
        a = list(args)
        if at is not None:
            a[at] = value
        pkv.paged_attention_tree(*a, kw.pop("mask", mask), V.SCALE, **kw)

    tree(kv_blocks_per_split=1 << 20)
    bad = [(0, args[0].float()), (0, args[0][:, :5]), (1, d["q"].cpu()), (1, d["q"].transpose(1, 2)),
           (2, d["k_cache"][:2]), (2, d["k_cache"].float()), (3, d["v_cache"][:, :1]), (4, d["block_tables"].long()),
           (4, d["block_tables"][:1]), (4, d["block_tables"][:, ::2]), (5, d["context_lens"].float()),
           (5, d["context_lens"][:1]), (0, None), (2, 7)]
    for at, value in bad:
        with pytest.raises((TypeError, ValueError)):
            tree(at, value)
        with pytest.raises((TypeError, ValueError)):
            a = list(args)
            a[at] = value
            pkv.paged_attention_window(*a, 6, 8, 0, V.SCALE)
    for kw in (dict(mask=mask[:, :5]), dict(mask=mask.int()), dict(mask=mask.repeat(1, 1, 2)), dict(mask=None),
               dict(tree_lens=d["context_lens"].long()), dict(tree_lens=d["context_lens"][:1]),
               dict(workspace=torch.empty(8)), dict(kv_blocks_per_split=1 << 40)):
        with pytest.raises((TypeError, ValueError)):
            tree(**kw)
    with pytest.raises(ValueError):
        pkv.paged_attention_window(*args, 5, 8, 0, V.SCALE)
    for window, sinks, scale in ((0, 0, 1.0), (8, -1, 1.0), (8, 0, 0.0), (8, 0, float("nan"))):
        with pytest.raises(pkv.PkvError):
            pkv.paged_attention_window(*args, 6, window, sinks, scale)
    with pytest.raises(pkv.PkvError):  # more than 8 splits without their workspace
        pkv.paged_attention_tree(*(list(args[:4]) + [torch.zeros((2, 100), dtype=torch.int32, device="cuda"), args[5]]),
                                 mask, V.SCALE, kv_blocks_per_split=4)
    x = torch.zeros((3, 12, 128), dtype=torch.bfloat16, device="cuda")
    q, k, v = x[:, :8], x[:, 8:10], x[:, 10:]
    slots = torch.tensor([-1, -1, -1], device="cuda")
    out = torch.empty((3, 8, 128), dtype=torch.bfloat16, device="cuda")
    table = torch.zeros((10, 64), device="cuda")
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")

    def rope(**kw):
        a = dict(q_out=out, k_cache=d["k_cache"], v_cache=d["v_cache"], slot_mapping=slots, q=q, k=k, v=v,
                 positions=pos, rope_table=table)
        a.update(kw)
        pkv.qk_norm_rope_append(**a)

    rope()
    for kw in (dict(q=q[:2]), dict(k=k[:, :1]), dict(v=v.float()), dict(q_out=out[:2]), dict(slot_mapping=slots.int()),
               dict(positions=None), dict(positions=pos.long()), dict(positions=pos[:2]), dict(rope_table=table[0]),
               dict(rope_table=table.double()), dict(q_weight=out[0, 0, :64]), dict(k_weight=table[0]),
               dict(q=x.transpose(0, 1)[:8].transpose(0, 1).flip(2)[..., ::2]), dict(kv_format=1), dict(kv_format=7),
               dict(q=q.cpu()), dict(k=k.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises((TypeError, ValueError)):
            rope(**kw)
    for kw in (dict(rope_table=torch.zeros((10, 24), device="cuda")), dict(eps=-1.0),
               dict(rope_table=torch.zeros((0, 64), device="cuda"))):
        with pytest.raises(pkv.PkvError):
            rope(**kw)

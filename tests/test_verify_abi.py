"""Refusals of the verification-step and sliding-window entry points, on the
host: bad arguments return the documented status before the GPU is touched."""
import ctypes

import pytest
import torch

import paged_kv_decode_attention_gb300 as pkv

P = ctypes.c_void_p(4096)


def _desc(**kw):
    d = dict(num_blocks=4, block_size=16, num_kv_heads=8, head_dim=128)
    d.update(kw)
    return pkv.CacheDesc(**d)


def _call(name, order, base, **kw):
    a = dict(base, **kw)
    return getattr(pkv.lib(), name)(*[a[k] for k in order])


ROPE_ORDER = ["qo", "kc", "vc", "desc", "fmt", "slots", "q", "qs", "k", "ks", "v", "vs", "hq", "qw", "kw", "eps",
              "table", "rows", "rot", "inter", "pos", "n", "stream"]
ROPE = dict(qo=P, kc=P, vc=P, desc=_desc(), fmt=0, slots=P, q=ctypes.c_void_p(8192), qs=4096, k=P, ks=1024, v=P,
            vs=1024, hq=32, qw=P, kw=P, eps=1e-6, table=P, rows=100, rot=128, inter=0, pos=P, n=3, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(desc=None), 1), (dict(desc=_desc(head_dim=64)), 3), (dict(desc=_desc(block_size=8)), 3),
    (dict(desc=_desc(num_blocks=-1)), 2), (dict(fmt=3), 3), (dict(fmt=-1), 3), (dict(hq=16), 3), (dict(n=-1), 2),
    (dict(eps=float("nan")), 2), (dict(eps=-1.0), 2), (dict(rot=-16), 2), (dict(rot=8), 3), (dict(rot=144), 3),
    (dict(rows=0), 2), (dict(rows=-1), 2), (dict(qs=4095), 2), (dict(ks=1000), 2), (dict(vs=0), 2),
    (dict(qs=4100), 3), (dict(vs=1028), 3), (dict(qo=None), 1), (dict(kc=None), 1), (dict(vc=None), 1),
    (dict(slots=None), 1), (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(table=None), 1),
    (dict(pos=None), 1), (dict(q=ctypes.c_void_p(8200)), 3), (dict(kw=ctypes.c_void_p(4098)), 3),
    (dict(table=ctypes.c_void_p(4100)), 3), (dict(q=P, qs=5000 * 8), 2), (dict(n=0), 0), (dict(n=0, qo=None), 0),
])
def test_qk_norm_rope_append(change, status):
    assert _call("pkv_qk_norm_rope_append", ROPE_ORDER, ROPE, **change) == status


TREE_ORDER = ["out", "q", "k", "v", "desc", "bt", "maxb", "cl", "tl", "mask", "b", "n", "hq", "scale", "bps", "ws",
              "wsb", "stream"]
TREE = dict(out=P, q=P, k=P, v=P, desc=_desc(), bt=P, maxb=64, cl=P, tl=None, mask=P, b=2, n=9, hq=32, scale=0.1,
            bps=4, ws=None, wsb=0, stream=None)
WIN_ORDER = ["out", "q", "k", "v", "desc", "bt", "maxb", "cl", "b", "n", "hq", "window", "sinks", "scale", "bps", "ws",
             "wsb", "stream"]
WIN = dict(out=P, q=P, k=P, v=P, desc=_desc(), bt=P, maxb=64, cl=P, b=2, n=9, hq=32, window=500, sinks=4, scale=0.1,
           bps=4, ws=None, wsb=0, stream=None)
MASKED = [
    (dict(desc=None), 1), (dict(desc=_desc(head_dim=64)), 3), (dict(hq=16), 3), (dict(n=0), 2), (dict(b=-1), 2),
    (dict(maxb=0), 2), (dict(maxb=1 << 27), 3), (dict(bps=-1), 2), (dict(scale=0.0), 2), (dict(scale=-0.1), 2),
    (dict(scale=float("nan")), 2), (dict(scale=float("inf")), 2), (dict(out=None), 1), (dict(q=None), 1),
    (dict(k=None), 1), (dict(v=None), 1), (dict(bt=None), 1), (dict(cl=None), 1), (dict(q=ctypes.c_void_p(4104)), 3),
    (dict(b=1 << 28), 3), (dict(desc=_desc(num_blocks=0)), 2), (dict(desc=_desc(num_blocks=1 << 30)), 3),
    (dict(), 4), (dict(ws=P, wsb=100), 4), (dict(ws=ctypes.c_void_p(4096 + 16), wsb=1 << 40), 4), (dict(b=0), 0),
]


@pytest.mark.parametrize("change,status", MASKED + [
    (dict(mask=None), 1), (dict(mask=ctypes.c_void_p(4100)), 3), (dict(n=1025), 3)])
def test_paged_attention_tree(change, status):
    assert _call("pkv_paged_attention_tree", TREE_ORDER, TREE, **change) == status


@pytest.mark.parametrize("change,status", MASKED + [
    (dict(window=0), 2), (dict(window=-5), 2), (dict(sinks=-1), 2), (dict(n=1 << 27, b=1), 3)])
def test_paged_attention_window(change, status):
    assert _call("pkv_paged_attention_window", WIN_ORDER, WIN, **change) == status


ARR = (ctypes.c_void_p * 2)(4096, 8192)
HOLE = (ctypes.c_void_p * 2)(4096, 0)
ODD = (ctypes.c_void_p * 2)(4096, 8200)
COMP_ORDER = ["kc", "vc", "layers", "desc", "fmt", "bt", "maxb", "cl", "tl", "b", "n", "acc", "num", "maxa", "stream"]
COMP = dict(kc=ARR, vc=ARR, layers=2, desc=_desc(), fmt=0, bt=P, maxb=64, cl=P, tl=None, b=2, n=9, acc=P, num=P,
            maxa=4, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(desc=None), 1), (dict(desc=_desc(block_size=32)), 3), (dict(fmt=5), 3), (dict(layers=-1), 2),
    (dict(b=-1), 2), (dict(maxb=0), 2), (dict(n=0), 2), (dict(n=1025), 3), (dict(maxa=0), 2), (dict(maxa=10), 2),
    (dict(layers=70000), 3), (dict(kc=None), 1), (dict(vc=None), 1), (dict(bt=None), 1), (dict(cl=None), 1),
    (dict(acc=None), 1), (dict(num=None), 1), (dict(kc=HOLE), 1), (dict(vc=ODD), 3), (dict(b=0), 0),
    (dict(layers=0), 0)])
def test_kv_compact(change, status):
    assert _call("pkv_kv_compact", COMP_ORDER, COMP, **change) == status


@pytest.mark.parametrize("name,order,base", [
    ("pkv_qk_norm_rope_append", ROPE_ORDER, dict(ROPE, hq=0, qs=0)), ("pkv_paged_attention_tree", TREE_ORDER, TREE),
    ("pkv_paged_attention_window", WIN_ORDER, WIN), ("pkv_kv_compact", COMP_ORDER, COMP)])
def test_head_counts_beyond_the_kernels_grids(name, order, base):
    # (4 << 30 heads would wrap to 0 in 32 bits)
    for heads in (65536, 1 << 30):
        assert _call(name, order, base, desc=_desc(num_kv_heads=heads)) == 3


def test_splits_and_workspaces_are_host_arithmetic():
    # enough row tiles: no split, no workspace
    assert pkv.choose_kv_blocks_per_split_tree(37, 8, 16, 144, 152) == 144
    assert pkv.workspace_size_tree(37, 16, 32, 144, 144) == 0
    assert pkv.workspace_size_window(37, 16, 32, 144, 100, 4, 200) == 0
    # one long request is split in whole tiles; partials and sums, each part 256-byte aligned
    bps = pkv.choose_kv_blocks_per_split_tree(1, 8, 16, 528, 152)
    assert 16 <= bps < 528 and bps % 4 == 0
    splits = -(-528 // bps)
    rows = 16 * 32
    assert pkv.workspace_size_tree(1, 16, 32, 528, bps) == rows * splits * 512 + -(-rows * splits * 4 // 256) * 256
    assert pkv.choose_kv_blocks_per_split_tree(1, 8, 64, 528, 152) % 4 == 0
    # up to 8 splits merge on chip
    assert pkv.workspace_size_tree(1, 16, 32, 528, 528 // 8) == 0
    assert pkv.workspace_size_tree(1, 16, 32, 528, 56) > 0
    # a window reads its own span, however long the table
    a = pkv.workspace_size_window(1, 1, 32, 1 << 20, 1000, 4)
    assert a == pkv.workspace_size_window(1, 1, 32, 1 << 24, 1000, 4) and a < 1 << 21
    # an endless window reads the table
    assert pkv.choose_kv_blocks_per_split_window(64, 8, 16, 144, (1 << 31) - 1, (1 << 31) - 1, 152) == 144
    for bad in ((0, 16, 32, 144), (1, 0, 32, 144), (1, 1025, 32, 144), (1, 16, 0, 144), (1, 16, 32, 0)):
        assert pkv.workspace_size_tree(*bad) == 0
    assert pkv.workspace_size_window(1, 1, 32, 100, 0, 4) == 0 and pkv.workspace_size_window(1, 1, 32, 100, 5, -1) == 0


def test_bindings_refuse_cpu_tensors():
    if torch.cuda.is_available():
        pytest.skip("the refusal of a device is tested where there is none")
    x = torch.zeros(4, 8, 16, 128, dtype=torch.bfloat16)
    q = torch.zeros(1, 1, 32, 128, dtype=torch.bfloat16)
    i = torch.zeros(1, 4, dtype=torch.int32)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        pkv.paged_attention_window(q, q, x, x, i, i[:, 0].contiguous(), 1, 8, 0, 0.1)
    with pytest.raises(ValueError):
        pkv.KvPools([x], [x.clone()])

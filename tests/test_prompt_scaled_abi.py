"""Refusals of the prompt attention and of the calls of the FP8 cache with block scales, on the host: bad arguments
return the documented status before the GPU is touched."""
import ctypes

import pytest
import torch

import paged_kv_decode_attention_gb300 as pkv

P = ctypes.c_void_p(4096)


def off(n):
    return ctypes.c_void_p(4096 + n)


def _desc(**kw):
    d = dict(num_blocks=4, block_size=16, num_kv_heads=8, head_dim=128)
    d.update(kw)
    return pkv.CacheDesc(**d)


def _call(name, order, base, **kw):
    a = dict(base, **kw)
    return getattr(pkv.lib(), name)(*[a[k] for k in order])


PROMPT_ORDER = ["out", "lse", "q", "qs", "k", "ks", "v", "vs", "cu", "b", "t", "hq", "hkv", "d", "scale", "stream"]
PROMPT = dict(out=P, lse=P, q=P, qs=4096, k=P, ks=1024, v=P, vs=1024, cu=P, b=3, t=100, hq=32, hkv=8, d=128, scale=0.1,
              stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(b=-1), 2), (dict(t=-1), 2), (dict(hq=0), 2), (dict(hkv=0), 2), (dict(hkv=-8), 2), (dict(d=64), 3),
    (dict(hq=31, qs=4096), 3), (dict(hq=129, hkv=1, qs=129 * 128, ks=128, vs=128), 3), (dict(hq=4, qs=4096), 3),
    (dict(scale=0.0), 2), (dict(scale=-0.1), 2), (dict(scale=float("nan")), 2), (dict(scale=float("inf")), 2),
    (dict(qs=4088), 2), (dict(ks=1016), 2), (dict(vs=0), 2), (dict(qs=4100), 3), (dict(ks=1028), 3),
    (dict(qs=1 << 39), 3), (dict(t=0x7fffffff), 3), (dict(out=None), 1), (dict(q=None), 1), (dict(k=None), 1),
    (dict(v=None), 1), (dict(cu=None), 1), (dict(out=off(8)), 3), (dict(q=off(8)), 3), (dict(k=off(2)), 3),
    (dict(v=off(4)), 3), (dict(lse=off(2)), 3), (dict(cu=off(1)), 3), (dict(b=0), 0), (dict(t=0, q=None), 0),
])
def test_prompt_attention(change, status):
    assert _call("pkv_prompt_attention", PROMPT_ORDER, PROMPT, **change) == status


APPEND_ORDER = ["kc", "vc", "ks", "vs", "desc", "bt", "maxb", "cl", "cu", "b", "k", "kst", "v", "vst", "t", "stream"]
APPEND = dict(kc=P, vc=P, ks=P, vs=P, desc=_desc(), bt=P, maxb=64, cl=P, cu=P, b=3, k=P, kst=1024, v=P, vst=1024, t=50,
              stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(desc=None), 1), (dict(desc=_desc(head_dim=64)), 3), (dict(desc=_desc(block_size=32)), 3),
    (dict(desc=_desc(num_blocks=-1)), 2), (dict(desc=_desc(num_kv_heads=0)), 2), (dict(b=-1), 2), (dict(t=-1), 2),
    (dict(maxb=0), 2), (dict(maxb=1 << 27), 3), (dict(cu=None), 2), (dict(cu=None, t=4), 2), (dict(kst=1016), 2),
    (dict(vst=1020), 2), (dict(vst=1028), 3), (dict(kc=None), 1), (dict(vc=None), 1), (dict(ks=None), 1),
    (dict(vs=None), 1), (dict(bt=None), 1), (dict(cl=None), 1), (dict(k=None), 1), (dict(v=None), 1),
    (dict(kc=off(8)), 3), (dict(k=off(8)), 3), (dict(v=off(2)), 3), (dict(ks=off(2)), 3), (dict(cu=off(2)), 3),
    (dict(b=0), 0), (dict(t=0), 0), (dict(t=0, b=0, cu=None, kc=None), 0),
])
def test_append(change, status):
    assert _call("pkv_kv_append_fp8_scaled", APPEND_ORDER, APPEND, **change) == status


ATT_ORDER = ["out", "q", "kc", "vc", "ks", "vs", "desc", "bt", "maxb", "cl", "b", "n", "hq", "scale", "ws", "wsb",
             "stream"]
ATT = dict(out=P, q=P, kc=P, vc=P, ks=P, vs=P, desc=_desc(), bt=P, maxb=4096, cl=P, b=2, n=1, hq=32, scale=0.1,
           ws=None, wsb=0, stream=None)


@pytest.mark.parametrize("n", [1, 9, 100])
@pytest.mark.parametrize("change,status", [
    (dict(desc=None), 1), (dict(desc=_desc(head_dim=64)), 3), (dict(hq=16), 3), (dict(n=0), 2), (dict(b=-1), 2),
    (dict(maxb=0), 2), (dict(maxb=1 << 27), 3), (dict(scale=0.0), 2), (dict(scale=-0.1), 2),
    (dict(scale=float("nan")), 2), (dict(scale=float("inf")), 2), (dict(out=None), 1), (dict(q=None), 1),
    (dict(kc=None), 1), (dict(vc=None), 1), (dict(ks=None), 1), (dict(vs=None), 1), (dict(bt=None), 1),
    (dict(cl=None), 1), (dict(q=off(8)), 3), (dict(out=off(4)), 3), (dict(ks=off(2)), 3), (dict(b=1 << 28), 3),
    (dict(desc=_desc(num_blocks=0)), 2), (dict(desc=_desc(num_blocks=1 << 30)), 3),
    (dict(b=2), 4), (dict(ws=P, wsb=100), 4), (dict(ws=off(16), wsb=1 << 40), 4), (dict(b=0), 0),
])
def test_attention(change, status, n):
    assert _call("pkv_paged_attention_fp8_scaled", ATT_ORDER, ATT, **{"n": n, **change}) == status


COPY_ORDER = ["kc", "vc", "ks", "vs", "desc", "src", "dst", "n", "stream"]
COPY = dict(kc=P, vc=P, ks=P, vs=P, desc=_desc(), src=P, dst=P, n=3, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(desc=None), 1), (dict(desc=_desc(head_dim=64)), 3), (dict(n=-1), 2), (dict(n=(1 << 30) + 1), 3),
    (dict(kc=None), 1), (dict(vc=None), 1), (dict(ks=None), 1), (dict(vs=None), 1), (dict(src=None), 1),
    (dict(dst=None), 1), (dict(kc=off(8)), 3), (dict(vs=off(2)), 3), (dict(n=0), 0),
])
def test_copy_blocks(change, status):
    assert _call("pkv_copy_blocks_fp8_scaled", COPY_ORDER, COPY, **change) == status


@pytest.mark.parametrize("b,n,heads,maxb", [(1, 1, 32, 520), (64, 1, 32, 1001), (128, 1, 32, 530), (37, 7, 32, 150),
                                            (4, 2000, 32, 500), (1, 300, 4, 4000), (1, 1, 4, 1)])
def test_workspace_is_bounded(b, n, heads, maxb):
    """Two partials of a CTA's rows and their bookkeeping at most, or the splits of single tokens."""
    size = pkv.workspace_size_fp8_scaled(b, n, heads, maxb)
    assert size % 256 == 0
    assert size <= (152 * 2 * 256 * 520 + 152 * 40 + 768 if n > 1 else b * heads * 64 * 520 + 512)


def test_sizes_of_nothing():
    assert pkv.workspace_size_fp8_scaled(0, 1, 32, 10) == 0
    assert pkv.workspace_size_fp8_scaled(1, 0, 32, 10) == 0
    assert pkv.workspace_size_fp8_scaled(1, 1, 32, 0) == 0
    assert pkv.workspace_size_fp8_scaled(1, 1, 32, -1) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="needs tensors that are not on the current device")
def test_python_refuses_host_tensors():
    try:
        pkv._binding()
    except RuntimeError as e:  # no compiler for the binding
        pytest.skip(str(e))
    q = torch.zeros((4, 8, 128), dtype=torch.bfloat16)
    with pytest.raises((ValueError, RuntimeError)):
        pkv.prompt_attention(q, q, q, q, torch.zeros(2, dtype=torch.int32), 0.1)

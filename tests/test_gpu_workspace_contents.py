"""Nothing of a workspace is read that the call has not written: every path
that merges splits through one gives the same bits whether it held zeros or
NaN (0xff bytes) before."""
import pytest
import torch

import test_gpu_cascade as cascade
import verify_util as V
import workloads as W

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import paged_kv_decode_attention_gb300 as pkv
else:  # collected on CPU-only machines, every test skipped
    pkv = None

CTX = [0, 1, 15, 16, 17, 333, 1000, 64, 2000, 5]


def _same(call, shape):
    """call(out, workspace) with either content."""
    pkv.get_device_error(reset=True)
    outs = []
    for byte in (0, 255):
        out = torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        call(out, torch.full((256 << 20,), byte, dtype=torch.uint8, device="cuda"))
        torch.cuda.synchronize()
        assert torch.isfinite(out).all()
        outs.append(out)
    assert torch.equal(*outs)
    assert pkv.get_device_error(reset=True) == 0


@pytest.mark.parametrize("q_len", [1, 3, 16, 40])
@pytest.mark.parametrize("bps", [0, 1, 4, 13, 40])
def test_attention(q_len, bps):
    d = {k: v.cuda() for k, v in V.paged_case(CTX, q_len, 2, 1).items()}
    _same(lambda out, ws: pkv.paged_attention(out, d["q"], d["k_cache"], d["v_cache"], d["block_tables"],
                                              d["context_lens"], q_len, V.SCALE, kv_blocks_per_split=bps,
                                              workspace=ws), d["q"].shape)


@pytest.mark.parametrize("bps", [8, 16, 40])
def test_decode_of_a_large_batch(bps):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    ctx = CTX + [40] * (-(-2 * sms // 8) - len(CTX))
    d = {k: v.cuda() for k, v in V.paged_case(ctx, 1, 8, 1).items()}
    _same(lambda out, ws: pkv.paged_attention(out, d["q"], d["k_cache"], d["v_cache"], d["block_tables"],
                                              d["context_lens"], 1, V.SCALE, kv_blocks_per_split=bps, workspace=ws),
          d["q"].shape)


@pytest.mark.parametrize("bps", [0, 16, 40])
@pytest.mark.parametrize("fmt", ["e4m3", "q8_0"])
def test_quantised_decode(fmt, bps):
    d = {k: v.cuda() for k, v in V.paged_case(CTX, 1, 2, 1).items()}
    n = d["k_cache"].shape[0]
    gen = torch.Generator().manual_seed(7)
    pools = []
    for _ in range(2):
        x = torch.randn((n, 2, 16, 128), generator=gen)
        if fmt == "e4m3":
            pools.append(x.to(torch.float8_e4m3fn).view(torch.uint8).cuda())
        else:
            codes = (x * 30).clamp(-127, 127).to(torch.int8).view(n, 2, 2048).view(torch.uint8)
            scales = torch.full((n, 2, 64), 1 / 30, dtype=torch.float16).view(torch.uint8)
            pools.append(torch.cat([codes, scales], -1).contiguous().cuda())
    attend = pkv.paged_attention_fp8_e4m3 if fmt == "e4m3" else pkv.paged_attention_q8_0
    _same(lambda out, ws: attend(out, d["q"], *pools, d["block_tables"], d["context_lens"], V.SCALE,
                                 kv_blocks_per_split=bps, workspace=ws), d["q"].shape)


@pytest.mark.parametrize("q_len", [1, 16, 70])
@pytest.mark.parametrize("mask", ["tree", "window"])
def test_masked(mask, q_len):
    ctx = [max(c, q_len) if c else 0 for c in CTX]
    d = {k: v.cuda() for k, v in V.paged_case(ctx, q_len, 2, 1).items()}
    words = V.masks_to_words([[list(range(i + 1)) for i in range(q_len)]] * len(ctx), q_len).cuda()
    lens = torch.tensor([min(c, max(1, q_len - r)) for r, c in enumerate(ctx)], dtype=torch.int32).cuda()
    args = (d["q"], d["k_cache"], d["v_cache"], d["block_tables"], d["context_lens"])
    if mask == "tree":
        call = lambda out, ws: pkv.paged_attention_tree(out, *args, words, V.SCALE, lens, kv_blocks_per_split=4,
                                                        workspace=ws)
    else:
        call = lambda out, ws: pkv.paged_attention_window(out, *args, q_len, 900, 20, V.SCALE, kv_blocks_per_split=4,
                                                          workspace=ws)
    _same(call, d["q"].shape)


def _same_cascade(monkeypatch, w, gs, gb, sp, pbps, sbps):
    empty, outs = torch.empty, []
    for byte in (0, 255):

        def filled(*a, **kw):
            t = empty(*a, **kw)
            return t.fill_(byte) if t.dtype == torch.uint8 else t

        with monkeypatch.context() as m:
            m.setattr(torch, "empty", filled)  # (its workspace)
            outs.append(cascade.run_cascade(w, gs, gb, sp, pbps, sbps, append=False))
    assert torch.equal(*outs) and torch.isfinite(outs[0]).all()


@pytest.mark.parametrize("pbps,sbps", [(0, 0), (4, 3), (16, 1000), (1, 1)])
def test_cascade(monkeypatch, pbps, sbps):
    """A group and requests outside it, a padding row and a context that ends inside its prefix."""
    ctx = [130, 200, 129, 140, 300, 50, 77, 16, 1, 60]
    w = W.build("casc", ctx, 160, seed=50, shared_prefix_blocks=8, sharers=[True] * 5 + [False] * 5)
    groups = W.prefix_groups(w)
    w.context_lens[3], w.context_lens[8] = 70, 0
    _same_cascade(monkeypatch, w, *groups, pbps, sbps)


@pytest.mark.parametrize("pbps,sbps", [(0, 0), (3, 5), (4, 3)])
def test_cascade_of_a_large_batch(monkeypatch, pbps, sbps):
    _same_cascade(monkeypatch, *cascade.large_cascade_batch(seed=3), pbps, sbps)

"""A block table entry that names no block of the pool is reported, whatever
its value: the lowest 32-bit integer too, in the block ids that a kernel reads
first and in those that it reads later, and in the last block of a context."""
import pytest
import torch

import verify_util as V

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import paged_kv_decode_attention_gb300 as pkv
else:  # collected on CPU-only machines, every test skipped
    pkv = None

LOWEST = -2 ** 31
CTX = [1000, 1000]
PLACES = (0, 17, 31, 32, 50, 62)  # logical blocks of request 1


@pytest.fixture(autouse=True)
def _clear_device_error():
    if pkv is not None:
        pkv.get_device_error(reset=True)
    yield
    if pkv is not None:
        assert pkv.get_device_error(reset=True) == 0


def _case(q_len, hkv, seed, ctx=CTX):
    d = {k: v.cuda() for k, v in V.paged_case(ctx, q_len, hkv, seed).items()}
    d["k_cache"][0] = d["v_cache"][0] = 0.25  # what a bad id reads may be a block nobody holds
    return d


def _reported(call, out, tables):
    """call() with request 1's entries replaced one at a time: the error word is set, request 0 keeps its result, and
    request 1's is that of block 0 in the entry's place (what the kernels read for a bad id)."""
    call()
    good = out.clone()
    assert pkv.get_device_error(reset=True) == 0
    for at in PLACES:
        saved = int(tables[1, at])
        tables[1, at] = 0
        call()
        block0 = out.clone()
        assert pkv.get_device_error(reset=True) == 0
        for bad in (LOWEST, LOWEST + 1, -1):
            tables[1, at] = bad
            call()
            assert pkv.get_device_error(reset=True) == pkv.DEVERR_BLOCK_ID, (at, bad)
            assert torch.equal(out[0], good[0]), (at, bad)
            assert torch.equal(out[1], block0[1]), (at, bad)
        tables[1, at] = saved


@pytest.mark.parametrize("q_len", [1, 16, 40, 70])
@pytest.mark.parametrize("bps", [0, 4, 20, 1 << 20])
@pytest.mark.parametrize("mask", ["tree", "window"])
def test_masked_attention(mask, q_len, bps):
    d = _case(q_len, 2, q_len + bps % 7)
    out = torch.empty_like(d["q"])
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    words = V.masks_to_words([[list(range(i + 1)) for i in range(q_len)]] * 2, q_len).cuda()
    args = (out, d["q"], d["k_cache"], d["v_cache"], d["block_tables"], d["context_lens"])
    if mask == "tree":
        call = lambda: pkv.paged_attention_tree(*args, words, V.SCALE, kv_blocks_per_split=bps, workspace=ws)
    else:  # a window that sees every block
        call = lambda: pkv.paged_attention_window(*args, q_len, 2000, 4, V.SCALE, kv_blocks_per_split=bps,
                                                  workspace=ws)
    _reported(call, out, d["block_tables"])


@pytest.mark.parametrize("q_len", [1, 3])
@pytest.mark.parametrize("bps", [0, 1, 4, 13, 1 << 20])
def test_decode_one_cta_per_row(q_len, bps):
    """The CTA-per-row decode: one pass, splits merged in a cluster, splits through the workspace."""
    d = _case(q_len, 2, q_len + bps % 7)
    out = torch.empty_like(d["q"])
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    _reported(lambda: pkv.paged_attention(out, d["q"], d["k_cache"], d["v_cache"], d["block_tables"],
                                          d["context_lens"], q_len, V.SCALE, kv_blocks_per_split=bps, workspace=ws),
              out, d["block_tables"])


@pytest.mark.parametrize("q_len", [16, 40])
@pytest.mark.parametrize("bps", [0, 4, 13, 1 << 20])
def test_causal_chunk(q_len, bps):
    d = _case(q_len, 2, q_len + bps % 7)
    out = torch.empty_like(d["q"])
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    _reported(lambda: pkv.paged_attention(out, d["q"], d["k_cache"], d["v_cache"], d["block_tables"],
                                          d["context_lens"], q_len, V.SCALE, kv_blocks_per_split=bps, workspace=ws),
              out, d["block_tables"])


@pytest.mark.parametrize("bps", [0, 8, 20, 1 << 20])
def test_decode_of_a_large_batch(bps):
    """Enough rows for the tensor-core decode (two per SM)."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    d = _case(1, 8, 3, ctx=CTX + [40] * (-(-2 * sms // 8) - 2))
    out = torch.empty_like(d["q"])
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    _reported(lambda: pkv.paged_attention(out, d["q"], d["k_cache"], d["v_cache"], d["block_tables"],
                                          d["context_lens"], 1, V.SCALE, kv_blocks_per_split=bps, workspace=ws),
              out, d["block_tables"])


@pytest.mark.parametrize("bps", [0, 16, 20, 1 << 20])
@pytest.mark.parametrize("fmt", ["e4m3", "q8_0"])
def test_decode_of_quantised_caches(fmt, bps):
    d = _case(1, 2, 5)
    n = d["k_cache"].shape[0]
    gen = torch.Generator().manual_seed(7)
    pools = []
    for _ in range(2):
        x = torch.randn((n, 2, 16, 128), generator=gen)
        if fmt == "e4m3":
            pools.append(x.to(torch.float8_e4m3fn).view(torch.uint8).cuda())
        else:  # a tile: 16 x 128 codes, then 16 x 4 scales
            codes = (x * 30).clamp(-127, 127).to(torch.int8).view(n, 2, 2048).view(torch.uint8)
            scales = torch.full((n, 2, 64), 1 / 30, dtype=torch.float16).view(torch.uint8)
            pools.append(torch.cat([codes, scales], -1).contiguous().cuda())
    out = torch.empty_like(d["q"])
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    attend = pkv.paged_attention_fp8_e4m3 if fmt == "e4m3" else pkv.paged_attention_q8_0
    _reported(lambda: attend(out, d["q"], *pools, d["block_tables"], d["context_lens"], V.SCALE,
                             kv_blocks_per_split=bps, workspace=ws), out, d["block_tables"])

"""The FP8 cache with block scales at the edges of its calls: a workspace of just the stated size, rows cut into more
pieces than a warp has lanes, new tokens whose boundaries are wrong."""
import pytest
import torch

from test_gpu_fp8_scaled import (BLOCK, D, SCALE, _pkv, append_reference, attention_case, check, dev, pool, reference,
                                 run_attention, tables, values)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q_len,ctx", [(1, [1]), (1, [8300]), (1, [700] * 40), (1, [16000] + [30] * 63), (2, [40, 9]),
                                       (7, [2100] * 37), (16, [300, 5000]), (32, [1000] * 9), (33, [4000, 100]),
                                       (130, [3000, 200])])
def test_nothing_beyond_the_workspace(q_len, ctx):
    """A workspace of the stated size between guards: they stay, and the result is the usual one; a byte less is
    refused."""
    pkv = _pkv()
    q, kc, vc, ks, vs, t = attention_case(ctx, q_len, 2)
    size = pkv.workspace_size_fp8_scaled(len(ctx), q_len, 8, t.shape[1])
    guard = 1 << 16
    room = torch.full((size + 2 * guard,), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, 7.0)
    pkv.paged_attention_fp8_scaled(out, q, kc, vc, ks, vs, dev(t), dev(ctx), q_len, SCALE, room[guard:guard + size])
    assert pkv.get_device_error() == 0
    assert bool((room[:guard] == 0xA5).all()) and bool((room[guard + size:] == 0xA5).all())
    assert torch.equal(out, run_attention(q, kc, vc, ks, vs, t, ctx))
    with pytest.raises(RuntimeError):
        pkv.paged_attention_fp8_scaled(out, q, kc, vc, ks, vs, dev(t), dev(ctx), q_len, SCALE,
                                       room[guard:guard + size - 1])


@pytest.mark.parametrize("q_len,hkv,ctx", [(1, 1, [100000] + [3] * 19), (1, 1, [60000, 90000] + [500] * 30),
                                           (3, 2, [100000]), (20, 1, [70000, 9]), (40, 2, [100000])])
def test_rows_cut_into_many_pieces(q_len, hkv, ctx):
    """One long row over most of the CTAs: more than 32 partials, joined 32 at a time."""
    case = attention_case(ctx, q_len, hkv)
    out = run_attention(*case, ctx)
    assert _pkv().get_device_error() == 0
    check(out, reference(*case, ctx), ctx)
    assert torch.equal(out, run_attention(*case, ctx))


@pytest.mark.parametrize("cu,ctx", [([0, 100, 3, 8], [100, 30, 5]), ([0, 40, 20, 90], [40, 20, 75]),
                                    ([10, 60, 60, 201], [57, 0, 150]), ([-3, 50, 90, 200], [60, 43, 115]),
                                    ([150, 100, 50, 0], [50, 50, 50]), ([0, 64, 0, 64], [70, 64, 64])])
def test_wrong_boundaries_store_whole_blocks_or_nothing(cu, ctx):
    """Each block is what it was or what its request's tokens make of it, and a request whose own entries are wrong is
    left alone."""
    pkv = _pkv()
    tokens, hkv, nb = 200, 2, 40
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((2, tokens, hkv, D), generator=g, device="cuda").to(torch.bfloat16)
    t = tables([-(-c // BLOCK) for c in ctx], nb)
    kc, ks = pool(nb, hkv, 5)
    vc, vs = pool(nb, hkv, 6)
    before = [y.clone() for y in (kc, vc, ks, vs)]
    pkv.kv_append_fp8_scaled(kc, vc, ks, vs, dev(t), dev(ctx), x[0], x[1], dev(cu))
    assert pkv.get_device_error() == pkv.DEVERR_SEQLENS
    stored = 0
    for codes, scales, old, old_s, y in ((kc, ks, before[0], before[2], x[0]), (vc, vs, before[1], before[3], x[1])):
        got, got_s = values(codes), scales.double().cpu()
        was, was_s = values(old), old_s.double().cpu()
        left = torch.ones(nb, dtype=torch.bool)
        for r, c in enumerate(ctx):
            if not 0 <= cu[r] <= cu[r + 1] <= tokens:
                continue
            want, want_s = was.clone(), was_s.clone()
            append_reference(want, want_s, t[r:r + 1], [c], [0, cu[r + 1] - cu[r]], y[cu[r]:cu[r + 1]].double().cpu())
            for b in t[r][t[r] >= 0]:
                here = torch.equal(got[b], want[b]) and torch.equal(got_s[b], want_s[b])
                left[b] = not here
                stored += here
        assert torch.equal(got[left], was[left]) and torch.equal(got_s[left], was_s[left])
    assert stored > 0 or cu == [150, 100, 50, 0]

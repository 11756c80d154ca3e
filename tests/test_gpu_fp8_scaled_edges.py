"""The FP8 cache with block scales at the edges of its calls: a workspace of just the stated size, rows cut into more
pieces than a warp has lanes."""
import pytest
import torch

from test_gpu_fp8_scaled import SCALE, _pkv, attention_case, check, dev, reference, run_attention

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

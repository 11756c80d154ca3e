"""The FP8 cache with block scales where weights and scores span a wide range: one key that holds most of a long row's
weight, scores far from zero, queries that are not finite."""
import math

import pytest
import torch

from test_gpu_fp8_scaled import BLOCK, D, SCALE, attention_case, dev, run_attention

pytestmark = pytest.mark.gpu


def sink_case(requests, ctx, share, v_sink, q_len, hkv=1, seed=0):
    """Requests over one shared context whose first key takes `share` of the weight and whose V is `v_sink` of the
    others' size; the other weights are lognormal, V is normal with a mean of half a deviation."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    nb = -(-ctx // BLOCK)
    base = 2 * normal(hkv, D)
    q = base[None, None, :, None] + 0.2 * normal(requests, q_len, hkv, 4, D)
    size = float((base * base).sum(-1).mean())
    k = normal(nb * BLOCK, hkv, D) / (size ** 0.5 * SCALE)  # scores of deviation 1
    k[0] = base * (math.log(share / (1 - share) * ctx) + 0.5) / (size * SCALE)
    v = 0.5 + normal(nb * BLOCK, hkv, D)
    v[0] *= v_sink
    pools = []
    for x in (k, v):
        s = 2.0 ** math.ceil(math.log2(float(x.abs().max()) / 448))
        codes = (x / s).to(torch.float8_e4m3fn).view(torch.uint8)
        pools += [codes.view(nb, BLOCK, hkv, D).transpose(1, 2).contiguous(), torch.full((nb, hkv), s, device="cuda")]
    t = torch.arange(nb).expand(requests, nb).numpy()
    return q.reshape(requests, q_len, 4 * hkv, D).to(torch.bfloat16), pools[0], pools[2], pools[1], pools[3], t


def sink_error(case, out, ctx):
    """The rows' largest error, relative to the norm of their exact value, over some of the requests."""
    q, kc, vc, ks, vs, _ = case
    n, hkv = q.shape[1], kc.shape[1]
    some = sorted({*range(min(3, q.shape[0])), q.shape[0] // 2, q.shape[0] - 1})
    worst = 0.0
    for h in range(hkv):
        k, v = ((c.view(torch.float8_e4m3fn)[:, h].float().double() * s[:, h, None, None].double()).flatten(0, 1)[:ctx]
                for c, s in ((kc, ks), (vc, vs)))
        hidden = torch.arange(ctx, device="cuda")[None] > torch.arange(ctx - n, ctx, device="cuda")[:, None]
        for r in some:
            for g in range(4 * h, 4 * h + 4):
                x = (q[r, :, g].double() @ k.T * SCALE).masked_fill(hidden, -math.inf)
                want = torch.softmax(x, -1) @ v
                worst = max(worst, float(((out[r, :, g].double() - want).norm(dim=-1) / want.norm(dim=-1)).max()))
    return worst


# Requests: one (divided among CTAs), or one for each SM.
@pytest.mark.parametrize("requests", [1, 152])
@pytest.mark.parametrize("ctx,share,v_sink", [(2048, 0.9, 0.02), (8192, 0.9, 0.02), (32768, 0.5, 1.0), (32768, 0.9, 0.02),
                                              (131072, 0.5, 1.0), (131072, 0.99, 0.02)])
@pytest.mark.parametrize("q_len", [1, 2, 8, 9, 16, 17, 32, 40])
def test_most_of_the_weight_on_one_key(q_len, ctx, share, v_sink, requests):
    """Each weight is off by at most 2^-8 of itself, whatever the largest one is: of the row no more than that, and the
    result's rounding to BF16, 2^-8 of each value at most and evenly spread, 2^-8 / sqrt(3) of the row's norm."""
    case = sink_case(requests, ctx, share, v_sink, q_len)
    out = run_attention(*case, [ctx] * requests)
    assert sink_error(case, out, ctx) < 5e-3


@pytest.mark.parametrize("q_len", [1, 4, 8, 16, 20, 32, 40, 100])
@pytest.mark.parametrize("e", [-6, 10, 16, 18, 20, 25, 28, 32])
def test_scores_far_from_zero(q_len, e):
    """K scales up to the largest: the scores' differences are far beyond the rounding of the scores, so a row's result
    is the value of its highest key, to the rounding of that one weight (2^-8) and of the result (2^-8)."""
    ctx = [300, 64, 900]
    q, kc, vc, ks, vs, t = attention_case(ctx, q_len, 2)
    ks.fill_(2.0 ** e)
    out = run_attention(q, kc, vc, ks, vs, t, ctx)
    assert bool(out.isfinite().all())
    clear, rows = 0, 0
    for r, c in enumerate(ctx):
        at = torch.arange(c, device="cuda")
        blk, off = dev(t[r], torch.int64)[at // BLOCK], at % BLOCK
        seen = at[None] <= torch.arange(c - q_len, c, device="cuda")[:, None]
        for h in range(8):
            k, v = (z.view(torch.float8_e4m3fn).float()[blk, h // 4, off].double() * s[blk, h // 4, None].double()
                    for z, s in ((kc, ks), (vc, vs)))
            x = (q[r, :, h].double() @ k.T * SCALE).masked_fill(~seen, -math.inf)
            # a score is off by at most 2^-17 of sum |q| |k| twice over (see test_gpu_fp8_scaled.check), and its
            # rounding; 40 more: the other keys' weights are below 2^-50
            slack = SCALE * 2.0 ** -16 * (q[r, :, h].double().abs().amax(-1, keepdim=True) * k.abs().sum(-1)).amax(-1)
            exp = x.amax(-1) - slack * 4 - 40
            one = ((x > exp[:, None]).sum(-1) == 1) & (seen.sum(-1) > 0)
            want = v[x.argmax(-1)]
            err = (out[r, :, h].double() - want).abs()
            assert bool((err[one] <= 2.0 ** -7 * 1.01 * want[one].abs()).all())
            clear += int(one.sum())
            rows += int((seen.sum(-1) > 0).sum())
    if e >= 10:
        assert clear > 0.9 * rows


@pytest.mark.parametrize("small", [False, True])
@pytest.mark.parametrize("q_len", [1, 7, 20, 32, 40])
@pytest.mark.parametrize("count", [2, 40])
def test_queries_that_are_not_finite(q_len, count, small):
    """A query with an infinity or NaN gives NaN, however small the keys are; the others' rows are what they were, bit
    for bit."""
    ctx = ([300, 70] * count)[:count]
    case = attention_case(ctx, q_len, 2)
    q, kc = case[:2]
    if small:
        kc[:] = (2.0 ** -7 * torch.randn(kc.shape, device="cuda")).to(torch.float8_e4m3fn).view(torch.uint8)
    want = run_attention(*case, ctx)
    assert bool(want.isfinite().all())
    bad = torch.zeros(q.shape[:3], dtype=torch.bool, device="cuda")
    for i, x in enumerate((math.inf, -math.inf, math.nan)):
        r, at, h = i % count, (3 * i) % q_len, (3 * i + 1) % 8
        q[r, at, h, 17 * i + 5] = x
        bad[r, at, h] = True
    out = run_attention(*case, ctx)
    assert bool(out[bad].isnan().all())
    assert torch.equal(out[~bad], want[~bad])

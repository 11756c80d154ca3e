"""The FP8 cache with block scales: append, attention and block copies against their definitions in 64 bits."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BLOCK, D = 16, 128
SCALE = D ** -0.5


def _pkv():
    import paged_kv_decode_attention_gb300 as pkv
    return pkv


def dev(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x)).to(device="cuda", dtype=dtype)


def tables(counts, total, seed=0, spare=1):
    perm = np.random.default_rng(seed).permutation(total)
    t = np.full((len(counts), max(counts) + spare), -1, np.int32)
    at = 0
    for r, n in enumerate(counts):
        t[r, :n] = perm[at:at + n]
        at += n
    return t


def round_e4m3(x):
    """64-bit: to the nearest of 4 significant bits, no bit below 2^-9, ties to even, at most 448."""
    a = x.abs().clamp(min=2.0 ** -60)
    p = torch.floor(torch.log2(a)).clamp(min=-6)
    step = torch.exp2(p - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def scale_of(amax):
    if amax == 0:
        return 2.0 ** -32
    e = math.ceil(math.log2(amax / 448.0))
    while amax > 448.0 * 2.0 ** e:
        e += 1
    while amax <= 448.0 * 2.0 ** (e - 1):
        e -= 1
    return 2.0 ** min(max(e, -32), 32)


def append_reference(codes, scales, table, ctx, starts, x):
    """codes [nb][Hkv][16][128] and scales [nb][Hkv] as 64-bit values on the host, changed in place."""
    for r in range(len(ctx)):
        n = starts[r + 1] - starts[r]
        if n == 0 or ctx[r] <= 0:
            continue
        p0 = ctx[r] - n
        for lb in range(p0 // BLOCK, -(-ctx[r] // BLOCK)):
            a, b = max(p0, lb * BLOCK), min(ctx[r], (lb + 1) * BLOCK)
            rows = x[starts[r] + a - p0:starts[r] + b - p0]
            blk, off = table[r][lb], a - lb * BLOCK
            for h in range(codes.shape[1]):
                s = scale_of(float(rows[:, h].abs().max()))
                if off > 0 and float(scales[blk, h]) > s:
                    s = float(scales[blk, h])
                if off > 0 and s != float(scales[blk, h]):
                    codes[blk, h, :off] = round_e4m3(codes[blk, h, :off] * (float(scales[blk, h]) / s))
                scales[blk, h] = s
                codes[blk, h, off:off + b - a] = round_e4m3(rows[:, h] / s)


def values(codes):
    return codes.view(torch.float8_e4m3fn).float().double().cpu()


def pool(nb, hkv, seed, power=True, lo=-6, hi=6):
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = (torch.randn((nb, hkv, BLOCK, D), generator=g, device="cuda") * 100).clamp(-448, 448)
    codes = codes.to(torch.float8_e4m3fn).view(torch.uint8)
    e = torch.randint(lo, hi + 1, (nb, hkv), generator=g, device="cuda").double()
    scales = torch.exp2(e - 6).float()
    if not power:
        scales *= 1 + torch.rand((nb, hkv), generator=g, device="cuda")
    return codes, scales


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("hkv", [1, 3, 8])
@pytest.mark.parametrize("before,new", [
    ([0], [1]), ([15], [1]), ([16], [1]), ([7, 0, 31, 100], [1, 1, 1, 1]), ([0, 3, 16], [16, 13, 32]),
    ([5, 0, 40, 8, 0], [0, 500, 3, 24, 17]), ([1] * 70, list(range(70))), ([9] * 1100, [1] * 1100)])
def test_append(before, new, hkv):
    pkv = _pkv()
    g = torch.Generator(device="cuda").manual_seed(len(before) + hkv)
    ctx = [b + n for b, n in zip(before, new)]
    counts = [-(-c // BLOCK) for c in ctx]
    nb = sum(counts) + 3
    t = tables(counts, nb)
    starts = [0] + np.cumsum(new).tolist()
    x = [torch.randn((starts[-1], hkv, D), generator=g, device="cuda") *
         torch.exp2(4 * torch.randn((starts[-1], 1, 1), generator=g, device="cuda")) for _ in range(2)]
    x = [y.to(torch.bfloat16) for y in x]
    kc, ks = pool(nb, hkv, 1)
    vc, vs = pool(nb, hkv, 2, power=False)
    want = []
    for codes, scales, y in ((kc, ks, x[0]), (vc, vs, x[1])):
        c, s = values(codes), scales.double().cpu()
        if scales is vs:  # (64-bit quotients of other scales round elsewhere than the 32-bit ones)
            s = torch.exp2(torch.round(torch.log2(s)))
            vs.copy_(s.float())
        append_reference(c, s, t, ctx, starts, y.double().cpu())
        want.append((c, s))
    pkv.kv_append_fp8_scaled(kc, vc, ks, vs, dev(t), dev(ctx), x[0], x[1], dev(starts))
    assert pkv.get_device_error() == 0
    for (c, s), codes, scales in zip(want, (kc, vc), (ks, vs)):
        assert torch.equal(scales.double().cpu(), s)
        assert torch.equal(values(codes), c)
    if all(n == 1 for n in new):  # the single-token form: the same bits
        again = [z.clone() for z in (kc, vc, ks, vs)]
        pkv.kv_append_fp8_scaled(kc, vc, ks, vs, dev(t), dev(ctx), x[0], x[1])
        assert all(torch.equal(a, b) for a, b in zip(again, (kc, vc, ks, vs)))


def test_append_into_blocks_of_other_scales():
    """Scales that are no powers of two, as calibrated pools have: kept or outgrown, in FP32 arithmetic."""
    pkv = _pkv()
    kc, ks = pool(8, 2, 1, power=False)
    vc, vs = pool(8, 2, 2, power=False)
    x = (30 * torch.randn((8, 2, D), device="cuda")).to(torch.bfloat16)
    want = []
    for codes, scales in ((kc, ks), (vc, vs)):
        c, s, y = codes.cpu().view(torch.float8_e4m3fn).float(), scales.cpu().clone(), x.cpu().float()
        for b in range(8):
            for h in range(2):
                new = max(float(s[b, h]), scale_of(float(y[b, h].abs().max())))
                grown = torch.tensor(new)
                if new != float(s[b, h]):
                    f = s[b, h] / grown
                    c[b, h, :5] = (c[b, h, :5] * f).to(torch.float8_e4m3fn).float()
                c[b, h, 5] = (y[b, h] / grown).clamp(-448, 448).to(torch.float8_e4m3fn).float()
                s[b, h] = grown
        want.append((c, s))
    grew = sum(int((w[1] != z.cpu()).sum()) for w, z in zip(want, (ks, vs)))
    assert 0 < grew < 32
    pkv.kv_append_fp8_scaled(kc, vc, ks, vs, dev(np.arange(8)[:, None]), dev([6] * 8), x, x)
    for (c, s), codes, scales in zip(want, (kc, vc), (ks, vs)):
        assert torch.equal(scales.cpu(), s)
        assert torch.equal(values(codes), c.double())


def test_append_token_by_token_keeps_the_block_accurate():
    """A block filled one token at a time, each larger than the ones before: every value stays within E4M3's rounding
    of the block's final scale."""
    pkv = _pkv()
    hkv = 2
    x = (torch.randn((BLOCK, hkv, D), device="cuda") * torch.exp2(torch.arange(BLOCK, device="cuda") - 8.0)[:, None, None]).to(torch.bfloat16)
    kc, ks = pool(1, hkv, 3)
    vc, vs = pool(1, hkv, 4)
    for i in range(BLOCK):
        pkv.kv_append_fp8_scaled(kc, vc, ks, vs, dev([[0]]), dev([i + 1]), x[i:i + 1], x[i:i + 1])
    for codes, scales in ((kc, ks), (vc, vs)):
        for h in range(hkv):
            s = scale_of(float(x[:, h].float().abs().max()))
            assert float(scales[0, h]) == s
            got = values(codes)[0, h] * s
            y = x[:, h].double().cpu()
            # one rounding per growth in E4M3's subnormal range (its steps halve each time: at most twice the last),
            # half a step of the normal range (2^-4) once
            assert bool(((got - y).abs() <= 2.0 ** -4 * y.abs() + 2.0 ** -9 * s).all())


def test_append_extremes():
    pkv = _pkv()
    x = torch.zeros((6, 1, D), dtype=torch.bfloat16, device="cuda")
    x[1, 0, 0] = 448.0
    x[2, 0, 0] = 450.0
    x[3, 0, 0] = 3.0e38
    x[4, 0, 5] = 1e-30
    x[5, 0, 7] = -448.0 * 2.0 ** 32
    kc, ks = pool(6, 1, 3)
    vc, vs = pool(6, 1, 4)
    pkv.kv_append_fp8_scaled(kc, vc, ks, vs, dev(np.arange(6)[:, None]), dev([1] * 6), x, x)
    for codes, scales in ((kc, ks), (vc, vs)):
        assert scales[:, 0].tolist() == [2.0 ** -32, 1.0, 2.0, 2.0 ** 32, 2.0 ** -32, 2.0 ** 32]
        c = values(codes)
        assert float(c[1, 0, 0, 0]) == 448 and float(c[3, 0, 0, 0]) == 448 and float(c[5, 0, 0, 7]) == -448
        assert bool((c[0, 0, 0] == 0).all()) and bool((c[4, 0, 0] == 0).all())


def test_append_leaves_the_rest():
    """Slots past the new tokens, other blocks, padding rows and bad requests keep their bytes."""
    pkv = _pkv()
    hkv, nb = 2, 12
    t = np.full((6, 3), -1, np.int32)
    t[0, :2], t[1, :1], t[2, :3], t[3, :2], t[4, :3], t[5, 0] = [1, 2], [3], [4, 5, 6], [7, 99], [8, 9, 10], 11
    ctx = [20, 0, 60, 18, 3, 2]  # 2: longer than its table; 3: its second block is bad; 4: shorter than its tokens
    starts = [0, 3, 5, 9, 13, 17, 17]  # 1 is a padding row with tokens, 5 has none
    x = torch.randn((20, hkv, D), device="cuda").to(torch.bfloat16)
    kc, ks = pool(nb, hkv, 5)
    vc, vs = pool(nb, hkv, 6)
    before = [y.clone() for y in (kc, vc, ks, vs)]
    want = [(values(kc), ks.double().cpu()), (values(vc), vs.double().cpu())]
    good = [20, 0, 0, 0, 0, 2]
    for c, s in want:
        append_reference(c, s, t, good, starts, x.double().cpu())
        tt = t.copy()
        append_reference(c, s, tt, [0, 0, 0, 16, 0, 0], [0, 0, 0, 9, 11, 11, 11], x.double().cpu())
    pkv.kv_append_fp8_scaled(kc, vc, ks, vs, dev(t), dev(ctx), x, x, dev(starts))
    assert pkv.get_device_error() == pkv.DEVERR_CONTEXT | pkv.DEVERR_BLOCK_ID
    for (c, s), codes, scales in zip(want, (kc, vc), (ks, vs)):
        assert torch.equal(values(codes), c) and torch.equal(scales.double().cpu(), s)
    for y, z in zip((kc, vc, ks, vs), before):
        keep = [0, 1, 3, 4, 5, 6, 8, 9, 10, 11]
        assert torch.equal(y[keep], z[keep])


@pytest.mark.parametrize("cu", [[0, 5, 3, 8], [0, 2, 4, 99], [-1, 2, 4, 8], [8, 6, 4, 2]])
def test_append_bad_boundaries_are_reported(cu):
    pkv = _pkv()
    kc, ks = pool(8, 2, 5)
    vc, vs = pool(8, 2, 6)
    x = torch.randn((8, 2, D), device="cuda").to(torch.bfloat16)
    pkv.kv_append_fp8_scaled(kc, vc, ks, vs, dev([[0, 1], [2, 3], [4, 5]]), dev([20, 20, 20]), x, x, dev(cu))
    assert pkv.get_device_error() & pkv.DEVERR_SEQLENS


def test_append_strided():
    pkv = _pkv()
    wide = torch.randn((40, 6 * D + 8), device="cuda").to(torch.bfloat16)
    k, v = wide[:, : 2 * D].view(40, 2, D), wide[:, 3 * D:5 * D].view(40, 2, D)
    outs = []
    for a, b in ((k, v), (k.contiguous(), v.contiguous())):
        kc, ks = pool(5, 2, 5)
        vc, vs = pool(5, 2, 6)
        pkv.kv_append_fp8_scaled(kc, vc, ks, vs, dev([[4, 2, 0], [1, 3, -1]]), dev([30, 10]), a, b, dev([0, 30, 40]))
        outs.append((kc, vc, ks, vs))
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_copy_blocks():
    pkv = _pkv()
    kc, ks = pool(9, 3, 5)
    vc, vs = pool(9, 3, 6)
    before = [y.clone() for y in (kc, vc, ks, vs)]
    pkv.copy_blocks_fp8_scaled(kc, vc, ks, vs, dev([1, 4]), dev([8, 0]))
    for y, z in zip((kc, vc, ks, vs), before):
        z[8], z[0] = z[1].clone(), z[4].clone()
        assert torch.equal(y, z)
    assert pkv.get_device_error() == 0
    pkv.copy_blocks_fp8_scaled(kc, vc, ks, vs, dev([1, 9, -1]), dev([2, 3, 5]))
    assert pkv.get_device_error() == pkv.DEVERR_BLOCK_ID
    before[0][2] = before[0][1]
    assert torch.equal(kc, before[0])


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def reference(q, kc, vc, ks, vs, t, ctx, scale=SCALE):
    """out [B][q_len][Hq][128] in 64 bits; sum of w |v|; the largest w |v scale| 448 and what the scores may be off."""
    b, n, hq, _ = q.shape
    hkv = kc.shape[1]
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    mass, floor = torch.zeros_like(out), torch.zeros(q.shape[:3], dtype=torch.float64, device="cuda")
    score = torch.zeros_like(floor)
    for r in range(b):
        if ctx[r] <= 0:
            continue
        at = torch.arange(ctx[r], device="cuda")
        blk, off = dev(t[r], torch.int64)[at // BLOCK], at % BLOCK
        k, v = (c.view(torch.float8_e4m3fn).float()[blk, :, off].double() * s[blk].double()[..., None]
                for c, s in ((kc, ks), (vc, vs)))
        for h in range(hq):
            kh, vh, sv = k[:, h // (hq // hkv)], v[:, h // (hq // hkv)], vs[blk, h // (hq // hkv)].double()
            x = q[r, :, h].double() @ kh.T * scale
            seen = at[None] <= torch.arange(ctx[r] - n, ctx[r], device="cuda")[:, None]
            x = x.masked_fill(~seen, -math.inf)
            w = torch.softmax(x, -1).nan_to_num(0.0)
            out[r, :, h], mass[r, :, h] = w @ vh, w @ vh.abs()
            floor[r, :, h] = (w * sv).amax(-1) * 448
            score[r, :, h] = scale * torch.where(seen, 2.0 ** -17 * q[r, :, h].double().abs().amax(-1, keepdim=True) *
                                                 kh.abs().sum(-1) + 2.0 ** -17 * (q[r, :, h].double().abs() @ kh.abs().T),
                                                 torch.zeros_like(x)).amax(-1)
    return out, mass, floor, score


def check(out, ref, ctx, rel=5e-3):
    """Queries: two E4M3 parts, off by at most 2^-17 of the head's largest value; FP32 sums of 128 products.  Weights:
    two E4M3 parts, 2^-8 relative (chunks: by way of FP16, 2^-11 more), down to 2^-16 of the largest weight with its
    scale.  The result: BF16, 2^-8 relative."""
    want, mass, floor, score = ref
    n = max(max(ctx), 1)
    w_err = 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -20 + 2 * score + n * 2.0 ** -23
    tol = 2.0 ** -8 * want.abs() + 1.02 * (w_err[..., None] * mass + n * 2.0 ** -16 * floor[..., None]) + 1e-30
    err = (out.double() - want).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    if float(want.norm()) > 0:
        assert float(err.norm() / want.norm()) < rel


def attention_case(ctx, q_len, hkv, seed=0, power=True, spread=6, extra=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    counts = [max(-(-c // BLOCK), 0) for c in ctx]
    nb = sum(counts) + 2
    t = tables(counts, nb, seed, extra) if max(counts) else np.full((len(ctx), 1), -1, np.int32)
    kc, ks = pool(nb, hkv, seed + 1, power)
    vc, vs = pool(nb, hkv, seed + 2, power, -spread, spread)
    ks *= 0.25
    q = (2 * torch.randn((len(ctx), q_len, 4 * hkv, D), generator=g, device="cuda")).to(torch.bfloat16)
    # slots past the context hold NaN codes
    for r, c in enumerate(ctx):
        if c % BLOCK and c > 0:
            for z in (kc, vc):
                z[t[r][c // BLOCK], :, c % BLOCK:] = 0x7F
    return q, kc, vc, ks, vs, t


def run_attention(q, kc, vc, ks, vs, t, ctx):
    pkv = _pkv()
    b, n, hq, _ = q.shape
    out = torch.full_like(q, 7.0)
    ws = torch.full((max(pkv.workspace_size_fp8_scaled(b, n, hq, t.shape[1]), 1),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    pkv.paged_attention_fp8_scaled(out, q, kc, vc, ks, vs, dev(t), dev(ctx), n, SCALE, ws)
    return out


@pytest.mark.parametrize("hkv", [1, 2, 8])
@pytest.mark.parametrize("q_len,ctx", [
    (1, [1]), (1, [16, 17, 15, 0]), (1, [300, 1, 255, 256, 257, 1000]), (1, [5000]), (1, [33] * 60),
    (2, [2, 1, 0, 40]), (3, [700, 2]), (4, [65, 600]), (5, [66, 300]), (7, [129, 128, 7, 3, 0, 260]), (8, [8, 400, 64]),
    (9, [9, 63, 400]), (16, [16, 500]), (17, [17, 900]), (31, [31, 200]), (32, [32, 33, 500]), (33, [33, 40, 1000]), (64, [300, 64, 20]), (65, [65, 1500]), (200, [200, 777])])
def test_attention(q_len, ctx, hkv):
    case = attention_case(ctx, q_len, hkv)
    out = run_attention(*case, ctx)
    assert _pkv().get_device_error() == 0
    check(out, reference(*case, ctx), ctx)


@pytest.mark.parametrize("q_len", [1, 5, 40])
@pytest.mark.parametrize("ctx", [[1100, 40, 0, 513], [9000], [20000, 3, 3, 3, 3, 3], [60] * 300, [1] * 500,
                                 [129, 0, 0, 4000, 257, 0] * 9])
def test_cuts(q_len, ctx):
    """Work cut anywhere: within one long context over all CTAs, between short ones, several to a CTA."""
    case = attention_case(ctx, q_len, 2, extra=7)
    out = run_attention(*case, ctx)
    assert _pkv().get_device_error() == 0
    check(out, reference(*case, ctx), ctx)
    assert torch.equal(out, run_attention(*case, ctx))


@pytest.mark.parametrize("q_len", [1, 4, 50])
def test_scales_of_any_value_and_wide_spread(q_len):
    """Scales that are no powers of two; V scales that differ by 2^40 between blocks."""
    ctx = [600, 90]
    case = attention_case(ctx, q_len, 2, power=False)
    check(run_attention(*case, ctx), reference(*case, ctx), ctx)
    case = attention_case(ctx, q_len, 2, spread=20)
    check(run_attention(*case, ctx), reference(*case, ctx), ctx)
    # scales at both ends of the range, in different requests and heads
    case = attention_case(ctx, q_len, 2)
    vs = case[4]
    vs[:, 0], vs[:, 1] = 2.0 ** -32, 2.0 ** 32
    case[3].fill_(2.0 ** -6)
    out, ref = run_attention(*case, ctx), reference(*case, ctx)
    for heads in (slice(0, 4), slice(4, 8)):
        check(out[:, :, heads], tuple(x[:, :, heads] for x in ref), ctx)


@pytest.mark.parametrize("q_len", [1, 6, 48])
def test_small_v_scale_under_most_of_the_weight(q_len):
    """The block that takes nearly all the weight has a V scale 2^-14 of the others': its values still come out."""
    ctx = [256]
    q, kc, vc, ks, vs, t = attention_case(ctx, q_len, 1)
    vs.fill_(1.0)
    vs[t[0][0]] = 2.0 ** -14
    ks.fill_(2.0 ** -6)
    k0 = q[0, 0, 0].float()
    q[:] = q[:, :1, :1]
    kc[:] = 0
    kc[t[0][0], :, :] = (k0 * 30).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    case = (q, kc, vc, ks, vs, t)
    check(run_attention(*case, ctx), reference(*case, ctx), ctx)


@pytest.mark.parametrize("q_len", [1, 3, 12, 20, 48])
def test_queries_and_scales_whose_product_vanishes(q_len):
    """Scores whose factor leaves FP32's range: the masked places stay masked, the others weigh the same."""
    ctx = [200, 70]
    q, kc, vc, ks, vs, t = attention_case(ctx, q_len, 2)
    q = (q.float() * 2.0 ** -124).to(torch.bfloat16)
    ks.fill_(2.0 ** -32)
    case = (q, kc, vc, ks, vs, t)
    check(run_attention(*case, ctx), reference(*case, ctx), ctx)


@pytest.mark.parametrize("count", [3, 40])
@pytest.mark.parametrize("q_len", [1, 2, 12, 24, 50])
def test_a_broken_request_breaks_no_other(q_len, count):
    """NaN codes in one request's context: its rows are NaN, the others' are what they were, bit for bit."""
    ctx = ([300, 70, 500] * count)[:count]
    q, kc, vc, ks, vs, t = attention_case(ctx, q_len, 2)
    want = run_attention(q, kc, vc, ks, vs, t, ctx)
    for broken in (kc, vc):
        kept = broken.clone()
        broken[t[1][0], :, 3] = 0x7F
        out = run_attention(q, kc, vc, ks, vs, t, ctx)
        broken.copy_(kept)
        assert bool(out[1].isnan().all())
        rest = [r for r in range(count) if r != 1]
        assert torch.equal(out[rest], want[rest])


@pytest.mark.parametrize("q_len", [1, 5, 70])
def test_bad_tables_and_contexts_are_reported(q_len):
    pkv = _pkv()
    ctx = [200, 90]
    q, kc, vc, ks, vs, t = attention_case(ctx, q_len, 2)
    for bad in (kc.shape[0], -1, -2 ** 31, 2 ** 31 - 1):
        u = t.copy()
        u[0, 3] = bad
        run_attention(q, kc, vc, ks, vs, u, ctx)
        assert pkv.get_device_error() == pkv.DEVERR_BLOCK_ID
    run_attention(q, kc, vc, ks, vs, t[:, :3].copy(), [200, 40])
    assert pkv.get_device_error() == pkv.DEVERR_CONTEXT


@pytest.mark.parametrize("q_len", [1, 4, 80])
def test_captured_and_two_streams(q_len):
    pkv = _pkv()
    ctxs = [[700, 100], [90, 1300]]
    cases = [attention_case(c, q_len, 2, seed=i) for i, c in enumerate(ctxs)]
    want = [run_attention(*case, c) for case, c in zip(cases, ctxs)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(4):
        got = []
        for case, c, s in zip(cases, ctxs, streams):
            with torch.cuda.stream(s):
                got.append(run_attention(*case, c))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    q, kc, vc, ks, vs, t = cases[0]
    out, lens, table = torch.zeros_like(q), dev(ctxs[0]), dev(t)
    ws = torch.empty(max(pkv.workspace_size_fp8_scaled(2, q_len, 8, t.shape[1]), 1), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.paged_attention_fp8_scaled(out, q, kc, vc, ks, vs, table, lens, q_len, SCALE, workspace=ws)
    for c in ([700, 100], [333, 1], [0, 64]):
        lens.copy_(dev(c))
        graph.replay()
        torch.cuda.synchronize()
        check(out, reference(q, kc, vc, ks, vs, t, c), c)


def test_pools_beyond_32_bits():
    """Blocks whose codes lie past 4 GiB of their pool: appended to, copied and attended."""
    pkv = _pkv()
    hkv, nb = 16, 140000  # 4.6 GB a pool
    kc, vc = (torch.zeros((nb, hkv, BLOCK, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((nb, hkv), device="cuda") for _ in range(2))
    t = np.array([[nb - 1, 7, nb - 2, nb - 3], [nb - 9, nb - 5, 3, -1]], np.int32)
    ctx = [60, 33]
    x = [torch.randn((93, hkv, D), device="cuda").to(torch.bfloat16) for _ in range(2)]
    pkv.kv_append_fp8_scaled(kc, vc, ks, vs, dev(t), dev(ctx), x[0], x[1], dev([0, 60, 93]))
    pkv.copy_blocks_fp8_scaled(kc, vc, ks, vs, dev([nb - 3]), dev([nb - 4]))
    t[0, 3] = nb - 4
    used = sorted({int(b) for b in t.reshape(-1) if b >= 0})
    small = {b: i for i, b in enumerate(used)}
    u = np.vectorize(lambda b: small.get(int(b), -1))(t).astype(np.int32)
    parts = [z[dev(used, torch.int64)] for z in (kc, vc, ks, vs)]
    for q_len in (1, 6, 40):
        q = torch.randn((2, q_len, 4 * hkv, D), device="cuda").to(torch.bfloat16)
        out = run_attention(q, kc, vc, ks, vs, t, ctx)
        check(out, reference(q, *parts, u, ctx), ctx)
    assert pkv.get_device_error() == 0


# ---------------------------------------------------------------------------
# a prompt, then its decode
# ---------------------------------------------------------------------------
def test_prompt_then_decode():
    """The prompts' attention, their store, and decode steps that append and attend, as a serving loop runs them; a
    request that shares its prompt takes its own copy of the last block."""
    pkv = _pkv()
    hkv, hq, lens = 2, 8, [50, 7, 128]
    g = torch.Generator(device="cuda").manual_seed(1)
    steps = 20
    nb = 64
    bp = pkv.BlockPool(nb)
    rows = [bp.alloc(-(-n // BLOCK)) for n in lens]
    width = 16
    kc, vc = (torch.full((nb, hkv, BLOCK, D), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((nb, hkv), math.nan, device="cuda") for _ in range(2))

    def table():
        t = np.full((len(rows), width), -1, np.int32)
        for r, row in enumerate(rows):
            t[r, : len(row)] = row
        return t

    def proj(n):
        x = torch.randn((n, (hq + 2 * hkv) * D), generator=g, device="cuda").to(torch.bfloat16)
        return (x[:, : hq * D].view(n, hq, D), x[:, hq * D:(hq + hkv) * D].view(n, hkv, D),
                x[:, (hq + hkv) * D:].view(n, hkv, D))

    q, k, v = proj(sum(lens))
    cu = dev([0] + np.cumsum(lens).tolist())
    out = torch.empty_like(q)
    pkv.prompt_attention(out, q, k, v, cu, SCALE)
    pkv.kv_append_fp8_scaled(kc, vc, ks, vs, dev(table()), dev(lens), k, v, cu)
    kept = [k[:50], k[50:57], k[57:]], [v[:50], v[50:57], v[57:]]
    # the cache, attended as a chunk, gives the prompts' attention up to the codes' rounding: evenly spread over
    # +-2^-4 relative at most, 0.026 of a value on average, in V and (over 128 products of size 1, times 128^-0.5) in
    # the scores, so about 0.037 of the result's norm
    chunk = run_attention(q[:50].unsqueeze(0).contiguous(), kc, vc, ks, vs, table()[:1], [50])
    assert float((chunk[0].double() - out[:50].double()).norm() / out[:50].double().norm()) < 0.06
    # request 3 starts from request 0's prompt
    bp.share(rows[0])
    rows.append(list(rows[0]))
    ctx = lens + [50]
    for z in kept:
        z.append(z[0])
    for _ in range(steps):
        src, dst = [], []
        for r in range(4):
            for a, b in bp.reserve(rows[r], ctx[r], 1, width):
                src.append(a)
                dst.append(b)
        if src:
            pkv.copy_blocks_fp8_scaled(kc, vc, ks, vs, dev(src), dev(dst))
        q1, k1, v1 = proj(4)
        ctx = [c + 1 for c in ctx]
        pkv.kv_append_fp8_scaled(kc, vc, ks, vs, dev(table()), dev(ctx), k1, v1)
        for r in range(4):
            kept[0][r], kept[1][r] = torch.cat([kept[0][r], k1[r:r + 1]]), torch.cat([kept[1][r], v1[r:r + 1]])
        qq = q1.unsqueeze(1).contiguous()
        got = run_attention(qq, kc, vc, ks, vs, table(), ctx)
        check(got, reference(qq, kc, vc, ks, vs, table(), ctx), ctx)
    assert pkv.get_device_error() == 0
    # what the cache holds is the tokens, to E4M3's rounding of the block's scale
    t = table()
    for r in range(4):
        at = np.arange(ctx[r])
        for codes, scales, x in ((kc, ks, kept[0][r]), (vc, vs, kept[1][r])):
            blk, off = t[r][at // BLOCK], at % BLOCK
            s = scales.double().cpu()[blk][..., None]
            got = values(codes)[blk, :, off] * s
            y = x.double().cpu()
            assert bool(((got - y).abs() <= 2.0 ** -4 * y.abs() + 2.0 ** -9 * s).all())
    bp.close()

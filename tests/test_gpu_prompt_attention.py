"""prompt_attention against the definition in 64 bits: lengths, head groups, strides, padding, captured calls."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

D = 128
SCALE = D ** -0.5


def _pkv():
    import paged_kv_decode_attention_gb300 as pkv
    return pkv


def _inputs(lens, hkv, group, pad=0, seed=0, q_scale=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t, hq = sum(lens) + pad, hkv * group
    qkv = torch.randn((t, (hq + 2 * hkv) * D), generator=g, device="cuda").to(torch.bfloat16)
    q = qkv[:, : hq * D].view(t, hq, D)
    q *= q_scale
    k = qkv[:, hq * D:(hq + hkv) * D].view(t, hkv, D)
    v = qkv[:, (hq + hkv) * D:].view(t, hkv, D)
    cu = torch.tensor([0] + [sum(lens[: i + 1]) for i in range(len(lens))], dtype=torch.int32, device="cuda")
    return q, k, v, cu


def _reference(q, k, v, lens, scale=SCALE):
    """out, lse, and what the tolerances need: sum of w |v| and the largest sum |q||k| scale of each row."""
    hq, hkv = q.shape[1], k.shape[1]
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    mass = torch.zeros_like(out)
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device="cuda")
    size = torch.zeros_like(lse)
    at = 0
    for n in lens:
        if n == 0:
            continue
        qs, ks, vs = (x[at:at + n].double().transpose(0, 1) for x in (q, k, v))
        ks, vs = (x.repeat_interleave(hq // hkv, 0) for x in (ks, vs))
        hidden = torch.ones((n, n), dtype=torch.bool, device="cuda").triu(1)
        x = (qs @ ks.transpose(1, 2) * scale).masked_fill(hidden, -math.inf)
        w = torch.softmax(x, -1)
        out[at:at + n] = (w @ vs).transpose(0, 1)
        mass[at:at + n] = (w @ vs.abs()).transpose(0, 1)
        lse[at:at + n] = torch.logsumexp(x, -1).T
        size[at:at + n] = (qs.abs() @ ks.abs().transpose(1, 2) * scale).masked_fill(hidden, 0).amax(-1).T
        at += n
    return out, lse, mass, size


def _check(out, lse, ref, lens):
    """Scores: FP32 sums of 128 exact products, off by at most 128 * 2^-24 of sum |q||k|; the exponential 2^-22
    relative; the weights' rounding to BF16 2^-8 relative; the result's 2^-8 relative.  FP32 sums over n keys:
    n * 2^-24 relative."""
    want, want_lse, mass, size = ref
    t = sum(lens)
    n = max(lens)
    score = 128 * 2.0 ** -24 * size
    w_err = 2.0 ** -8 + 2.0 ** -21 + 2 * score + n * 2.0 ** -23
    tol = 2.0 ** -8 * want.abs() + w_err[..., None] * mass * 1.01 + 1e-30
    err = (out.double() - want).abs()
    assert bool((err[:t] <= tol[:t]).all()), float((err[:t] / tol[:t]).max())
    # the errors average out: far below the worst case over all values
    assert float(err[:t].norm() / want[:t].norm()) < 5e-3
    if lse is not None:
        tol = score + n * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -21 * want_lse.abs()
        err = (lse.double() - want_lse).abs()[:t]
        assert bool((err <= tol[:t]).all()), float((err / tol[:t]).max())


def _run(lens, hkv, group, pad=0, seed=0, lse=True, q_scale=2.0):
    pkv = _pkv()
    q, k, v, cu = _inputs(lens, hkv, group, pad, seed, q_scale)
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    l = torch.full(q.shape[:2], 7.0, device="cuda") if lse else None
    pkv.prompt_attention(out, q, k, v, cu, SCALE, out_lse=l)
    assert pkv.get_device_error() == 0
    return out, l, (q, k, v, cu)


@pytest.mark.parametrize("lens", [[1], [2, 0, 1], [0, 0, 5, 0], [31, 32, 33], [63, 64, 65, 127, 128, 129, 130], [200],
                                  [255, 256, 257], [1000, 3, 500], [2600], [1, 4001, 17, 640]])
def test_lengths(lens):
    out, lse, (q, k, v, _) = _run(lens, 8, 4)
    _check(out, lse, _reference(q, k, v, lens), lens)


@pytest.mark.parametrize("hkv,group", [(1, 1), (5, 1), (4, 2), (2, 3), (1, 4), (3, 5), (2, 6), (4, 7), (2, 8), (1, 16),
                                       (1, 33), (1, 71), (1, 128)])
def test_groups(hkv, group):
    lens = [37, 1, 300, 129]
    out, lse, (q, k, v, _) = _run(lens, hkv, group, pad=3)
    _check(out, lse, _reference(q, k, v, lens), lens)


@pytest.mark.parametrize("count,most", [(33, 90), (200, 40), (700, 9), (64, 700)])
def test_many_prompts(count, most):
    g = torch.Generator().manual_seed(count)
    lens = torch.randint(0, most + 1, (count,), generator=g).tolist()
    lens[count // 2] = most
    out, lse, (q, k, v, _) = _run(lens, 2, 4, pad=11)
    _check(out, lse, _reference(q, k, v, lens), lens)


def test_rows_of_no_prompt_stay_and_may_hold_anything():
    pkv = _pkv()
    lens = [70, 5, 200]
    q, k, v, cu = _inputs(lens, 2, 4, pad=150)
    want = _reference(q, k, v, lens)
    t = sum(lens)
    for x in (q, k, v):
        x[t:] = math.nan
        x[t + 1::2] = math.inf
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    pkv.prompt_attention(out, q, k, v, cu, SCALE, out_lse=lse)
    _check(out, lse, want, lens)
    assert bool((out[t:] == 7).all()) and bool((lse[t:] == 7).all())


def test_prompts_do_not_see_each_other():
    """A prompt of NaN leaves its neighbours as they are, bit for bit."""
    pkv = _pkv()
    lens = [70, 45, 200]
    q, k, v, cu = _inputs(lens, 2, 4)
    clean = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
    pkv.prompt_attention(clean, q, k, v, cu, SCALE)
    for x in (q, k, v):
        x[70:115] = math.nan
    out = torch.empty_like(clean)
    pkv.prompt_attention(out, q, k, v, cu, SCALE)
    assert torch.equal(out[:70], clean[:70]) and torch.equal(out[115:], clean[115:])
    assert bool(out[70:115].isnan().all())


def test_alone_or_among_others_bit_for_bit():
    pkv = _pkv()
    lens = [300, 900, 17]
    q, k, v, cu = _inputs(lens, 4, 4)
    out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
    pkv.prompt_attention(out, q, k, v, cu, SCALE)
    again = torch.empty_like(out)
    pkv.prompt_attention(again, q, k, v, cu, SCALE)
    assert torch.equal(out, again)
    one = torch.empty((900, 16, D), dtype=torch.bfloat16, device="cuda")
    pkv.prompt_attention(one, q[300:1200], k[300:1200], v[300:1200],
                         torch.tensor([0, 900], dtype=torch.int32, device="cuda"), SCALE)
    assert torch.equal(one, out[300:1200])


def test_rising_scores():
    """Each tile's scores far above the ones before, so that the running maximum moves and O is rescaled."""
    pkv = _pkv()
    lens = [700]
    q, k, v, cu = _inputs(lens, 2, 4)
    base = q[:1, :1].clone()
    q[:] = base
    k[:] = base[:, :1] * torch.linspace(0.02, 1.0, 700, device="cuda").to(torch.bfloat16)[:, None, None]
    out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(q.shape[:2], device="cuda")
    pkv.prompt_attention(out, q, k, v, cu, SCALE, out_lse=lse)
    _check(out, lse, _reference(q, k, v, lens), lens)
    # and falling ones: the first key keeps nearly all the weight
    k.copy_(k.flip(0))
    pkv.prompt_attention(out, q, k, v, cu, SCALE, out_lse=lse)
    _check(out, lse, _reference(q, k, v, lens), lens)


def test_layouts():
    """Separate contiguous tensors, a padded token stride, an output 16 bytes off a 32-byte boundary, no lse."""
    pkv = _pkv()
    lens = [90, 210]
    q, k, v, cu = _inputs(lens, 2, 4)
    want = _reference(q, k, v, lens)
    plain = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
    pkv.prompt_attention(plain, q, k, v, cu, SCALE)
    _check(plain, None, want, lens)
    wide = torch.zeros((300, 2 * D + 8), dtype=torch.bfloat16, device="cuda")
    wide[:, : 2 * D] = k.reshape(300, 2 * D)
    store = torch.empty(q.numel() + 8, dtype=torch.bfloat16, device="cuda")
    out = store[8:].view(q.shape)
    pkv.prompt_attention(out, q.contiguous(), wide[:, : 2 * D].view(300, 2, D), v.contiguous(), cu, SCALE)
    assert torch.equal(out, plain)


def test_captured_with_other_lengths_and_on_another_stream():
    pkv = _pkv()
    q, k, v, cu = _inputs([100, 200, 100], 2, 4)
    out = torch.zeros(q.shape, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(q.shape[:2], device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pkv.prompt_attention(out, q, k, v, cu, SCALE, out_lse=lse)
    torch.cuda.current_stream().wait_stream(side)
    _check(out, lse, _reference(q, k, v, [100, 200, 100]), [100, 200, 100])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.prompt_attention(out, q, k, v, cu, SCALE, out_lse=lse)
    for lens in ([100, 200, 100], [1, 398, 1], [0, 13, 0]):
        cu.copy_(torch.tensor([0, lens[0], lens[0] + lens[1], sum(lens)], dtype=torch.int32))
        q.normal_()
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        _check(out, lse, _reference(q, k, v, lens), lens)
        assert bool((out[sum(lens):] == 7).all())


def test_rows_beyond_32_bits():
    """A prompt whose rows lie past 4 GiB of q and of out, behind rows of none."""
    pkv = _pkv()
    t, n = 560000, 300
    q, k, v, _ = _inputs([n], 8, 4)
    big = [torch.empty((t, x.shape[1], D), dtype=torch.bfloat16, device="cuda") for x in (q, k, v)]
    for b, x in zip(big, (q, k, v)):
        b[t - n - 5:t - 5] = x
    out = torch.empty_like(big[0])
    pkv.prompt_attention(out, *big, torch.tensor([t - n - 5, t - 5], dtype=torch.int32, device="cuda"), SCALE)
    want = torch.empty_like(q.contiguous())
    pkv.prompt_attention(want, q, k, v, torch.tensor([0, n], dtype=torch.int32, device="cuda"), SCALE)
    assert pkv.get_device_error() == 0
    assert torch.equal(out[t - n - 5:t - 5], want)


def test_two_streams_at_once():
    pkv = _pkv()
    lens = [[700, 300], [64, 1100]]
    data = [_inputs(n, 4, 4, seed=i) for i, n in enumerate(lens)]
    outs = [torch.empty(d[0].shape, dtype=torch.bfloat16, device="cuda") for d in data]
    streams = [torch.cuda.Stream() for _ in data]
    torch.cuda.synchronize()
    for _ in range(5):
        for d, o, s in zip(data, outs, streams):
            pkv.prompt_attention(o, *d, SCALE, stream=s)
    torch.cuda.synchronize()
    for d, o, n in zip(data, outs, lens):
        _check(o, None, _reference(*d[:3], n), n)


@pytest.mark.parametrize("cu", [[0, 50, 30, 60], [0, 10, 20, 999], [-5, 10, 20, 30], [40, 30, 20, 10]])
def test_bad_boundaries_are_reported(cu):
    pkv = _pkv()
    q, k, v, _ = _inputs([60], 2, 4)
    out = torch.zeros(q.shape, dtype=torch.bfloat16, device="cuda")
    pkv.prompt_attention(out, q, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"), SCALE)
    assert pkv.get_device_error() == pkv.DEVERR_SEQLENS


def test_partials_join_with_attn_combine():
    """out_lse is what attn_combine takes: a prompt's halves, each over its own keys, joined."""
    pkv = _pkv()
    n, half = 256, 128
    q, k, v, cu = _inputs([n], 2, 4)
    out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(q.shape[:2], device="cuda")
    pkv.prompt_attention(out, q, k, v, cu, SCALE, out_lse=lse)
    # the second half's queries over their own half, and (all of it visible) over the first half
    own = torch.empty((half, 8, D), dtype=torch.bfloat16, device="cuda")
    own_lse = torch.empty((half, 8), device="cuda")
    pkv.prompt_attention(own, q[half:], k[half:], v[half:], torch.tensor([0, half], dtype=torch.int32, device="cuda"),
                         SCALE, out_lse=own_lse)
    ks, vs = (x[:half].double().transpose(0, 1).repeat_interleave(4, 0) for x in (k, v))
    x = q[half:].double().transpose(0, 1) @ ks.transpose(1, 2) * SCALE
    parts = torch.stack([(torch.softmax(x, -1) @ vs).transpose(0, 1).float(), own.float()], 2).contiguous()
    lses = torch.stack([torch.logsumexp(x, -1).T.float(), own_lse], 2).contiguous()
    joined = torch.empty((half * 8, D), dtype=torch.bfloat16, device="cuda")
    pkv.attn_combine(joined, parts.view(half * 8, 2, D), lses.view(half * 8, 2))
    err = (joined.view(half, 8, D).double() - out[half:].double()).norm() / out[half:].double().norm()
    assert float(err) < 6e-3

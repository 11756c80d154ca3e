"""pkv_qk_norm_rope_append against its definition in 64 bits: norms, rotations
of both pairings and of a part of the head, the three pool formats, strided
inputs, padding tokens, and the tokens and positions that it reports."""
import numpy as np
import pytest
import torch

import verify_util as V

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import paged_kv_decode_attention_gb300 as pkv
    FORMATS = {"bf16": pkv.KV_BF16, "q8_0": pkv.KV_Q8_0, "e4m3": pkv.KV_FP8_E4M3}
else:  # collected on CPU-only machines, every test skipped
    pkv = None

EPS = 1e-6


@pytest.fixture(autouse=True)
def _clear_device_error():
    if pkv is not None:
        pkv.get_device_error(reset=True)
    yield
    if pkv is not None:
        assert pkv.get_device_error(reset=True) == 0


def make(tokens, hkv, fmt, rot, seed, fused=True, norm=True, max_pos=5000):
    gen = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    hq = 4 * hkv
    blocks = -(-tokens // 16) + 3
    slots = torch.from_numpy(rng.permutation(blocks * 16)[:tokens].astype(np.int64))
    slots[3::11] = -1
    gain = torch.ones((hq + 2 * hkv) * 128)
    gain[torch.randperm(gain.numel(), generator=gen)[:20]] = 9.0
    qkv = (torch.randn((tokens, (hq + 2 * hkv) * 128 + 24), generator=gen)[:, :(hq + 2 * hkv) * 128 + 24])
    qkv[:, :gain.numel()] *= gain
    qkv = qkv.to(torch.bfloat16).cuda()
    d = {"q": qkv[:, :hq * 128].view(tokens, hq, 128),
         "k": qkv[:, hq * 128:(hq + hkv) * 128].view(tokens, hkv, 128),
         "v": qkv[:, (hq + hkv) * 128:(hq + 2 * hkv) * 128].view(tokens, hkv, 128)}
    if not fused:
        d = {n: t.contiguous() for n, t in d.items()}
    d["qw"] = (1 + 0.3 * torch.randn(128, generator=gen)).to(torch.bfloat16).cuda() if norm else None
    d["kw"] = (1 + 0.3 * torch.randn(128, generator=gen)).to(torch.bfloat16).cuda() if norm else None
    d["pos"] = torch.from_numpy(rng.integers(0, max_pos, tokens).astype(np.int32)).cuda()
    d["table"] = None
    if rot:
        ang = np.arange(max_pos, dtype=np.float64)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
        d["table"] = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)).cuda()
    d["slots"] = slots.cuda()
    shape = {"bf16": (blocks, hkv, 16, 128), "q8_0": (blocks, hkv, 2176), "e4m3": (blocks, hkv, 16, 128)}[fmt]
    if fmt == "bf16":
        pools = [V.randn_bf16(gen, *shape).cuda() for _ in range(2)]
    else:
        pools = [torch.randint(0, 120, shape, generator=gen, dtype=torch.uint8).cuda() for _ in range(2)]
    return d, pools


def call(d, pools, fmt, interleaved=False, q_out=None):
    q_out = torch.full(d["q"].shape, float("nan"), dtype=torch.bfloat16, device="cuda") if q_out is None else q_out
    pkv.qk_norm_rope_append(q_out, pools[0], pools[1], d["slots"], d["q"], d["k"], d["v"], d["pos"], d["table"],
                            d["qw"], d["kw"], EPS, interleaved, FORMATS[fmt])
    torch.cuda.synchronize()
    return q_out


def definition(x, w, pos, table, interleaved):
    """(z, sum of the magnitudes added into z) in 64 bits."""
    x = x.double()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.double()
    mag = x.abs()
    if table is not None:
        rot = table.shape[1]
        cos, sin = (t[:, None] for t in table[pos.long()].double().split(rot // 2, 1))
        a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
        z = x.clone()
        z[..., a] = x[..., a] * cos - x[..., b] * sin
        z[..., b] = x[..., b] * cos + x[..., a] * sin
        m = mag.clone()
        m[..., a] = mag[..., a] * cos.abs() + mag[..., b] * sin.abs()
        m[..., b] = mag[..., b] * cos.abs() + mag[..., a] * sin.abs()
        x, mag = z, m
    return x, mag


# FP32 steps before the rounding: 128 squares summed (128 * 2^-24 relative at most, halved by the root), the root's
# approximation and four products and sums: less than 2^-16 of the magnitudes.
FP32 = 2.0 ** -16


def rows_of(pool, slots):
    """Rows [T][Hkv][...] of a [block][Hkv][16][...] pool at slots."""
    return pool[slots // 16, :, slots % 16]


def dequantised(pool):
    codes = pool[..., :2048].view(torch.int8).unflatten(2, (16, 128)).double()
    scales = pool[..., 2048:].contiguous().view(torch.float16).unflatten(2, (16, 4)).double()
    return codes * scales.repeat_interleave(32, -1), scales


def check(d, pools, fmt, interleaved=False, q_out=None):
    q0 = {n: d[n].clone() for n in ("q", "k", "v")}
    before = [p.clone() for p in pools]
    q_out = call(d, pools, fmt, interleaved, q_out)
    z, mag = definition(q0["q"], d["qw"], d["pos"], d["table"], interleaved)
    V.assert_within(q_out, z, 2.0 ** -8 * z.abs() + FP32 * mag, "queries")
    stored = d["slots"] >= 0
    slots = d["slots"][stored]
    z, mag = definition(q0["k"], d["kw"], d["pos"], d["table"], interleaved)
    z, mag = z[stored], mag[stored]
    if fmt == "bf16":
        V.assert_within(rows_of(pools[0], slots), z, 2.0 ** -8 * z.abs() + FP32 * mag, "keys")
    elif fmt == "e4m3":
        z = z.clamp(-448, 448)
        got = rows_of(pools[0].view(torch.float8_e4m3fn).float(), slots)
        V.assert_within(got, z, 2.0 ** -4 * z.abs() + 2.0 ** -10 + FP32 * mag, "keys")
    else:
        # half a code step, 127 codes of a scale rounded to FP16 (2^-11), and the FP32 steps
        step = z.abs().unflatten(-1, (4, 32)).amax(-1, keepdim=True).expand(-1, -1, -1, 32).flatten(-2) / 127
        magg = mag.unflatten(-1, (4, 32)).amax(-1, keepdim=True).expand(-1, -1, -1, 32).flatten(-2)
        got = rows_of(dequantised(pools[0])[0], slots)
        V.assert_within(got, z, step * (0.5 + 127 * 2.0 ** -11) * (1 + 2.0 ** -10) + 2 * FP32 * magg, "keys")
    # V as the append stores it; everything else as it was
    after_append = [before[0].clone(), before[1].clone()]
    append = {"bf16": pkv.kv_append, "q8_0": pkv.kv_append_q8_0, "e4m3": pkv.kv_append_fp8_e4m3}[fmt]
    append(after_append[0], after_append[1], d["slots"], q0["k"].contiguous(), q0["v"].contiguous())
    as_int = torch.int16 if fmt == "bf16" else torch.uint8
    assert torch.equal(pools[1].view(as_int), after_append[1].view(as_int)), "values differ from the append's"
    changed = pools[0].view(as_int) != before[0].view(as_int)
    would = torch.ones(before[0].shape[0] * 16, dtype=torch.bool, device="cuda")
    would[slots] = False
    would = would.view(-1, 16)
    if fmt == "q8_0":
        codes, scales = changed[..., :2048].unflatten(2, (16, 128)), changed[..., 2048:].unflatten(2, (16, 8))
        assert not (codes & would[:, None, :, None]).any() and not (scales & would[:, None, :, None]).any()
    else:
        assert not (changed & would[:, None, :, None]).any(), "a slot outside the mapping changed"
    return after_append


@pytest.mark.parametrize("fmt", ["bf16", "q8_0", "e4m3"])
@pytest.mark.parametrize("tokens", [1, 2, 7, 37, 300])
@pytest.mark.parametrize("hkv", [1, 3, 8])
def test_sizes_and_formats(fmt, tokens, hkv):
    d, pools = make(tokens, hkv, fmt, 128, seed=tokens + hkv)
    check(d, pools, fmt)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [0, 16, 32, 64, 80, 96, 112, 128])
@pytest.mark.parametrize("norm", [False, True])
def test_rotations(interleaved, rot, norm):
    d, pools = make(53, 2, "bf16", rot, seed=rot, norm=norm)
    check(d, pools, "bf16", interleaved)


@pytest.mark.parametrize("fmt", ["bf16", "q8_0", "e4m3"])
def test_without_norm_and_rotation_it_is_the_append(fmt):
    d, pools = make(100, 4, fmt, 0, seed=2, norm=False)
    q = d["q"].clone()
    plain = check(d, pools, fmt)
    as_int = torch.int16 if fmt == "bf16" else torch.uint8
    assert torch.equal(pools[0].view(as_int), plain[0].view(as_int)) and torch.equal(call(d, pools, fmt), q)


def test_one_norm_only_and_contiguous_inputs():
    d, pools = make(40, 2, "bf16", 128, seed=4, fused=False)
    d["kw"] = None
    check(d, pools, "bf16")


def test_queries_in_place():
    d, pools = make(40, 2, "bf16", 64, seed=5, fused=False)
    check(d, pools, "bf16", q_out=d["q"])


def test_large_and_zero_heads():
    """A zero head stays zero (eps keeps the root finite); heads of 2^60 and 2^-60 are normed all the same as long
    as their squares are FP32 values."""
    d, pools = make(8, 1, "bf16", 128, seed=6, fused=False)
    d["q"][0] = 0
    d["k"][0] = 0
    d["q"][1] *= 2.0 ** 55
    check(d, pools, "bf16")


def test_saturating_keys_in_e4m3():
    d, pools = make(16, 2, "e4m3", 32, seed=7, norm=False)
    d["k"].mul_(300)
    check(d, pools, "e4m3")


def test_many_tokens():
    d, pools = make(4099, 8, "bf16", 128, seed=8)
    check(d, pools, "bf16", True)


@pytest.mark.parametrize("fmt", ["bf16", "q8_0", "e4m3"])
def test_slots_and_positions_out_of_range_are_reported(fmt):
    d, pools = make(30, 2, fmt, 64, seed=9)
    d["slots"][3], d["slots"][4] = pools[0].shape[0] * 16, 2 ** 40
    before = [p.clone() for p in pools]
    keep = d["slots"].clone()
    call(d, pools, fmt)
    assert pkv.get_device_error(reset=True) == pkv.DEVERR_SLOT
    d["slots"] = keep.clone()
    d["slots"][3] = d["slots"][4] = -1
    other = [p.clone() for p in before]
    call(d, other, fmt)
    as_int = torch.int16 if fmt == "bf16" else torch.uint8
    assert all(torch.equal(a.view(as_int), b.view(as_int)) for a, b in zip(pools, other))
    for bad, nearest in ((-1, 0), (5000, 4999), (-2 ** 31, 0), (2 ** 31 - 1, 4999)):
        d["pos"][2] = bad
        got = call(d, other, fmt)
        assert pkv.get_device_error(reset=True) == pkv.DEVERR_POSITION
        d["pos"][2] = nearest
        assert torch.equal(got, call(d, other, fmt))


def test_captured_and_on_another_stream():
    d, pools = make(64, 8, "bf16", 128, seed=10)
    base = [p.clone() for p in pools]
    want = call(d, pools, "bf16")
    other = [p.clone() for p in base]
    out = torch.empty_like(want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    pkv.qk_norm_rope_append(out, other[0], other[1], d["slots"], d["q"], d["k"], d["v"], d["pos"], d["table"],
                            d["qw"], d["kw"], EPS, False, pkv.KV_BF16, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(other[0], pools[0]) and torch.equal(other[1], pools[1])
    g = torch.cuda.CUDAGraph()
    out.zero_()
    with torch.cuda.graph(g):
        pkv.qk_norm_rope_append(out, other[0], other[1], d["slots"], d["q"], d["k"], d["v"], d["pos"], d["table"],
                                d["qw"], d["kw"], EPS)
    d["q"].mul_(-1)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, -want)

"""Cases of the prompt attention and of the 8-bit KV cache with block scales.

Three operators, as a serving loop runs them on each layer:

  prompt  causal attention of whole prompts of different lengths, packed one
          behind the other, with grouped heads (pkv.prompt_attention).
  append  the new tokens' K and V into a paged cache of E4M3 codes with one
          scale for each block of 16 tokens and KV head; a scale that grows
          takes the block's earlier tokens along (pkv.kv_append_fp8_scaled).
  paged   attention over that cache, single tokens and causal chunks
          (pkv.paged_attention_fp8_scaled).

`run` computes a case with elementary torch operations, or, where `own` is
true, with the library's entry points.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 16
DIM = 128
GROUP = 4  # query heads per KV head over the cache
SCALE = 1.0 / math.sqrt(DIM)
TOP = 448.0  # the largest E4M3 value
LOWEST = -32  # the scales' smallest exponent
HIGHEST = 32


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one short question: latency counts
        dict(name="prompt_1x200", op="prompt", seqs=1, shortest=200, longest=200, kv_heads=8, group=4, pad=0, shape=1),
        # 64 questions of a few dozen to a few hundred tokens, padded to a fixed buffer
        dict(name="prompt_64_short", op="prompt", seqs=64, shortest=16, longest=500, kv_heads=8, group=4, pad=37,
             shape=2),
        # 24 prompts whose lengths span two orders, seven query heads to a KV head
        dict(name="prompt_24_uneven_gqa7", op="prompt", seqs=24, shortest=40, longest=4000, kv_heads=4, group=7, pad=5,
             shape=3),
        # two long documents
        dict(name="prompt_2x16000", op="prompt", seqs=2, shortest=16000, longest=16000, kv_heads=8, group=4, pad=0,
             shape=4),
        # a decode step of 37 chats: latency counts
        dict(name="append_decode_37", op="append", seqs=37, shortest=1, longest=1, kv_heads=8, first=2048, spread=256,
             shape=5),
        # prefill chunks of 24 requests that start inside a block
        dict(name="append_24_chunks", op="append", seqs=24, shortest=5, longest=700, kv_heads=8, first=1, spread=3000,
             shape=6),
        # 4 prompts of about 8192 tokens
        dict(name="append_prefill_4x8192", op="append", seqs=4, shortest=8100, longest=8192, kv_heads=8, first=0,
             spread=1, shape=7),
        # one decode token of one long request: latency counts
        dict(name="paged_decode_1", op="paged", seqs=1, q_len=1, kv_heads=8, first=8300, spread=1, shape=8),
        # a decode step of 64 requests of very different lengths
        dict(name="paged_decode_64_uneven", op="paged", seqs=64, q_len=1, kv_heads=8, first=16, spread=16000, shape=9),
        # a decode step of 128 requests with long contexts
        dict(name="paged_decode_128_long", op="paged", seqs=128, q_len=1, kv_heads=8, first=8192, spread=256, shape=10),
        # a chain of 7 drafted tokens of each of 37 chats
        dict(name="paged_verify_37x7", op="paged", seqs=37, q_len=7, kv_heads=8, first=2048, spread=256, shape=11),
        # prefill chunks of 2000 tokens behind cached ones: the products, not the bytes, bound it
        dict(name="paged_chunk_4x2000", op="paged", seqs=4, q_len=2000, kv_heads=8, first=4000, spread=4000, shape=12),
    ]


def _logu(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        cost = most.setdefault(c["op"], {"bytes": 0, "flops": 0})
        for k in cost:
            cost[k] = max(cost[k], w[k])
    op = rng.choice(["prompt", "append", "paged", "paged"])
    while True:
        heads = rng.choice([1, 2, 4, 8, 8, 8, 16])
        shape = rng.randrange(1 << 30)
        if op == "prompt":
            lengths = sorted((_logu(rng, 1, 16000), _logu(rng, 1, 16000)))
            c = dict(op=op, seqs=_logu(rng, 1, 64), shortest=lengths[0], longest=lengths[1], kv_heads=heads,
                     group=rng.choice([1, 2, 3, 4, 4, 4, 5, 7, 8]), pad=rng.choice([0, rng.randrange(1, 100)]),
                     shape=shape)
        elif op == "append":
            lengths = sorted((_logu(rng, 1, 8192), _logu(rng, 1, 8192)))
            if rng.random() < 0.3:
                lengths = [1, 1]
            c = dict(op=op, seqs=_logu(rng, 1, 128), shortest=lengths[0], longest=lengths[1], kv_heads=heads,
                     first=_logu(rng, 1, 8000) - 1, spread=_logu(rng, 1, 4000), shape=shape)
        else:
            c = dict(op=op, seqs=_logu(rng, 1, 128), q_len=rng.choice([1, 1, _logu(rng, 1, 16), _logu(rng, 1, 2048)]),
                     kv_heads=heads, first=_logu(rng, 1, 16000), spread=_logu(rng, 1, 16000), shape=shape)
        w = work(c)
        if w["bytes"] <= most[op]["bytes"] and w["flops"] <= most[op]["flops"]:
            return c


def _uneven(g, lo, hi, n):
    """n lengths of [lo, hi], uniform in the logarithm, the longest among them."""
    out = np.floor(np.exp(g.uniform(math.log(lo), math.log(hi + 0.99), size=n))).astype(np.int64).clip(lo, hi)
    out[int(g.integers(n))] = hi
    return out


def _lengths(case):
    """What a scheduler knows on the host: per request, the tokens cached before this step and the new ones."""
    g = np.random.default_rng(case["shape"])
    n = case["seqs"]
    if case["op"] == "prompt":
        return np.zeros(n, np.int64), _uneven(g, case["shortest"], case["longest"], n)
    if case["spread"] > 4096:  # lengths over several orders
        before = _uneven(g, max(1, case["first"]), case["first"] + case["spread"], n)
    else:
        before = case["first"] + g.integers(0, case["spread"], size=n)
    if case["op"] == "append":
        return before, _uneven(g, case["shortest"], case["longest"], n)
    return before, np.full(n, case["q_len"])


def _pairs(before, new):
    """Keys that the causal queries see, summed."""
    return int((before * new + new * (new + 1) // 2).sum())


def work(case):
    before, new = _lengths(case)
    hkv, tokens = case["kv_heads"], int(new.sum())
    if case["op"] == "prompt":
        hq = hkv * case["group"]
        return {"bytes": tokens * (2 * hq + 2 * hkv) * DIM * 2 + 4 * (len(new) + 1), "flops": 4 * DIM * hq * _pairs(before, new)}
    if case["op"] == "append":
        blocks = int((-(-(before + new) // BLOCK) - before // BLOCK).sum())
        return {"bytes": tokens * 2 * hkv * DIM * 3 + blocks * (2 * hkv * 4 + 4) + 8 * len(new),
                "flops": tokens * 2 * hkv * DIM * 2}
    hq = hkv * GROUP
    keys, blocks = int((before + new).sum()), int((-(-(before + new) // BLOCK)).sum())
    return {"bytes": keys * hkv * DIM * 2 + blocks * (2 * hkv * 4 + 4) + 2 * tokens * hq * DIM * 2,
            "flops": 4 * DIM * hq * _pairs(before, new)}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _tables(counts, total, seed):
    """Block tables of a pool that is handed out in a shuffled order; -1 past a request's blocks."""
    perm = np.random.default_rng(seed).permutation(total)
    table = np.full((len(counts), max(counts) + 1), -1, dtype=np.int32)
    at = 0
    for r, n in enumerate(counts):
        table[r, :n] = perm[at:at + n]
        at += n
    return table


def _exponent(amax):
    """The smallest e of [LOWEST, HIGHEST] with amax <= 448 * 2^e (the highest where there is none)."""
    m, x = torch.frexp(amax)  # amax = m * 2^x, 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, x - 9, x - 8)
    return torch.where(amax > 0, e, torch.full_like(e, LOWEST)).clamp(LOWEST, HIGHEST)


def _power(e):
    """2^e in FP32 for whole numbers e."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _pool(gen, blocks, hkv):
    """A pool as appends leave it: every block's largest value fills its scale's last binade."""
    codes = torch.empty((blocks, hkv, BLOCK, DIM), dtype=torch.uint8, device="cuda")
    scales = torch.empty((blocks, hkv), dtype=torch.float32, device="cuda")
    for at in range(0, blocks, 8192):
        x = torch.empty((min(8192, blocks - at), hkv, BLOCK, DIM), device="cuda").normal_(generator=gen)
        size = torch.empty((x.shape[0], hkv, 1, 1), device="cuda").normal_(generator=gen)
        x *= torch.exp2(1.5 * size)  # blocks of unlike size
        s = _power(_exponent(x.abs().amax((2, 3))))
        codes[at:at + 8192] = (x / s[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        scales[at:at + 8192] = s
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def dev(a, dtype):
        return torch.from_numpy(np.ascontiguousarray(a)).to(device="cuda", dtype=dtype)

    before, new = _lengths(case)
    ctx = before + new
    seqs, hkv = case["seqs"], case["kv_heads"]
    s = {"case": case, "before": [int(x) for x in before], "new": [int(x) for x in new],
         "ctx": [int(x) for x in ctx], "starts": [0] + [int(x) for x in np.cumsum(new)]}
    if case["op"] in ("prompt", "append"):
        # the projection's output: some channels much larger than the others
        hq = hkv * case["group"] if case["op"] == "prompt" else 0
        tokens = s["starts"][-1] + case.get("pad", 0)
        qkv = torch.empty((tokens, (hq + 2 * hkv) * DIM), device="cuda", dtype=torch.bfloat16).normal_(generator=gen)
        gain = torch.ones(qkv.shape[1], device="cuda")
        gain[torch.randperm(gain.numel(), generator=gen, device="cuda")[: gain.numel() // 64]] = 4.0
        gain[: hq * DIM] *= 2.0  # some keys get much of the weight
        qkv *= gain
        s["q"] = qkv[:, : hq * DIM].unflatten(1, (hq, DIM)) if hq else None
        s["k"] = qkv[:, hq * DIM:(hq + hkv) * DIM].unflatten(1, (hkv, DIM))
        s["v"] = qkv[:, (hq + hkv) * DIM:].unflatten(1, (hkv, DIM))
        s["cu"] = dev(np.asarray(s["starts"]), torch.int32)
    if case["op"] == "prompt":
        s["out"] = torch.zeros((tokens, hq, DIM), device="cuda", dtype=torch.bfloat16)
        s["lse"] = torch.zeros((tokens, hq), device="cuda")
    else:
        counts = [-(-int(c) // BLOCK) for c in ctx]
        total = sum(counts) + 8
        table = _tables(counts, total, seed)
        s["tables"], s["lens"] = dev(table, torch.int32), dev(ctx, torch.int32)
        s["k_cache"], s["k_scales"] = _pool(gen, total, hkv)
        s["v_cache"], s["v_scales"] = _pool(gen, total, hkv)
    if case["op"] == "append":
        pos = np.concatenate([np.arange(b, c) for b, c in zip(before, ctx)])
        row = np.repeat(np.arange(seqs), new)
        s["blk"] = dev(table[row, pos // BLOCK], torch.int64)
        s["off"] = dev(pos % BLOCK, torch.int64)
        started = np.flatnonzero(before % BLOCK)  # requests whose first new token joins earlier ones
        s["started"] = dev(table[started, before[started] // BLOCK], torch.int64)
        s["held"] = dev(before[started] % BLOCK, torch.int64)
        s["fresh"] = dev(np.setdiff1d(table[row, pos // BLOCK], table[started, before[started] // BLOCK]), torch.int64)
    elif case["op"] == "paged":
        hq = hkv * GROUP
        q = torch.empty((seqs, case["q_len"], hq, DIM), device="cuda").normal_(generator=gen)
        s["q"] = (2.0 * q).to(torch.bfloat16)  # some keys get much of the weight
        s["out"] = torch.empty_like(s["q"])
    if own:
        import paged_kv_decode_attention_gb300 as pkv
        s["pkv"] = pkv
        if case["op"] == "paged":
            size = pkv.workspace_size_fp8_scaled(seqs, case["q_len"], hq, table.shape[1])
            s["workspace"] = torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(s):
    if own:
        return _run_own(s)
    return {"prompt": _plain_prompt, "append": _plain_append, "paged": _plain_paged}[s["case"]["op"]](s)


def _run_own(s):
    pkv, case = s["pkv"], s["case"]
    if case["op"] == "prompt":
        pkv.prompt_attention(s["out"], s["q"], s["k"], s["v"], s["cu"], SCALE, out_lse=s["lse"])
        return s["out"], s["lse"]
    if case["op"] == "append":
        pkv.kv_append_fp8_scaled(s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["tables"], s["lens"],
                                 s["k"], s["v"], s["cu"])
        return _append_outputs(s)
    pkv.paged_attention_fp8_scaled(s["out"], s["q"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"],
                                   s["tables"], s["lens"], case["q_len"], SCALE, workspace=s["workspace"])
    return s["out"]


def _append_outputs(s):
    return (s["k_cache"].view(torch.float8_e4m3fn), s["v_cache"].view(torch.float8_e4m3fn), s["k_scales"],
            s["v_scales"])


def _causal(q, k, v, first):
    """q [H][n][G][128], k and v [H][keys][128], all FP32; query i sees the keys 0 .. first + i.
    Returns the outputs [H][n][G][128] and the scores' log-sum-exp [H][n][G]."""
    h, n, g, _ = q.shape
    keys = k.shape[1]
    out, lse = torch.empty_like(q), torch.empty((h, n, g), device=q.device)
    step = max(1, (1 << 29) // (h * g * keys))  # bounds the scores held at once
    for i in range(0, n, step):
        j = min(n, i + step)
        end = min(keys, first + j)
        x = torch.matmul(q[:, i:j].reshape(h, -1, DIM), k[:, :end].transpose(1, 2)).view(h, j - i, g, end) * SCALE
        hidden = torch.arange(end, device=q.device) > torch.arange(first + i, first + j, device=q.device)[:, None]
        x = x.masked_fill(hidden[:, None], -math.inf)
        top = x.amax(-1, keepdim=True)
        e = torch.exp(x - top)
        total = e.sum(-1, keepdim=True)
        out[:, i:j] = (torch.matmul(e.view(h, -1, end), v[:, :end]).view(h, j - i, g, DIM)) / total
        lse[:, i:j] = (top + torch.log(total))[..., 0]
    return out, lse


def _plain_prompt(s):
    hkv, group = s["case"]["kv_heads"], s["case"]["group"]
    for a, b in zip(s["starts"], s["starts"][1:]):
        q = s["q"][a:b].float().view(b - a, hkv, group, DIM).transpose(0, 1)
        k, v = s["k"][a:b].float().transpose(0, 1), s["v"][a:b].float().transpose(0, 1)
        out, lse = _causal(q.contiguous(), k.contiguous(), v.contiguous(), 0)
        s["out"][a:b] = out.transpose(0, 1).reshape(b - a, hkv * group, DIM).to(torch.bfloat16)
        s["lse"][a:b] = lse.transpose(0, 1).reshape(b - a, hkv * group)
    return s["out"], s["lse"]


def _plain_append(s):
    hkv = s["case"]["kv_heads"]
    inside = torch.arange(BLOCK, device="cuda")[None, :] < s["held"][:, None]  # the earlier tokens
    for cache, scales, x in ((s["k_cache"], s["k_scales"], s["k"]), (s["v_cache"], s["v_scales"], s["v"])):
        x = x.float()
        amax = torch.zeros((cache.shape[0], hkv), device="cuda")
        amax.scatter_reduce_(0, s["blk"][:, None].expand(-1, hkv), x.abs().amax(-1), "amax")
        need = _power(_exponent(amax))
        old = scales[s["started"]]
        grown = torch.maximum(old, need[s["started"]])
        held = cache[s["started"]].view(torch.float8_e4m3fn).float()
        again = (held * (old / grown)[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        cache[s["started"]] = torch.where(inside[:, None, :, None], again, cache[s["started"]])
        scales[s["fresh"]] = need[s["fresh"]]
        scales[s["started"]] = grown
        y = (x / scales[s["blk"]][..., None]).clamp(-TOP, TOP).to(torch.float8_e4m3fn).view(torch.uint8)
        cache[s["blk"], :, s["off"]] = y
    return _append_outputs(s)


def _plain_paged(s):
    case, hkv = s["case"], s["case"]["kv_heads"]
    n = case["q_len"]
    for r, ctx in enumerate(s["ctx"]):
        blk = s["tables"][r, : -(-ctx // BLOCK)].long()
        k, v = ((c[blk].view(torch.float8_e4m3fn).float() * x[blk][..., None, None]).transpose(0, 1).flatten(1, 2)[:, :ctx]
                for c, x in ((s["k_cache"], s["k_scales"]), (s["v_cache"], s["v_scales"])))
        q = s["q"][r].float().view(n, hkv, GROUP, DIM).transpose(0, 1).contiguous()
        out, _ = _causal(q, k, v, ctx - n)
        s["out"][r] = out.transpose(0, 1).reshape(n, hkv * GROUP, DIM).to(torch.bfloat16)
    return s["out"]


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    before, new = _lengths(case)
    if case["op"] != "append" and 8 * DIM * case["kv_heads"] * case.get("group", GROUP) * _pairs(before, new) > 1.2e13:
        return None  # too long in 64 bits
    s = prepare(case, seed)
    return {"prompt": _exact_prompt, "append": _exact_append, "paged": _exact_paged}[case["op"]](s)


def _exact_rows(q, k, v, first):
    """q [n][Hq][128], k and v [keys][Hkv][128]: row i's softmax over the keys 0 .. first + i, head by head."""
    n, hq, _ = q.shape
    hkv = k.shape[1]
    out = torch.empty(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.empty((n, hq), dtype=torch.float64, device="cuda")
    at = torch.arange(k.shape[0], device="cuda")
    for h in range(hq):
        kh, vh = k[:, h // (hq // hkv)].double(), v[:, h // (hq // hkv)].double()
        for i in range(0, n, 2048):
            rows = torch.arange(i, min(n, i + 2048), device="cuda")
            top = int(first + rows[-1]) + 1
            x = q[rows, h].double() @ kh[:top].T / math.sqrt(DIM)
            x[at[None, :top] > first + rows[:, None]] = -math.inf
            norm = torch.logsumexp(x, 1)
            out[rows, h] = torch.exp(x - norm[:, None]) @ vh[:top]
            lse[rows, h] = norm
    return out, lse


def _exact_prompt(s):
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    for a, n in zip(s["starts"], s["new"]):
        out[a:a + n], lse[a:a + n] = _exact_rows(s["q"][a:a + n], s["k"][a:a + n], s["v"][a:a + n], 0)
    return out, lse


def _round_e4m3(x):
    """To the nearest value with 4 significant bits and no bit below 2^-9, ties to even, at most 448 (64 bits)."""
    power = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -40))).clamp(min=-6.0)
    step = torch.exp2(power - 3.0)
    return (torch.round(x / step) * step).clamp(-TOP, TOP)


def _exact_append(s):
    """Request by request and block by block, on the host."""
    tables = s["tables"].cpu()
    values, sizes = [], []
    for cache, scales, x in ((s["k_cache"], s["k_scales"], s["k"]), (s["v_cache"], s["v_scales"], s["v"])):
        codes = cache.view(torch.float8_e4m3fn).float().cpu().double()
        scales, x = scales.double().cpu(), x.float().cpu().double()
        for r, (b, c) in enumerate(zip(s["before"], s["ctx"])):
            for lb in range(b // BLOCK, -(-c // BLOCK)):
                p0, p1 = max(b, lb * BLOCK), min(c, (lb + 1) * BLOCK)
                rows = x[s["starts"][r] + p0 - b:s["starts"][r] + p1 - b]  # [n][Hkv][128]
                blk, off = int(tables[r, lb]), p0 - lb * BLOCK
                amax = rows.abs().amax((0, 2))
                e = torch.ceil(torch.log2((amax / TOP).clamp(min=2.0 ** LOWEST))).clamp(max=HIGHEST)
                size = torch.exp2(e)
                if off > 0:
                    size = torch.maximum(size, scales[blk])
                    codes[blk, :, :off] = _round_e4m3(codes[blk, :, :off] * (scales[blk] / size)[:, None, None])
                scales[blk] = size
                codes[blk, :, off:off + p1 - p0] = _round_e4m3(rows / size[:, None]).transpose(0, 1)
        values.append(codes.cuda())
        sizes.append(scales.cuda())
    return (*values, *sizes)


def _exact_paged(s):
    n = s["case"]["q_len"]
    out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
    for r, ctx in enumerate(s["ctx"]):
        at = torch.arange(ctx, device="cuda")
        blk, off = s["tables"][r].long()[at // BLOCK], at % BLOCK
        k, v = (c.view(torch.float8_e4m3fn)[blk, :, off].double() * x[blk].double()[..., None]
                for c, x in ((s["k_cache"], s["k_scales"]), (s["v_cache"], s["v_scales"])))
        out[r], _ = _exact_rows(s["q"][r], k, v, ctx - n)
    return out

"""Cases of the verification-step and sliding-window operators of the paged KV cache.

Four operators, as a serving loop runs them on each layer of a model with 4
query heads per KV head, 128 dims and 16-token blocks:

  norm_rope  RMS norms of the new tokens' query and key heads, the position
             rotation, and the store of K and V into the paged cache, in one
             pass (pkv.qk_norm_rope_append).
  tree       attention of a tree of drafted tokens over the cache
             (pkv.paged_attention_tree).
  window     attention with a sliding window whose first tokens stay visible
             (pkv.paged_attention_window).
  compact    after verification, the accepted path's K and V rows move to the
             places behind the committed context, in every layer
             (pkv.kv_compact).

`run` computes a case with elementary torch operations, or, where `own` is
true, with the library's entry points.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 16
DIM = 128
GROUP = 4
SCALE = 1.0 / math.sqrt(DIM)
EPS = 1e-6
THETA = 1.0e6
LAYERS = 36
TILE_BYTES = {"bf16": 4096, "q8_0": 2176, "e4m3": 2048}  # one (block, KV head) of K or of V


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one decode step of 37 chats with 2048 input tokens: latency counts
        dict(name="norm_rope_decode_37", op="norm_rope", seqs=37, per_seq=1, kv_heads=8, fmt="bf16", first=2048,
             spread=256, rot=128, interleaved=False, norm=True, shape=1),
        # verifying 25 drafted tokens of each of the 37 chats over an 8-bit cache
        dict(name="norm_rope_verify_37x25_e4m3", op="norm_rope", seqs=37, per_seq=25, kv_heads=8, fmt="e4m3",
             first=2048, spread=256, rot=128, interleaved=False, norm=True, shape=2),
        # a prefill chunk: 4 prompts of 8192 tokens, rotated in neighbouring pairs
        dict(name="norm_rope_prefill_4x8192", op="norm_rope", seqs=4, per_seq=8192, kv_heads=8, fmt="bf16", first=0,
             spread=1, rot=128, interleaved=True, norm=True, shape=3),
        # one chat, 26 drafted nodes, a short context: latency counts
        dict(name="tree_1x26_short", op="tree", seqs=1, nodes=26, kv_heads=8, first=600, spread=1, shape=4),
        # 37 chats of 2048 input tokens, up to 16 drafted nodes each
        dict(name="tree_37x16_chat", op="tree", seqs=37, nodes=16, kv_heads=8, first=2048, spread=256, shape=5),
        # 16 long requests, up to 61 drafted nodes each
        dict(name="tree_16x61_long", op="tree", seqs=16, nodes=61, kv_heads=8, first=8192, spread=256, shape=6),
        # one decode token of one long request: latency counts
        dict(name="window_decode_1", op="window", seqs=1, q_len=1, window=1024, sinks=4, kv_heads=8, first=8300,
             spread=1, shape=7),
        # a decode step of 64 requests of very different lengths
        dict(name="window_decode_64", op="window", seqs=64, q_len=1, window=2000, sinks=4, kv_heads=8, first=16,
             spread=32000, shape=8),
        # 128 streams that feed 16 tokens at a time
        dict(name="window_chunk_128x16", op="window", seqs=128, q_len=16, window=4096, sinks=64, kv_heads=8,
             first=1024, spread=31744, shape=9),
        # prefill chunks of 2000 tokens: the products, not the bytes, bound it
        dict(name="window_prefill_4x2000", op="window", seqs=4, q_len=2000, window=4096, sinks=4, kv_heads=8,
             first=6000, spread=6000, shape=10),
        # one chat's accepted path in 36 layers: latency counts
        dict(name="compact_1", op="compact", seqs=1, nodes=26, accept=5, kv_heads=8, fmt="bf16", layers=LAYERS,
             first=2048, spread=256, shape=11),
        # 128 chats' accepted paths in 36 layers of an 8-bit cache with scales
        dict(name="compact_128_q8_0", op="compact", seqs=128, nodes=61, accept=8, kv_heads=8, fmt="q8_0",
             layers=LAYERS, first=2048, spread=256, shape=12),
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
    op = rng.choice(["norm_rope", "tree", "window", "compact"])
    while True:
        heads = rng.choice([1, 2, 4, 8, 8, 8, 16])
        shape = rng.randrange(1 << 30)
        if op == "norm_rope":
            c = dict(op=op, seqs=_logu(rng, 1, 64), per_seq=_logu(rng, 1, 8192), kv_heads=heads,
                     fmt=rng.choice(["bf16", "bf16", "e4m3"]), first=_logu(rng, 1, 24000), spread=_logu(rng, 1, 4000),
                     rot=rng.choice([128, 128, 96, 64, 32]), interleaved=rng.random() < 0.3, norm=rng.random() < 0.8,
                     shape=shape)
        elif op == "tree":
            c = dict(op=op, seqs=_logu(rng, 1, 64), nodes=_logu(rng, 1, 128), kv_heads=heads,
                     first=_logu(rng, 128, 12000), spread=_logu(rng, 1, 4000), shape=shape)
        elif op == "window":
            c = dict(op=op, seqs=_logu(rng, 1, 128), q_len=rng.choice([1, _logu(rng, 1, 2048)]),
                     window=_logu(rng, 16, 4096), sinks=rng.choice([0, 1, 4, rng.randrange(65)]), kv_heads=heads,
                     first=_logu(rng, 1, 16000), spread=_logu(rng, 1, 16000), shape=shape)
        else:
            nodes = _logu(rng, 2, 128)
            c = dict(op=op, seqs=_logu(rng, 1, 128), nodes=nodes, accept=_logu(rng, 1, min(nodes, 16)),
                     kv_heads=heads, fmt=rng.choice(["bf16", "q8_0", "e4m3"]), layers=_logu(rng, 1, LAYERS),
                     first=_logu(rng, 1, 8000), spread=_logu(rng, 1, 4000), shape=shape)
        w = work(c)
        if w["bytes"] <= most[op]["bytes"] and w["flops"] <= most[op]["flops"]:
            return c


def _lengths(case):
    """What a scheduler knows on the host: per request, the committed tokens before this step and the new ones."""
    g = np.random.default_rng(case["shape"])
    before = case["first"] + g.integers(0, case["spread"], size=case["seqs"])
    if case["op"] == "window" and case["spread"] > 4096:  # lengths over several orders: uniform in the logarithm
        lo, hi = math.log(case["first"]), math.log(case["first"] + case["spread"])
        before = np.floor(np.exp(g.uniform(lo, hi, size=case["seqs"]))).astype(np.int64)
    if case["op"] in ("tree", "compact"):
        n = case["nodes"]
        new = g.integers(max(1, n - n // 4), n + 1, size=case["seqs"])  # a padded batch of trees
        new[0] = n
    else:
        new = np.full(case["seqs"], case["q_len"] if case["op"] == "window" else case["per_seq"])
    return before.astype(np.int64), new.astype(np.int64)


def _parents(case):
    """A tree for each request: every node hangs under an earlier one, most of them near the front."""
    g = np.random.default_rng(case["shape"] + 1)
    n = case["nodes"]
    return [[-1] + [int(g.integers(max(0, i // 3 - 1), max(1, (2 * i) // 3))) for i in range(1, n)]
            for _ in range(case["seqs"])]


def _accepted(case):
    """Each request's accepted nodes, rising: a few that are in place already, then later ones."""
    g = np.random.default_rng(case["shape"] + 2)
    _, new = _lengths(case)
    rows = []
    for n in new:
        m = int(g.integers(1, min(case["accept"], int(n)) + 1))
        keep = int(g.integers(0, min(2, m) + 1))
        keep = max(keep, m - max(0, int(n) - m))  # enough later nodes to choose from
        rows.append(list(range(keep)) + sorted(m + g.choice(int(n) - m, size=m - keep, replace=False)))
    return [[int(x) for x in row] for row in rows]


def _window_parts(case, ctx):
    """[0, sink_end) and [start, ctx): the keys that some query of the call sees."""
    first_pos = max(0, ctx - case["q_len"])
    start = max(0, first_pos - case["window"] + 1)
    return min(case["sinks"], start), start


def work(case):
    hkv, hq = case["kv_heads"], case["kv_heads"] * GROUP
    before, new = _lengths(case)
    if case["op"] == "norm_rope":
        tokens = int(new.sum())
        stored = 2 * hkv * (DIM * 2 if case["fmt"] == "bf16" else DIM)
        per_token = (hq + 2 * hkv) * DIM * 2 + hq * DIM * 2 + stored + case["rot"] * 4 + 12
        return {"bytes": tokens * per_token, "flops": tokens * (hq + hkv) * DIM * 8}
    if case["op"] == "compact":
        moved = sum(1 for row in _accepted(case) for j, i in enumerate(row) if i != j)
        row = hkv * TILE_BYTES[case["fmt"]] // BLOCK
        return {"bytes": 2 * 2 * moved * row * case["layers"] + 8 * sum(map(len, _accepted(case))), "flops": 0}
    if case["op"] == "tree":
        parents = _parents(case)
        pairs = 0
        for b, n, par in zip(before, new, parents):
            depth = []
            for i in range(int(n)):
                depth.append(1 if par[i] < 0 else depth[par[i]] + 1)
            pairs += int(n) * int(b) + sum(depth)
        keys = int((before + new).sum())
        rows = case["seqs"] * case["nodes"]
    else:
        pairs = keys = 0
        for b, n in zip(before, new):
            ctx = int(b + n)
            sink_end, start = _window_parts(case, ctx)
            keys += sink_end + ctx - start
            p = np.arange(int(b), ctx)
            lo = np.maximum(0, p - case["window"] + 1)
            pairs += int((p - lo + 1 + np.minimum(case["sinks"], lo)).sum())
        rows = int(new.sum())
    return {"bytes": keys * hkv * DIM * 2 * 2 + 2 * rows * hq * DIM * 2, "flops": 4 * DIM * hq * pairs}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _tables(needed, total, seed):
    """Block tables of a pool that is handed out in a shuffled order; -1 where a request holds no block.
    needed: for each request, the logical blocks that it holds."""
    perm = np.random.default_rng(seed).permutation(total)
    width = max(max(n) for n in needed) + 1
    table = np.full((len(needed), width), -1, dtype=np.int32)
    at = 0
    for r, blocks in enumerate(needed):
        table[r, blocks] = perm[at:at + len(blocks)]
        at += len(blocks)
    return table


def _rope_table(rot, length):
    inv = THETA ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    ang = torch.arange(length, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, scale=1.0):
        return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(torch.bfloat16)

    def randn_pool(*shape):
        return torch.empty(shape, device="cuda", dtype=torch.bfloat16).normal_(generator=gen)

    def dev(a, dtype):
        return torch.from_numpy(np.ascontiguousarray(a)).to(device="cuda", dtype=dtype)

    hkv, hq, seqs = case["kv_heads"], case["kv_heads"] * GROUP, case["seqs"]
    before, new = _lengths(case)
    ctx = before + new
    s = {"case": case, "ctx": [int(c) for c in ctx], "new": [int(n) for n in new]}
    if case["op"] == "norm_rope":
        need = [list(range(int(b) // BLOCK, -(-int(c) // BLOCK))) for b, c in zip(before, ctx)]
        total = sum(map(len, need)) + 8
        table = _tables(need, total, seed)
        pos, slots = [], []
        for r in range(seqs):
            p = np.arange(before[r], ctx[r])
            pos.append(p)
            slots.append(table[r, p // BLOCK].astype(np.int64) * BLOCK + p % BLOCK)
        pos, slots = np.concatenate(pos), np.concatenate(slots)
        slots[5::97] = -1  # tokens of a padded batch: nothing is stored for them
        tokens = len(pos)
        # the projection's output: some channels much larger than the others
        gain = torch.ones((hq + 2 * hkv) * DIM, device="cuda")
        gain[torch.randperm(gain.numel(), generator=gen, device="cuda")[: gain.numel() // 64]] = 8.0
        qkv = torch.empty((tokens, (hq + 2 * hkv) * DIM), device="cuda", dtype=torch.bfloat16).normal_(generator=gen)
        qkv *= gain
        s["q"] = qkv[:, : hq * DIM].view(tokens, hq, DIM)
        s["k"] = qkv[:, hq * DIM:(hq + hkv) * DIM].view(tokens, hkv, DIM)
        s["v"] = qkv[:, (hq + hkv) * DIM:].view(tokens, hkv, DIM)
        s["q_weight"] = s["k_weight"] = None
        if case["norm"]:
            s["q_weight"] = (1 + 0.2 * randn(DIM).float()).to(torch.bfloat16)
            s["k_weight"] = (1 + 0.2 * randn(DIM).float()).to(torch.bfloat16)
        s["rope_table"] = _rope_table(case["rot"], int(ctx.max()))
        s["positions"] = dev(pos, torch.int32)
        s["slots"] = dev(slots, torch.int64)
        stored = np.flatnonzero(slots >= 0)
        s["stored"] = dev(stored, torch.int64)
        s["blk"], s["off"] = dev(slots[stored] // BLOCK, torch.int64), dev(slots[stored] % BLOCK, torch.int64)
        if case["fmt"] == "bf16":
            s["k_cache"], s["v_cache"] = (randn_pool(total, hkv, BLOCK, DIM) for _ in range(2))
        else:
            s["k_cache"], s["v_cache"] = (randn_pool(total, hkv, BLOCK, DIM).to(torch.float8_e4m3fn).view(torch.uint8)
                                          for _ in range(2))
        s["q_out"] = torch.empty((tokens, hq, DIM), device="cuda", dtype=torch.bfloat16)
    elif case["op"] == "compact":
        need = [list(range(int(b) // BLOCK, -(-int(c) // BLOCK))) for b, c in zip(before, ctx)]
        total = sum(map(len, need)) + 8
        table = _tables(need, total, seed)
        rows = _accepted(case)
        width = max(map(len, rows))
        acc = np.zeros((seqs, width), np.int32)
        src, dst = [], []
        for r, row in enumerate(rows):
            acc[r, : len(row)] = row
            for j, i in enumerate(row):
                a, b = int(before[r]) + i, int(before[r]) + j
                src.append(int(table[r, a // BLOCK]) * BLOCK + a % BLOCK)
                dst.append(int(table[r, b // BLOCK]) * BLOCK + b % BLOCK)
        s["src"], s["dst"] = dev(np.asarray(src), torch.int64), dev(np.asarray(dst), torch.int64)
        s["accepted"], s["num_accepted"] = dev(acc, torch.int32), dev(np.asarray([len(r) for r in rows]), torch.int32)
        for name in ("k", "v"):  # one allocation for all layers
            if case["fmt"] == "bf16":
                s[name] = randn_pool(case["layers"], total, hkv, BLOCK, DIM)
            else:
                tile = (2176,) if case["fmt"] == "q8_0" else (BLOCK, DIM)
                s[name] = torch.randint(0, 127, (case["layers"], total, hkv, *tile), generator=gen, device="cuda",
                                        dtype=torch.uint8)
    else:
        if case["op"] == "tree":
            need = [list(range(-(-int(c) // BLOCK))) for c in ctx]
            width = case["nodes"]
        else:
            need = []
            for c in ctx:
                sink_end, start = _window_parts(case, int(c))
                need.append(sorted(set(range(-(-sink_end // BLOCK))) | set(range(start // BLOCK, -(-int(c) // BLOCK)))))
            width = case["q_len"]
        total = sum(map(len, need)) + 8
        table = _tables(need, total, seed)
        s["k_cache"], s["v_cache"] = randn_pool(total, hkv, BLOCK, DIM), randn_pool(total, hkv, BLOCK, DIM)
        s["q"] = randn(seqs, width, hq, DIM, scale=2.0)  # some keys get much of the weight
        s["out"] = torch.empty_like(s["q"])
        if case["op"] == "tree":
            words = -(-width // 64)
            mask = np.zeros((seqs, width, words), np.uint64)
            for r, par in enumerate(_parents(case)):
                for i in range(int(new[r])):
                    if par[i] >= 0:
                        mask[r, i] = mask[r, par[i]]
                    mask[r, i, i // 64] |= np.uint64(1 << (i % 64))
            s["mask"] = torch.from_numpy(mask.view(np.int64)).cuda()
    s["tables"] = dev(table, torch.int32)
    s["lens"] = dev(ctx, torch.int32)
    s["tree_lens"] = dev(new, torch.int32)
    if own:
        import paged_kv_decode_attention_gb300 as pkv
        s["pkv"] = pkv
        if case["op"] == "tree":
            size = pkv.workspace_size_tree(seqs, width, hq, table.shape[1])
            s["workspace"] = torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")
        elif case["op"] == "window":
            size = pkv.workspace_size_window(seqs, width, hq, table.shape[1], case["window"], case["sinks"])
            s["workspace"] = torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")
        elif case["op"] == "compact":
            fmt = {"bf16": pkv.KV_BF16, "q8_0": pkv.KV_Q8_0, "e4m3": pkv.KV_FP8_E4M3}[case["fmt"]]
            s["pools"] = pkv.KvPools(list(s["k"]), list(s["v"]), fmt)
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(s):
    case = s["case"]
    if own:
        return _run_own(s)
    return {"norm_rope": _plain_norm_rope, "tree": _plain_attention, "window": _plain_attention,
            "compact": _plain_compact}[case["op"]](s)


def _run_own(s):
    pkv, case = s["pkv"], s["case"]
    if case["op"] == "norm_rope":
        pkv.qk_norm_rope_append(s["q_out"], s["k_cache"], s["v_cache"], s["slots"], s["q"], s["k"], s["v"],
                                s["positions"], s["rope_table"], s["q_weight"], s["k_weight"], EPS,
                                case["interleaved"], pkv.KV_BF16 if case["fmt"] == "bf16" else pkv.KV_FP8_E4M3)
        return _norm_rope_outputs(s)
    if case["op"] == "tree":
        pkv.paged_attention_tree(s["out"], s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["mask"],
                                 SCALE, s["tree_lens"], workspace=s["workspace"])
        return s["out"]
    if case["op"] == "window":
        pkv.paged_attention_window(s["out"], s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"],
                                   case["q_len"], case["window"], case["sinks"], SCALE, workspace=s["workspace"])
        return s["out"]
    pkv.kv_compact(s["pools"], s["tables"], s["lens"], s["accepted"], s["num_accepted"], case["nodes"],
                   s["tree_lens"])
    return _compact_outputs(s)


def _norm_rope_outputs(s):
    if s["case"]["fmt"] == "bf16":
        return s["q_out"], s["k_cache"], s["v_cache"]
    return s["q_out"], s["k_cache"].view(torch.float8_e4m3fn), s["v_cache"].view(torch.float8_e4m3fn)


def _compact_outputs(s):
    as_int = torch.int16 if s["case"]["fmt"] == "bf16" else torch.uint8
    return s["k"].view(as_int), s["v"].view(as_int)


def _rotate(x, cos, sin, rot, interleaved):
    """x [T][H][128]; cos, sin [T][1][rot / 2]: pairs (2i, 2i + 1), or (i, i + rot / 2)."""
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2] = a * cos - b * sin
        y[..., 1:rot:2] = b * cos + a * sin
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        y[..., : rot // 2] = a * cos - b * sin
        y[..., rot // 2: rot] = b * cos + a * sin
    return y


def _plain_norm_rope(s):
    case = s["case"]
    t = s["rope_table"][s["positions"].long()]
    cos, sin = t[:, None, : case["rot"] // 2], t[:, None, case["rot"] // 2:]
    done = []
    for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
        done.append(_rotate(x, cos, sin, case["rot"], case["interleaved"]))
    s["q_out"].copy_(done[0])
    for cache, x in ((s["k_cache"], done[1]), (s["v_cache"], s["v"].float())):
        x = x[s["stored"]]
        if case["fmt"] == "bf16":
            cache[s["blk"], :, s["off"]] = x.to(torch.bfloat16)
        else:
            cache[s["blk"], :, s["off"]] = x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    return _norm_rope_outputs(s)


def _visible(s, r, t):
    """Which of the keys at positions t request r's queries see: [new][len(t)]."""
    case, ctx, n = s["case"], s["ctx"][r], s["new"][r]
    if case["op"] == "tree":
        j = (t - (ctx - n)).clamp(min=0)
        bits = (s["mask"][r, :n][:, j // 64] >> (j % 64)) & 1
        return (t < ctx - n) | (bits == 1)
    p = torch.arange(ctx - n, ctx, device="cuda")[:, None]
    return (t <= p) & ((t > p - case["window"]) | (t < case["sinks"]))


def _plain_attention(s):
    case = s["case"]
    hkv = case["kv_heads"]
    s["out"].zero_()
    for r, (ctx, n) in enumerate(zip(s["ctx"], s["new"])):
        if case["op"] == "tree":
            t = torch.arange(ctx, device="cuda")
        else:
            sink_end, start = _window_parts(case, ctx)
            t = torch.cat([torch.arange(sink_end, device="cuda"), torch.arange(start, ctx, device="cuda")])
        blk, off = s["tables"][r, t // BLOCK].long(), t % BLOCK
        k = s["k_cache"][blk, :, off].float().transpose(0, 1)  # [Hkv][keys][128]
        v = s["v_cache"][blk, :, off].float().transpose(0, 1)
        seen = _visible(s, r, t).repeat_interleave(GROUP, 0)  # [n * 4][keys]
        q = s["q"][r, :n].float().view(n, hkv, GROUP, DIM).transpose(0, 1).reshape(hkv, n * GROUP, DIM)
        x = torch.matmul(q, k.transpose(1, 2)) * SCALE
        x = x.masked_fill(~seen, -math.inf)
        e = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-1e30))
        o = torch.matmul(e, v) / e.sum(-1, keepdim=True).clamp(min=1e-30)
        s["out"][r, :n] = o.view(hkv, n, GROUP, DIM).transpose(0, 1).reshape(n, hkv * GROUP, DIM).to(torch.bfloat16)
    return s["out"]


def _plain_compact(s):
    src, dst = s["src"], s["dst"]
    for t in (s["k"], s["v"]):
        if s["case"]["fmt"] == "q8_0":  # codes [16][128], then scales [16][4] of 2 bytes
            parts = (t[..., :2048].unflatten(3, (BLOCK, DIM)), t[..., 2048:].unflatten(3, (BLOCK, 8)))
        else:
            parts = (t,)
        for p in parts:
            p[:, dst // BLOCK, :, dst % BLOCK] = p[:, src // BLOCK, :, src % BLOCK]
    return _compact_outputs(s)


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "compact":
        return None  # copies: there is nothing to compute
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        return _exact_norm_rope(s)
    return _exact_attention(s)


def _exact_norm_rope(s):
    case = s["case"]
    half, width = case["rot"] // 2, case["rot"]
    table = s["rope_table"].double()[s["positions"].long()]
    turn = torch.complex(table[:, :half], table[:, half:])[:, None]  # one unit complex number per pair

    def head(x, w):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / DIM + EPS) * w.double()
        front = x[..., :width]
        pairs = front.unflatten(-1, (half, 2)) if case["interleaved"] else front.unflatten(-1, (2, half)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        z = z.flatten(-2) if case["interleaved"] else z.transpose(-1, -2).flatten(-2)
        return torch.cat([z, x[..., width:]], -1)

    outs = [head(s["q"], s["q_weight"])]
    slots = s["slots"]
    for cache, x in ((s["k_cache"], head(s["k"], s["k_weight"])), (s["v_cache"], s["v"].double())):
        if case["fmt"] == "e4m3":
            cache = cache.view(torch.float8_e4m3fn)
            x = x.clamp(-448.0, 448.0)
        pool = cache.to(torch.float32).double()
        flat = pool.transpose(1, 2).flatten(0, 1).contiguous()  # [slot][Hkv][128]
        flat[slots[slots >= 0]] = x[slots >= 0]
        outs.append(flat.unflatten(0, (-1, BLOCK)).transpose(1, 2).contiguous())
    return tuple(outs)


def _exact_attention(s):
    case = s["case"]
    hkv, hq = case["kv_heads"], case["kv_heads"] * GROUP
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for r, (ctx, n) in enumerate(zip(s["ctx"], s["new"])):
        base = ctx - n
        pos = np.arange(ctx)
        if case["op"] == "window":  # the keys between the sinks and the window have no page
            pos = pos[(pos < case["sinks"]) | (pos > base - case["window"])]
        at = torch.from_numpy(pos).cuda()
        slot = s["tables"][r].long()[at // BLOCK] * BLOCK + at % BLOCK
        k = s["k_cache"][slot // BLOCK, :, slot % BLOCK].double()
        v = s["v_cache"][slot // BLOCK, :, slot % BLOCK].double()
        if case["op"] == "tree":
            allowed = torch.ones((n, len(pos)), dtype=torch.bool, device="cuda")
            words = s["mask"][r, :n].cpu().numpy().view(np.uint64)
            for i in range(n):
                number = sum(int(w) << (64 * k2) for k2, w in enumerate(words[i]))
                seen = torch.tensor([(number >> j) & 1 == 1 for j in range(n)], device="cuda")
                allowed[i, base:] = seen
        else:
            back = torch.arange(base, ctx, device="cuda")[:, None] - at[None]
            allowed = (back >= 0) & ((back < case["window"]) | (at < case["sinks"])[None])
        step = max(1, (1 << 26) // (hq * max(1, len(pos))))  # bounds the scores held at once
        for i in range(0, n, step):
            q = s["q"][r, i:min(n, i + step)].double()
            x = torch.einsum("nhgd,thd->nhgt", q.unflatten(1, (hkv, GROUP)), k) * SCALE
            ok = allowed[i:i + step, None, None]
            x = torch.where(ok, x, torch.full_like(x, -math.inf))
            top = x.max(-1, keepdim=True).values
            e = torch.where(ok, torch.exp(x - torch.where(top.isfinite(), top, torch.zeros_like(top))),
                            torch.zeros_like(x))
            total = e.sum(-1, keepdim=True)
            o = torch.einsum("nhgt,thd->nhgd", e, v) / torch.where(total > 0, total, torch.ones_like(total))
            out[r, i:i + q.shape[0]] = o.flatten(1, 2)
    return out

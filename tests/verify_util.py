"""Plain 64-bit forms of the verification-step and sliding-window operators,
and input builders, for their tests (torch float64 on the device the inputs
are on; nothing of the library)."""
import math

import numpy as np
import torch

SCALE = 1.0 / math.sqrt(128)


def randn_bf16(gen, *shape, scale=1.0):
    return (torch.randn(shape, generator=gen, dtype=torch.float32) * scale).to(torch.bfloat16)


def paged_case(ctx, width, hkv, seed, spare=5, hold=None, max_blocks=None, q_scale=1.5):
    """Pools, tables and queries (CPU).  hold(r): the logical blocks request r holds (default: all of its context);
    other table entries are -1 and pool blocks nobody holds are NaN, as are slots past a context."""
    gen = torch.Generator().manual_seed(seed)
    blocks = [list(range(-(-max(c, 0) // 16))) if hold is None else sorted(hold(r)) for r, c in enumerate(ctx)]
    total = sum(map(len, blocks)) + spare
    maxb = max_blocks or max([b[-1] + 1 for b in blocks if b] + [1]) + 2
    perm = torch.randperm(total, generator=gen).tolist()
    table = torch.full((len(ctx), maxb), -1, dtype=torch.int32)
    k, v = randn_bf16(gen, total, hkv, 16, 128), randn_bf16(gen, total, hkv, 16, 128)
    at = 0
    for r, bl in enumerate(blocks):
        for b in bl:
            table[r, b] = perm[at]
            at += 1
        if ctx[r] % 16 and bl and bl[-1] == ctx[r] // 16:
            for t in (k, v):
                t[perm[at - 1], :, ctx[r] % 16:] = float("nan")
    for b in perm[at:]:
        k[b] = float("nan")
        v[b] = float("nan")
    q = randn_bf16(gen, len(ctx), width, 4 * hkv, 128, scale=q_scale)
    return {"q": q, "k_cache": k, "v_cache": v, "block_tables": table,
            "context_lens": torch.tensor(ctx, dtype=torch.int32)}


def masks_to_words(rows, width):
    """rows[r][i] = iterable of visible drafts -> int64 [B][width][ceil(width/64)]."""
    words = np.zeros((len(rows), width, -(-width // 64)), np.uint64)
    for r, req in enumerate(rows):
        for i, seen in enumerate(req):
            for j in seen:
                words[r, i, j // 64] |= np.uint64(1 << (j % 64))
    return torch.from_numpy(words.view(np.int64))


def random_tree(rng, n):
    rows = []
    for i in range(n):
        parent = int(rng.integers(-1, i)) if i else -1
        rows.append(([] if parent < 0 else list(rows[parent])) + [i])
    return rows


def attention64(d, allowed, scale=SCALE, weights=2.0 ** -8):
    """allowed(r) -> (query rows, positions, visible [rows][positions]) for request r.  Returns the outputs in 64 bits
    and, per output, a bound of the kernels' error from the format's roundings:

    half a BF16 step of the output (2^-8 |o|); the weights' own rounding, at most `weights` of each weight (2^-8 as
    one BF16 value, 2^-16 as a BF16 value and the BF16 rounding of the remainder), so that much of A = sum p |v|; and
    the FP32 logits and sums: a dot product of 128 exact products is off by at most 128 * 2^-24 *
    sum |q k|, which moves every weight by that much (x scale), numerator and denominator; the base-2 exponential and
    the sums add less than 2^-16 of A."""
    q = d["q"].double()
    b, width, hq, dim = q.shape
    hkv = d["k_cache"].shape[1]
    out = torch.zeros_like(q)
    tol = torch.zeros_like(q)
    for r in range(b):
        rows, pos, seen = allowed(r)
        if len(rows) == 0 or len(pos) == 0:
            continue
        rows, pos = torch.as_tensor(rows, device=q.device), torch.as_tensor(pos, device=q.device)
        seen = torch.as_tensor(seen, device=q.device)
        blk = d["block_tables"][r].to(q.device).long()[pos // 16]
        k = d["k_cache"][blk, :, pos % 16].double()
        v = d["v_cache"][blk, :, pos % 16].double()
        qr = q[r, rows].view(len(rows), hkv, 4, dim)
        x = torch.einsum("nhgd,thd->nhgt", qr, k) * scale
        e_s = torch.einsum("nhgd,thd->nhgt", qr.abs(), k.abs()).amax(-1, keepdim=True) * (scale * 2.0 ** -17)
        x = x.masked_fill(~seen[:, None, None], -math.inf)
        m = x.amax(-1, keepdim=True)
        e = torch.where(seen[:, None, None], torch.exp(x - m.clamp(min=-1e300)), 0.0)
        l = e.sum(-1, keepdim=True)
        p = e / torch.where(l > 0, l, 1.0)
        o = torch.einsum("nhgt,thd->nhgd", p, v)
        a = torch.einsum("nhgt,thd->nhgd", p, v.abs())
        out[r, rows] = o.reshape(len(rows), hq, dim)
        tol[r, rows] = (2.0 ** -8 * o.abs() + a * (weights + 2 * e_s + 2.0 ** -16)).reshape(len(rows), hq, dim)
    return out, tol


def tree_allowed(ctx, tree_lens, rows):
    def f(r):
        c, n = ctx[r], tree_lens[r]
        if c <= 0 or n <= 0:
            return [], [], []
        seen = np.zeros((n, c), bool)
        for i in range(n):
            seen[i, :max(0, c - n)] = True
            for j in rows[r][i]:
                if j < n and 0 <= c - n + j:
                    seen[i, c - n + j] = True
        return np.arange(n), np.arange(c), seen
    return f


def window_allowed(ctx, q_len, window, sinks):
    def f(r):
        c = ctx[r]
        if c <= 0:
            return [], [], []
        rows = np.arange(max(0, q_len - c), q_len)
        p = (c - q_len + rows)[:, None]
        t = np.arange(c)
        keep = (t < sinks) | (t > p[0, 0] - window)
        t = t[keep]
        return rows, t, (t[None] <= p) & ((t[None] > p - window) | (t[None] < sinks))
    return f


def window_hold(ctx, q_len, window, sinks):
    def hold(r):
        c = ctx[r]
        if c <= 0:
            return []
        start = max(0, max(0, c - q_len) - window + 1)
        return set(range(-(-min(sinks, start) // 16))) | set(range(start // 16, -(-c // 16)))
    return hold


def assert_within(got, ref, tol, what=""):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: non-finite output"
    over = (got - ref).abs() - tol
    assert (over <= 0).all(), f"{what}: off by {float((got - ref).abs().max()):.3e}, {float(over.max()):.3e} beyond the bound"

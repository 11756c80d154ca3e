"""A verification step as a serving loop runs it -- the drafts' queries, keys
and values normed, rotated and stored, each draft attending to its ancestors,
the accepted path kept -- and the decode step after it, against a request that
was fed the accepted tokens one by one."""
import numpy as np
import pytest
import torch

import verify_util as V

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import paged_kv_decode_attention_gb300 as pkv
else:  # collected on CPU-only machines, every test skipped
    pkv = None

HKV, LAYERS, EPS, MAX_POS = 2, 2, 1e-6, 600


@pytest.mark.parametrize("width,window", [(12, None), (40, None), (12, 64), (40, 64)])
def test_accepted_path_equals_the_tokens_fed_one_by_one(width, window):
    pkv.get_device_error(reset=True)
    rng = np.random.default_rng(width)
    gen = torch.Generator().manual_seed(width)
    committed, lens = [37, 0, 500, 16, 130], [width, width, 5, width - 1, 1]
    ctx = [c + n for c, n in zip(committed, lens)]
    trees = [V.random_tree(rng, n) for n in lens]
    # the accepted path: the ancestors of some node, itself included
    paths = [t[int(rng.integers(len(t) // 2, len(t)))] for t in trees]
    b, maxb = len(ctx), -(-(max(ctx) + 1) // 16) + 1
    blocks = [-(-(c + 1) // 16) for c in ctx]
    total = sum(blocks)
    perm, at = rng.permutation(total), 0
    table = np.full((b, maxb), -1, np.int32)
    for r, n in enumerate(blocks):
        table[r, :n] = perm[at:at + n]
        at += n
    slot = lambda r, p: int(table[r, p // 16]) * 16 + p % 16
    tables = torch.from_numpy(table).cuda()
    ang = np.arange(MAX_POS)[:, None] * 10000.0 ** (-np.arange(0, 128, 2) / 128)
    rope = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)).cuda()
    weights = [(1 + 0.2 * torch.randn(128, generator=gen)).to(torch.bfloat16).cuda() for _ in range(2)]
    base = [[V.randn_bf16(gen, total, HKV, 16, 128).cuda() for _ in range(2)] for _ in range(LAYERS)]
    qkv = [V.randn_bf16(gen, b, width + 1, 6 * HKV * 128, scale=1.5).cuda() for _ in range(LAYERS)]  # drafts, then the next token
    split = lambda t: (t[:, :4 * HKV * 128].unflatten(1, (4 * HKV, 128)),
                       t[:, 4 * HKV * 128:5 * HKV * 128].unflatten(1, (HKV, 128)),
                       t[:, 5 * HKV * 128:].unflatten(1, (HKV, 128)))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()

    def store(pools, t, q_out, slots, pos):
        q, k, v = split(t)
        pkv.qk_norm_rope_append(q_out, pools[0], pools[1], torch.tensor(slots, dtype=torch.int64).cuda(), q, k, v,
                                i32(pos), rope, weights[0], weights[1], EPS)

    def decode(pools, layer, lens_now):
        """The next token of every request, at position lens_now - 1."""
        q = torch.empty((b, 1, 4 * HKV, 128), dtype=torch.bfloat16, device="cuda")
        store(pools, qkv[layer][:, width].contiguous(), q.view(b, 4 * HKV, 128),
              [slot(r, n - 1) for r, n in enumerate(lens_now)], [n - 1 for n in lens_now])
        out = torch.empty_like(q)
        if window is None:
            pkv.paged_attention(out, q, pools[0], pools[1], tables, i32(lens_now), 1, V.SCALE,
                                kv_blocks_per_split=1 << 20)
        else:
            pkv.paged_attention_window(out, q, pools[0], pools[1], tables, i32(lens_now), 1, window, 4, V.SCALE,
                                       kv_blocks_per_split=1 << 20)
        return out

    # the verification step
    pools = [[p.clone() for p in layer] for layer in base]
    depth = [[len(row) - 1 for row in t] for t in trees]
    slots = [slot(r, committed[r] + i) if i < lens[r] else -1 for r in range(b) for i in range(width)]
    pos = [committed[r] + depth[r][i] if i < lens[r] else 0 for r in range(b) for i in range(width)]
    mask = V.masks_to_words(trees, width).cuda()
    tree_out = []
    for layer in range(LAYERS):
        q = torch.empty((b, width, 4 * HKV, 128), dtype=torch.bfloat16, device="cuda")
        store(pools[layer], qkv[layer][:, :width].reshape(b * width, -1), q.view(b * width, 4 * HKV, 128), slots, pos)
        out = torch.full_like(q, float("nan"))
        ws = torch.empty(max(1, pkv.workspace_size_tree(b, width, 4 * HKV, maxb)), dtype=torch.uint8, device="cuda")
        pkv.paged_attention_tree(out, q, pools[layer][0], pools[layer][1], tables, i32(ctx), mask, V.SCALE, i32(lens),
                                 workspace=ws)
        tree_out.append(out)
    acc = torch.zeros((b, max(map(len, paths))), dtype=torch.int32)
    for r, p in enumerate(paths):
        acc[r, :len(p)] = torch.tensor(p)
    pkv.kv_compact(pkv.KvPools([p[0] for p in pools], [p[1] for p in pools]), tables, i32(ctx), acc.cuda(),
                   i32([len(p) for p in paths]), width, i32(lens))
    after = [c + len(p) for c, p in zip(committed, paths)]
    got = [decode(pools[layer], layer, [n + 1 for n in after]) for layer in range(LAYERS)]

    # the same tokens one by one
    serial = [[p.clone() for p in layer] for layer in base]
    for layer in range(LAYERS):
        for r, path in enumerate(paths):
            for j, i in enumerate(path):
                q = torch.empty((1, 1, 4 * HKV, 128), dtype=torch.bfloat16, device="cuda")
                store(serial[layer], qkv[layer][r:r + 1, i].contiguous(), q.view(1, 4 * HKV, 128),
                      [slot(r, committed[r] + j)], [committed[r] + j])
                one = torch.empty_like(q)
                pkv.paged_attention(one, q, serial[layer][0], serial[layer][1], tables[r:r + 1].contiguous(),
                                    i32([committed[r] + j + 1]), 1, V.SCALE, kv_blocks_per_split=1 << 20)
                d = {"q": q, "k_cache": serial[layer][0], "v_cache": serial[layer][1],
                     "block_tables": tables[r:r + 1], "context_lens": None}
                n = committed[r] + j + 1
                _, tol = V.attention64(d, lambda _: ([0], np.arange(n), np.ones((1, n), bool)))
                draft = tree_out[layer][r, i].double()
                assert ((draft - one[0, 0].double()).abs() <= 2 * tol[0, 0]).all(), (layer, r, i)
        for t in range(b):  # the kept rows are the same bits
            for p in range(after[t]):
                s = slot(t, p)
                for a, c in zip(pools[layer], serial[layer]):
                    assert torch.equal(a[s // 16, :, s % 16], c[s // 16, :, s % 16])
    want = [decode(serial[layer], layer, [n + 1 for n in after]) for layer in range(LAYERS)]
    torch.cuda.synchronize()
    assert pkv.get_device_error(reset=True) == 0
    for a, c in zip(got, want):
        assert torch.equal(a, c)
    for layer in range(LAYERS):
        for r in range(b):
            assert not tree_out[layer][r, lens[r]:].any()

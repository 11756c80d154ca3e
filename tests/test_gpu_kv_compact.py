"""pkv_kv_compact: the accepted drafts' rows, bit for bit, in every pool
format and layer; and the lists, lengths and tables that it refuses."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import paged_kv_decode_attention_gb300 as pkv
    FORMATS = {"bf16": pkv.KV_BF16, "q8_0": pkv.KV_Q8_0, "e4m3": pkv.KV_FP8_E4M3}
else:  # collected on CPU-only machines, every test skipped
    pkv = None


@pytest.fixture(autouse=True)
def _clear_device_error():
    if pkv is not None:
        pkv.get_device_error(reset=True)
    yield
    if pkv is not None:
        assert pkv.get_device_error(reset=True) == 0


def parts(pool, fmt):
    """Views [block][Hkv][16][...] of a pool's token rows."""
    if fmt == "q8_0":
        return [pool[..., :2048].unflatten(2, (16, 128)), pool[..., 2048:].unflatten(2, (16, 8))]
    return [pool]


def make(committed, tree_lens, tree_len, lists, fmt, layers, hkv=2, seed=0):
    rng = np.random.default_rng(seed)
    ctx = [c + n for c, n in zip(committed, tree_lens)]
    blocks = [-(-c // 16) for c in ctx]
    total, maxb = sum(blocks) + 4, max(blocks) + 1
    perm = rng.permutation(total)
    table = np.full((len(ctx), maxb), -1, np.int32)
    at = 0
    for r, n in enumerate(blocks):
        table[r, :n] = perm[at:at + n]
        at += n
    width = max(1, max(len(x) for x in lists))
    acc = rng.integers(-5, 2000, (len(ctx), width)).astype(np.int32)  # entries behind a list are never read
    for r, x in enumerate(lists):
        acc[r, :len(x)] = x
    shape = (total, hkv, 2176) if fmt == "q8_0" else (total, hkv, 16, 128)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    def pool():
        if fmt == "bf16":
            return torch.randint(-2 ** 15, 2 ** 15, shape, generator=gen, device="cuda", dtype=torch.int16)
        return torch.randint(0, 256, shape, generator=gen, device="cuda", dtype=torch.uint8)
    d = {"k": [pool() for _ in range(layers)], "v": [pool() for _ in range(layers)], "table_np": table, "ctx": ctx,
         "tables": torch.from_numpy(table).cuda(), "lens": torch.tensor(ctx, dtype=torch.int32).cuda(),
         "tree_lens": torch.tensor(tree_lens, dtype=torch.int32).cuda(), "acc": torch.from_numpy(acc).cuda(),
         "num": torch.tensor([len(x) for x in lists], dtype=torch.int32).cuda(), "tree_len": tree_len}
    return d


def expected(d, committed, lists, fmt, skip=()):
    want = {n: [p.clone() for p in d[n]] for n in ("k", "v")}
    for r, x in enumerate(lists):
        if r in skip or not x:
            continue
        src = np.array([committed[r] + i for i in x])
        dst = committed[r] + np.arange(len(x))
        sb, db = (torch.from_numpy(d["table_np"][r][p // 16].astype(np.int64)).cuda() for p in (src, dst))
        so, do = torch.from_numpy(src % 16).cuda(), torch.from_numpy(dst % 16).cuda()
        for n in ("k", "v"):
            for p in want[n]:
                for part in parts(p, fmt):
                    part[db, :, do] = part[sb, :, so].clone()
    return want


def run(d, fmt, use_lens=True):
    pools = pkv.KvPools(d["k"], d["v"], FORMATS[fmt])
    pkv.kv_compact(pools, d["tables"], d["lens"], d["acc"], d["num"], d["tree_len"],
                   d["tree_lens"] if use_lens else None)
    torch.cuda.synchronize()


def same(d, want):
    return all(torch.equal(a, b) for n in ("k", "v") for a, b in zip(d[n], want[n]))


def rising(rng, n, m):
    return sorted(int(x) for x in rng.choice(n, m, replace=False))


@pytest.mark.parametrize("fmt", ["bf16", "q8_0", "e4m3"])
@pytest.mark.parametrize("hkv", [1, 5, 8, 16])
def test_random_lists(fmt, hkv):
    rng = np.random.default_rng(hkv)
    tree_len = 61
    tree_lens = [61, 1, 30, 61, 17, 61, 5, 61, 0]
    committed = [0, 15, 16, 100, 1, 33, 500, 7, 64]
    lists = [rising(rng, n, int(rng.integers(0, n + 1))) for n in tree_lens]
    d = make(committed, tree_lens, tree_len, lists, fmt, 3, hkv, seed=hkv)
    want = expected(d, committed, lists, fmt)
    run(d, fmt)
    assert same(d, want)


@pytest.mark.parametrize("fmt", ["bf16", "q8_0", "e4m3"])
def test_every_length_of_the_list(fmt):
    """Lists of 0 to 40 entries: whole batches, parts of one, and rows that overlap sources and destinations."""
    rng = np.random.default_rng(1)
    n = 45
    lists = [rising(rng, n, m) for m in range(41)] + [list(range(1, m + 1)) for m in (1, 3, 4, 5, 8, 33, 44)] + \
        [list(range(n)), [0], [n - 1]]
    committed = rng.integers(0, 90, len(lists)).tolist()
    d = make(committed, [n] * len(lists), n, lists, fmt, 2, seed=3)
    want = expected(d, committed, lists, fmt)
    run(d, fmt, use_lens=False)
    assert same(d, want)


def test_wide_trees():
    rng = np.random.default_rng(2)
    n = 1024
    lists = [rising(rng, n, 700), rising(rng, n, 3), list(range(1, 1024))]
    committed = [11, 0, 16]
    d = make(committed, [n] * 3, n, lists, "bf16", 1, 1, seed=4)
    want = expected(d, committed, lists, "bf16")
    run(d, "bf16")
    assert same(d, want)


def test_more_layers_than_one_launch_takes():
    lists = [[0, 3, 4], [2]]
    d = make([20, 30], [6, 4], 6, lists, "bf16", 67, seed=5)
    want = expected(d, [20, 30], lists, "bf16")
    run(d, "bf16")
    assert same(d, want)


@pytest.mark.parametrize("fmt", ["bf16", "q8_0", "e4m3"])
def test_bad_requests_are_left_as_they_are(fmt):
    """A list that falls, repeats, leaves the tree or is too long, lengths that contradict one another, and a table
    without the block: each is reported and nothing of its request moves; the others are served."""
    cases = [
        ("falls", [3, 1], None, 32), ("repeats", [2, 2], None, 32), ("negative", [-1, 2], None, 32),
        ("past the tree", [1, 8], None, 32), ("far past", [1, 2 ** 31 - 1], None, 32),
        ("falls late", [1, 2, 4, 5, 6, 7, 7], None, 32),
        ("longer than the list's room", [1, 2], ("num", 8), 32), ("negative count", [1, 2], ("num", -3), 32),
        ("more than drafts", [1, 2, 3], ("tree_lens", 2), 32), ("negative tree", [1, 2], ("tree_lens", -1), 32),
        ("tree too wide", [1, 2], ("tree_lens", 9), 32),
        ("shorter than its tree", [1, 2], ("lens", 7), 4), ("empty context", [1, 2], ("lens", 0), 4),
        ("longer than the table", [1, 2], ("lens", 10 ** 6), 4),
    ]
    for name, bad, change, bit in cases:
        lists = [[1, 4], bad, [0, 5]]
        d = make([20, 14, 30], [8, 8, 8], 8, lists, fmt, 2, seed=6)
        if change:
            d[change[0]][1] = change[1]
        want = expected(d, [20, 14, 30], lists, fmt, skip=(1,))
        run(d, fmt)
        assert pkv.get_device_error(reset=True) == bit, name
        assert same(d, want), name
    for entry in (-1, 10 ** 6):
        lists = [[1, 4], [1, 4], [0, 5]]
        d = make([20, 14, 30], [8, 8, 8], 8, lists, fmt, 2, seed=6)
        want = expected(d, [20, 14, 30], lists, fmt, skip=(1,))
        d["tables"][1, 1] = entry
        run(d, fmt)
        assert pkv.get_device_error(reset=True) == pkv.DEVERR_BLOCK_ID
        assert same(d, want)


def test_captured():
    lists = [[1, 4], [0, 2, 7]]
    d = make([20, 14], [8, 8], 8, lists, "bf16", 2, seed=7)
    pools = pkv.KvPools(d["k"], d["v"])
    want = expected(d, [20, 14], lists, "bf16")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.kv_compact(pools, d["tables"], d["lens"], d["acc"], d["num"], 8, d["tree_lens"])
    g.replay()
    torch.cuda.synchronize()
    assert same(d, want)
    lists = [[3, 5], [6, 7]]
    d["acc"][:, :2] = torch.tensor(lists, dtype=torch.int32).cuda()
    d["num"].fill_(2)
    want = expected(d, [20, 14], lists, "bf16")
    g.replay()
    torch.cuda.synchronize()
    assert same(d, want)


def test_pools_are_checked():
    a, b = (torch.zeros((4, 2, 16, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for k, v, f in (([a], [a], 0), ([a], [], 0), ([], [], 0), ([a], [b[:2]], 0), ([a], [b], 1), ([a], [b], 9),
                    ([a.cpu()], [b.cpu()], 0), ([a], [b.transpose(0, 1)], 0)):
        with pytest.raises((ValueError, TypeError)):
            pkv.KvPools(k, v, f)

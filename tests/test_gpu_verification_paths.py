"""The verification step's calls in the surroundings a serving loop gives
them: all of them on two streams at once, a chain of drafts in a
sliding-window layer, pools of 8-bit formats between the append and the next
decode, heads at the ends of the FP32 range, and the same bits on every run."""
import numpy as np
import pytest
import torch

import verify_util as V

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import paged_kv_decode_attention_gb300 as pkv
else:  # collected on CPU-only machines, every test skipped
    pkv = None

HKV = 2


@pytest.fixture(autouse=True)
def _clear_device_error():
    if pkv is not None:
        pkv.get_device_error(reset=True)
    yield
    if pkv is not None:
        assert pkv.get_device_error(reset=True) == 0


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def rope_table(positions, rot=128):
    ang = np.arange(positions)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
    return torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)).cuda()


class Step:
    """One verification step's buffers: norms, rotation and append, both attentions, compaction."""

    def __init__(self, width, seed, stream=None):
        rng = np.random.default_rng(seed)
        self.width, self.stream = width, stream
        self.ctx = [2000, 31 + width, 700, width]
        rows = [V.random_tree(rng, width) for _ in self.ctx]
        d = {k: v.cuda() for k, v in V.paged_case(self.ctx, width, HKV, seed).items()}
        self.d, self.mask = d, V.masks_to_words(rows, width).cuda()
        self.start = [d["k_cache"].clone(), d["v_cache"].clone()]
        b = len(self.ctx)
        gen = torch.Generator().manual_seed(seed)
        x = V.randn_bf16(gen, b * width, 6 * HKV, 128).cuda()
        self.q, self.k, self.v = x[:, :4 * HKV], x[:, 4 * HKV:5 * HKV], x[:, 5 * HKV:]
        table = d["block_tables"].cpu()
        pos = [c - width + i for c in self.ctx for i in range(width)]
        self.slots = torch.tensor([int(table[r, p // 16]) * 16 + p % 16
                                   for r, c in enumerate(self.ctx) for p in range(c - width, c)], device="cuda")
        self.pos, self.rope = i32(pos), rope_table(2100)
        self.w = [(1 + 0.2 * torch.randn(128, generator=gen)).to(torch.bfloat16).cuda() for _ in range(2)]
        self.acc, self.num = i32([[0, 2, 4]] * b), i32([3, 2, 1, 3])
        self.pools = pkv.KvPools([d["k_cache"]], [d["v_cache"]])
        self.rot = torch.empty((b, width, 4 * HKV, 128), dtype=torch.bfloat16, device="cuda")
        self.tree, self.window = torch.empty_like(self.rot), torch.empty_like(self.rot)
        self.ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")

    def run(self):
        d, b = self.d, len(self.ctx)
        args = (self.rot, d["k_cache"], d["v_cache"], d["block_tables"], d["context_lens"])
        pkv.qk_norm_rope_append(self.rot.view(b * self.width, 4 * HKV, 128), d["k_cache"], d["v_cache"], self.slots,
                                self.q, self.k, self.v, self.pos, self.rope, *self.w, stream=self.stream)
        for bps in (4, 12):  # through the workspace, then in clusters: the one that stays
            pkv.paged_attention_tree(self.tree, *args, self.mask, V.SCALE, kv_blocks_per_split=bps, workspace=self.ws,
                                     stream=self.stream)
            pkv.paged_attention_window(self.window, *args, self.width, 500, 4, V.SCALE, kv_blocks_per_split=bps,
                                       workspace=self.ws, stream=self.stream)
        pkv.kv_compact(self.pools, d["block_tables"], d["context_lens"], self.acc, self.num, self.width,
                       stream=self.stream)

    def results(self):
        return [t.clone().view(torch.int16) for t in (self.rot, self.tree, self.window, self.d["k_cache"],
                                                      self.d["v_cache"])]

    def restore(self):
        self.d["k_cache"].copy_(self.start[0])
        self.d["v_cache"].copy_(self.start[1])


def test_every_operator_on_two_streams_at_once():
    """Each stream's results are those of its step run alone, whatever runs beside it."""
    steps = [Step(26, 1, torch.cuda.Stream()), Step(50, 2, torch.cuda.Stream())]
    want = []
    for s in steps:
        torch.cuda.synchronize()
        s.run()
        torch.cuda.synchronize()
        want.append(s.results())
    for _ in range(10):
        for s in steps:
            s.restore()
        torch.cuda.synchronize()
        for _ in range(3):  # (the append puts the drafts back, so a step may be run again)
            for s in steps:
                s.run()
        torch.cuda.synchronize()
        for s, w in zip(steps, want):
            assert all(torch.equal(a, b) for a, b in zip(s.results(), w))


def test_the_same_bits_on_every_run():
    """No result depends on the order in which CTAs run."""
    for width in (1, 30, 64):
        ctx = np.random.default_rng(width).integers(width, 1500, 60).tolist()
        d = {k: v.cuda() for k, v in V.paged_case(ctx, width, 8, width).items()}
        mask = V.masks_to_words([[list(range(i + 1)) for i in range(width)]] * 60, width).cuda()
        args = (d["q"], d["k_cache"], d["v_cache"], d["block_tables"], d["context_lens"])
        for bps in (0, 8, 24, 1 << 20):
            ws = torch.empty(max(256, pkv.workspace_size_tree(60, width, 32, args[3].shape[1], bps),
                                 pkv.workspace_size_window(60, width, 32, args[3].shape[1], 300, 4, bps)),
                             dtype=torch.uint8, device="cuda")
            first = None
            for _ in range(5):
                out = [torch.empty_like(d["q"]) for _ in range(2)]
                pkv.paged_attention_tree(out[0], *args, mask, V.SCALE, kv_blocks_per_split=bps, workspace=ws)
                pkv.paged_attention_window(out[1], *args, width, 300, 4, V.SCALE, kv_blocks_per_split=bps, workspace=ws)
                ws.random_(0, 255)
                first = first or out
                assert all(torch.equal(a, b) for a, b in zip(first, out)), (width, bps)


@pytest.mark.parametrize("n", [6, 40])
def test_a_chain_of_drafts_in_a_sliding_window_layer(n):
    """Where drafts form a chain, slot order is ancestor order, and the window call verifies them: each draft as the
    decode step of the same window gives it, the rejected ones behind it notwithstanding."""
    window, sinks, ctx = 64, 4, [n, n + 37, n + 500]
    step = Step(n, n)
    step.ctx = ctx
    gen = torch.Generator().manual_seed(n)
    d = {k: v.cuda() for k, v in V.paged_case(ctx, n, HKV, n).items()}
    b, table = len(ctx), d["block_tables"].cpu()
    places = [(r, p) for r, c in enumerate(ctx) for p in range(c - n, c)]
    slots = torch.tensor([int(table[r, p // 16]) * 16 + p % 16 for r, p in places], device="cuda")
    x = V.randn_bf16(gen, b * n, 6 * HKV, 128, scale=1.5).cuda()
    q = torch.empty((b, n, 4 * HKV, 128), dtype=torch.bfloat16, device="cuda")
    pkv.qk_norm_rope_append(q.view(b * n, 4 * HKV, 128), d["k_cache"], d["v_cache"], slots, x[:, :4 * HKV],
                            x[:, 4 * HKV:5 * HKV], x[:, 5 * HKV:], i32([p for _, p in places]), rope_table(600),
                            *step.w)
    out = torch.empty_like(q)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    args = (d["k_cache"], d["v_cache"], d["block_tables"])
    pkv.paged_attention_window(out, q, *args, d["context_lens"], n, window, sinks, V.SCALE, workspace=ws)
    ref, tol = V.attention64(dict(d, q=q), V.window_allowed(ctx, n, window, sinks))
    V.assert_within(out, ref, tol, "chain")
    one = torch.empty((b, 1, 4 * HKV, 128), dtype=torch.bfloat16, device="cuda")
    for i in range(n):
        pkv.paged_attention_window(one, q[:, i:i + 1].contiguous(), *args, d["context_lens"] - (n - 1 - i), 1, window,
                                   sinks, V.SCALE, workspace=ws)
        assert ((one[:, 0].double() - out[:, i].double()).abs() <= 2 * tol[:, i]).all(), i


@pytest.mark.parametrize("fmt", ["bf16", "q8_0", "e4m3"])
def test_kept_drafts_in_every_format(fmt):
    """Drafts normed, rotated and stored in a pool, the accepted ones kept: the pools' rows and the next token's
    attention are those of a cache that was fed the accepted tokens alone, bit for bit."""
    kv_format = {"bf16": pkv.KV_BF16, "q8_0": pkv.KV_Q8_0, "e4m3": pkv.KV_FP8_E4M3}[fmt]
    rng = np.random.default_rng(4)
    gen = torch.Generator().manual_seed(4)
    committed, width, paths = [37, 0, 200], 12, [[0, 3, 7, 11], [1, 2], [0, 1, 2, 3, 4, 5, 9]]
    b, total = len(paths), 50
    table = torch.from_numpy(rng.permutation(total)[:45].reshape(3, 15).astype(np.int32))
    table = torch.cat([table, torch.full((3, 3), -1, dtype=torch.int32)], 1).contiguous()
    tables = table.cuda()
    slot = lambda r, p: int(table[r, p // 16]) * 16 + p % 16
    rope = rope_table(300)
    w = [(1 + 0.2 * torch.randn(128, generator=gen)).to(torch.bfloat16).cuda() for _ in range(2)]
    shape = (total, HKV, 2176) if fmt == "q8_0" else (total, HKV, 16, 128)
    zeros = lambda: torch.zeros(shape, dtype=torch.bfloat16 if fmt == "bf16" else torch.uint8, device="cuda")

    def feed(pools, x, places, positions):
        q = torch.empty((len(places), 4 * HKV, 128), dtype=torch.bfloat16, device="cuda")
        pkv.qk_norm_rope_append(q, *pools, torch.tensor([slot(r, p) for r, p in places], device="cuda"),
                                x[:, :4 * HKV], x[:, 4 * HKV:5 * HKV], x[:, 5 * HKV:], i32(positions), rope, *w,
                                kv_format=kv_format)
        return q

    def attend(pools, q, lens):
        out = torch.empty((b, 1, 4 * HKV, 128), dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(16 << 20, dtype=torch.uint8, device="cuda")
        args = (out, q.view(b, 1, 4 * HKV, 128), *pools, tables, i32(lens))
        if fmt == "bf16":
            pkv.paged_attention(*args, 1, V.SCALE, workspace=ws)
        else:
            (pkv.paged_attention_q8_0 if fmt == "q8_0" else pkv.paged_attention_fp8_e4m3)(*args, V.SCALE, workspace=ws)
        return out

    old = [(r, p) for r, c in enumerate(committed) for p in range(c)]
    x_old = V.randn_bf16(gen, len(old), 6 * HKV, 128, scale=1.5).cuda()
    drafts = [(r, c + i) for r, c in enumerate(committed) for i in range(width)]
    x_new = V.randn_bf16(gen, len(drafts), 6 * HKV, 128, scale=1.5).cuda()
    depth = [paths[r].index(i) if i in paths[r] else 0 for r in range(b) for i in range(width)]
    x_next = V.randn_bf16(gen, b, 6 * HKV, 128, scale=1.5).cuda()
    after = [c + len(p) for c, p in zip(committed, paths)]

    got = [zeros(), zeros()]
    feed(got, x_old, old, [p for _, p in old])
    feed(got, x_new, drafts, [committed[r] + depth[r * width + i] for r in range(b) for i in range(width)])
    acc = torch.zeros((b, max(map(len, paths))), dtype=torch.int32)
    for r, p in enumerate(paths):
        acc[r, :len(p)] = torch.tensor(p)
    pkv.kv_compact(pkv.KvPools([got[0]], [got[1]], kv_format), tables, i32([c + width for c in committed]), acc.cuda(),
                   i32([len(p) for p in paths]), width)
    want = [zeros(), zeros()]
    feed(want, x_old, old, [p for _, p in old])
    kept = [(r, j, i) for r, p in enumerate(paths) for j, i in enumerate(p)]
    feed(want, x_new[[r * width + i for r, _, i in kept]], [(r, committed[r] + j) for r, j, _ in kept],
         [committed[r] + j for r, j, _ in kept])

    def rows(pool, r):
        blk, off = torch.tensor([(slot(r, p) // 16, p % 16) for p in range(after[r])], device="cuda").T
        if fmt != "q8_0":
            return [pool[blk, :, off].contiguous().view(torch.int16 if fmt == "bf16" else torch.uint8)]
        return [part[blk, :, off] for part in (pool[..., :2048].unflatten(2, (16, 128)),
                                               pool[..., 2048:].unflatten(2, (16, 8)))]

    for r in range(b):
        for a, c in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(rows(a, r), rows(c, r))), r
    outs = [attend(p, feed(p, x_next, [(r, n) for r, n in enumerate(after)], after), [n + 1 for n in after])
            for p in (got, want)]
    assert torch.equal(*outs) and outs[0].any()


@pytest.mark.parametrize("power,eps", [(60, 0.0), (60, 1e-6), (-60, 0.0), (-60, 1e-38), (-60, 1e-6), (0, 0.0)])
def test_heads_at_the_ends_of_the_range(power, eps):
    """Heads whose largest values are 2^60 or 2^-60: their squares and the sum of 128 of them are FP32 values."""
    gen = torch.Generator().manual_seed(3)
    x = torch.randn((5, 6 * HKV, 128), generator=gen)
    x = (x / x.abs().amax(-1, keepdim=True) * 2.0 ** power).to(torch.bfloat16).cuda()
    w = [(1 + 0.2 * torch.randn(128, generator=gen)).to(torch.bfloat16).cuda() for _ in range(2)]
    k, v = (torch.zeros((1, HKV, 16, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q_out = torch.empty((5, 4 * HKV, 128), dtype=torch.bfloat16, device="cuda")
    pkv.qk_norm_rope_append(q_out, k, v, torch.arange(5, device="cuda"), x[:, :4 * HKV], x[:, 4 * HKV:5 * HKV],
                            x[:, 5 * HKV:], q_weight=w[0], k_weight=w[1], eps=eps)
    eps32 = float(np.float32(eps))
    for got, raw, gain in ((q_out, x[:, :4 * HKV], w[0]), (k[0, :, :5].transpose(0, 1), x[:, 4 * HKV:5 * HKV], w[1])):
        raw = raw.double()
        z = raw * torch.rsqrt(raw.square().mean(-1, keepdim=True) + eps32) * gain.double()
        # half a BF16 step; 128 squares, the root and three products in FP32 (less than 2^-16 of the value); and what
        # a square below FP32's normal numbers loses of the mean, 2^-150 against 2^-127 at least
        V.assert_within(got, z, 2.0 ** -8 * z.abs() + 2.0 ** -16 * z.abs(), f"2^{power}, eps {eps}")
    assert torch.equal(v[0, :, :5].transpose(0, 1), x[:, 5 * HKV:])

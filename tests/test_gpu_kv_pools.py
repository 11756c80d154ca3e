"""KvPools: the pools of a model's layers may be parts of one allocation, but
not parts that share memory (a row would be moved twice).  And the shapes in
which kv_compact takes its lengths."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import paged_kv_decode_attention_gb300 as pkv
else:  # collected on CPU-only machines, every test skipped
    pkv = None


def test_pools_that_overlap_are_refused():
    whole = torch.zeros((12, 2, 16, 128), dtype=torch.bfloat16, device="cuda")
    for k, v in (([whole[:4]], [whole[3:7]]), ([whole[:4], whole[8:]], [whole[4:8], whole[7:11]]),
                 ([whole[1:5]], [whole[:4]]), ([whole[:4]], [whole[:4]])):
        with pytest.raises(ValueError):
            pkv.KvPools(k, v)
    for shape, fmt in (((6, 2, 2176), pkv.KV_Q8_0), ((6, 2, 16, 128), pkv.KV_FP8_E4M3)):
        x = torch.zeros(shape, dtype=torch.uint8, device="cuda")
        pkv.KvPools([x[:3]], [x[3:]], fmt)
        with pytest.raises(ValueError):
            pkv.KvPools([x[:3]], [x[2:5]], fmt)


def test_pools_that_are_parts_of_one_allocation():
    pkv.get_device_error(reset=True)
    layers, hkv = 3, 2
    whole = torch.randn((layers, 2, 4, hkv, 16, 128), device="cuda").to(torch.bfloat16)
    want = whole.clone()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    pools = pkv.KvPools([whole[i, 0] for i in range(layers)], [whole[i, 1] for i in range(layers)])
    # positions 10 + (0 .. 7) are drafts in blocks 2 and 1; drafts 1, 3 and 7 are kept
    pkv.kv_compact(pools, i32([[2, 1]]), i32([18]), i32([[1, 3, 7]]), i32([3]), 8)
    place = lambda p: ([2, 1][p // 16], p % 16)
    for j, i in enumerate((1, 3, 7)):
        (db, do), (sb, so) = place(10 + j), place(10 + i)
        want[:, :, db, :, do] = want[:, :, sb, :, so]
    assert torch.equal(whole, want)
    assert pkv.get_device_error(reset=True) == 0


@pytest.mark.parametrize("shape", [(3,), (1, 3), (3, 1), (1, 3, 1)])
def test_lengths_of_any_shape_cover_every_request(shape):
    """One length per request is asked for, in whatever shape: the other calls take them so too."""
    pkv.get_device_error(reset=True)
    k, v = (torch.randn((3, 2, 16, 128), device="cuda").to(torch.bfloat16) for _ in range(2))
    want = [t.clone() for t in (k, v)]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    pkv.kv_compact(pkv.KvPools([k], [v]), i32([[2], [0], [1]]), i32([8, 9, 10]).view(shape), i32([[1, 4], [2, 3], [0, 3]]),
                   i32([2, 1, 2]).view(shape), 5, i32([5, 4, 5]).view(shape))
    for t in want:
        for blk, base, acc in ((2, 3, (1, 4)), (0, 5, (2,)), (1, 5, (0, 3))):
            for j, i in enumerate(acc):
                t[blk, :, base + j] = t[blk, :, base + i].clone()
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])
    assert pkv.get_device_error(reset=True) == 0

"""The split that the tree and window calls choose by themselves is the one
that their choose functions name: asking for it gives the same plan."""
import pytest
import torch

import paged_kv_decode_attention_gb300 as pkv
import verify_util as V


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (3, 2), (16, 16), (17, 33), (40, 5), (100, 64), (1 << 30, 4)])
def test_window_choice_is_its_own_plan(window, sinks):
    for max_blocks in list(range(1, 50)) + [100, 1000]:
        for seqs, heads, q_len in ((1, 1, 1), (1, 8, 1), (3, 8, 40), (1, 2, 64), (1, 1, 200), (40, 8, 5)):
            bps = pkv.choose_kv_blocks_per_split_window(seqs, heads, q_len, max_blocks, window, sinks)
            # one pass is named by max_blocks, and anything below is a split in whole tiles
            assert bps == max_blocks or (bps < max_blocks and bps % 4 == 0), (max_blocks, seqs, heads, q_len, bps)
            size = lambda b: pkv.workspace_size_window(seqs, q_len, 4 * heads, max_blocks, window, sinks, b)
            assert size(0) == size(bps)


def test_tree_choice_is_its_own_plan():
    for max_blocks in list(range(1, 50)) + [100, 1000, 8192]:
        for seqs, heads, width in ((1, 1, 1), (1, 8, 26), (3, 8, 40), (1, 2, 64), (1, 1, 200), (40, 8, 5)):
            bps = pkv.choose_kv_blocks_per_split_tree(seqs, heads, width, max_blocks)
            assert bps == max_blocks or (bps < max_blocks and bps % 4 == 0), (max_blocks, seqs, heads, width, bps)
            size = lambda b: pkv.workspace_size_tree(seqs, width, 4 * heads, max_blocks, b)
            assert size(0) == size(bps)


@pytest.mark.gpu
@pytest.mark.parametrize("q_len", [1, 40])
@pytest.mark.parametrize("max_blocks,window,sinks", [(1, 1, 1), (2, 3, 2), (4, 8, 17), (5, 8, 30), (8, 40, 20),
                                                     (60, 300, 40)])
def test_window_choice_gives_the_same_bits(q_len, max_blocks, window, sinks):
    pkv.get_device_error(reset=True)
    ctx = [max_blocks * 16 - 1, max_blocks * 16]
    d = {k: v.cuda() for k, v in V.paged_case(ctx, q_len, 1, 3, max_blocks=max_blocks).items()}
    ws = torch.empty(8 << 20, dtype=torch.uint8, device="cuda")
    outs = []
    for bps in (0, pkv.choose_kv_blocks_per_split_window(2, 1, q_len, max_blocks, window, sinks)):
        out = torch.empty_like(d["q"])
        pkv.paged_attention_window(out, d["q"], d["k_cache"], d["v_cache"], d["block_tables"], d["context_lens"], q_len,
                                   window, sinks, V.SCALE, kv_blocks_per_split=bps, workspace=ws)
        outs.append(out)
    assert torch.equal(*outs)
    ref, tol = V.attention64(d, V.window_allowed(ctx, q_len, window, sinks))
    V.assert_within(outs[0], ref, tol)
    assert pkv.get_device_error(reset=True) == 0

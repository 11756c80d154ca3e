"""E4M3 decode where one key holds most of a long row's weight."""
import pytest
import torch

from test_gpu_fp8_scaled import SCALE, _pkv, dev
from test_gpu_fp8_scaled_range import sink_case, sink_error

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("append", [False, True])
@pytest.mark.parametrize("requests", [1, 152])
@pytest.mark.parametrize("ctx,share,v_sink", [(2048, 0.9, 0.02), (8192, 0.9, 0.02), (32768, 0.5, 1.0), (32768, 0.9, 0.02),
                                              (131072, 0.5, 1.0), (131072, 0.99, 0.02)])
def test_most_of_the_weight_on_one_key(ctx, share, v_sink, requests, append):
    """Each weight is off by at most 2^-8 of itself, whatever the largest one is: of the row no more than that, and the
    result's rounding to BF16, 2^-8 of each value at most and evenly spread, 2^-8 / sqrt(3) of the row's norm."""
    pkv = _pkv()
    q, kc, vc, ks, vs, t = sink_case(requests, ctx, share, v_sink, 1)
    q = (q.float() * ks[0, 0]).to(torch.bfloat16)  # a power of two
    one = torch.ones_like(ks)
    blocks = pkv.choose_kv_blocks_per_split_fp8_e4m3(requests, 1, t.shape[1])
    size = max(pkv.workspace_size_q8_0(requests, 4, t.shape[1], blocks), 1)
    args = dict(kv_blocks_per_split=blocks, workspace=torch.empty(size, dtype=torch.uint8, device="cuda"))
    out = torch.full_like(q, 7.0)
    tables, lens = dev(t), dev([ctx] * requests)
    if append:  # the last token's row again, stored by the request whose table it is; the others store nothing
        slots = torch.full((requests,), -1, dtype=torch.int64, device="cuda")
        slots[0] = int(t[0][-1]) * 16 + 15
        new = [c[t[0][-1], :, 15].view(torch.float8_e4m3fn).to(torch.bfloat16).expand(requests, 1, 128).contiguous()
               for c in (kc, vc)]
        pkv.paged_attention_fp8_e4m3_append(out, q, kc, vc, tables, lens, SCALE, slots, *new, **args)
    else:
        pkv.paged_attention_fp8_e4m3(out, q, kc, vc, tables, lens, SCALE, **args)
    assert pkv.get_device_error() == 0
    assert sink_error((q, kc, vc, one, one, t), out, ctx) < 5e-3

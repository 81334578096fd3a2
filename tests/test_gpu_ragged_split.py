"""The split of ragged batches over the workers, call after call: every cut stream is merged, every call gives
the same bits."""
import pytest
import torch

from kv_cache_decode_kvc_gb300 import kvc

from ragged_util import Batch, attention64, check_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("dtype,D,math", [("f32", 64, 0), ("f32", 4, 0), ("bf16", 256, 0), ("bf16", 128, 1),
                                          ("bf16", 128, 0)])
@pytest.mark.parametrize("ctas", [0, 37])
def test_every_cut_stream_is_merged(dtype, D, math, ctas):
    # few streams of many tiles: nearly every worker ends in the middle of one and leaves it for the merge.  An
    # output that no merge wrote keeps its NaN; scratch starts as NaN too.
    bt = Batch([1, 2, 40], [4000, 2500, 900], 32, 4, 1, D, dtype, seed=31)
    c, d = bt.cache(kvc), bt.dev()
    c.set_ctas(ctas)
    c.set_math(math)
    ws = torch.full((c.attn_workspace_bytes(bt.rows),), 255, dtype=torch.uint8, device="cuda")
    outs = [torch.full((bt.rows, 4, D), float("nan"), dtype=bt.dtype, device="cuda") for _ in range(200)]
    for o in outs:
        c.attn_ragged(0, d["q"], o, d["table"], d["cu"], d["lens"], workspace=ws)
    assert c.last_error() == (kvc.KVC_OK, 0)
    check_attention(outs[0], bt, attention64(bt), dtype == "bf16" and D < 256 and math == 0)
    for o in outs[1:]:
        assert torch.equal(o, outs[0])


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f32", 64)])
@pytest.mark.parametrize("groups", [33, 100, 341])
def test_many_groups_call_after_call(dtype, D, groups):
    # more groups than a warp has lanes, of three sequences or an odd one: their bounds and prefixes are read by
    # other threads than those that fetched them, in every worker
    B = 3 * groups
    start = [3 * g - g % 2 for g in range(groups)] + [B]
    prefix = [16 * (1 + g % 4) for g in range(groups)]
    hist = [0] * B
    for g, (a, b) in enumerate(zip(start, start[1:])):
        for s in range(a, b):
            hist[s] = prefix[g] + (5 * s) % 23
    bt = Batch([s % 3 for s in range(B)], hist, 16, 2, 1, D, dtype, start, prefix, seed=32)
    c, d = bt.cache(kvc), bt.dev()
    ws = torch.full((c.attn_workspace_bytes(bt.rows, groups),), 255, dtype=torch.uint8, device="cuda")
    outs = [torch.full((bt.rows, 2, D), float("nan"), dtype=bt.dtype, device="cuda") for _ in range(100)]
    for o in outs:
        c.attn_shared(0, d["q"], o, d["table"], d["cu"], d["lens"], d["groups"], d["prefix"], workspace=ws)
    assert c.last_error() == (kvc.KVC_OK, 0)
    check_attention(outs[0], bt, attention64(bt), dtype == "bf16")
    for o in outs[1:]:
        assert torch.equal(o, outs[0])

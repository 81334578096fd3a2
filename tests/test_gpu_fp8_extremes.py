"""Attention over the paged cache held in 8 bits where scales, queries and values are at the ends of their ranges."""
import pytest
import torch

from fp8_util import Batch8, smallest_weights, values
from ragged_util import attention64, check_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc():
    import __graft_entry__
    __graft_entry__.build()
    from kv_cache_decode_kvc_gb300 import kvc
    return kvc


def attend(kvc, bt, shared=False, math=0):
    c, d = bt.cache(kvc), bt.dev()
    c.set_math(math)
    out = torch.full_like(d["q"], 7.0)
    a = (0, d["q"], out, d["table"], d["cu"], d["lens"])
    c.attn_shared(*a, d["groups"], d["prefix"]) if shared else c.attn_ragged(*a)
    assert c.last_error() == (kvc.KVC_OK, 0)
    assert (out[bt.n:] == 7).all()
    return out


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("size", [-40, -75, -100, -126])
@pytest.mark.parametrize("keys", ["zero", "never written", "zero beside others"])
@pytest.mark.parametrize("shared", [False, True])
def test_tiny_queries_before_zero_keys(kvc, D, size, keys, shared):
    # scores of 0 or next to it at every position that a row sees, none at the others of its last tile
    kw = dict(start=[0, 2, 4], prefix=[32, 0]) if shared else {}
    bt = Batch8([3, 1, 1, 9], [200, 77, 500, 0], 16, 8, 2, D, pad=1, **kw)
    bt.q = (bt.q.double() * 2.0 ** size).to(torch.bfloat16)
    some = slice(None, None, 2) if keys == "zero beside others" else slice(None)
    bt.K8[some] = 0
    bt.Ks[some] = 0.0 if keys == "never written" else 2.0 ** -64
    bt.K = values(bt.K8, bt.Ks)
    check_attention(attend(kvc, bt, shared), bt, attention64(bt), tensor_cores=True)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("math", [0, 1])
@pytest.mark.parametrize("value", [2.0 ** 60, 3e20, 5e37, 3e38])
@pytest.mark.parametrize("before", ["ordinary", "zero"])
def test_a_large_value_of_a_later_token(kvc, D, math, value, before):
    # token 1 begins a block, which token 0 does not see: in token 0's tile, and in a tile of its own
    for hist in ([15, 255], [143, 15]):
        bt = Batch8([6, 3], hist, 16, 8, 2, D, pad=1)
        bt.K *= 0.25
        if before == "zero":
            bt.V.zero_()
        for b in (0, 1):
            bt.V[int(bt.table[b, (hist[b] + 1) // 16]), 1, 0, 9] = value
        bt.requantize()
        out = attend(kvc, bt, math=math)
        ref, tol, A = attention64(bt)
        if math == 0:
            tol = tol + smallest_weights(bt)
        check_attention(out, bt, (ref, tol, A), tensor_cores=math == 0)
        assert before != "zero" or ((out[0] == 0).all() and (out[6] == 0).all())


@pytest.mark.parametrize("D", [64, 128])
def test_large_and_small_values_seen_together(kvc, D):
    # scales of V 2^140 and more apart in one sequence, the large ones first, last and in between; every weight finite
    for at in ([0], [18], [0, 9, 18]):
        bt = Batch8([2, 1], [300, 40], 16, 8, 2, D)
        bt.V *= 2.0 ** -50
        for j in at:
            bt.V[int(bt.table[0, j])] *= 2.0 ** 150
        bt.requantize()
        check_attention(attend(kvc, bt), bt, attention64(bt), tensor_cores=True)

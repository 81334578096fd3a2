"""Attention over the paged cache held in 8 bits where scales, queries and values are at the ends of their ranges."""
import pytest
import torch

from fp8_util import Batch8, values
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

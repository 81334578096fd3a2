"""Results of ragged attention over the plain paged cache, to the bit: a change of the split, of a kernel's order of sums or
of the merge that is not meant to change results leaves these as they are."""
import hashlib

import pytest
import torch

from ragged_util import Batch

pytestmark = pytest.mark.gpu

# first 16 digits of the outputs' SHA-256 by (dtype, D, CTAs at most)
WANT = {
    ("bf16", 128, 2): "c7f31726443ad5dc",
    ("bf16", 128, 5): "08cfd7f5475a518e",
    ("bf16", 128, 11): "a11d1708113a5362",
    ("bf16", 128, 24): "5cef28854b6321ba",
    ("bf16", 128, 60): "0e237fac7a9bf10f",
    ("bf16", 64, 2): "76e8c7deb4cbbfb2",
    ("bf16", 64, 5): "88bd32d96e62002a",
    ("bf16", 64, 11): "d8ef73eaf2f47cee",
    ("bf16", 64, 24): "ae243a5224c70c17",
    ("bf16", 64, 60): "173ceaa8aacab0ab",
    ("f32", 64, 2): "7cc295e438354cbe",
    ("f32", 64, 5): "5ac21e1668436dfa",
    ("f32", 64, 11): "b041bef49b2005ca",
    ("f32", 64, 24): "7afce33961b8ddc0",
    ("f32", 64, 60): "2f530e90160cfc07",
}


def digest(kvc, dtype, D, ctas):
    # few rows, 40 tokens and 200, streams in one piece, two, three, four and more (the fewer CTAs the fewer pieces)
    bt = Batch([1, 40, 200, 1, 2], [700, 1500, 300, 2500, 60], 32, 8, 2, D, dtype)
    g = torch.Generator().manual_seed(5)
    bt.q, bt.K, bt.V = (torch.randint(-64, 65, x.shape, generator=g).div(32).to(bt.dtype) for x in (bt.q, bt.K, bt.V))
    c, d = bt.cache(kvc), bt.dev()
    c.set_ctas(ctas)
    out = torch.zeros_like(d["q"])
    c.attn_ragged(0, d["q"], out, d["table"], d["cu"], d["lens"])
    assert c.last_error() == (kvc.KVC_OK, 0)
    return hashlib.sha256(out.cpu().view(torch.uint8).numpy().tobytes()).hexdigest()[:16]


CASES = [(dtype, D, ctas) for dtype, D in (("bf16", 128), ("bf16", 64), ("f32", 64)) for ctas in (2, 5, 11, 24, 60)]


@pytest.mark.parametrize("dtype,D,ctas", CASES)
def test_results_stay_what_they_were(dtype, D, ctas):
    import __graft_entry__
    __graft_entry__.build()
    from kv_cache_decode_kvc_gb300 import kvc
    assert digest(kvc, dtype, D, ctas) == WANT[dtype, D, ctas]

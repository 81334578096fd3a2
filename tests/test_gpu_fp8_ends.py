"""The 8-bit paged cache at the last positions a sequence can have, and calls whose rows are all padding: what is written, and
where nothing is."""
import pytest
import torch

from fp8_util import Cache64, quantize, values

pytestmark = pytest.mark.gpu

BS = 16
BLOCKS = 2 ** 27 - 1  # of one sequence, at most


@pytest.fixture(scope="module")
def kvc():
    import __graft_entry__
    __graft_entry__.build()
    from kv_cache_decode_kvc_gb300 import kvc
    return kvc


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Table:
    """The last block of the sequence is pool block 1, the others 0."""

    def __getitem__(self, j):
        return int(j == BLOCKS - 1)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("f32", 128)])
@pytest.mark.parametrize("short", [0, 3])
@pytest.mark.parametrize("n", [1, 5, 13])
@pytest.mark.parametrize("size", [0.25, 40.0])
def test_rows_at_the_last_positions(kvc, dtype, D, short, n, size):
    dt, top = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype], BS * BLOCKS - short
    g = torch.Generator().manual_seed(D + n)
    c, r = kvc.PagedFP8KVCache(1, 2, BS, 1, BLOCKS, 2, 2, D, dtype), Cache64(2, 2, BS, D)
    for x in "KV":
        r.codes[x], r.scales[x] = quantize(torch.randn(2, 2, BS, D, generator=g))
    for view, x in zip(c.layer_views(0), (r.codes["K"], r.codes["V"], r.scales["K"], r.scales["V"])):
        view.copy_(x)
    table = torch.zeros(1, BLOCKS, dtype=torch.int32, device="cuda")
    table[:, -1] = 1
    k, v = ((torch.randn(n, 2, D, generator=g) * size).to(dt) for _ in range(2))
    r.append(Table(), top - n, n, k, v)
    c.append_rope(0, None, None, k.cuda(), v.cuda(), table, i32([0, n]), i32([top]))
    assert c.last_error() == (kvc.KVC_OK, 0)
    for view, x in zip(c.layer_views(0), (r.codes["K"], r.codes["V"], r.scales["K"], r.scales["V"])):
        assert torch.equal(view.cpu(), x)
    m = min(n + 2, BS - short)  # read back with rows held before
    k_out, v_out = (torch.zeros(m, 2, D, dtype=dt, device="cuda") for _ in range(2))
    c.read(0, k_out, v_out, table, i32([0, m]), i32([top]))
    assert c.last_error() == (kvc.KVC_OK, 0)
    for out, x in ((k_out, "K"), (v_out, "V")):
        want = values(r.codes[x], r.scales[x])[1, :, BS - short - m:BS - short].transpose(0, 1)
        assert torch.equal(out.cpu().double(), want)


@pytest.mark.parametrize("N", [3, 1400])
@pytest.mark.parametrize("fp8,D,dtype", [(True, 128, "bf16"), (True, 64, "f32"), (False, 128, "bf16")])
def test_reading_padding_alone_writes_neither_output(kvc, N, fp8, D, dtype):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    c = (kvc.PagedFP8KVCache if fp8 else kvc.PagedKVCache)(1, 6, 16, 2, 3, 8, 2, D, dtype)
    for x in c.layer_views(0):
        x.fill_(3)
    table, cu, lens = torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3), i32([0, 0, 0]), i32([20, 0])
    k_out, v_out = (torch.full((N, 2, D), 7.0, dtype=dt, device="cuda") for _ in range(2))
    c.read(0, k_out, v_out, table, cu, lens)
    assert c.last_error() == (kvc.KVC_OK, 0)
    assert (k_out == 7).all() and (v_out == 7).all()

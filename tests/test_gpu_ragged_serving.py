"""Ragged attention and rotary append as a server runs them: many short sequences, many groups, layers
behind the first, caches past 32-bit offsets, graphs with scratch of their own, scratch used again."""
import pytest
import torch

from kv_cache_decode_kvc_gb300 import kvc

from ragged_util import Batch, attention64, check_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _call(c, bt, d, out, shared, **kw):
    if shared:
        c.attn_shared(0, d["q"], out, d["table"], d["cu"], d["lens"], d["groups"], d["prefix"], **kw)
    else:
        c.attn_ragged(0, d["q"], out, d["table"], d["cu"], d["lens"], **kw)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("f32", 64)])
@pytest.mark.parametrize("H_q,H_kv", [(8, 2), (32, 1), (4, 4)])
@pytest.mark.parametrize("ctas", [3, 0])
def test_many_short_streams(dtype, D, H_q, H_kv, ctas):
    # workers that take many streams of a tile or two each, of 1 to 70 rows a head in every order: a
    # stream's products must not touch the rows of the one before, call after call
    new = [(1, 2, 1, 17, 1, 1, 9, 1, 3, 0)[i % 10] for i in range(60)]
    hist = [(37 * i) % 250 for i in range(60)]
    bt = Batch(new, hist, 16, H_q, H_kv, D, dtype, pad=1, seed=21)
    c, d = bt.cache(kvc), bt.dev()
    c.set_ctas(ctas)
    ref = attention64(bt)
    outs = [torch.full((bt.rows, H_q, D), 7.0, dtype=bt.dtype, device="cuda") for _ in range(12)]
    for o in outs:
        _call(c, bt, d, o, False)
    assert c.last_error() == (kvc.KVC_OK, 0)
    check_attention(outs[0], bt, ref, dtype == "bf16")
    for o in outs[1:]:
        assert torch.equal(o, outs[0])


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f32", 64)])
@pytest.mark.parametrize("size", [1, 2, 3])
def test_as_many_groups_as_a_batch_has(dtype, D, size):
    # 1024 sequences, the most a cache takes, in groups of one (which share nothing) to three
    B = 1024
    start = sorted(set(range(0, B, size)) | {B})
    prefix = [16 * (g % 3) for g in range(len(start) - 1)]
    hist = [0] * B
    for g, (a, b) in enumerate(zip(start, start[1:])):
        for s in range(a, b):
            hist[s] = prefix[g] + s % 11
    bt = Batch([1] * B, hist, 16, 2, 1, D, dtype, start, prefix, seed=22)
    c, d = bt.cache(kvc), bt.dev()
    out = torch.zeros(bt.rows, 2, D, dtype=bt.dtype, device="cuda")
    _call(c, bt, d, out, True)
    assert c.last_error() == (kvc.KVC_OK, 0)
    check_attention(out, bt, attention64(bt), dtype == "bf16")


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("f32", 128)])
def test_later_layers(dtype, D):
    bt = Batch([3, 80, 1], [40, 0, 129], 32, 4, 2, D, dtype, seed=23)
    c, d = bt.cache(kvc, layers=3, layer=2), bt.dev()
    for l in (0, 1):
        for x in c.layer_views(l):
            x.fill_(float("nan"))
    out = torch.zeros(bt.rows, 4, D, dtype=bt.dtype, device="cuda")
    c.attn_ragged(2, d["q"], out, d["table"], d["cu"], d["lens"])
    check_attention(out, bt, attention64(bt), dtype == "bf16")
    # an append to layer 1 leaves the others as they are
    before = [x.clone() for x in c.layer_views(2)]
    c.append_rope(1, kvc.Rope([1.0, 0.5]), d["q"], d["k"], d["v"], d["table"], d["cu"], d["lens"])
    assert c.last_error() == (kvc.KVC_OK, 0)
    assert all(torch.equal(a, b) for a, b in zip(before, c.layer_views(2)))
    K, V = c.layer_views(1)
    row = bt.cu[1] + 79
    blk, at = int(bt.table[1, 79 // 32]), 79 % 32
    assert torch.equal(V[blk, :, at].cpu(), bt.v[row])
    assert torch.equal(K[blk, :, at, 4:].cpu(), bt.k[row, :, 4:])  # dimensions behind the rotated ones


@pytest.mark.parametrize("dtype,D,blocks", [("bf16", 128, 18000), ("f32", 64, 36000)])
def test_blocks_past_32_bit_offsets(dtype, D, blocks):
    # 128 rows x 8 heads a block: the pools hold more than 2^31 values, the sequences lie at both ends
    bt = Batch([5, 1, 90], [200, 300, 0], 128, 8, 8, D, dtype, [0, 2, 3], [128, 0], seed=24)
    c = kvc.PagedKVCache(1, blocks, 128, bt.B, bt.max_blocks, 8, 8, D, dtype)
    assert blocks * 8 * 128 * D > 2 ** 31
    far = torch.arange(bt.nblocks) % 2 == 0
    where = torch.where(far, blocks - 1 - torch.arange(bt.nblocks), torch.arange(bt.nblocks))
    d = bt.dev()
    d["table"] = where[bt.table.long()].to(torch.int32).cuda()
    K, V = c.layer_views(0)
    K[where.cuda()], V[where.cuda()] = bt.K.cuda(), bt.V.cuda()
    ref = attention64(bt)
    for shared in (False, True):
        out = torch.zeros(bt.rows, 8, D, dtype=bt.dtype, device="cuda")
        _call(c, bt, d, out, shared)
        assert c.last_error() == (kvc.KVC_OK, 0)
        check_attention(out, bt, ref, dtype == "bf16")
    c.append_rope(0, kvc.Rope([0.0]), d["q"], d["k"], d["v"], d["table"], d["cu"], d["lens"])
    for b, n in enumerate(bt.new):
        for i in (0, n - 1):
            t = bt.hist[b] + i
            blk = int(d["table"][b, t // 128])
            assert torch.equal(K[blk, :, t % 128].cpu(), bt.k[bt.cu[b] + i])
            assert torch.equal(V[blk, :, t % 128].cpu(), bt.v[bt.cu[b] + i])


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("f32", 64)])
@pytest.mark.parametrize("new", [[1], [3], [2, 1]])
@pytest.mark.parametrize("ctas", [0, 19, 600])
def test_few_long_sequences(dtype, D, new, ctas):
    # one KV head, a stream or two cut into a piece for every worker: merges of up to hundreds of pieces, of 32
    # to 96 rows
    bt = Batch(new, [20011, 9000][:len(new)], 64, 32, 1, D, dtype, seed=29)
    c, d = bt.cache(kvc), bt.dev()
    c.set_ctas(ctas)
    ref = attention64(bt)
    out = torch.zeros(bt.rows, 32, D, dtype=bt.dtype, device="cuda")
    _call(c, bt, d, out, False)
    assert c.last_error() == (kvc.KVC_OK, 0)
    check_attention(out, bt, ref, dtype == "bf16")
    out.zero_()
    _call(c, bt, d, out, True)  # one group of all, no prefix: merged row by row
    assert c.last_error() == (kvc.KVC_OK, 0)
    check_attention(out, bt, ref, dtype == "bf16")


def test_graphs_with_scratch_of_their_own_run_at_once():
    bt = Batch([1] * 30 + [40], [200 + 17 * i for i in range(31)], 32, 8, 2, 128, "bf16", [0, 31], [192], seed=25)
    c, d = bt.cache(kvc), bt.dev()
    ref = attention64(bt)
    outs = [torch.zeros(bt.rows, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ws = [torch.empty(c.attn_workspace_bytes(bt.rows, 1), dtype=torch.uint8, device="cuda") for _ in range(2)]
    for k in range(2):
        _call(c, bt, d, outs[k], k == 1, workspace=ws[k])
    torch.cuda.synchronize()
    graphs = []
    for k in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _call(c, bt, d, outs[k], k == 1, workspace=ws[k])
        graphs.append(g)
    want = []
    for k in range(2):
        outs[k].zero_()
        graphs[k].replay()
        torch.cuda.synchronize()
        want.append(outs[k].clone())
        check_attention(want[k], bt, ref, True)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                outs[k].zero_()
                graphs[k].replay()
        torch.cuda.synchronize()
        for k in range(2):
            assert torch.equal(outs[k], want[k])


def test_scratch_is_used_again_by_calls_of_other_kinds():
    # one workspace, large enough for every call, dirty from the call before: ragged and shared, both
    # kernels, other splits
    bt = Batch([4, 1, 70, 1], [300, 280, 256, 500], 32, 8, 2, 128, "bf16", [0, 3, 4], [256, 0], seed=26)
    c, d = bt.cache(kvc), bt.dev()
    ref = attention64(bt)
    need = []
    for math in (0, 1):
        c.set_math(math)
        need += [c.attn_workspace_bytes(bt.rows, 0), c.attn_workspace_bytes(bt.rows, 2)]
    ws = torch.full((max(need),), 255, dtype=torch.uint8, device="cuda")  # NaN in every float
    for math, ctas, shared in [(0, 0, True), (1, 0, False), (0, 5, False), (1, 7, True), (0, 1, True), (0, 0, False)]:
        c.set_math(math)
        c.set_ctas(ctas)
        out = torch.zeros(bt.rows, 8, 128, dtype=torch.bfloat16, device="cuda")
        _call(c, bt, d, out, shared, workspace=ws)
        assert c.last_error() == (kvc.KVC_OK, 0)
        check_attention(out, bt, ref, math == 0)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f32", 64)])
def test_a_block_named_twice(dtype, D):
    # sequences that name the same blocks without being told of it, and one that names a block twice
    bt = Batch([2, 2, 1], [60, 60, 90], 16, 4, 2, D, dtype, seed=27)
    bt.table[1] = bt.table[0]
    bt.table[2, 3] = bt.table[2, 1]
    c, d = bt.cache(kvc), bt.dev()
    ref = attention64(bt)
    for shared in (False, True):
        out = torch.zeros(bt.rows, 4, D, dtype=bt.dtype, device="cuda")
        _call(c, bt, d, out, shared)
        assert c.last_error() == (kvc.KVC_OK, 0)
        check_attention(out, bt, ref, dtype == "bf16")


@pytest.mark.parametrize("shared", [False, True])
def test_an_empty_batch_writes_nothing(shared):
    bt = Batch([0, 0, 0], [0, 5, 40], 16, 4, 2, 128, "bf16", [0, 3], [0], pad=3, seed=28)
    c, d = bt.cache(kvc), bt.dev()
    out = torch.full((3, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    _call(c, bt, d, out, shared)
    before = [x.clone() for x in c.layer_views(0)]
    c.append_rope(0, kvc.Rope([1.0]), d["q"], d["k"], d["v"], d["table"], d["cu"], d["lens"])
    assert c.last_error() == (kvc.KVC_OK, 0)
    assert (out == 7.0).all()
    assert all(torch.equal(a, b) for a, b in zip(before, c.layer_views(0)))


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("bf16", 256), ("f32", 64)])
def test_tensors_aligned_to_16_bytes_only(dtype, D):
    # base pointers 16 bytes past a multiple of 32 and row strides of an odd number of 16-byte pieces
    bt = Batch([3, 70, 1, 2], [100, 30, 400, 64], 16, 4, 2, D, dtype, [0, 2, 4], [16, 64], pad=2, seed=30)
    c, d = bt.cache(kvc), bt.dev()
    piece = 16 // bt.K.element_size()

    def odd(x=None, heads=4):
        row = heads * D + piece
        buf = torch.full((bt.rows * row + piece,), 7.0, dtype=bt.dtype, device="cuda")
        v = buf[piece:].view(bt.rows, row)[:, :heads * D].unflatten(1, (heads, D))
        assert v.data_ptr() % 32 == 16
        if x is not None:
            v.copy_(x)
        return v, buf

    ref = attention64(bt)
    for shared in (False, True):
        q, out, buf = odd(d["q"])[0], *odd()
        _call(c, bt, dict(d, q=q), out, shared)
        assert c.last_error() == (kvc.KVC_OK, 0)
        check_attention(out, bt, ref, dtype == "bf16" and D < 256)
        out.fill_(7.0)
        assert (buf == 7.0).all()  # nothing between the rows is written
    q, k, v = odd(d["q"])[0], odd(d["k"], 2)[0], odd(d["v"], 2)[0]
    rope = kvc.Rope([1.0, 0.25] * (D // 4))
    c.append_rope(0, rope, q, k, v, d["table"], d["cu"], d["lens"])
    got = [x.clone() for x in c.layer_views(0)]
    c.append_rope(0, rope, d["q"], d["k"], d["v"], d["table"], d["cu"], d["lens"])
    assert c.last_error() == (kvc.KVC_OK, 0)
    assert torch.equal(q[:bt.n], d["q"][:bt.n])
    assert all(torch.equal(a, b) for a, b in zip(got, c.layer_views(0)))

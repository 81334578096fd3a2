"""Attention of ragged new tokens over the paged cache held in 8 bits, against the definition in 64 bits."""
import pytest
import torch

from fp8_util import F8, Batch8
from ragged_util import attention64, check_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc():
    import __graft_entry__
    __graft_entry__.build()
    from kv_cache_decode_kvc_gb300 import kvc
    return kvc


def attend(kvc, bt, c=None, shared=False, ws=None, math=0, stream=None):
    c = c or bt.cache(kvc)
    c.set_math(math)
    d = bt.dev()
    out = torch.full_like(d["q"], 7.0)
    if shared:
        c.attn_shared(0, d["q"], out, d["table"], d["cu"], d["lens"], d["groups"], d["prefix"], workspace=ws)
    else:
        c.attn_ragged(0, d["q"], out, d["table"], d["cu"], d["lens"], workspace=ws)
    assert c.last_error() == (kvc.KVC_OK, 0)
    assert (out[bt.n:] == 7).all()
    return out


CASES = [
    # new, hist, bs, H_q, H_kv, D, dtype
    ([1, 1, 1], [0, 127, 300], 16, 32, 8, 128, "bf16"),       # the first token, whole tiles, a ragged end
    ([1, 1, 1, 1], [128, 129, 255, 6000], 64, 8, 1, 128, "bf16"),
    ([1, 2, 3, 5], [0, 1, 2, 700], 32, 32, 1, 128, "bf16"),   # 32 heads of one
    ([1], [9000], 128, 4, 4, 128, "bf16"),                    # split over the whole GPU
    ([17, 1, 64, 33], [5, 1000, 0, 130], 16, 8, 2, 128, "bf16"),
    ([300, 1, 129], [0, 50, 200], 256, 16, 2, 128, "bf16"),   # chunks beside a token
    ([0, 3, 0, 1], [5, 40, 0, 3], 16, 2, 2, 128, "bf16"),     # sequences without new tokens
    ([1, 4, 70], [100, 333, 12], 32, 4, 2, 64, "bf16"),
    ([1] * 40, list(range(0, 800, 20)), 16, 8, 8, 64, "bf16"),
    ([1, 9], [70, 20], 64, 4, 1, 256, "bf16"),
    ([1, 400, 2, 65, 64], [300, 100, 0, 60, 7], 32, 8, 2, 128, "bf16"),  # 260 and 256 rows a head: either side of a rule
    ([1, 400, 2, 65, 64], [300, 100, 0, 60, 7], 128, 8, 2, 64, "bf16"),
    ([0] * 150 + [140] + [0] * 49, [3] * 150 + [500] + [9] * 49, 64, 4, 2, 128, "bf16"),  # a chunk alone in a wide batch
    ([1, 6, 40], [200, 0, 77], 32, 4, 2, 64, "f32"),
    ([2, 1], [0, 130], 16, 2, 1, 128, "f32"),
]


@pytest.mark.parametrize("new,hist,bs,H_q,H_kv,D,dtype", CASES)
@pytest.mark.parametrize("math", [0, 1])
def test_against_64_bits(kvc, new, hist, bs, H_q, H_kv, D, dtype, math):
    bt = Batch8(new, hist, bs, H_q, H_kv, D, dtype, pad=2, q_scale=2.0, mag=3)
    out = attend(kvc, bt, math=math)
    check_attention(out, bt, attention64(bt), tensor_cores=dtype == "bf16" and math == 0)


@pytest.mark.parametrize("new,hist,start,prefix,bs,H_q,H_kv,D", [
    ([1] * 6, [300, 310, 290, 288, 700, 301], [0, 6], [288], 32, 32, 8, 128),
    ([1, 2, 1, 3], [200, 210, 64, 90], [0, 2, 4], [160, 64], 16, 8, 1, 128),
    ([1, 5, 1], [600, 513, 512], [0, 3], [512], 128, 32, 1, 64),
    ([40, 1, 1], [130, 129, 400], [0, 3], [128], 64, 8, 2, 128),
    # prefixes and sequences of more than 256 rows a head, in every combination with fewer
    ([1] * 80 + [70, 1], [300 + i for i in range(80)] + [70, 90], [0, 80, 82], [272, 64], 16, 8, 2, 128),
    ([1] * 80 + [70, 1, 1], [300 + i for i in range(80)] + [70, 90, 3], [0, 80, 82, 83], [256, 0, 0], 32, 8, 2, 64),
    ([3, 1, 2, 1, 1, 4], [2050, 2048, 3000, 2200, 2300, 2064], [0, 6], [2048], 64, 32, 1, 128),
])
@pytest.mark.parametrize("math", [0, 1])
def test_shared_prefixes(kvc, new, hist, start, prefix, bs, H_q, H_kv, D, math):
    bt = Batch8(new, hist, bs, H_q, H_kv, D, start=start, prefix=prefix, pad=1, q_scale=2.0, mag=2)
    out = attend(kvc, bt, shared=True, math=math)
    check_attention(out, bt, attention64(bt), tensor_cores=math == 0)


def test_scales_far_apart(kvc):
    # blocks of one sequence whose scales are 2^80 apart: values near 2^40 beside 2^-40, equal weights
    bt = Batch8([1, 1], [400, 90], 16, 8, 2, 128, q_scale=0.5)
    g = torch.Generator().manual_seed(1)
    f = torch.exp2(torch.randint(-40, 41, (bt.nblocks, 2), generator=g).double())[..., None, None]
    bt.V = bt.V * f
    bt.requantize()
    check_attention(attend(kvc, bt), bt, attention64(bt), tensor_cores=True)


def test_peaked_rows(kvc):
    # one key far above the rest, first in the last tile, then in the first; and rows of equal scores
    for at in (0, 130, 517):
        bt = Batch8([1, 2], [517, 40], 32, 8, 2, 128, q_scale=1.0)
        e, o = int(bt.table[0, at // 32]), at % 32
        bt.K[e, :, o] = bt.q[0, ::4].double() * 8
        bt.q[1:] = 0
        bt.requantize()
        check_attention(attend(kvc, bt), bt, attention64(bt), tensor_cores=True)


@pytest.mark.parametrize("D,new,hist", [(128, [1, 3, 9], [200, 130, 5]), (64, [1, 3, 40], [200, 130, 5]),
                                        (128, [80, 1], [10, 127])])
def test_values_that_no_row_sees_do_not_matter(kvc, D, new, hist):
    # NaN codes, and NaN or infinite scales, in blocks and slots behind the sequences' ends
    bt = Batch8(new, hist, 16, 8, 2, D)
    good = attend(kvc, bt)
    seen = bt.seen()
    for x in (bt.K8, bt.V8):
        x[~seen[:, None].expand(-1, 2, -1)] = 0x7F
    unused = ~seen.any(1)
    bt.Ks[unused] = float("nan")
    bt.Vs[unused] = float("inf")
    assert torch.equal(attend(kvc, bt), good)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("i", [1, 2])  # (the second token of a pair in memory, and the first)
def test_nan_codes_reach_the_rows_that_see_them_and_no_others(kvc, D, i):
    t, d = 125 + i, 9  # new token i's value in dimension 9 of KV head 1

    def batch():
        return Batch8([6, 1], [125, 300], 16, 8, 2, D)
    bt = batch()
    good = attend(kvc, bt).cpu()
    bt.V8[int(bt.table[0, t // 16]), 1, t % 16, d] = 0x7F
    out = attend(kvc, bt).cpu()
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[i:6, 4:, d] = True
    assert torch.isnan(out[hit]).all() and torch.equal(out[~hit], good[~hit])
    bt = batch()
    bt.K8[int(bt.table[0, t // 16]), 1, t % 16, d] = 0xFF
    out = attend(kvc, bt).cpu()
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[i:6, 4:] = True
    assert torch.isnan(out[hit]).all() and torch.equal(out[~hit], good[~hit])


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_a_query_that_is_not_finite_spoils_its_own_row(kvc, value):
    bt = Batch8([2, 1], [125, 300], 16, 8, 2, 128)
    good = attend(kvc, bt).cpu()
    bt.q[1, 3, 5] = value
    out = attend(kvc, bt).cpu()
    assert torch.isnan(out[1, 3]).all()
    out[1, 3] = good[1, 3]
    assert torch.equal(out, good)


def test_large_and_small_queries_in_one_tile(kvc):
    bt = Batch8([4], [500], 16, 8, 1, 128)
    bt.q *= torch.exp2(torch.arange(8.0) * 2 - 12).to(torch.bfloat16)[None, :, None]
    check_attention(attend(kvc, bt), bt, attention64(bt), tensor_cores=True)


def test_views_strides_and_scratch(kvc):
    bt = Batch8([1, 20, 3], [200, 0, 64], 32, 8, 2, 128)
    good = attend(kvc, bt)
    c, d = bt.cache(kvc), bt.dev()
    wide = torch.zeros(bt.rows, 24, 128, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:16] = d["q"]
    out = torch.zeros(bt.rows, 16, 128, dtype=torch.bfloat16, device="cuda")
    n = c.attn_workspace_bytes(bt.rows)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")  # scratch as the last user left it
    c.attn_ragged(0, wide[:, 8:16], out[:, 8:], d["table"], d["cu"], d["lens"], workspace=ws)
    assert torch.equal(out[:, 8:], good) and (out[:, :8] == 0).all()
    with pytest.raises(kvc.KvcError):
        c.attn_ragged(0, wide[:, 8:16], out[:, 8:], d["table"], d["cu"], d["lens"], workspace=ws[:256])


def test_device_errors(kvc):
    bt = Batch8([1, 2, 1], [40, 30, 20], 16, 8, 2, 128)
    good = attend(kvc, bt)

    def call(**edit):
        c, d = bt.cache(kvc), bt.dev()
        for k, (i, x) in edit.items():
            d[k][i] = x
        out = torch.full_like(d["q"], 7.0)
        c.attn_ragged(0, d["q"], out, d["table"], d["cu"], d["lens"])
        return out, c.last_error()[1]
    for L in (1, 10 ** 6):
        out, bits = call(lens=(1, L))
        assert bits == kvc.KVC_DEV_BAD_LENS and (out[1:3] == 0).all()
        assert torch.equal(out[0], good[0]) and torch.equal(out[3], good[3])
    for e in (-1, 10 ** 6):
        out, bits = call(table=((2, 1), e))
        assert bits == kvc.KVC_DEV_BAD_BLOCK and torch.equal(out[:3], good[:3])
    for i, x in ((1, 4), (0, 1), (3, 5), (1, -1)):
        out, bits = call(cu=(i, x))
        assert bits == kvc.KVC_DEV_BAD_SEQ and (out == 7).all()


@pytest.mark.parametrize("new", [[1, 1, 1], [1, 60, 1]])
def test_graph_and_two_streams(kvc, new):
    # a captured call replayed on other lengths, and two calls at once with scratch of their own
    bt = Batch8(new, [300, 20, 129], 16, 8, 2, 128)
    c, d = bt.cache(kvc), bt.dev()
    out = torch.zeros_like(d["q"])
    ws = torch.empty(c.attn_workspace_bytes(bt.rows), dtype=torch.uint8, device="cuda")
    c.attn_ragged(0, d["q"], out, d["table"], d["cu"], d["lens"], workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.attn_ragged(0, d["q"], out, d["table"], d["cu"], d["lens"], workspace=ws)
    for hist in ([300, 20, 129], [17, 0, 280]):
        b2 = Batch8(new, [300, 20, 129], 16, 8, 2, 128)
        b2.hist, b2.lens = hist, [a + b for a, b in zip(new, hist)]
        d["lens"].copy_(torch.tensor(b2.lens, dtype=torch.int32))
        out.zero_()
        graph.replay()
        check_attention(out, b2, attention64(b2), tensor_cores=True)
    want = out.clone()
    outs = [torch.zeros_like(out) for _ in range(2)]
    wss = [torch.empty_like(ws) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, o, w in zip(streams, outs, wss):
            with torch.cuda.stream(s):
                c.attn_ragged(0, d["q"], o, d["table"], d["cu"], d["lens"], workspace=w)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_calls_repeat_bit_for_bit(kvc):
    bt = Batch8([1, 30, 1, 2], [3000, 100, 0, 700], 64, 32, 8, 128, q_scale=2.0)
    c = bt.cache(kvc)
    a = attend(kvc, bt, c)
    assert all(torch.equal(a, attend(kvc, bt, c)) for _ in range(3))


def test_a_serving_step(kvc):
    """Prompts, then single tokens: append with norms and rotation, attention, reading back; the keys and
    values that attention sees are those that are read back."""
    B, bs, H_q, H_kv, D = 3, 16, 8, 2, 128
    c = kvc.PagedFP8KVCache(2, 60, bs, B, 20, H_q, H_kv, D)
    g = torch.Generator().manual_seed(2)
    table = torch.randperm(60, generator=g).view(B, 20).to(torch.int32).cuda()
    rope = kvc.Rope([10000.0 ** (-i / 64) for i in range(64)])
    w = (1 + 0.2 * torch.randn(D, generator=g)).to(torch.bfloat16).cuda()
    lens = [0, 0, 0]
    for new in ([100, 33, 16], [1, 1, 1], [1, 0, 1], [4, 1, 64]):
        n = sum(new)
        lens = [a + b for a, b in zip(lens, new)]
        cu = torch.tensor([0, new[0], new[0] + new[1], n], dtype=torch.int32, device="cuda")
        ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
        for layer in range(2):
            q, k, v = (torch.randn(n, h, D, generator=g).to(torch.bfloat16).cuda() for h in (H_q, H_kv, H_kv))
            out = torch.empty_like(q)
            c.append_rope(layer, rope, q, k, v, table, cu, ln, q_norm=w, k_norm=w)
            c.attn_ragged(layer, q, out, table, cu, ln)
            # all positions back, and the definition over them
            full = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device="cuda")
            ks, vs = (torch.empty(sum(lens), H_kv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
            c.read(layer, ks, vs, table, full, ln)
            r = p = 0
            for b in range(B):
                for i in range(new[b]):
                    m = lens[b] - new[b] + i + 1
                    s = torch.einsum("hgd,thd->hgt", q[r].double().view(H_kv, 4, D), ks[p:p + m].double()) / D ** 0.5
                    o = torch.einsum("hgt,thd->hgd", s.softmax(-1), vs[p:p + m].double()).reshape(H_q, D)
                    a = torch.einsum("hgt,thd->hgd", s.softmax(-1), vs[p:p + m].double().abs()).reshape(H_q, D)
                    assert ((out[r].double() - o).abs() <= 2.0 ** -8 * o.abs() + 2.0 ** -7 * a).all()
                    r += 1
                p += lens[b]
    assert c.last_error() == (kvc.KVC_OK, 0)

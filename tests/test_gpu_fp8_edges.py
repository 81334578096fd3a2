"""The paged cache held in 8 bits at its edges: long and strided appends, positions of several axes, blocks never
written, wide batches, many KV heads, splits over few and many CTAs, the last positions a cache takes."""
import math

import pytest
import torch

from fp8_util import F8, Batch8, Cache64, quantize, turned, values
from ragged_util import HALF_STEP, attention64, check_attention

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def kvc():
    import __graft_entry__
    __graft_entry__.build()
    from kv_cache_decode_kvc_gb300 import kvc
    return kvc


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def near(codes, scales, exact, err):
    """Codes are the nearest to the exact values, `err` (absolute) aside."""
    s = scales.double()[..., None, None].clamp(min=2.0 ** -64)
    c, x = codes.view(F8).double(), exact / s
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))) / 8
    return ((c - x).abs() <= step / 2 * (1 + 2.0 ** -20) + err / s).all()


@pytest.mark.parametrize("dtype,new,H_q,H_kv", [("bf16", [900, 0, 500], 8, 2), ("f32", [700, 600], 4, 4), ("bf16", [5, 3], 8, 2)])
def test_fused_rows_rotated_in_place_along_three_axes(kvc, dtype, new, H_q, H_kv):
    # q, k, v side by side in one tensor, q rotated where it lies and read by the next call on the stream at once
    D, bs, n = 128, 64, sum(new)
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    g = torch.Generator().manual_seed(n)
    x = torch.randn(n + 3, (H_q + 2 * H_kv), D, generator=g).to(dt)
    w = [(1 + 0.3 * torch.randn(D, generator=g)).to(dt) for _ in range(2)]
    freq = [10000.0 ** (-i / 64) for i in range(64)]
    axis = [i % 3 for i in range(64)]
    pos = torch.randint(0, 100000, (3, n + 3), generator=g, dtype=torch.int32)
    hist = [7 * (b + 1) if T else 0 for b, T in enumerate(new)]
    mb = -(-(max(new) + 40) // bs)
    table = torch.randperm(len(new) * mb, generator=g).view(len(new), mb).to(torch.int32)
    cu = [0]
    for T in new:
        cu.append(cu[-1] + T)
    c = kvc.PagedFP8KVCache(2, len(new) * mb, bs, len(new), mb, H_q, H_kv, D, dtype)
    y = x.cuda()
    q, k, v = y[:, :H_q], y[:, H_q:H_q + H_kv], y[:, H_q + H_kv:]
    c.append_rope(1, kvc.Rope(freq, axis=axis), q, k, v, table.cuda(), i32(cu), i32([a + b for a, b in zip(hist, new)]),
                  positions=pos.cuda(), q_norm=w[0].cuda(), k_norm=w[1].cuda(), norm_eps=EPS)
    got = q.clone()
    assert c.last_error() == (kvc.KVC_OK, 0)
    p = pos[:, :n].T.double()
    ref, tol = turned(x[:n, :H_q], w[0], EPS, p, freq, False, axis)
    assert ((got[:n].cpu().double() - ref).abs() <= tol + HALF_STEP[dt] * (ref.abs() + tol)).all()
    assert torch.equal(y[n:].cpu(), x[n:]) and torch.equal(y[:, H_q:].cpu(), x[:, H_q:])
    kk, ktol = turned(x[:n, H_q:H_q + H_kv], w[1], EPS, p, freq, False, axis)
    r = Cache64(len(new) * mb, H_kv, bs, D)
    exact, err = torch.zeros(r.exact["K"].shape, dtype=torch.float64), torch.zeros(r.exact["K"].shape, dtype=torch.float64)
    for b, T in enumerate(new):
        if T:
            s = slice(cu[b], cu[b + 1])
            # blocks start with zeros of scale 0 before the new rows
            r.append(table[b], hist[b], T, kk[s], x[:n, H_q + H_kv:][s].double())
            t = torch.arange(hist[b], hist[b] + T)
            at = table[b, t // bs].long(), slice(None), t % bs
            exact[at], err[at] = kk[s], ktol[s]
    K, V, Ks, Vs = (a.cpu() for a in c.layer_views(1))
    assert torch.equal(V, r.codes["V"]) and torch.equal(Ks, r.scales["K"]) and torch.equal(Vs, r.scales["V"])
    assert near(K, Ks, exact, err)
    assert all((a == 0).all() for a in c.layer_views(0))


def test_axes_that_share_a_row_of_positions(kvc):
    n, D = 40, 128
    g = torch.Generator().manual_seed(2)
    freq, axis = [10000.0 ** (-i / 64) for i in range(64)], [i % 2 for i in range(64)]
    row = torch.randint(0, 5000, (n,), generator=g, dtype=torch.int32).cuda()
    k, v = (torch.randn(n, 2, D, generator=g).bfloat16().cuda() for _ in range(2))
    table = torch.arange(2, dtype=torch.int32, device="cuda").view(1, 2)
    views = []
    for positions in (row.expand(2, n), row.repeat(2, 1)):
        c = kvc.PagedFP8KVCache(1, 2, 32, 1, 2, 8, 2, D)
        c.append_rope(0, kvc.Rope(freq, axis=axis), None, k, v, table, i32([0, n]), i32([n]), positions=positions)
        assert c.last_error() == (kvc.KVC_OK, 0)
        views.append(c.layer_views(0))
    assert all(torch.equal(a, b) for a, b in zip(*views))


@pytest.mark.parametrize("new", [[1, 1, 1], [900, 1, 600]])  # (queries in the keys' launch, or in one of their own beside it)
def test_steps_captured_and_side_by_side(kvc, new):
    # append and attention in one graph, replayed on other lengths, rows and positions; then two layers on two streams at
    # once: all as one call after the other
    D, H_q, H_kv, bs, mb, n = 128, 8, 2, 32, 64, sum(new)
    g = torch.Generator().manual_seed(n)
    table = torch.randperm(3 * mb, generator=g).view(3, mb).to(torch.int32).cuda()
    rope = kvc.Rope([10000.0 ** (-i / 64) for i in range(64)])
    cu = i32([0] + [sum(new[:b + 1]) for b in range(3)])
    w = [(1 + 0.3 * torch.randn(D, generator=g)).bfloat16().cuda() for _ in range(2)]

    def rows():
        return [torch.randn(n, h, D, generator=g).bfloat16().cuda() for h in (H_q, H_kv, H_kv)]

    def step(c, layer, x, out, lens, ws, stream=None):
        c.append_rope(layer, rope, x[0], x[1], x[2], table, cu, lens, q_norm=w[0], k_norm=w[1], norm_eps=EPS, stream=stream)
        c.attn_ragged(layer, x[0], out, table, cu, lens, workspace=ws, stream=stream)

    steps = [(rows(), i32([h + T for h, T in zip(hist, new)])) for hist in ([0, 0, 0], [900, 40, 600], [100, 1, 33])]
    want, views = [], []
    c = kvc.PagedFP8KVCache(2, 3 * mb, bs, 3, mb, H_q, H_kv, D)
    ws = torch.empty(c.attn_workspace_bytes(n), dtype=torch.uint8, device="cuda")
    for x, lens in steps:
        out = torch.zeros(n, H_q, D, dtype=torch.bfloat16, device="cuda")
        step(c, 0, [t.clone() for t in x], out, lens, ws)
        torch.cuda.synchronize()
        want.append(out)
    views = [t.clone() for t in c.layer_views(0)]
    assert c.last_error() == (kvc.KVC_OK, 0)

    c = kvc.PagedFP8KVCache(2, 3 * mb, bs, 3, mb, H_q, H_kv, D)
    x, lens, out = [t.clone() for t in steps[0][0]], steps[0][1].clone(), torch.zeros_like(want[0])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(c, 0, x, out, lens, ws)
    for (rows_, lens_), o in zip(steps, want):
        for t, r in zip(x, rows_):
            t.copy_(r)
        lens.copy_(lens_)
        graph.replay()
        assert torch.equal(out, o)
    assert all(torch.equal(a, b) for a, b in zip(c.layer_views(0), views))

    c = kvc.PagedFP8KVCache(2, 3 * mb, bs, 3, mb, H_q, H_kv, D)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs, wss = [torch.zeros_like(out) for _ in range(2)], [torch.empty_like(ws) for _ in range(2)]
    for (rows_, lens_), o in zip(steps, want):
        xs = [[t.clone() for t in rows_] for _ in range(2)]
        torch.cuda.synchronize()
        for layer, s in enumerate(streams):
            step(c, layer, xs[layer], outs[layer], lens_, wss[layer], stream=s)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], o) and torch.equal(outs[1], o)
    for layer in range(2):
        assert all(torch.equal(a, b) for a, b in zip(c.layer_views(layer), views))
    assert c.last_error() == (kvc.KVC_OK, 0)


def attend(kvc, bt, shared=False, ctas=None, math=0):
    c, d = bt.cache(kvc), bt.dev()
    c.set_math(math)
    if ctas:
        c.set_ctas(ctas)
    out = torch.full_like(d["q"], 7.0)
    a = (0, d["q"], out, d["table"], d["cu"], d["lens"])
    c.attn_shared(*a, d["groups"], d["prefix"]) if shared else c.attn_ragged(*a)
    assert c.last_error() == (kvc.KVC_OK, 0)
    assert (out[bt.n:] == 7).all()
    return out


@pytest.mark.parametrize("D", [64, 128])
def test_blocks_never_written(kvc, D):
    # a new cache is zeros with scales of zero: keys and values 0
    bt = Batch8([1, 5, 80], [300, 70, 200], 32, 8, 2, D, pad=1)
    for x in (bt.K8, bt.V8, bt.Ks, bt.Vs):
        x[::2] = 0
    bt.K, bt.V = values(bt.K8, bt.Ks), values(bt.V8, bt.Vs)
    check_attention(attend(kvc, bt), bt, attention64(bt), tensor_cores=True)


@pytest.mark.parametrize("ctas", [1, 5, 600])
@pytest.mark.parametrize("D,shared", [(128, False), (64, False), (128, True)])
def test_splits_over_few_and_many_ctas(kvc, ctas, D, shared):
    new, hist = [1, 2, 90, 1], [900, 200, 170, 0]
    kw = dict(start=[0, 2, 4], prefix=[160, 0]) if shared else {}
    bt = Batch8(new, hist, 32, 8, 2, D, pad=1, **kw)
    out = attend(kvc, bt, shared, ctas)
    check_attention(out, bt, attention64(bt), tensor_cores=True)


MIXES = [  # new, H_q, H_kv, D: which rows are attended on codes and which on widened blocks depends on D and on their mean
    ([1] * 11 + [140], 8, 2, 128),            # one chunk beside single tokens
    ([1] * 11 + [140], 8, 2, 64),
    ([1] * 11 + [140], 8, 1, 64),             # (more rows to a token)
    ([1, 2, 3, 5, 4, 5, 1, 1, 5], 32, 1, 64),  # drafts, all of them
    ([1, 2, 3, 5, 4, 5, 1, 1, 5], 32, 1, 128),
    ([7, 8, 9, 8, 1, 9, 8], 32, 1, 128),
    ([40, 60, 0, 50, 33], 4, 1, 128),
    ([40, 60, 0, 50, 33], 4, 1, 64),
]


def with_room(bt, blocks):
    """The batch in a cache whose sequences may grow to that many blocks (what is widened depends on it)."""
    bt.table = torch.cat([bt.table, torch.full((bt.B, blocks - bt.max_blocks), -1, dtype=torch.int32)], 1)
    bt.max_blocks = blocks
    return bt


@pytest.mark.parametrize("new,H_q,H_kv,D", MIXES)
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("blocks", [64, 1 << 16])
def test_rows_on_codes_beside_widened_blocks(kvc, new, H_q, H_kv, D, shared, blocks):
    hist = [(211 * i) % 300 + 40 for i in range(len(new))]
    kw = dict(start=[0, 2, len(new)], prefix=[40, 32]) if shared else {}
    bt = with_room(Batch8(new, hist, 16, H_q, H_kv, D, pad=3, mag=2, **kw), blocks)
    check_attention(attend(kvc, bt, shared), bt, attention64(bt), tensor_cores=True)


@pytest.mark.parametrize("math", [0, 1])
@pytest.mark.parametrize("D", [64, 128])
def test_many_kv_heads(kvc, D, math):
    bt = Batch8([1, 9, 70], [130, 0, 33], 16, 64, 64, D, pad=1)
    check_attention(attend(kvc, bt, math=math), bt, attention64(bt), tensor_cores=math == 0)


@pytest.mark.parametrize("shared", [False, True])
def test_wide_batches(kvc, shared):
    # chunks far apart in a batch of 700 slots, most of them empty or with a token
    new = [i % 3 == 0 for i in range(700)]
    new = [int(x) for x in new]
    new[5], new[300], new[699] = 150, 80, 140
    hist = [(37 * i) % 90 for i in range(700)]
    kw = {}
    if shared:
        start = list(range(0, 701, 2))
        prefix = [min(hist[a:a + 2]) for a in start[:-1]]
        kw = dict(start=start, prefix=prefix)
    bt = Batch8(new, hist, 16, 4, 1, 64, pad=2, **kw)
    check_attention(attend(kvc, bt, shared), bt, attention64(bt), tensor_cores=True)


@pytest.mark.parametrize("new,hist,start,prefix,bs,H_q,H_kv,D", [
    ([300, 1, 129], [0, 50, 200], None, None, 256, 16, 2, 128),
    ([1, 400, 2, 65, 64], [300, 100, 0, 60, 7], None, None, 32, 8, 2, 128),   # a rule's either side: 260 and 256 rows
    ([1, 400, 2, 65, 64], [300, 100, 0, 60, 7], None, None, 128, 8, 2, 64),
    ([0, 600, 0, 0], [5, 0, 90, 0], None, None, 16, 2, 1, 128),
    ([2] * 90 + [300], [70] * 90 + [3], None, None, 16, 4, 2, 128),
    # prefixes and sequences of many rows, in every combination with few
    ([300, 2, 1], [200, 180, 150], [0, 2, 3], [128, 64], 32, 8, 2, 128),
    ([30] * 12, [97] * 12, [0, 12], [96], 32, 4, 2, 64),
    ([400, 500], [300, 280], [0, 1, 2], [256, 0], 64, 4, 2, 64),
    ([1] * 300, [50 + i % 7 for i in range(300)], [0, 150, 300], [48, 32], 16, 4, 2, 128),
])
@pytest.mark.parametrize("ctas", [None, 7])
def test_widened_entries(kvc, new, hist, start, prefix, bs, H_q, H_kv, D, ctas):
    kw = dict(start=start, prefix=prefix) if start else {}
    bt = with_room(Batch8(new, hist, bs, H_q, H_kv, D, pad=2, mag=2, q_scale=1.5, **kw), (1 << 21) // bs)
    c = bt.cache(kvc)
    assert c.attn_workspace_bytes(bt.rows, len(start) - 1 if start else 0) > 2 * 2 * bt.K8.numel()  # (two pools in bf16)
    out = attend(kvc, bt, start is not None, ctas)
    check_attention(out, bt, attention64(bt), tensor_cores=True)


def test_math_modes(kvc):
    for dtype, D, tensor in (("bf16", 128, True), ("bf16", 64, True), ("bf16", 256, False), ("f32", 128, False)):
        c = kvc.PagedFP8KVCache(1, 2, 16, 1, 2, 8, 2, D, dtype)
        assert c.math() == (3 if tensor else 1)
        before = c.attn_workspace_bytes(1)
        c.set_math(1)
        assert c.math() == 1
        # two widened pools more on CUDA cores, whose scratch the other call is refused without
        assert c.attn_workspace_bytes(1) >= 2 * 2 * 2 * 16 * D
        for bad in (2, 4) if tensor else (2, 3, 4):
            with pytest.raises(kvc.KvcError):
                c.set_math(bad)
        c.set_math(3 if tensor else 0)
        assert c.attn_workspace_bytes(1) == before


@pytest.mark.parametrize("blocks", [8, 1 << 16])
def test_scratch_grows_with_rows_and_groups(kvc, blocks):
    c = kvc.PagedFP8KVCache(1, 8, 16, 6, blocks, 8, 2, 128)
    for groups in (0, 1, 6):
        sizes = [c.attn_workspace_bytes(n, groups) for n in (1, 6, 64, 128, 129, 130, 134, 135, 500)]
        assert sizes == sorted(sizes)
    assert c.attn_workspace_bytes(64, 0) <= c.attn_workspace_bytes(64, 1) <= c.attn_workspace_bytes(64, 6)


BS = 16
BLOCKS = 2 ** 27 - 1  # of one sequence, at most


# The test looks for positions lost or read from elsewhere: the last block holds half of a row's weight.  Sums this long
# are allowed what a worker's can lose.  A tile of up to 32 rows sees all 2^31 positions; with n such tiles 304 CTAs share
# n 2^31 of them (D = 64 with 32 rows: 152, of twice the positions a product), so n 220,753 products of 32 positions lie one after the
# other in a sum, each off by up to 2^-23 of it (added and cut off), and n 55,189 additions (2^-24) in a thread's
# denominator; the weights' rounding and the rest are below 2 %.
def tolerance(rows):
    n = -(-rows // 32)
    return n * (220753 * 2.0 ** -23 + 55189 * 2.0 ** -24) + 0.02


@pytest.mark.parametrize("D,H_q,new", [(128, 1, 3), (64, 1, 3), (128, 4, 17), (64, 1, 40)])
@pytest.mark.parametrize("short", [0, 3])
def test_the_last_positions(kvc, D, H_q, new, short):
    TOP = BS * BLOCKS
    g = torch.Generator().manual_seed(D)
    u = torch.nn.functional.normalize(torch.randn(D, generator=g, dtype=torch.float64), dim=0)
    a = math.sqrt(math.log(2.0 ** 31) * math.sqrt(D))  # a^2 / sqrt(D) = log of the number of positions
    q = (a * u + 0.1 * torch.randn(new, H_q, D, generator=g)).bfloat16()
    K = torch.randn(2, 1, BS, D, generator=g).double()
    K[0] -= (K[0] @ u)[..., None] * u  # block 0: scores near 0
    K[1] = a * u + 0.1 * torch.randn(1, BS, D, generator=g)
    K8, Ks = quantize(K)
    V8, Vs = quantize(torch.randn(2, 1, BS, D, generator=g))
    K, V = values(K8, Ks), values(V8, Vs)
    V8[1, :, BS - short:] = 0x7F  # NaN behind the last position
    c = kvc.PagedFP8KVCache(1, 2, BS, 1, BLOCKS, H_q, 1, D)
    for view, x in zip(c.layer_views(0), (K8, V8, Ks, Vs)):
        view.copy_(x)
    out, A = torch.zeros(new, H_q, D, dtype=torch.float64), torch.zeros(new, H_q, D, dtype=torch.float64)
    for i in range(new):
        n = TOP - short - new + i + 1  # positions the token sees
        times = [(min(n, TOP - BS) - j + BS - 1) // BS for j in range(BS)] + [1] * max(0, n - (TOP - BS))
        k, v = torch.cat([K[0, 0], K[1, 0]])[:len(times)], torch.cat([V[0, 0], V[1, 0]])[:len(times)]
        w = torch.softmax(q[i].double() @ k.T / math.sqrt(D) + torch.tensor(times, dtype=torch.float64).log(), -1)
        out[i], A[i] = w @ v, w @ v.abs()
    table = torch.zeros(1, BLOCKS, dtype=torch.int32, device="cuda")
    table[:, -1] = 1
    got = torch.full((new, H_q, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    c.attn_ragged(0, q.cuda(), got, table, i32([0, new]), i32([TOP - short]))
    assert c.last_error() == (kvc.KVC_OK, 0)
    err = (got.cpu().double() - out).abs()
    assert (err <= tolerance(new * H_q) * A).all(), float((err / A).max())
    # and read back and appended to there
    k_out, v_out = (torch.zeros(new, 1, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    n = min(new, BS - short)
    c.read(0, k_out[:n], v_out[:n], table, i32([0, n]), i32([TOP - short]))
    assert torch.equal(k_out[:n, 0].cpu(), K[1, 0, BS - short - n:BS - short].bfloat16())
    before = [x.clone() for x in c.layer_views(0)]
    x = torch.randn(new, 1, D, device="cuda").bfloat16()
    c.append_rope(0, None, None, x[:n], x[:n], table, i32([0, n]), i32([TOP - short]))
    assert c.last_error() == (kvc.KVC_OK, 0)
    for y, old in zip(c.layer_views(0), before):
        assert torch.equal(y[0], old[0])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("shared", [False, True])
def test_more_work_than_a_call_takes_is_refused(kvc, D, shared):
    # one token of 64 KV heads at the last position: 64 x 2^24 tiles of 128 keys (2^23 of 256), 4 units each
    heads = 64 if D == 128 else 128
    c = kvc.PagedFP8KVCache(1, 2, BS, 1, BLOCKS, heads, heads, D)
    table, q = torch.zeros(1, BLOCKS, dtype=torch.int32, device="cuda"), torch.randn(1, heads, D, device="cuda").bfloat16()
    out = torch.full_like(q, 7.0)
    ws = torch.full((c.attn_workspace_bytes(1, 1),), 255, dtype=torch.uint8, device="cuda")
    a = (0, q, out, table, i32([0, 1]), i32([BS * BLOCKS]))
    c.attn_shared(*a, i32([0, 1]), i32([BS]), workspace=ws) if shared else c.attn_ragged(*a, workspace=ws)
    assert c.last_error() == (kvc.KVC_EDEVICE, kvc.KVC_DEV_TOO_LARGE)
    assert (out == 7.0).all()


@pytest.mark.parametrize("N", [3, 1400])
@pytest.mark.parametrize("D,dtype", [(128, "bf16"), (64, "bf16"), (128, "f32")])
def test_a_batch_of_padding_alone(kvc, N, D, dtype):
    # no sequence has a new token: every call returns, and leaves all as it was
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    c = kvc.PagedFP8KVCache(1, 6, 16, 2, 3, 8, 2, D, dtype)
    for x in c.layer_views(0):
        x.fill_(3)
    table, cu, lens = torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3), i32([0, 0, 0]), i32([20, 0])
    q, k = torch.randn(N, 8, D, device="cuda").to(dt), torch.randn(N, 2, D, device="cuda").to(dt)
    w = torch.ones(D, dtype=dt, device="cuda")
    out, k_out = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    c.append_rope(0, kvc.Rope([1.0] * (D // 2)), q, k, k, table, cu, lens, q_out=out, q_norm=w, k_norm=w)
    c.read(0, k_out, k_out.clone(), table, cu, lens)
    c.attn_ragged(0, q, out, table, cu, lens)
    c.attn_shared(0, q, out, table, cu, lens, i32([0, 2]), i32([0]))
    assert c.last_error() == (kvc.KVC_OK, 0)
    assert (out == 7).all() and (k_out == 7).all() and all((x == 3).all() for x in c.layer_views(0))

"""Attention of ragged new tokens over a paged cache (kvc_paged_attn_ragged, kvc_paged_attn_shared)
against the definition in 64 bits: dtypes, head counts, block sizes, odd lengths, single tokens,
every kind of split; values in unseen places; what is left untouched; what is flagged; streams,
graphs, and the run of append, chunk attention and shared decode together."""
import pytest
import torch

from kv_cache_decode_kvc_gb300 import kvc

from ragged_util import Batch, attention64, check_attention, rotate64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _tc(bt, math):
    return bt.name == "bf16" and bt.D in (64, 128) and math != 1


def _run(bt, shared=False, ctas=0, math=0, c=None, q=None, out=None):
    c = bt.cache(kvc) if c is None else c
    d = bt.dev()
    c.set_ctas(ctas)
    if math == 1:
        c.set_math(1)
    q = d["q"] if q is None else q
    out = torch.full((bt.rows, bt.H_q, bt.D), 7.0, dtype=bt.dtype, device="cuda") if out is None else out
    if shared:
        c.attn_shared(0, q, out, d["table"], d["cu"], d["lens"], d["groups"], d["prefix"])
    else:
        c.attn_ragged(0, q, out, d["table"], d["cu"], d["lens"])
    assert c.last_error() == (kvc.KVC_OK, 0)
    assert (out[bt.n:] == 7.0).all()  # padding
    return out


PATHS = [("bf16", 128, 0), ("bf16", 64, 0), ("bf16", 128, 1), ("bf16", 256, 0), ("f32", 128, 0), ("f32", 64, 0),
         ("f32", 4, 0), ("f32", 256, 0)]


@pytest.mark.parametrize("dtype,D,math", PATHS)
@pytest.mark.parametrize("H_q,H_kv", [(2, 2), (8, 2), (32, 1)])
@pytest.mark.parametrize("bs", [16, 128, 256])
def test_ragged_matches_64_bits(dtype, D, math, H_q, H_kv, bs):
    bt = Batch([1, 0, 37, 1, 130, 5], [0, 9, 0, 300, 61, 255], bs, H_q, H_kv, D, dtype, pad=2, seed=D + bs)
    check_attention(_run(bt, math=math), bt, attention64(bt), _tc(bt, math))


@pytest.mark.parametrize("dtype,D,math", [("bf16", 128, 0), ("bf16", 64, 0), ("f32", 64, 0)])
@pytest.mark.parametrize("ctas", [1, 2, 7, 40, 152, 600])
def test_ragged_any_split(dtype, D, math, ctas):
    # streams of one row tile and of several, cut into pieces of one tile up to none at all
    bt = Batch([300, 1, 2, 0, 64], [500, 900, 0, 3, 127], 32, 8, 2, D, dtype, seed=ctas)
    check_attention(_run(bt, ctas=ctas, math=math), bt, attention64(bt), _tc(bt, math))


@pytest.mark.parametrize("n,hist", [(1, 0), (1, 1), (1, 127), (1, 128), (1, 129), (2, 126), (64, 64), (65, 63),
                                    (127, 0), (128, 0), (129, 0), (257, 0), (255, 1)])
@pytest.mark.parametrize("G", [1, 4])
def test_ragged_tile_edges(n, hist, G):
    bt = Batch([n], [hist], 16, G, 1, 128, seed=n)
    check_attention(_run(bt), bt, attention64(bt), True)


@pytest.mark.parametrize("G", [1, 2, 4, 8, 16, 32])
@pytest.mark.parametrize("bs", [16, 32, 64, 128, 256])
def test_ragged_groups_and_blocks(G, bs):
    bt = Batch([1, 20, 3], [700, 200, 0], bs, 2 * G, 2, 128, seed=G + bs)
    check_attention(_run(bt), bt, attention64(bt), True)


SHARED = [
    # new, hist, start, prefix
    ([1] * 6, [256, 300, 256, 411, 700, 257], [0, 6], [256]),
    ([1] * 40, [160 + 7 * i for i in range(40)], [0, 40], [160]),              # more than 128 rows at G = 4
    ([1, 0, 5, 2, 1, 0, 1], [100, 130, 97, 64, 200, 64, 31], [0, 3, 5, 7], [96, 64, 0]),  # groups, odd prefixes
    ([1, 2, 1], [300, 290, 300], [0, 1, 1, 3], [300, 5, 290]),                 # a group of one, an empty group
    ([130, 3, 70], [515, 520, 512], [0, 3], [512]),                            # prompts behind a prefix
    ([0, 0, 1, 1], [64, 64, 20, 30], [0, 2, 4], [64, 16]),                     # a group without new tokens
    ([1, 1], [15, 14], [0, 2], [14]),                                          # a prefix below one block
]


@pytest.mark.parametrize("dtype,D,math", [("bf16", 128, 0), ("bf16", 64, 0), ("bf16", 128, 1), ("f32", 64, 0),
                                          ("bf16", 256, 0)])
@pytest.mark.parametrize("case", range(len(SHARED)))
@pytest.mark.parametrize("ctas", [0, 1, 13])
def test_shared_matches_64_bits(dtype, D, math, case, ctas):
    new, hist, start, prefix = SHARED[case]
    bt = Batch(new, hist, 16, 8, 2, D, dtype, start, prefix, pad=1, seed=case)
    check_attention(_run(bt, True, ctas, math), bt, attention64(bt), _tc(bt, math))


@pytest.mark.parametrize("G,bs", [(1, 32), (16, 64), (32, 256), (2, 128)])
def test_shared_groups_and_blocks(G, bs):
    bt = Batch([1, 3, 1, 1, 2], [600, 520, 512, 900, 513], bs, 2 * G, 2, 128, "bf16", [0, 3, 5], [512, 513], seed=G)
    check_attention(_run(bt, True), bt, attention64(bt), True)


@pytest.mark.parametrize("dtype,D,math", [("bf16", 128, 0), ("bf16", 64, 0), ("f32", 64, 0), ("f32", 4, 0)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("shared", [False, True])
def test_unseen_values_do_not_leak(dtype, D, math, value, shared):
    # every row of the pool that no sequence holds: the ends of last blocks, other blocks
    bt = Batch([1, 40, 3], [77, 70, 64], 32, 4, 2, D, dtype, [0, 3], [64], seed=11)
    ref = attention64(bt)
    bt.K, bt.V = bt.K.clone(), bt.V.clone()
    hidden = ~bt.seen()
    for x in (bt.K, bt.V):
        x.transpose(1, 2)[hidden] = value
    check_attention(_run(bt, shared, math=math), bt, ref, _tc(bt, math))


@pytest.mark.parametrize("dtype,D,math", [("bf16", 128, 0), ("bf16", 64, 0), ("f32", 64, 0)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("ctas", [0, 1])
def test_later_tokens_values_do_not_leak(dtype, D, math, value, ctas):
    # a value that is not finite at position `at` reaches exactly the rows at or behind it
    new, hist, at, dim = 200, 60, 153, 5
    bt = Batch([new], [hist], 32, 4, 2, D, dtype, seed=12)
    ref = attention64(bt)
    bt.V = bt.V.clone()
    bt.V[bt.table[0, at // 32].long(), 1, at % 32, dim] = value
    got = _run(bt, ctas=ctas, math=math)
    before = torch.arange(at - hist)
    check_attention(got, bt, ref, _tc(bt, math), before)
    g = got.cpu()[at - hist:].float()
    want = torch.full_like(g[:, 2:, dim], value)
    assert torch.equal(g[:, 2:, dim].nan_to_num(nan=9e9), want.nan_to_num(nan=9e9))
    g[:, 2:, dim] = 0
    assert g.isfinite().all()
    # and a key that is not finite
    bt.V = Batch([new], [hist], 32, 4, 2, D, dtype, seed=12).V
    bt.K = bt.K.clone()
    bt.K[bt.table[0, at // 32].long(), 1, at % 32, dim] = float("nan")
    got = _run(bt, ctas=ctas, math=math)
    check_attention(got, bt, ref, _tc(bt, math), before)
    assert got[at - hist:, 2:].isnan().all() and got[:, :2].isfinite().all()


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_scores_that_rise_fall_and_jump(dtype, D):
    # histories whose maximum moves (the running maximum is raised again and again), and large scores
    for kind in range(4):
        bt = Batch([50, 1], [400, 900], 32, 4, 2, D, dtype, seed=20 + kind, q_scale=4.0 if kind == 3 else 1.0)
        if kind < 3:
            u = torch.randn(bt.H_kv, D, generator=torch.Generator().manual_seed(1))
            u = u / u.norm(dim=-1, keepdim=True)
            for b, L in enumerate(bt.lens):
                t = torch.arange(L)
                tau = (0.05 * t, 45 - 0.05 * t, 12.0 * ((t // 97) % 5))[kind]
                at = bt.table[b, t // 32].long(), t % 32
                K = bt.K[at[0], :, at[1]].float() + (tau * D ** 0.5)[:, None, None] * u
                bt.K[at[0], :, at[1]] = K.to(bt.dtype)
            bt.q = (0.3 * bt.q.float() + u.repeat_interleave(2, 0)).to(bt.dtype)
        check_attention(_run(bt), bt, attention64(bt), _tc(bt, 0))


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f32", 64)])
@pytest.mark.parametrize("shared", [False, True])
def test_invalid_lengths_give_zero_rows(dtype, D, shared):
    bt = Batch([2, 3, 1, 4], [64, 70, 80, 64], 16, 4, 2, D, dtype, [0, 4], [64], seed=6)
    ref = attention64(bt)
    for bad in (2, -1, 2 ** 31 - 1, bt.max_blocks * 16 + 1) + ((66,) if shared else ()):
        c, d = bt.cache(kvc), bt.dev()
        d["lens"][1] = bad
        out = torch.full((bt.rows, 4, D), 7.0, dtype=bt.dtype, device="cuda")
        if shared:
            c.attn_shared(0, d["q"], out, d["table"], d["cu"], d["lens"], d["groups"], d["prefix"])
        else:
            c.attn_ragged(0, d["q"], out, d["table"], d["cu"], d["lens"])
        assert c.last_error() == (kvc.KVC_EDEVICE, kvc.KVC_DEV_BAD_LENS)
        assert not out[2:5].any()
        check_attention(out, bt, ref, _tc(bt, 0), [0, 1, 5, 6, 7, 8, 9])


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f32", 64)])
def test_bad_arrays_write_nothing(dtype, D):
    bt = Batch([2, 3, 1], [64, 70, 80], 16, 4, 2, D, dtype, [0, 2, 3], [64, 16], seed=7)
    for name, vals in [("cu", [1, 2, 5, 6]), ("cu", [0, 3, 2, 6]), ("cu", [0, 2, 5, 7]), ("cu", [0, -1, 5, 6]),
                       ("groups", [0, 2, 2]), ("groups", [1, 2, 3]), ("groups", [0, 4, 3]), ("groups", [0, -1, 3])]:
        c, d = bt.cache(kvc), bt.dev()
        d[name].copy_(torch.tensor(vals, dtype=torch.int32))
        out = torch.full((bt.rows, 4, D), 7.0, dtype=bt.dtype, device="cuda")
        ws = torch.full((c.attn_workspace_bytes(bt.rows, 2),), 255, dtype=torch.uint8, device="cuda")
        c.attn_shared(0, d["q"], out, d["table"], d["cu"], d["lens"], d["groups"], d["prefix"], workspace=ws)
        assert c.last_error() == (kvc.KVC_EDEVICE, kvc.KVC_DEV_BAD_SEQ), (name, vals)
        assert (out == 7.0).all()
        if name == "cu":
            c.attn_ragged(0, d["q"], out, d["table"], d["cu"], d["lens"], workspace=ws)
            assert c.last_error() == (kvc.KVC_EDEVICE, kvc.KVC_DEV_BAD_SEQ), (name, vals)
            assert (out == 7.0).all()


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_bad_blocks_and_prefixes_are_flagged(dtype, D):
    bt = Batch([2, 3, 1], [64, 70, 80], 16, 4, 2, D, dtype, [0, 2, 3], [64, 16], seed=8)
    ref = attention64(bt)
    for bad in (-1, bt.nblocks, 2 ** 31 - 1):
        c, d = bt.cache(kvc), bt.dev()
        d["table"][2, 3] = bad
        out = torch.full((bt.rows, 4, D), 7.0, dtype=bt.dtype, device="cuda")
        c.attn_ragged(0, d["q"], out, d["table"], d["cu"], d["lens"])
        assert c.last_error() == (kvc.KVC_EDEVICE, kvc.KVC_DEV_BAD_BLOCK)
        check_attention(out, bt, ref, _tc(bt, 0), range(5))
    for bad in (-1, bt.max_blocks * 16 + 1, 2 ** 31 - 1):
        c, d = bt.cache(kvc), bt.dev()
        d["prefix"][0] = bad
        out = torch.full((bt.rows, 4, D), 7.0, dtype=bt.dtype, device="cuda")
        c.attn_shared(0, d["q"], out, d["table"], d["cu"], d["lens"], d["groups"], d["prefix"])
        assert c.last_error() == (kvc.KVC_EDEVICE, kvc.KVC_DEV_BAD_LENS)
        assert not out[:5].any()
        check_attention(out, bt, ref, _tc(bt, 0), [5])


def test_strided_queries_and_outputs():
    bt = Batch([3, 60, 1], [100, 0, 33], 16, 4, 2, 128, pad=2, seed=9)
    q = torch.randn(bt.rows, 5, 4, 128).to(torch.bfloat16).cuda()
    q[:, 1] = bt.q.cuda()
    out = torch.full((bt.rows, 3, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    got = _run(bt, q=q[:, 1], out=out[:, 2])
    check_attention(got, bt, attention64(bt), True)
    assert (out[:, :2] == 7.0).all()


def test_results_are_reproducible_and_streams_do_not_disturb_each_other():
    bt = Batch([1] * 20 + [90], [300 + 31 * i for i in range(21)], 32, 8, 2, 128, "bf16", [0, 21], [288], seed=10)
    c, d = bt.cache(kvc), bt.dev()
    first = [_run(bt, False, c=c), _run(bt, True, c=c)]
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[torch.zeros_like(first[0]) for _ in range(8)] for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(8):  # the two calls at once, each with scratch of its own
        c.attn_ragged(0, d["q"], outs[0][i], d["table"], d["cu"], d["lens"], stream=s[0])
        c.attn_shared(0, d["q"], outs[1][i], d["table"], d["cu"], d["lens"], d["groups"], d["prefix"], stream=s[1])
    torch.cuda.synchronize()
    for k in range(2):
        for o in outs[k]:
            assert torch.equal(o, first[k])


def test_captured_calls_follow_the_arrays():
    # a graph of append, ragged and shared attention, replayed with other lengths, tables and groups
    a = Batch([1, 5, 2, 1], [200, 100, 128, 140], 16, 8, 2, 128, "bf16", [0, 2, 4], [96, 128], pad=3, seed=13)
    b = Batch([2, 1, 0, 9], [60, 48, 51, 300], 16, 8, 2, 128, "bf16", [0, 3, 4], [48, 0], pad=0, seed=14)
    T = max(a.max_blocks, b.max_blocks)
    c = kvc.PagedKVCache(1, 200, 16, 4, T, 8, 2, 128)
    Kv, Vv = c.layer_views(0)
    freq = [10000.0 ** (-i / 64) for i in range(64)]
    rope = kvc.Rope(freq)
    N = 12
    assert a.rows == b.rows == N
    live = {k: torch.zeros_like(v) for k, v in a.dev().items()}
    live["table"] = torch.zeros(4, T, dtype=torch.int32, device="cuda")
    qr, o1, o2 = (torch.zeros(N, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    ws = torch.empty(c.attn_workspace_bytes(N, 2), dtype=torch.uint8, device="cuda")

    def load(bt):
        for k, v in bt.dev().items():
            (live[k][:, :bt.max_blocks] if k == "table" else live[k]).copy_(v)
        Kv[:bt.nblocks].copy_(bt.K)
        Vv[:bt.nblocks].copy_(bt.V)

    def step():
        c.append_rope(0, rope, live["q"], live["k"], live["v"], live["table"], live["cu"], live["lens"], qr)
        c.attn_ragged(0, qr, o1, live["table"], live["cu"], live["lens"], workspace=ws)
        c.attn_shared(0, qr, o2, live["table"], live["cu"], live["lens"], live["groups"], live["prefix"], workspace=ws)

    load(a)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for bt in (b, a, b):
        load(bt)
        graph.replay()
        assert c.last_error() == (kvc.KVC_OK, 0)
        ref = attention64(bt, qr.cpu(), Kv[:bt.nblocks].cpu(), Vv[:bt.nblocks].cpu())
        check_attention(o1, bt, ref, True)
        check_attention(o2, bt, ref, True)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f32", 64)])
def test_prompt_in_chunks_then_shared_decode(dtype, D):
    """A prompt taken in as ragged chunks, then decode steps of sequences sharing it: each step is
    append_rope, then attention; compared with the whole history in 64 bits, and the decode step with
    the cache's own single-token attention."""
    bs, H_q, H_kv, S = 16, 8, 2, 4
    g = torch.Generator().manual_seed(15)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    freq = [10000.0 ** (-2 * i / D) for i in range(D // 2)]
    rope = kvc.Rope(freq)
    prompt, max_blocks = 150, 20
    c = kvc.PagedKVCache(1, 100, bs, S, max_blocks, H_q, H_kv, D, dtype)
    table = torch.randperm(100, generator=g)[:S * max_blocks].view(S, max_blocks).to(torch.int32)
    x = {n: torch.randn(400, h, D, generator=g).to(dt) for n, h in (("q", H_q), ("k", H_kv), ("v", H_kv))}

    def step(new, hist, rows, tab, shared=None):
        bt = Batch(new, hist, bs, H_q, H_kv, D, dtype, seed=0)
        bt.table, i32 = tab, dict(dtype=torch.int32, device="cuda")
        d = {n: t[rows].cuda() for n, t in x.items()}
        cu, lens, tb = torch.tensor(bt.cu, **i32), torch.tensor(bt.lens, **i32), tab.cuda()
        c.append_rope(0, rope, d["q"], d["k"], d["v"], tb, cu, lens)
        out = torch.empty_like(d["q"])
        if shared is None:
            c.attn_ragged(0, d["q"], out, tb, cu, lens)
        else:
            c.attn_shared(0, d["q"], out, tb, cu, lens, torch.tensor([0, S], **i32), torch.tensor([shared], **i32))
        assert c.last_error() == (kvc.KVC_OK, 0)
        K, V = (t.cpu() for t in c.layer_views(0))
        check_attention(out, bt, attention64(bt, d["q"].cpu(), K, V), _tc(bt, 0))
        # the rotated rows are what a 64-bit rotation gives, so positions ran on from chunk to chunk
        pos = torch.cat([torch.arange(h, h + n) for n, h in zip(new, hist)])[:, None]
        y, _ = rotate64(x["q"][rows], pos, freq, [0] * (D // 2), False)
        assert (d["q"].cpu().double() - y).abs().max() <= (0.04 if dtype == "bf16" else 1e-4)
        return d["q"], out, tb, lens

    at, h = 0, 0
    for n in (64, 1, 85):  # sequence 0 takes the prompt in
        step([n, 0, 0, 0], [h, 0, 0, 0], torch.arange(at, at + n), table)
        at, h = at + n, h + n
    # the others share its whole blocks and copy the last, partial one
    whole = prompt // bs
    shared_table = table.clone()
    shared_table[1:, :whole] = table[0, :whole]
    K, V = c.layer_views(0)
    for s in range(1, S):
        K[int(table[s, whole])] = K[int(table[0, whole])]
        V[int(table[s, whole])] = V[int(table[0, whole])]
    hist = [prompt] * S
    for i in range(3):
        new = [1, 1, 1, 1] if i != 1 else [2, 1, 3, 0]
        n = sum(new)
        q, out, tb, lens = step(new, hist, torch.arange(at, at + n), shared_table, shared=prompt)
        hist = [a + b for a, b in zip(hist, new)]
        at += n
        if n == S:  # one token each: the cache's own decode attention on the same state
            ref = torch.empty_like(out)
            c.decode_attn(0, q, ref, tb, lens)
            assert c.last_error() == (kvc.KVC_OK, 0)
            assert (out.float() - ref.float()).abs().max() <= (0.03 if dtype == "bf16" else 2e-5)


def test_refusals_on_the_host():
    bt = Batch([2, 1], [20, 3], 16, 4, 2, 64, seed=1)
    c, d = bt.cache(kvc), bt.dev()
    h, L = c.h, kvc.load()
    out, ws = torch.zeros_like(d["q"]), torch.empty(c.attn_workspace_bytes(3, 2), dtype=torch.uint8, device="cuda")
    P = {k: v.data_ptr() for k, v in d.items()}
    rope = kvc.Rope([1.0] * 32)

    def ragged(layer=0, q=P["q"], qs=256, o=out.data_ptr(), os_=256, t=P["table"], cu=P["cu"], lens=P["lens"], n=3,
               w=ws.data_ptr(), nb=ws.numel(), handle=h):
        return L.kvc_paged_attn_ragged(handle, layer, q, qs, o, os_, t, cu, lens, n, w, nb, None)

    def shared(ng=2, gr=P["groups"], pf=P["prefix"], nb=ws.numel()):
        return L.kvc_paged_attn_shared(h, 0, P["q"], 256, out.data_ptr(), 256, P["table"], P["cu"], P["lens"], 3, gr, pf,
                                       ng, ws.data_ptr(), nb, None)

    def append(layer=0, r=rope.r, q=P["q"], qs=256, qo=P["q"], qos=256, k=P["k"], ks=128, v=P["v"], vs=128, pos=None,
               ps=0, n=3, handle=h):
        return L.kvc_paged_append_rope(handle, layer, r, q, qs, qo, qos, k, ks, v, vs, pos, ps, P["table"], P["cu"],
                                       P["lens"], n, None)

    need = c.attn_workspace_bytes(3)
    for kw in (dict(layer=1), dict(layer=-1), dict(q=None), dict(q=P["q"] + 2), dict(qs=252), dict(qs=255), dict(qs=260),
               dict(o=None), dict(o=out.data_ptr() + 8), dict(os_=0), dict(t=None), dict(cu=None), dict(lens=None),
               dict(cu=P["cu"] + 2), dict(n=0), dict(n=-1), dict(w=None), dict(w=ws.data_ptr() + 16), dict(nb=need - 1)):
        assert ragged(**kw) == kvc.KVC_EINVAL, kw
    for kw in (dict(ng=0), dict(ng=3), dict(gr=None), dict(pf=None), dict(gr=P["groups"] + 1), dict(nb=need)):
        assert shared(**kw) == kvc.KVC_EINVAL, kw
    wide = kvc.Rope([1.0] * 33)
    two = kvc.Rope([1.0] * 32, axis=[0, 1] * 16)
    for kw in (dict(layer=1), dict(r=None), dict(r=wide.r), dict(q=None), dict(qo=None), dict(qos=264), dict(qs=200),
               dict(k=None), dict(k=P["k"] + 2), dict(ks=120), dict(vs=129), dict(n=0), dict(pos=P["lens"] + 1),
               dict(r=two.r, pos=P["lens"], ps=2)):
        assert append(**kw) == kvc.KVC_EINVAL, kw
    plain = kvc.KVCache(1, 2, 4, 2, 64, 32)
    assert ragged(handle=plain.h) == kvc.KVC_EINVAL and append(handle=plain.h) == kvc.KVC_EINVAL
    import ctypes
    n = ctypes.c_uint64()
    for args in ((plain.h, 3, 0), (h, 0, 0), (h, 3, -1), (h, 3, 3)):
        assert L.kvc_paged_attn_workspace(*args, ctypes.byref(n)) == kvc.KVC_EINVAL
    assert c.last_error() == (kvc.KVC_OK, 0)
    with pytest.raises(ValueError):
        c.attn_ragged(0, d["q"].transpose(1, 2), out, d["table"], d["cu"], d["lens"])
    with pytest.raises(ValueError):
        c.attn_ragged(0, d["q"].float(), out, d["table"], d["cu"], d["lens"])
    with pytest.raises(ValueError):
        c.attn_ragged(0, d["q"], out[:2], d["table"], d["cu"], d["lens"])
    with pytest.raises(ValueError):
        c.attn_ragged(0, d["q"], out, d["table"], d["cu"].long(), d["lens"])
    with pytest.raises(ValueError):
        c.append_rope(0, rope, d["q"], d["k"], d["v"][:2], d["table"], d["cu"], d["lens"])
    with pytest.raises(ValueError):
        c.append_rope(0, rope, d["q"], d["k"], d["v"], d["table"], d["cu"], d["lens"],
                      positions=torch.zeros(2, 3, dtype=torch.int32, device="cuda"))

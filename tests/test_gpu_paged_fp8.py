"""The paged cache held in 8 bits: append and reading back, against the definition in 64 bits."""
import pytest
import torch

from fp8_util import F8, Batch8, Cache64, turned, values
from ragged_util import HALF_STEP, Batch

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


class Run:
    """A cache on the GPU and its definition on the CPU, taken through steps of new tokens per sequence."""

    def __init__(self, kvc, B, bs, H_q, H_kv, D, dtype="bf16", rot=None, adjacent=False, norm=False, T_max=600, seed=0):
        self.kvc, self.B, self.bs, self.H_q, self.H_kv, self.D = kvc, B, bs, H_q, H_kv, D
        self.dtype = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
        self.mb = -(-T_max // bs)
        self.nb = B * self.mb + 2
        self.g = torch.Generator().manual_seed(seed)
        self.table = torch.randperm(self.nb, generator=self.g)[:B * self.mb].view(B, self.mb).to(torch.int32)
        self.c = kvc.PagedFP8KVCache(1, self.nb, bs, B, self.mb, H_q, H_kv, D, dtype)
        self.ref = Cache64(self.nb, H_kv, bs, D)
        rot = D if rot is None else rot
        self.freq = [10000.0 ** (-2 * i / rot) for i in range(rot // 2)] if rot else None
        self.rope = kvc.Rope(self.freq, layout="adjacent" if adjacent else "half") if rot else None
        self.adjacent, self.lens = adjacent, [0] * B
        self.w = [(1 + 0.3 * torch.randn(D, generator=self.g)).to(self.dtype) if norm else None for _ in range(2)]

    def step(self, new, mag=1.0, pad=2, edit=None, stream=None):
        n, D = sum(new), self.D
        q = torch.randn(n + pad, self.H_q, D, generator=self.g).to(self.dtype)
        k = (torch.randn(n + pad, self.H_kv, D, generator=self.g) * mag).to(self.dtype)
        v = (torch.randn(n + pad, self.H_kv, D, generator=self.g) * mag).to(self.dtype)
        if edit:
            edit(k, v)
        cu = [0]
        for x in new:
            cu.append(cu[-1] + x)
        before = [x.cpu() for x in self.c.layer_views(0)]
        lens = [a + b for a, b in zip(self.lens, new)]
        out = torch.full(q.shape, 7.0, dtype=self.dtype, device="cuda")
        w = [None if x is None else x.cuda() for x in self.w]
        self.c.append_rope(0, self.rope, q.cuda(), k.cuda(), v.cuda(), self.table.cuda(), i32(cu), i32(lens), q_out=out,
                           q_norm=w[0], k_norm=w[1], norm_eps=EPS)
        assert self.c.last_error() == (self.kvc.KVC_OK, 0)
        pos = torch.cat([torch.arange(h, L) for h, L in zip(self.lens, lens)])
        ref, tol = turned(q[:n], self.w[0], EPS, pos, self.freq, self.adjacent)
        tol = tol + HALF_STEP[self.dtype] * (ref.abs() + tol)
        assert ((out[:n].cpu().double() - ref).abs() <= tol).all() and (out[n:] == 7).all()
        kk, ktol = turned(k[:n], self.w[1], EPS, pos, self.freq, self.adjacent)
        err = torch.zeros(self.nb, self.H_kv, self.bs, D, dtype=torch.float64)
        for b in range(self.B):
            if new[b] == 0:
                continue
            s = slice(cu[b], cu[b + 1])
            self.ref.append(self.table[b], self.lens[b], new[b], kk[s], v[:n][s].double())
            t = torch.arange(self.lens[b], lens[b])
            err[self.table[b, t // self.bs].long(), :, t % self.bs] = ktol[s]
        self.check(err, before)
        self.lens = lens

    def check(self, err, before):
        """Scales and V's codes are the definition's; K's codes too, but where the fp32 error of a new value
        reaches the next code."""
        K, V, Ks, Vs = (x.cpu() for x in self.c.layer_views(0))
        r = self.ref
        assert torch.equal(Ks, r.scales["K"]) and torch.equal(Vs, r.scales["V"])
        assert torch.equal(V, r.codes["V"])
        differ = K != r.codes["K"]
        if differ.any():
            x, c = r.exact["K"], K.view(F8).double()
            slack = err / Ks.double()[..., None, None].clamp(min=2.0 ** -64)
            # nearest within the slack: no further from the exact value than half of the larger step about it
            step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))) / 8
            ok = (err > 0) & ((c - x).abs() <= step / 2 * (1 + 2.0 ** -20) + slack)
            assert (ok | ~differ).all(), int((differ & ~ok).sum())
            assert differ.float().mean() < 1e-3
            r.codes["K"] = K.clone()


@pytest.mark.parametrize("dtype,D,H_q,H_kv,bs,rot,adjacent,norm", [
    ("bf16", 128, 8, 2, 16, None, False, False),
    ("bf16", 128, 8, 8, 64, None, True, True),
    ("bf16", 64, 4, 1, 32, 32, False, True),
    ("bf16", 256, 2, 2, 128, 64, False, False),
    ("bf16", 128, 32, 1, 256, None, False, True),
    ("f32", 128, 2, 2, 16, None, False, True),
    ("f32", 64, 8, 4, 64, 16, True, False),
    ("f32", 256, 2, 1, 256, None, False, False),
    ("bf16", 128, 6, 3, 32, 0, False, True),   # heads that no group divides, no rotation
    ("bf16", 64, 40, 40, 16, None, False, False),
])
def test_steps(kvc, dtype, D, H_q, H_kv, bs, rot, adjacent, norm):
    if (H_q // H_kv) & (H_q // H_kv - 1):
        pytest.skip("group sizes are powers of two")
    r = Run(kvc, 3, bs, H_q, H_kv, D, dtype, rot, adjacent, norm, T_max=5 * bs + 200)
    r.step([37, 0, 5])
    r.step([1, 1, 1], mag=8.0)       # blocks that hold tokens take a larger scale
    r.step([1, 1, 1], mag=0.01)      # ... and keep it
    r.step([bs, 3 * bs + 1, 2], mag=100.0)
    r.step([0, 1, 70])


def test_growth_many_times(kvc):
    # each token twice as large as the one before: the codes move down a binade each time, in a block of
    # their own until the next begins; what is left stays within a step of 2^-9 of the last scale
    r = Run(kvc, 1, 32, 2, 1, 128, rot=0, T_max=64)
    xs = []
    for i in range(32):
        r.step([1], mag=2.0 ** (i - 16), pad=0, edit=lambda k, v: xs.append(v[0, 0].clone()))
    V, s = r.c.layer_views(0)[1].cpu(), r.c.layer_views(0)[3].cpu()
    e = int(r.table[0, 0])
    got = values(V, s)[e, 0]
    want = torch.stack(xs).double()
    bound = want.abs() * 2.0 ** -4 + float(s[e, 0]) * 2.0 ** -9
    assert ((got - want).abs() <= bound).all()


def test_rows_are_quantized_alike_in_one_call_and_in_many(kvc):
    a, b = Run(kvc, 1, 16, 2, 2, 64, rot=0, seed=3), Run(kvc, 1, 16, 2, 2, 64, rot=0, seed=3)
    g = torch.Generator().manual_seed(9)
    x = torch.randn(16, 2, 64, generator=g).to(torch.bfloat16)
    x[0] = x.abs().amax()  # the first token sets the scale
    a.step([16], pad=0, edit=lambda k, v: (k.copy_(x), v.copy_(x)))
    for i in range(16):
        b.step([1], pad=0, edit=lambda k, v: (k.copy_(x[i:i + 1]), v.copy_(x[i:i + 1])))
    for p, q in zip(a.c.layer_views(0), b.c.layer_views(0)):
        assert torch.equal(p[int(a.table[0, 0])], q[int(b.table[0, 0])])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_values_at_the_ends(kvc, dtype):
    # zeros, the smallest values, the largest finite ones (codes stay below what reads back as infinite),
    # infinities and NaN (stored as NaN, outside the maximum)
    big = float(torch.finfo(Batch([1], [0], 16, 1, 1, 64, dtype).dtype).max)

    def edit(k, v):
        v[0] = 0
        v[1] = 2.0 ** -70
        v[2, 0] = big
        v[2, 1] = 448
        v[3, 0] = 449
        v[4, 0, 3] = float("inf")
        v[5, 0, 4] = float("-inf")
        v[6, 0, 5] = float("nan")
        k[0] = 0
    for new in ([7], [1, 0, 0, 0, 0, 0, 6]):
        r = Run(kvc, len(new), 16, 2, 2, 64, dtype, rot=0)
        r.step(new, edit=edit)
        V = r.c.layer_views(0)[1].cpu()
        out = torch.zeros(sum(new), 2, 64, dtype=r.dtype, device="cuda")
        cu = [0]
        for x in new:
            cu.append(cu[-1] + x)
        r.c.read(0, None, out, r.table.cuda(), i32(cu), i32(new))
        if len(new) == 1:
            got = out.cpu()
            assert not torch.isinf(got).any() and int(torch.isnan(got).sum()) == 3
            assert abs(float(got[2, 0, 0]) / big - 1) < 2.0 ** -4 + 2.0 ** -8
        assert V.any()


def test_a_block_begun_anew_forgets_its_scale(kvc):
    r = Run(kvc, 1, 16, 2, 2, 64, rot=0)
    r.step([20], mag=1000.0)
    r.lens = [0]  # the sequence ended; its blocks are handed out again
    r.step([3], mag=0.5)
    assert float(r.c.layer_views(0)[3][int(r.table[0, 0])].max()) < 0.1


@pytest.mark.parametrize("dtype,D,H_kv,bs", [("bf16", 128, 8, 16), ("bf16", 64, 1, 64), ("f32", 128, 2, 32),
                                             ("f32", 256, 1, 256), ("bf16", 256, 3, 128)])
def test_read(kvc, dtype, D, H_kv, bs):
    bt = Batch8([5, 0, 1, 300], [17, 3, 0, 210], bs, H_kv, H_kv, D, dtype, pad=4, mag=10)
    c, d = bt.cache(kvc), bt.dev()
    k, v = (torch.full((bt.rows, H_kv, D), 7.0, dtype=bt.dtype, device="cuda") for _ in range(2))
    c.read(0, k, v, d["table"], d["cu"], d["lens"])
    for got, pool in ((k, bt.K), (v, bt.V)):
        got = got.cpu()
        for b in range(bt.B):
            t = torch.arange(bt.hist[b], bt.lens[b])
            want = pool[bt.table[b, t // bs].long(), :, t % bs]
            assert torch.equal(got[bt.cu[b]:bt.cu[b + 1]].double(), want)
        assert (got[bt.n:] == 7).all()
    only = torch.zeros(bt.rows, H_kv, D, dtype=bt.dtype, device="cuda")
    c.read(0, None, only, d["table"], d["cu"], d["lens"])
    assert torch.equal(only[:bt.n], v[:bt.n])
    wide = torch.full((bt.rows, 2 * H_kv, D), 7.0, dtype=bt.dtype, device="cuda")  # strided rows
    c.read(0, wide[:, :H_kv], wide[:, H_kv:], d["table"], d["cu"], d["lens"])
    assert torch.equal(wide[:bt.n, :H_kv], k[:bt.n]) and torch.equal(wide[:bt.n, H_kv:], v[:bt.n])
    assert c.last_error() == (kvc.KVC_OK, 0)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f32", 4), ("f32", 64)])
def test_read_of_a_plain_cache(kvc, dtype, D):
    bt = Batch([5, 0, 1, 90], [17, 3, 0, 210], 32, 2, 2, D, dtype, pad=4)
    c, d = bt.cache(kvc), bt.dev()
    k, v = (torch.full((bt.rows, 2, D), 7.0, dtype=bt.dtype, device="cuda") for _ in range(2))
    c.read(0, k, v, d["table"], d["cu"], d["lens"])
    for got, pool in ((k, bt.K), (v, bt.V)):
        for b in range(bt.B):
            t = torch.arange(bt.hist[b], bt.lens[b])
            assert torch.equal(got[bt.cu[b]:bt.cu[b + 1]].cpu(), pool[bt.table[b, t // 32].long(), :, t % 32])
        assert (got[bt.n:] == 7).all()


def test_device_errors(kvc):
    def fresh():
        bt = Batch8([3, 2], [10, 20], 16, 4, 2, 64)
        return bt, bt.cache(kvc), bt.dev()
    rope = kvc.Rope([1.0, 0.3, 0.1, 0.01, 1e-3, 1e-4, 1e-5, 1e-6])

    def append(c, d):
        q = torch.full_like(d["q"], 7.0)
        c.append_rope(0, rope, d["q"], d["k"], d["v"], d["table"], d["cu"], d["lens"], q_out=q)
        return q

    def read(c, d):
        k = torch.full_like(d["k"], 7.0)
        c.read(0, k, None, d["table"], d["cu"], d["lens"])
        return k

    def only_block_changed(before, c, seen):  # its codes; its scales may stay
        for i, (x, y) in enumerate(zip(before, c.layer_views(0))):
            same = (x == y).flatten(1).all(1).cpu()
            assert i >= 2 or not same[seen]
            same[seen] = True
            assert same.all()
    # too many new tokens, too long a sequence: that sequence alone is left out (read: zeros)
    for L in (2, 10 ** 6):
        bt, c, d = fresh()
        d["lens"][0] = L
        before = [x.clone() for x in c.layer_views(0)]
        append(c, d)
        assert c.last_error() == (kvc.KVC_EDEVICE, kvc.KVC_DEV_BAD_LENS)
        seen = bt.table[1, 20 // 16].item()
        only_block_changed(before, c, seen)
        k = read(c, d)
        assert c.last_error() == (kvc.KVC_EDEVICE, kvc.KVC_DEV_BAD_LENS)
        assert (k[:3] == 0).all() and (k[3:] != 0).any()
    # a block out of range: its rows are not stored, and read as zeros
    for e in (-1, 10 ** 6):
        bt, c, d = fresh()
        d["table"][1, 1] = e
        before = [x.clone() for x in c.layer_views(0)]
        append(c, d)
        assert c.last_error() == (kvc.KVC_EDEVICE, kvc.KVC_DEV_BAD_BLOCK)
        seen = bt.table[0, 0].item()
        only_block_changed(before, c, seen)
        k = read(c, d)
        assert c.last_error() == (kvc.KVC_EDEVICE, kvc.KVC_DEV_BAD_BLOCK)
        assert (k[3:] == 0).all() and (k[:3] != 0).any()
    # sequences that do not ascend: nothing is written
    for cu in ([0, 4, 3], [1, 3, 5], [0, 3, 6], [-1, 3, 5]):
        bt, c, d = fresh()
        d["cu"].copy_(torch.tensor(cu, dtype=torch.int32))
        before = [x.clone() for x in c.layer_views(0)]
        q = append(c, d)
        assert c.last_error() == (kvc.KVC_EDEVICE, kvc.KVC_DEV_BAD_SEQ)
        assert all(torch.equal(x, y) for x, y in zip(before, c.layer_views(0))) and (q == 7).all()
        k = read(c, d)
        assert c.last_error() == (kvc.KVC_EDEVICE, kvc.KVC_DEV_BAD_SEQ) and (k == 7).all()


def test_refusals(kvc):
    bt = Batch8([3, 2], [10, 20], 16, 4, 2, 64)
    c, d = bt.cache(kvc), bt.dev()
    E = kvc.KvcError

    def status(f, *a):
        with pytest.raises(E) as x:
            f(*a)
        return x.value.status
    K = torch.zeros(2, 2, 8, 64, dtype=torch.bfloat16, device="cuda")
    one = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    for f, a in ((c.prefill_write, (0, K, K, d["table"], d["lens"])), (c.append, (0, one, one, d["table"], d["lens"])),
                 (c.decode_attn, (0, q, q, d["table"], d["lens"])),
                 (c.decode_step, (0, q, one, one, q, d["table"], d["lens"]))):
        assert status(f, *a) == kvc.KVC_EUNSUPPORTED
    rope = kvc.Rope([1.0, 0.1])  # pairs that no whole vector holds
    assert status(c.append_rope, 0, rope, d["q"], d["k"], d["v"], d["table"], d["cu"], d["lens"]) == kvc.KVC_EUNSUPPORTED
    with pytest.raises(ValueError):
        c.read(0, None, None, d["table"], d["cu"], d["lens"])
    with pytest.raises(ValueError):
        c.read(0, d["k"], d["v"][:4], d["table"], d["cu"], d["lens"])
    with pytest.raises(ValueError):
        c.read(0, d["k"].float(), None, d["table"], d["cu"], d["lens"])
    assert status(kvc.kvc_paged_read, c.h, 1, d["k"], 128, None, 0, d["table"], d["cu"], d["lens"], 5) == kvc.KVC_EINVAL
    assert status(kvc.kvc_paged_read, c.h, 0, d["k"], 64, None, 0, d["table"], d["cu"], d["lens"], 5) == kvc.KVC_EINVAL
    assert kvc.load().kvc_get_cache_format(c.h) == kvc.KVC_CACHE_FP8
    assert c.nbytes() >= 2 * bt.nblocks * 2 * (16 * 64 + 4)
    assert kvc.kvc_payload_bytes(c.h, bt.lens) == 2 * 2 * (64 * sum(bt.lens) + 4 * sum(-(-L // 16) for L in bt.lens))
    plain = kvc.KVCache(1, 2, 4, 2, 64, 32)
    assert status(kvc.kvc_paged_read, plain.h, 0, d["k"], 128, None, 0, d["table"], d["cu"], d["lens"], 5) == kvc.KVC_EINVAL
    for args in ((1, 4, 24, 2, 4, 4, 2, 64, 0), (1, 4, 16, 2, 4, 4, 2, 32, 0), (1, 4, 16, 2, 4, 4, 2, 4, 1)):
        with pytest.raises(E) as x:
            kvc.kvc_create_paged_fp8(*args)
        assert x.value.status == kvc.KVC_EUNSUPPORTED


def test_graph_replays_on_new_lengths(kvc):
    # one captured step, replayed while the sequences grow: the same bits as calls one by one
    r = Run(kvc, 2, 16, 4, 2, 128)
    r.step([20, 3])
    D = r.D
    g = torch.Generator().manual_seed(4)
    steps = [[(torch.randn(2, h, D, generator=g) * (1 + i)).to(torch.bfloat16).cuda() for h in (4, 2, 2)] for i in range(6)]
    base = [x.clone() for x in r.c.layer_views(0)]
    bufs = [torch.zeros_like(x) for x in steps[0]]
    out, table, cu, lens = torch.zeros_like(bufs[0]), r.table.cuda(), i32([0, 1, 2]), i32(r.lens)
    outs, pools = [], []
    for mode in ("eager", "graph"):
        for x, y in zip(r.c.layer_views(0), base):
            x.copy_(y)
        lens.copy_(i32(r.lens))
        if mode == "graph":
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                lens += 1
                r.c.append_rope(0, r.rope, *bufs, table, cu, lens, q_out=out)
            for x, y in zip(r.c.layer_views(0), base):
                x.copy_(y)
            lens.copy_(i32(r.lens))
        got = []
        for s in steps:
            for x, y in zip(bufs, s):
                x.copy_(y)
            if mode == "graph":
                graph.replay()
            else:
                lens += 1
                r.c.append_rope(0, r.rope, *bufs, table, cu, lens, q_out=out)
            got.append(out.clone())
        outs.append(got)
        pools.append([x.clone() for x in r.c.layer_views(0)])
    assert all(torch.equal(a, b) for a, b in zip(*outs)) and all(torch.equal(a, b) for a, b in zip(*pools))
    assert r.c.last_error() == (kvc.KVC_OK, 0)

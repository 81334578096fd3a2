"""Append with norms of the heads to plain paged caches, against the definition in 64 bits."""
import pytest
import torch

from fp8_util import turned
from ragged_util import Batch, HALF_STEP

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def kvc():
    import __graft_entry__
    __graft_entry__.build()
    from kv_cache_decode_kvc_gb300 import kvc
    return kvc


def _weights(D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (1 + 0.3 * torch.randn(D, generator=g)).to(dtype)


def run(kvc, bt, rot, adjacent, qn, kn, in_place=False, q=True, strided=False, seed=5):
    c, d = bt.cache(kvc), bt.dev()
    w = {x: _weights(bt.D, bt.dtype, seed + i) if on else None for i, (x, on) in enumerate((("q", qn), ("k", kn)))}
    freq = [10000.0 ** (-2 * i / rot) for i in range(rot // 2)] if rot else None
    rope = kvc.Rope(freq, layout="adjacent" if adjacent else "half") if rot else None
    if strided:  # views of a joint projection
        joint = torch.cat([d["q"].flatten(1), d["k"].flatten(1), d["v"].flatten(1)], 1)
        sizes = [bt.H_q * bt.D, bt.H_kv * bt.D, bt.H_kv * bt.D]
        d["q"], d["k"], d["v"] = (t.unflatten(1, (-1, bt.D)) for t in joint.split(sizes, 1))
    q_out = None if in_place else torch.full((bt.rows, bt.H_q, bt.D), 7.0, dtype=bt.dtype, device="cuda")
    dev = {x: t.cuda() if t is not None else None for x, t in w.items()}
    c.append_rope(0, rope, d["q"] if q else None, d["k"], d["v"], d["table"], d["cu"], d["lens"],
                  q_out=q_out if q else None, q_norm=dev["q"], k_norm=dev["k"], norm_eps=EPS)
    K, V = c.layer_views(0)
    assert c.last_error() == (kvc.KVC_OK, 0)
    got_q = (d["q"] if in_place else q_out).cpu() if q else None
    pos = torch.cat([torch.arange(h, h + n) for h, n in zip(bt.hist, bt.new)])
    return got_q, K.cpu(), V.cpu(), w, freq, pos


def close(got, ref, tol, dtype, what):
    err = (got.double() - ref).abs()
    tol = tol + HALF_STEP[dtype] * (ref.abs() + tol) + 2.0 ** -133
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / tol).max()):.2f}"


@pytest.mark.parametrize("dtype,D,H_q,H_kv,rot,adjacent,new,hist,bs", [
    ("bf16", 128, 32, 8, 128, False, [1, 1, 1], [300, 0, 17], 16),
    ("bf16", 128, 8, 2, 64, True, [5, 0, 130], [0, 9, 63], 64),
    ("bf16", 64, 4, 4, 64, False, [33, 1], [1, 500], 32),
    ("bf16", 256, 2, 1, 96, False, [9, 4], [0, 3], 128),
    ("bf16", 128, 4, 2, 18, False, [7, 3], [2, 0], 16),      # pairs that no whole vector holds
    ("f32", 64, 8, 8, 32, True, [1, 70], [10, 0], 32),
    ("f32", 4, 2, 1, 4, False, [3, 1], [0, 40], 16),
    ("f32", 256, 2, 2, 10, True, [3, 1], [0, 40], 16),
    ("bf16", 128, 64, 8, 128, False, [700, 600], [0, 5], 256),  # four rows a block
    ("bf16", 128, 8, 2, 0, False, [4, 1], [0, 7], 16),       # norms alone
])
@pytest.mark.parametrize("qn,kn", [(True, True), (False, True), (True, False)])
def test_against_64_bits(kvc, dtype, D, H_q, H_kv, rot, adjacent, new, hist, bs, qn, kn):
    bt = Batch(new, hist, bs, H_q, H_kv, D, dtype, pad=3)
    q, K, V, w, freq, pos = run(kvc, bt, rot, adjacent, qn, kn)
    n = bt.n
    ref, tol = turned(bt.q[:n], w["q"], EPS, pos, freq, adjacent)
    close(q[:n], ref, tol, bt.dtype, "q")
    assert (q[n:] == 7).all()
    ref, tol = turned(bt.k[:n], w["k"], EPS, pos, freq, adjacent)
    want_K, want_V = bt.K.clone(), bt.V.clone()
    blocks = torch.cat([bt.table[b, torch.arange(bt.hist[b], bt.lens[b]) // bs] for b in range(bt.B)]).long()
    close(K[blocks, :, pos % bs], ref, tol, bt.dtype, "K")
    want_K[blocks, :, pos % bs] = K[blocks, :, pos % bs]
    want_V[blocks, :, pos % bs] = bt.v[:n]
    assert torch.equal(K, want_K) and torch.equal(V, want_V)  # nothing else moved, values byte for byte


@pytest.mark.parametrize("rot,adjacent", [(128, False), (22, True)])
def test_in_place_strided_and_append_only(kvc, rot, adjacent):
    bt = Batch([40, 1, 3], [5, 100, 0], 32, 8, 2, 128)
    a = run(kvc, bt, rot, adjacent, True, True)
    b = run(kvc, bt, rot, adjacent, True, True, in_place=True)
    s = run(kvc, bt, rot, adjacent, True, True, strided=True)
    o = run(kvc, bt, rot, adjacent, False, True, q=False)
    for x in (b, s):
        assert torch.equal(a[0][:bt.n], x[0][:bt.n]) and torch.equal(a[1], x[1]) and torch.equal(a[2], x[2])
    assert torch.equal(a[1], o[1])


def test_without_norms_it_is_the_plain_append(kvc):
    bt = Batch([40, 1, 3], [5, 100, 0], 32, 8, 2, 128)
    c, c2, d = bt.cache(kvc), bt.cache(kvc), bt.dev()
    rope = kvc.Rope([10000.0 ** (-i / 64) for i in range(64)])
    q1, q2 = torch.zeros_like(d["q"]), torch.zeros_like(d["q"])
    c.append_rope(0, rope, d["q"], d["k"], d["v"], d["table"], d["cu"], d["lens"], q_out=q1)
    s = kvc._stream(None)
    D = bt.D
    kvc.kvc_paged_append_norm_rope(c2.h, 0, rope.r, None, None, 0.0, d["q"], 8 * D, q2, 8 * D, d["k"], 2 * D, d["v"], 2 * D,
                                   None, 0, d["table"], d["cu"], d["lens"], bt.n, s)
    assert torch.equal(q1, q2) and all(torch.equal(a, b) for a, b in zip(c.layer_views(0), c2.layer_views(0)))


def test_zero_rows_and_extreme_values(kvc):
    # a head of zeros is 0 / sqrt(eps); one of 2^60 overflows the sum of squares nowhere (2^120 128 < 2^128)
    bt = Batch([4], [0], 16, 2, 1, 128)
    bt.q[0] = 0
    bt.q[1] *= 2.0 ** 57
    bt.q[2] *= 2.0 ** -60
    bt.k[3] = 0
    q, K, V, w, freq, pos = run(kvc, bt, 128, False, True, True)
    ref, tol = turned(bt.q, w["q"], EPS, pos, freq, False)
    close(q, ref, tol, bt.dtype, "q")


def test_refusals(kvc):
    bt = Batch([2, 1], [0, 3], 16, 4, 2, 64)
    c, d = bt.cache(kvc), bt.dev()
    rope = kvc.Rope([1.0, 0.5])
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    args = (0, rope, d["q"], d["k"], d["v"], d["table"], d["cu"], d["lens"])
    for bad in (w.float(), w[:32], w.cpu(), torch.ones(128, dtype=torch.bfloat16, device="cuda")[::2]):
        with pytest.raises(ValueError, match="q_norm"):
            c.append_rope(*args, q_norm=bad)
        with pytest.raises(ValueError, match="k_norm"):
            c.append_rope(*args, k_norm=bad)
    for eps in (-1e-6, float("nan"), float("inf")):
        with pytest.raises(kvc.KvcError):
            c.append_rope(*args, q_norm=w, norm_eps=eps)
    with pytest.raises(kvc.KvcError):  # a norm of queries that are not there
        c.append_rope(0, rope, None, *args[3:], q_norm=w)
    odd = torch.ones(65, dtype=torch.bfloat16, device="cuda")[1:]  # not 16-byte aligned
    with pytest.raises(kvc.KvcError):
        c.append_rope(*args, q_norm=odd)
    with pytest.raises(ValueError, match="positions"):
        c.append_rope(0, None, *args[2:], positions=torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert c.last_error() == (kvc.KVC_OK, 0)

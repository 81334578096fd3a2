"""How exact attention on the codes of the 8-bit paged cache is: three E5M2 terms a weight, two E4M3 terms a query, errors over
whole sequences where many pieces are merged."""
import math

import pytest
import torch

from fp8_util import F8, Batch8, smallest_weights
from ragged_util import attention64, check_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc():
    import __graft_entry__
    __graft_entry__.build()
    from kv_cache_decode_kvc_gb300 import kvc
    return kvc


def attend(kvc, bt, shared=False, ctas=0):
    c, d = bt.cache(kvc), bt.dev()
    c.set_ctas(ctas)
    out = torch.full_like(d["q"], 7.0)
    a = (0, d["q"], out, d["table"], d["cu"], d["lens"])
    c.attn_shared(*a, d["groups"], d["prefix"]) if shared else c.attn_ragged(*a)
    assert c.last_error() == (kvc.KVC_OK, 0)
    return out


# A weight w, 2^k <= w < 2^(k + 1), is rounded to f16 (2^(k - 11) off at most).  Its first term, cut after two bits behind the
# leading one, leaves less than 2^(k - 2), the second, of that, less than 2^(k - 5), and the third is rounded to a step of
# 2^(k - 8) or less: 2^(k - 9) off.
THREE_TERMS = 2.0 ** -9 + 2.0 ** -11


def terms(w, n):
    """The first n terms' sum of weights w (fp32), as the kernel takes them."""
    def top(x):
        return (x.view(torch.int16) & -256).view(torch.float16)
    h, t, scale = w.half(), torch.zeros(w.shape, dtype=torch.float64), 1.0
    for i in range(n):
        u = top(h) if i < 2 else ((h.view(torch.int16) + 0x80) & -256).view(torch.float16)
        t, h, scale = t + u.double() * scale, (h - u) * 8, scale / 8
    return t


def on_codes(bt, weight_terms=3, query_terms=2):
    """The outputs with that many terms, and all else in 64 bits."""
    out = torch.zeros(bt.rows, bt.H_q, bt.D, dtype=torch.float64)
    G = bt.H_q // bt.H_kv
    for b in range(bt.B):
        for h in range(bt.H_kv):
            t = torch.arange(bt.lens[b])
            e = bt.table[b, t // bt.bs].long()
            K, V, s = bt.K[e, h, t % bt.bs], bt.V[e, h, t % bt.bs], bt.Vs[e, h].double()
            for i in range(bt.new[b]):
                n, r = bt.hist[b] + i + 1, bt.cu[b] + i
                q = bt.q[r, h * G:(h + 1) * G].double()
                up = torch.exp2(7 - torch.floor(torch.log2(q.abs().amax(-1, keepdim=True))))
                t0 = (q * up).float().to(F8).double()
                t1 = ((q * up - t0) * 16).float().to(F8).double() / 16
                x = (t0 + t1 * (query_terms > 1)) / up @ K[:n].T / math.sqrt(bt.D) * math.log2(math.e)
                la = torch.log2(s[:n])
                M = torch.ceil((x + la).amax(-1, keepdim=True)) - 4
                w = terms(torch.exp2(x + la - M).float(), weight_terms)
                m = x.amax(-1, keepdim=True)
                out[r, h * G:(h + 1) * G] = w @ (V[:n] / s[:n, None]) * torch.exp2(M - m) / torch.exp2(x - m).sum(-1, keepdim=True)
    return out


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H_q,H_kv", [(4, 4), (8, 2), (32, 1)])
@pytest.mark.parametrize("ctas", [0, 5])
@pytest.mark.parametrize("hist", [[0, 2, 5, 1, 3, 0], [900, 300, 0, 128, 5, 63]])
def test_weights_have_three_terms_and_queries_two(kvc, D, H_q, H_kv, ctas, hist):
    # values above 0: what a weight loses, the outputs lose
    bt = Batch8([1, 6, 2, 1, 0, 1], hist, 32, H_q, H_kv, D, seed=61)
    bt.V = bt.V.abs()
    bt.requantize()
    ref, tol, A = attention64(bt)
    bound = tol + THREE_TERMS * A + smallest_weights(bt)
    check_attention(attend(kvc, bt, ctas=ctas), bt, (ref, bound, A))
    # the bound holds for the terms as they are, and leaves no room for one fewer of either
    assert ((on_codes(bt) - ref).abs() <= bound).all()
    for fewer in (dict(weight_terms=2), dict(query_terms=1)):
        assert ((on_codes(bt, **fewer) - ref).abs() > bound).any(), fewer


def test_the_terms_of_all_weights():
    # every f16 weight that the kernel lets pass, and fp32 ones between: the two bounds of the header
    w = torch.cat([torch.arange(0x7400, dtype=torch.int16).view(torch.float16).float(),
                   torch.arange(1, 2, 2.0 ** -18).float() * 3, torch.tensor([1.14208984375, 16383.0])])
    err = (terms(w, 3) - w.double()).abs()
    assert (err <= (THREE_TERMS * w.double()).clamp(min=2.0 ** -23 + 2.0 ** -25)).all()
    assert (err > 2.0 ** -9 * w.double())[w > 2.0 ** -13].any()  # (the third term's rounding alone is not all)


# Per sequence || error || / || output ||: the output's rounding 0.0017 and the weights' errors below that of each other;
# one of n key tiles lost moves it by about sqrt(1 / n).
LIMIT = 1e-2


def relative(got, want):
    return float((got - want).norm() / want.norm())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,H_q,ctas", [([1], 32, 0), ([2, 1], 32, 0), ([1], 32, 19), ([3], 32, 600), ([20], 4, 0), ([40, 1], 4, 37),
                                          ([1], 1, 0)])
@pytest.mark.parametrize("shared", [False, True])
def test_long_sequences_lose_no_tile(kvc, D, new, H_q, ctas, shared):
    bt = Batch8(new, [20011, 9000][:len(new)], 64, H_q, 1, D, seed=54)
    out = attend(kvc, bt, shared, ctas).cpu().double()
    ref = attention64(bt)[0]
    for b in range(bt.B):
        rows = slice(bt.cu[b], bt.cu[b + 1])
        assert relative(out[rows], ref[rows]) <= LIMIT, b
    # the limit sees a lost tile: the first token's output without positions [128 j, 128 j + 128)
    n = bt.hist[0] + 1
    t = torch.arange(n)
    K, V = (x[bt.table[0, t // 64].long(), 0, t % 64].double() for x in (bt.K, bt.V))
    s = bt.q[0].double() @ K.T / math.sqrt(D)
    assert relative(torch.softmax(s, -1) @ V, ref[0]) < 1e-12
    for j in (0, 1, 77, 155):
        keep = (t < 128 * j) | (t >= 128 * j + 128)
        assert relative(torch.softmax(s[:, keep], -1) @ V[keep], ref[0]) > 3 * LIMIT

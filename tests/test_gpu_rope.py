"""kvc_paged_append_rope against the rotation in 64 bits: layouts, axes, dtypes, partial rotations,
odd lengths, strides, far positions; what it may not touch; what it flags."""
import pytest
import torch

from kv_cache_decode_kvc_gb300 import kvc

from ragged_util import HALF_STEP, U, Batch, rotate64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _freq(rot):
    return [10000.0 ** (-2 * i / rot) for i in range(rot // 2)]


def _slots(bt):
    return torch.cat([torch.arange(h, h + n) for h, n in zip(bt.hist, bt.new)])


def _close(got, want, w, dtype):
    err = (got.double() - want).abs()
    assert (err <= w * 12 * U + HALF_STEP[dtype] * want.abs()).all(), float(err.max())


def _check(bt, c, q_out, pos, freq, axis, adjacent, q0, scale=1.0):
    """q_out, the pool's new rows and everything else of the pool."""
    n = bt.n
    y, w = rotate64(bt.q[:n], pos, freq, axis, adjacent, scale)
    _close(q_out[:n].cpu(), y, w, bt.dtype)
    assert torch.equal(q_out[n:].cpu(), q0[n:])
    y, w = rotate64(bt.k[:n], pos, freq, axis, adjacent, scale)
    K, V = (x.cpu() for x in c.layer_views(0))
    slot = _slots(bt)
    b = torch.repeat_interleave(torch.arange(bt.B), torch.tensor(bt.new))
    at = bt.table[b, slot // bt.bs].long(), slot % bt.bs
    _close(K[at[0], :, at[1]], y, w, bt.dtype)
    assert torch.equal(V[at[0], :, at[1]], bt.v[:n])
    Kw, Vw = bt.K.clone(), bt.V.clone()
    Kw[at[0], :, at[1]], Vw[at[0], :, at[1]] = K[at[0], :, at[1]], V[at[0], :, at[1]]
    assert torch.equal(K, Kw) and torch.equal(V, Vw)  # nothing else changed


@pytest.mark.parametrize("dtype,D,rot", [("bf16", 128, 128), ("bf16", 128, 64), ("bf16", 64, 64), ("bf16", 256, 32),
                                         ("bf16", 128, 10), ("f32", 128, 128), ("f32", 64, 24), ("f32", 64, 6),
                                         ("f32", 4, 4), ("f32", 4, 2), ("f32", 256, 256)])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("axes", [1, 3])
def test_append_rope_matches_64_bits(dtype, D, rot, adjacent, axes):
    bt = Batch([3, 0, 1, 70, 0, 33], [0, 5, 40, 17, 0, 31], 32, 8, 2, D, dtype, pad=5, seed=rot + D)
    freq = _freq(rot)
    axis = [i % axes for i in range(rot // 2)]
    if rot // 2 < axes:
        pytest.skip("fewer pairs than axes")
    c, d = bt.cache(kvc), bt.dev()
    rope = kvc.Rope(freq, "adjacent" if adjacent else "half", axis)
    q0 = torch.full((bt.rows, 8, D), 7.0, dtype=bt.dtype)
    q_out = q0.cuda()
    pos = torch.randint(0, 5000, (axes, bt.rows), generator=torch.Generator().manual_seed(1)).to(torch.int32)
    c.append_rope(0, rope, d["q"], d["k"], d["v"], d["table"], d["cu"], d["lens"], q_out, pos.cuda())
    assert c.last_error() == (kvc.KVC_OK, 0)
    _check(bt, c, q_out, pos[:, :bt.n].T, freq, axis, adjacent, q0)


@pytest.mark.parametrize("bs", [16, 64, 256])
@pytest.mark.parametrize("many", [False, True])
def test_append_rope_slot_positions_joint_projection_and_in_place(bs, many):
    # q, k, v views of one projection, q rotated in place; many: over the row count where a block
    # takes several rows (16 per SM)
    new = [1, 700, 0, 2, 1999] if many else [1, 9, 0, 2, 30]
    bt = Batch(new, [100, 3, 50, 0, 77], bs, 4, 2, 128, pad=3, seed=bs)
    c, d = bt.cache(kvc), bt.dev()
    qkv = torch.cat([d["q"], d["k"], d["v"]], 1).flatten(1).contiguous()
    q = qkv[:, :512].unflatten(1, (4, 128))
    k = qkv[:, 512:768].unflatten(1, (2, 128))
    v = qkv[:, 768:].unflatten(1, (2, 128))
    freq = _freq(128)
    c.append_rope(0, kvc.Rope(freq, scale=1.25), q, k, v, d["table"], d["cu"], d["lens"])
    assert c.last_error() == (kvc.KVC_OK, 0)
    _check(bt, c, q, _slots(bt)[:, None], freq, [0] * 64, False, bt.q, 1.25)
    assert torch.equal(k.cpu(), bt.k) and torch.equal(v.cpu(), bt.v)


def test_append_rope_without_queries():
    bt = Batch([4, 1], [0, 20], 16, 8, 8, 64, seed=3)
    c, d = bt.cache(kvc), bt.dev()
    freq = _freq(64)
    c.append_rope(0, kvc.Rope(freq), None, d["k"], d["v"], d["table"], d["cu"], d["lens"])
    q_out, w = rotate64(bt.q, _slots(bt)[:, None], freq, [0] * 32, False)
    _check(bt, c, q_out.to(bt.dtype), _slots(bt)[:, None], freq, [0] * 32, False, bt.q)


def test_append_rope_far_and_negative_positions():
    # the bound holds at positions where an fp32 angle has no correct digit left; 64-bit angles of
    # 2^31 positions are themselves off by 2^31 2^-53 of a radian
    bt = Batch([6], [10], 16, 2, 1, 128, "f32", seed=4)
    c, d = bt.cache(kvc), bt.dev()
    freq = _freq(128)
    pos = torch.tensor([[0, 1, -1, -(2 ** 31), 2 ** 31 - 1, 1234567890]], dtype=torch.int32)
    q_out = torch.empty_like(d["q"])
    c.append_rope(0, kvc.Rope(freq), d["q"], d["k"], d["v"], d["table"], d["cu"], d["lens"], q_out, pos.cuda())
    y, w = rotate64(bt.q, pos.T, freq, [0] * 64, False)
    err = (q_out.cpu().double() - y).abs()
    # both sides' double angles: each product off by 2^-53 of itself at most, 2^31 2^-52 together
    assert (err <= w * (12 * U + 2.0 ** -21) + U * y.abs()).all(), float(err.max())


def test_append_rope_flags_and_skips_bad_sequences():
    bt = Batch([2, 3, 1], [4, 40, 9], 16, 4, 2, 64, seed=5)
    freq = _freq(64)
    rope = kvc.Rope(freq)
    for bad in (2, bt.max_blocks * 16 + 1, 2 ** 31 - 1, -5):  # lens[1] below its new tokens / past T_max
        c, d = bt.cache(kvc), bt.dev()
        d["lens"][1] = bad
        q_out = torch.zeros_like(d["q"])
        c.append_rope(0, rope, d["q"], d["k"], d["v"], d["table"], d["cu"], d["lens"], q_out)
        assert c.last_error() == (kvc.KVC_EDEVICE, kvc.KVC_DEV_BAD_LENS)
        K, V = (x.cpu() for x in c.layer_views(0))
        t = bt.table[1].long()
        assert torch.equal(K[t], bt.K[t]) and torch.equal(V[t], bt.V[t])
        assert not q_out[2:5].any() and q_out[:2].any() and q_out[5:].any()
    for bad in (-1, bt.nblocks, 2 ** 31 - 1):
        c, d = bt.cache(kvc), bt.dev()
        d["table"][1, 40 // 16] = bad
        q_out = torch.zeros_like(d["q"])
        c.append_rope(0, rope, d["q"], d["k"], d["v"], d["table"], d["cu"], d["lens"], q_out)
        assert c.last_error() == (kvc.KVC_EDEVICE, kvc.KVC_DEV_BAD_BLOCK)
        K, _ = (x.cpu() for x in c.layer_views(0))
        others = torch.ones(bt.nblocks, dtype=torch.bool)
        for b, slots in ((0, range(4, 6)), (2, range(9, 10))):
            others[[int(bt.table[b, s // 16]) for s in slots]] = False
        assert torch.equal(K[others], bt.K[others])
    for cu in ([1, 2, 5, 6], [0, 3, 2, 6], [0, 2, 5, 7], [0, -1, 5, 6]):
        c, d = bt.cache(kvc), bt.dev()
        d["cu"].copy_(torch.tensor(cu, dtype=torch.int32))
        q_out = torch.zeros_like(d["q"])
        c.append_rope(0, rope, d["q"], d["k"], d["v"], d["table"], d["cu"], d["lens"], q_out)
        assert c.last_error() == (kvc.KVC_EDEVICE, kvc.KVC_DEV_BAD_SEQ)
        K, V = (x.cpu() for x in c.layer_views(0))
        assert torch.equal(K, bt.K) and torch.equal(V, bt.V) and not q_out.any()


def test_append_rope_looks_nothing_up_for_rows_outside_their_sequence():
    # sequence bounds out of order or out of range in the middle: whichever sequence a row falls to, its
    # slot is looked up only if the row lies within it
    bt = Batch([2, 3, 1, 2, 1], [4, 40, 9, 0, 30], 16, 4, 2, 64, seed=6)
    rope = kvc.Rope(_freq(64))
    lo, hi = -2 ** 31, 2 ** 31 - 1
    for cu in ([0, 50, 6, 3, 8, 9], [0, lo, 5, 6, 8, 9], [0, 2, 5, hi, 8, 9], [0, 2, 5, 6, 8, hi], [0, hi, hi, lo, 8, 9],
               [lo, lo, lo, lo, lo, hi]):
        c, d = bt.cache(kvc), bt.dev()
        d["cu"].copy_(torch.tensor(cu, dtype=torch.int32))
        q_out = torch.zeros_like(d["q"])
        c.append_rope(0, rope, d["q"], d["k"], d["v"], d["table"], d["cu"], d["lens"], q_out)
        status, word = c.last_error()
        assert status == kvc.KVC_EDEVICE and word & kvc.KVC_DEV_BAD_SEQ
        K, V = (x.cpu() for x in c.layer_views(0))
        assert torch.equal(K, bt.K) and torch.equal(V, bt.V) and not q_out.any()


def test_append_rope_flags_unsound_bounds_alone():
    # lens below the new tokens and bad table entries say nothing where cu_seqlens is unsound elsewhere
    bt = Batch([2, 3, 1, 2, 1], [4, 40, 9, 0, 30], 16, 4, 2, 64, seed=7)
    rope = kvc.Rope(_freq(64))
    for cu in ([0, 2, 5, 6, 8, 7], [0, 2, 5, 6, 8, 10], [0, 2, 5, 6, 5, 9], [0, 2, -1, 6, 8, 9]):
        for bad in ("lens", "table", "both"):
            c, d = bt.cache(kvc), bt.dev()
            d["cu"].copy_(torch.tensor(cu, dtype=torch.int32))
            if bad != "table":
                d["lens"][:] = 0
            if bad != "lens":
                d["table"][:] = -1
            q_out = torch.zeros_like(d["q"])
            c.append_rope(0, rope, d["q"], d["k"], d["v"], d["table"], d["cu"], d["lens"], q_out)
            assert c.last_error() == (kvc.KVC_EDEVICE, kvc.KVC_DEV_BAD_SEQ), (cu, bad)
            assert not q_out.any()


def test_append_rope_negative_and_tiny_frequencies_at_far_positions():
    # a rate of -x turns back by exactly what x turns; small ones are not rounded to the next whole turn first
    bt = Batch([6], [10], 16, 2, 1, 128, "f32", seed=8)
    pos = torch.tensor([[0, 1, -1, -(2 ** 31), 2 ** 31 - 1, 1234567890]], dtype=torch.int32)
    rates = [1e-9 * 3.0 ** (i / 4) for i in range(64)]
    got = []
    for sign in (1, -1):
        c, d = bt.cache(kvc), bt.dev()
        freq = [sign * f for f in rates]
        q_out = torch.empty_like(d["q"])
        c.append_rope(0, kvc.Rope(freq), d["q"], d["k"], d["v"], d["table"], d["cu"], d["lens"], q_out,
                      (sign * pos.long()).clamp(-2 ** 31, 2 ** 31 - 1).to(torch.int32).cuda())
        y, w = rotate64(bt.q, (sign * pos.long()).clamp(-2 ** 31, 2 ** 31 - 1).T, freq, [0] * 64, False)
        err = (q_out.cpu().double() - y).abs()
        # the reference's angles reach 2^31 x 3.4e-2 < 2^27 radians in double: off by 2^27 2^-53; the fraction by
        # 2^31 2^-62 turns
        assert (err <= w * (12 * U + 2.0 ** -25) + U * y.abs()).all(), float(err.max())
        got.append(q_out)
    rows = [0, 1, 2, 4, 5]  # (-2^31 has no negative)
    assert (got[0][rows] - got[1][rows]).abs().max() < 1e-5


@pytest.mark.parametrize("N", [1, 40])
def test_append_rope_positions_shared_by_the_axes(N):
    # an expanded tensor: one row of positions for all axes, at the end of its memory
    bt = Batch([N], [10], 16, 2, 1, 64, seed=9)
    freq, axis = _freq(64), [i % 3 for i in range(32)]
    pos = torch.randint(0, 5000, (N,), generator=torch.Generator().manual_seed(2)).to(torch.int32)
    rope = kvc.Rope(freq, axis=axis)
    d = bt.dev()
    for p in (pos.cuda()[None].expand(3, N), pos.repeat(3, 2).cuda()[:, :N], pos.repeat(3, 1).cuda()):
        c = bt.cache(kvc)
        q_out = torch.zeros_like(d["q"])
        c.append_rope(0, rope, d["q"], d["k"], d["v"], d["table"], d["cu"], d["lens"], q_out, p)
        assert c.last_error() == (kvc.KVC_OK, 0)
        _check(bt, c, q_out, pos[:, None].expand(N, 3), freq, axis, False, bt.q)
    c = bt.cache(kvc)
    if N > 1:
        overlapping = torch.zeros(200, dtype=torch.int32, device="cuda").as_strided((3, N), (N - 1, 1))
        with pytest.raises(ValueError, match="overlap"):
            c.append_rope(0, rope, d["q"], d["k"], d["v"], d["table"], d["cu"], d["lens"], None, overlapping)

"""Ragged batches at the end of the longest history a paged cache takes, 2^31 - 16 positions of one sequence: tiles
and boxes that reach past 2^31, where a signed sum would turn negative.  The histories repeat one block; each
sequence's last block is its own, its keys score high enough to weigh as much as all positions before it."""
import math

import pytest
import torch

from kv_cache_decode_kvc_gb300 import kvc

pytestmark = pytest.mark.gpu

BS = 16
ONE, TWO = 2 ** 27 - 1, 2 ** 26 - 1  # blocks of a sequence, at most, in a cache of one and of two


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _batch(dtype, D, H_q, new, short):
    """cache, q, block table, cu, lens, and the exact outputs with A = sum p |v|: new[b] tokens that end `short`
    positions before the cache's last."""
    MB = ONE if len(new) == 1 else TWO
    TOP = BS * MB
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator().manual_seed(D)
    u = torch.nn.functional.normalize(torch.randn(D, generator=g, dtype=torch.float64), dim=0)
    a = math.sqrt(math.log(2.0 ** 31) * math.sqrt(D))  # a^2 / sqrt(D) = log of the number of positions
    rows = sum(new)
    q = (a * u + 0.1 * torch.randn(rows, H_q, D, generator=g)).to(dt)
    K = torch.randn(3, 1, BS, D, generator=g)
    K = (K - (K.double() @ u)[..., None] * u).to(dt)  # block 0: scores near 0
    K[1:] = (a * u + 0.1 * torch.randn(2, 1, BS, D, generator=g)).to(dt)
    V = torch.randn(3, 1, BS, D, generator=g).to(dt)
    V[1:, :, BS - short:] = float("nan")  # behind the last position
    c = kvc.PagedKVCache(1, 3, BS, len(new), MB, H_q, 1, D, dtype)
    Kv, Vv = c.layer_views(0)
    Kv.copy_(K)
    Vv.copy_(V)
    out, A = torch.zeros(rows, H_q, D, dtype=torch.float64), torch.zeros(rows, H_q, D, dtype=torch.float64)
    r = 0
    for b, T in enumerate(new):
        for i in range(T):
            n = TOP - short - T + i + 1  # positions the token sees
            times = [(min(n, TOP - BS) - j + BS - 1) // BS for j in range(BS)] + [1] * max(0, n - (TOP - BS))
            k = torch.cat([K[0, 0], K[1 + b, 0]])[:len(times)].double()
            v = torch.cat([V[0, 0], V[1 + b, 0]])[:len(times)].double()
            w = torch.softmax(q[r].double() @ k.T / math.sqrt(D) + torch.tensor(times, dtype=torch.float64).log(), -1)
            out[r], A[r] = w @ v, w @ v.abs()
            r += 1
    i32 = dict(dtype=torch.int32, device="cuda")
    cu = [0]
    for T in new:
        cu.append(cu[-1] + T)
    table = torch.zeros(len(new), MB, **i32)
    table[:, -1] = 1 + torch.arange(len(new))
    return c, q.cuda(), table, torch.tensor(cu, **i32), torch.tensor([TOP - short] * len(new), **i32), out, A


# The test looks for positions lost or read from elsewhere: the last block holds half of a row's weight.  Sums this
# long are allowed what a tensor-core worker's can lose: it adds at most 2^31 / 152 / 16 = 883,012 products of 16
# positions one after the other, each addition off by up to 2^-24 of the sum (no direction is assumed, so 5 %);
# the weights' rounding and the rest are below 2 %.
TOLERANCE = 883012 * 2.0 ** -24 + 0.02


def _check(got, out, A):
    err = (got.cpu().double() - out).abs()
    assert (err <= TOLERANCE * A).all(), float((err / A).max())


@pytest.mark.parametrize("dtype,D,H_q,new", [("bf16", 128, 1, 3), ("bf16", 64, 1, 3), ("bf16", 128, 1, 70),
                                             ("bf16", 64, 4, 33), ("f32", 4, 1, 3), ("f32", 64, 1, 70)])
@pytest.mark.parametrize("short", [0, 3])
def test_the_last_positions(dtype, D, H_q, new, short):
    c, q, table, cu, lens, out, A = _batch(dtype, D, H_q, [new], short)
    got = torch.full_like(q, float("nan"))
    c.attn_ragged(0, q, got, table, cu, lens)
    assert c.last_error() == (kvc.KVC_OK, 0)
    _check(got, out, A)


@pytest.mark.parametrize("dtype,D,H_q", [("bf16", 128, 32), ("bf16", 64, 1), ("f32", 64, 2)])
def test_a_prefix_of_all_but_the_last_block(dtype, D, H_q):
    c, q, table, cu, lens, out, A = _batch(dtype, D, H_q, [3, 2], 3)
    got = torch.full_like(q, float("nan"))
    i32 = dict(dtype=torch.int32, device="cuda")
    c.attn_shared(0, q, got, table, cu, lens, torch.tensor([0, 2], **i32), torch.tensor([BS * (TWO - 1)], **i32))
    assert c.last_error() == (kvc.KVC_OK, 0)
    _check(got, out, A)


def test_append_to_the_last_slots():
    c, q, table, cu, lens, _, _ = _batch("bf16", 128, 2, [5], 0)
    k, v = torch.randn(5, 1, 128, device="cuda").bfloat16(), torch.randn(5, 1, 128, device="cuda").bfloat16()
    before = [x.clone() for x in c.layer_views(0)]
    c.append_rope(0, kvc.Rope([0.0]), q, k, v, table, cu, lens)
    assert c.last_error() == (kvc.KVC_OK, 0)
    for x, old, new in zip(c.layer_views(0), before, (k, v)):
        old[1, :, BS - 5:] = new.transpose(0, 1)
        assert torch.equal(x, old)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("f32", 64)])
@pytest.mark.parametrize("shared", [False, True])
def test_more_work_than_a_call_takes_is_refused(dtype, D, shared):
    # one token of 64 KV heads at the last position: 64 x 2^24 tiles of 128 keys (2^25 of 64)
    dt, i32 = torch.bfloat16 if dtype == "bf16" else torch.float32, dict(dtype=torch.int32, device="cuda")
    c = kvc.PagedKVCache(1, 2, BS, 1, ONE, 64, 64, D, dtype)
    table, q = torch.zeros(1, ONE, **i32), torch.randn(1, 64, D, device="cuda").to(dt)
    out = torch.full_like(q, 7.0)
    cu, lens = torch.tensor([0, 1], **i32), torch.tensor([BS * ONE], **i32)
    ws = torch.full((c.attn_workspace_bytes(1, 1),), 255, dtype=torch.uint8, device="cuda")
    if shared:
        c.attn_shared(0, q, out, table, cu, lens, torch.tensor([0, 1], **i32), torch.tensor([BS], **i32), workspace=ws)
    else:
        c.attn_ragged(0, q, out, table, cu, lens, workspace=ws)
    assert c.last_error() == (kvc.KVC_EDEVICE, kvc.KVC_DEV_TOO_LARGE)
    assert (out == 7.0).all()

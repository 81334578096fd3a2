"""Blocks of the 8-bit paged cache whose scale grows: all codes that they hold move down, whoever writes the scale."""
import pytest
import torch

from fp8_util import Cache64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvc():
    import __graft_entry__
    __graft_entry__.build()
    from kv_cache_decode_kvc_gb300 import kvc
    return kvc


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# a head's keys or values of a block are one warp's, two warps' or four warps'
@pytest.mark.parametrize("bs,H_kv,dtype,D", [(16, 8, "bf16", 128), (64, 8, "bf16", 128), (64, 4, "f32", 64), (32, 4, "bf16", 256),
                                             (64, 2, "bf16", 64), (128, 4, "bf16", 128), (256, 1, "f32", 128)])
@pytest.mark.parametrize("rounds", [1, 2])
def test_all_held_codes_follow_the_scale(kvc, bs, H_kv, dtype, D, rounds):
    # every sequence holds all but the last few rows of a block; the next row is 2^1 to 2^6 times as large, by head
    B, dt = 48, {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    g = torch.Generator().manual_seed(bs + H_kv + D)
    c = kvc.PagedFP8KVCache(1, B, bs, B, 1, H_kv, H_kv, D, dtype)
    r = Cache64(B, H_kv, bs, D)
    table = torch.randperm(B, generator=g).view(B, 1).to(torch.int32)
    lens = [0] * B
    for step in range(1 + rounds):
        new = [bs - rounds - b % 3 for b in range(B)] if step == 0 else [1] * B
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        size = torch.exp2(torch.randint(1, 7, (cu[-1], H_kv, 1), generator=g).float()) ** step
        k, v = ((torch.randn(cu[-1], H_kv, D, generator=g) * size).to(dt) for _ in range(2))
        for b in range(B):
            r.append(table[b], lens[b], new[b], k[cu[b]:cu[b + 1]], v[cu[b]:cu[b + 1]])
            lens[b] += new[b]
        c.append_rope(0, None, None, k.cuda(), v.cuda(), table.cuda(), i32(cu), i32(lens))
        assert c.last_error() == (kvc.KVC_OK, 0)
        K, V, Ks, Vs = (x.cpu() for x in c.layer_views(0))
        assert torch.equal(Ks, r.scales["K"]) and torch.equal(Vs, r.scales["V"])
        assert torch.equal(K, r.codes["K"]) and torch.equal(V, r.codes["V"])

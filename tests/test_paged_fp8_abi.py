"""The 8-bit paged cache: host-side refusals, and the definition that the GPU tests compare with."""
import ctypes
import struct

import pytest
import torch

from fp8_util import F8, Cache64, exponent, quantize, values
from kv_cache_decode_kvc_gb300 import kvc


@pytest.fixture(scope="module")
def lib():
    from kv_cache_decode_kvc_gb300 import build
    build.build()
    return kvc.load()


def test_null_arguments_are_refused(lib):
    out = ctypes.c_void_p(5)
    assert lib.kvc_create_paged_fp8(None, 1, 1, 16, 1, 1, 1, 1, 64, 0) == kvc.KVC_EINVAL
    assert lib.kvc_paged_read(None, 0, 16, 64, 16, 64, 16, 16, 16, 1, None) == kvc.KVC_EINVAL
    assert lib.kvc_paged_append_norm_rope(None, 0, None, 16, 16, 0.0, 16, 16, 16, 16, 16, 16, 16, 16, None, 0, 16, 16, 16,
                                          1, None) == kvc.KVC_EINVAL
    for args, status in (((0, 4, 16, 2, 4, 4, 2, 64, 0), kvc.KVC_EINVAL), ((1, 0, 16, 2, 4, 4, 2, 64, 0), kvc.KVC_EINVAL),
                         ((1, 4, 16, 2, 0, 4, 2, 64, 0), kvc.KVC_EINVAL), ((1, 4, 16, 2, 4, 4, 0, 64, 0), kvc.KVC_EINVAL),
                         ((1, 4, 16, 2, 4, 4, 2, 64, 5), kvc.KVC_EINVAL), ((1, 4, 24, 2, 4, 4, 2, 64, 0), kvc.KVC_EUNSUPPORTED),
                         ((1, 4, 16, 2, 4, 4, 2, 32, 0), kvc.KVC_EUNSUPPORTED), ((1, 4, 16, 2, 4, 4, 2, 4, 1), kvc.KVC_EUNSUPPORTED),
                         ((1, 4, 256, 2, 1 << 23, 4, 2, 64, 0), kvc.KVC_ERANGE),
                         ((1, 4, 256, 2, 4, 1 << 15, 1 << 15, 256, 0), kvc.KVC_ERANGE)):
        out = ctypes.c_void_p(5)
        assert lib.kvc_create_paged_fp8(ctypes.byref(out), *args) == status and out.value is None


def test_calls_by_a_block_of_arguments_are_refused(lib):
    # an unknown call, another number of arguments, none, not aligned, an int past 32 bits; the calls' own refusals (no handle)
    counts = {0: 18, 1: 21, 2: 11, 3: 13, 4: 16}
    for call, n in counts.items():
        words = struct.pack(f"={n + 1}q", *[0] * (n + 1))
        for c, w, m in ((call, words, n), (call, words, n - 1), (call, words, n + 1), (call, None, n), (-1, words, n), (5, words, n)):
            assert lib.kvc_call(c, w, m) == kvc.KVC_EINVAL
        buf = ctypes.create_string_buffer(8 * n + 8)
        assert lib.kvc_call(call, ctypes.addressof(buf) + 4, n) == kvc.KVC_EINVAL
        wide = [0] * n
        wide[1] = 1 << 32
        assert lib.kvc_call(call, struct.pack(f"={n}q", *wide), n) == kvc.KVC_EINVAL


@pytest.mark.parametrize("amax,e", [(448.0, 0), (449.0, 1), (448 * 2.0 ** -64, -64), (0.0, -64), (1e-30, -64), (1.0, -8),
                                    (1.75, -8), (1.76, -7), (2.0, -7), (3.38e38, 120), (448 * 2.0 ** -63, -63)])
def test_exponent(amax, e):
    assert int(exponent(torch.tensor(amax))) == e


def test_quantized_values_are_within_half_a_step():
    g = torch.Generator().manual_seed(0)
    x = torch.randn(5, 2, 16, 64, generator=g) * torch.exp2(torch.randint(-30, 30, (5, 2, 1, 1), generator=g).float())
    c, s = quantize(x)
    err = (values(c, s) - x.double()).abs()
    assert (err <= x.double().abs() * 2.0 ** -4 + s.double()[..., None, None] * 2.0 ** -10).all()
    assert (c.view(F8).float().abs().amax((2, 3)) > 223).all()


def test_the_definition_token_by_token():
    # a block's scale only grows while it holds tokens, and earlier codes follow it
    c = Cache64(2, 1, 16, 64)
    g = torch.Generator().manual_seed(0)
    x = torch.randn(16, 1, 64, generator=g).double() * torch.exp2(torch.arange(16.0) - 8).double()[:, None, None]
    last = 0.0
    for i in range(16):
        c.append([0], i, 1, x[i:i + 1], x[i:i + 1])
        assert float(c.scales["K"][0, 0]) >= last
        last = float(c.scales["K"][0, 0])
        got = values(c.codes["K"], c.scales["K"])[0, 0, :i + 1]
        assert ((got - x[:i + 1, 0]).abs() <= x[:i + 1, 0].abs() * 2.0 ** -4 + last * 2.0 ** -9).all()


class _On:
    """What the binding's checks see of a tensor on GPU `device` (no GPU needed)."""

    def __init__(self, t, device):
        self.t, self.n, self.device = t, device, f"cuda:{device}"
        self.is_cuda, self.shape, self.dtype = True, t.shape, t.dtype

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return self.n


def test_tensors_on_another_device_are_refused(monkeypatch):
    called = []
    monkeypatch.setattr(kvc, "_device", lambda: 0)
    monkeypatch.setattr(kvc, "_current_stream", lambda device=None: 0)
    for name in ("kvc_paged_append_norm_rope", "kvc_paged_read"):
        monkeypatch.setattr(kvc, name, lambda *a, name=name: called.append(name))
    c = kvc.PagedFP8KVCache.__new__(kvc.PagedFP8KVCache)
    c.h, c.dtype_code = None, kvc.KVC_BF16
    c.B, c.max_blocks, c.H_q, c.H_kv, c.D = 2, 5, 4, 2, 64
    rope = kvc.Rope.__new__(kvc.Rope)
    rope.r, rope.n_axes = None, 2

    def i32(*shape):
        return torch.zeros(shape, dtype=torch.int32)

    bf = dict(dtype=torch.bfloat16)
    batch = dict(block_table=i32(2, 5), cu_seqlens=i32(3), lens=i32(2))
    append = dict(batch, q=torch.zeros(3, 4, 64, **bf), k=torch.zeros(3, 2, 64, **bf), v=torch.zeros(3, 2, 64, **bf),
                  q_out=torch.zeros(3, 4, 64, **bf), positions=i32(2, 3), q_norm=torch.zeros(64, **bf),
                  k_norm=torch.zeros(64, **bf))
    read = dict(batch, k_out=append["k"], v_out=append["v"])
    for call, args in ((lambda **a: c.append_rope(0, rope, **a), append), (lambda **a: c.read(0, **a), read)):
        here = {k: _On(v, 0) for k, v in args.items()}
        called.clear()
        call(**here)
        assert len(called) == 1
        for k in args:
            with pytest.raises(ValueError, match="current device"):
                call(**dict(here, **{k: _On(args[k], 1)}))
        assert len(called) == 1

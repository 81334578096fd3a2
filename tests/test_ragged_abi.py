"""Host-side checks of the ragged calls: rotary tables and refusals that need no GPU."""
import ctypes

import pytest

from kv_cache_decode_kvc_gb300 import kvc


@pytest.fixture(scope="module")
def lib():
    from kv_cache_decode_kvc_gb300 import build
    build.build()
    return kvc.load()


def test_rope_create_and_destroy(lib):
    r = kvc.Rope([1.0, 0.1, 0.01], layout="adjacent", axis=[0, 2, 1], scale=0.5)
    assert r.rot_dim == 6 and r.n_axes == 3 and r.r
    r.close()
    assert lib.kvc_rope_destroy(None) == kvc.KVC_OK


@pytest.mark.parametrize("rot,freq,layout,axes,axis,scale,status", [
    (0, [1.0], 0, 1, None, 1.0, kvc.KVC_EINVAL),
    (3, [1.0, 1.0], 0, 1, None, 1.0, kvc.KVC_EINVAL),
    (4, [1.0, float("inf")], 0, 1, None, 1.0, kvc.KVC_EINVAL),
    (4, [1.0, float("nan")], 0, 1, None, 1.0, kvc.KVC_EINVAL),
    (4, [1.0, 1.0], 2, 1, None, 1.0, kvc.KVC_EINVAL),
    (4, [1.0, 1.0], 0, 0, None, 1.0, kvc.KVC_EINVAL),
    (4, [1.0, 1.0], 0, 2, [0, 2], 1.0, kvc.KVC_EINVAL),
    (4, [1.0, 1.0], 0, 2, [0, -1], 1.0, kvc.KVC_EINVAL),
    (4, [1.0, 1.0], 0, 1, None, float("nan"), kvc.KVC_EINVAL),
    (258, [1.0] * 129, 0, 1, None, 1.0, kvc.KVC_EUNSUPPORTED),
    (4, [1.0, 1.0], 0, 9, None, 1.0, kvc.KVC_EUNSUPPORTED),
])
def test_rope_create_refuses(lib, rot, freq, layout, axes, axis, scale, status):
    out = ctypes.c_void_p(5)
    f = (ctypes.c_double * len(freq))(*freq)
    a = None if axis is None else (ctypes.c_int32 * len(axis))(*axis)
    assert lib.kvc_rope_create(ctypes.byref(out), rot, f, layout, axes, a, scale) == status
    assert out.value is None


def test_rope_create_refuses_null(lib):
    out = ctypes.c_void_p(5)
    assert lib.kvc_rope_create(None, 4, None, 0, 1, None, 1.0) == kvc.KVC_EINVAL
    assert lib.kvc_rope_create(ctypes.byref(out), 4, None, 0, 1, None, 1.0) == kvc.KVC_EINVAL
    with pytest.raises(ValueError):
        kvc.kvc_rope_create(4, [1.0])
    with pytest.raises(kvc.KvcError):
        kvc.Rope([1.0, float("inf")])


def test_null_handles_are_refused(lib):
    r = kvc.Rope([1.0])
    n = ctypes.c_uint64()
    assert lib.kvc_paged_append_rope(None, 0, r.r, 16, 16, 16, 16, 16, 16, 16, 16, None, 0, 16, 16, 16, 1,
                                     None) == kvc.KVC_EINVAL
    assert lib.kvc_paged_attn_ragged(None, 0, 16, 16, 16, 16, 16, 16, 16, 1, 256, 1 << 40, None) == kvc.KVC_EINVAL
    assert lib.kvc_paged_attn_shared(None, 0, 16, 16, 16, 16, 16, 16, 16, 1, 16, 16, 1, 256, 1 << 40,
                                     None) == kvc.KVC_EINVAL
    assert lib.kvc_paged_attn_workspace(None, 1, 0, ctypes.byref(n)) == kvc.KVC_EINVAL


def test_tensors_on_the_host_are_refused():
    import torch
    x, i = torch.zeros(3, 2, 64), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="on the GPU"):
        kvc._packed(x, 2, 64, torch.float32, "q")
    with pytest.raises(ValueError, match="on the GPU"):
        kvc._index(i, "lens", torch.int32, 4)


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
    # every tensor of the two calls in turn, on device 1 while the cache and the current device are 0; a call whose
    # tensors are all in place reaches the library
    import torch
    called = []
    monkeypatch.setattr(kvc, "_device", lambda: 0)
    monkeypatch.setattr(kvc, "_current_stream", lambda device=None: 0)
    for name in ("kvc_paged_append_rope", "kvc_paged_attn_ragged", "kvc_paged_attn_shared"):
        monkeypatch.setattr(kvc, name, lambda *a, name=name: called.append(name))
    c = kvc.PagedKVCache.__new__(kvc.PagedKVCache)
    c.h, c.dtype_code = None, kvc.KVC_BF16
    c.B, c.max_blocks, c.H_q, c.H_kv, c.D = 2, 5, 4, 2, 64
    rope = kvc.Rope.__new__(kvc.Rope)
    rope.r, rope.n_axes = None, 2

    def i32(*shape):
        return torch.zeros(shape, dtype=torch.int32)

    bf = dict(dtype=torch.bfloat16)
    batch = dict(block_table=i32(2, 5), cu_seqlens=i32(3), lens=i32(2))
    append = dict(batch, q=torch.zeros(3, 4, 64, **bf), k=torch.zeros(3, 2, 64, **bf), v=torch.zeros(3, 2, 64, **bf),
                  q_out=torch.zeros(3, 4, 64, **bf), positions=i32(2, 3))
    attn = dict(batch, q=append["q"], out=append["q_out"], workspace=torch.zeros(64, dtype=torch.uint8))
    shared = dict(attn, groups=i32(2), prefix_lens=i32(1))
    for call, args in ((lambda **a: c.append_rope(0, rope, **a), append), (lambda **a: c.attn_ragged(0, **a), attn),
                       (lambda **a: c.attn_shared(0, **a), shared)):
        here = {k: _On(v, 0) for k, v in args.items()}
        called.clear()
        call(**here)
        assert len(called) == 1
        for k in args:
            with pytest.raises(ValueError, match="current device"):
                call(**dict(here, **{k: _On(args[k], 1)}))
        assert len(called) == 1

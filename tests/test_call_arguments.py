"""What the binding takes for a handle and an address: integers of any subclass, ctypes pointers, None."""
import ctypes
import enum
import struct

import pytest

from kv_cache_decode_kvc_gb300 import kvc


class Address(int):
    pass


class Number(enum.IntEnum):
    FIVE = 5


class Words:
    """Stands for the library: keeps the words of a call."""

    def kvc_call(self, call, words, n):
        self.words = struct.unpack(f"={n}q", words)
        return 0


CALLS = {  # name, arguments up to the stream: handles h and r, an address a
    "kvc_paged_append_rope": lambda h, r, a: (h, 0, r, a, 64, a, 64, a, 64, a, 64, None, 0, a, a, a, 1),
    "kvc_paged_append_norm_rope": lambda h, r, a: (h, 0, r, a, a, 0.0, a, 64, a, 64, a, 64, a, 64, None, 0, a, a, a, 1),
    "kvc_paged_read": lambda h, r, a: (h, 0, a, 64, a, 64, a, a, a, 1),
    "kvc_paged_attn_ragged": lambda h, r, a: (h, 0, a, 64, a, 64, a, a, a, 1, a, 256),
    "kvc_paged_attn_shared": lambda h, r, a: (h, 0, a, 64, a, 64, a, a, a, 1, a, a, 1, a, 256),
}


@pytest.mark.parametrize("name", CALLS)
def test_steps_take_integers_of_a_subclass_and_ctypes_handles(monkeypatch, name):
    lib = Words()
    monkeypatch.setattr(kvc, "_lib", lib)
    call = getattr(kvc, name)
    call(*CALLS[name](48, 80, 4096), stream=0)
    want = lib.words
    assert want[0] == 48 and 4096 in want
    for h, r, a in ((Address(48), Address(80), Address(4096)), (ctypes.c_void_p(48), ctypes.c_void_p(80), 4096),
                    (ctypes.c_void_p(48), Address(80), Address(4096))):
        call(*CALLS[name](h, r, a), stream=Address(0))
        assert lib.words == want
    call(*CALLS[name](ctypes.c_void_p(), None, Number.FIVE), stream=0)
    assert lib.words[0] == 0 and 5 in lib.words


def test_addresses():
    assert kvc._ptr(Address(7)) == 7 and kvc._ptr(Number.FIVE) == 5 and kvc._ptr(None) is None
    assert kvc._addr(None) == 0 and kvc._addr(ctypes.c_void_p()) == 0 and kvc._addr(ctypes.c_void_p(9)) == 9
    for wrong in ("x", 1.5, object()):
        with pytest.raises(TypeError):
            kvc._addr(wrong)

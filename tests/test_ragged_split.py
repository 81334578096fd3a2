"""Host arithmetic of the ragged calls, compiled from their headers and compared with exact values: the cost sums that
split a batch over the workers (a wrong sum would put a stream's start, and with it every lookup of its keys,
in the wrong place), and the rotary frequencies as fractions of a turn."""
import ctypes
import decimal
import random
import subprocess

import pytest

from kv_cache_decode_kvc_gb300 import build

SOURCE = r"""
#include "kvc_ragged.cuh"
using namespace kvc;
static Entry entry(int T, int L, int pfx, int group) {
    Entry s;
    s.row0 = 0; s.T = T; s.L = L; s.pfx = pfx; s.seq = 0; s.group = group != 0; s.ok = true; s.bad = false;
    return s;
}
template <class R> static int units(int lgG, int T, int L, int pfx, int group) {
    RaggedParams p{};
    p.lgG = lgG;
    const Entry s = entry(T, L, pfx, group);
    return R::cost(p, s, R::cls(p, s));
}
template <class R> static float about(int lgG, int T, int L, int pfx, int group) {
    RaggedParams p{};
    p.lgG = lgG;
    const Entry s = entry(T, L, pfx, group);
    return R::cost_about(p, s, R::cls(p, s));
}
extern "C" float ragged_about(int kind, int lgG, int T, int L, int pfx, int group) {
    return kind == 0   ? about<Ragged<8, 7, true, true>>(lgG, T, L, pfx, group)
           : kind == 1 ? about<Ragged<6, 6, false, true>>(lgG, T, L, pfx, group)
                       : about<Ragged<6, 5, false, true>>(lgG, T, L, pfx, group);
}
extern "C" uint64_t turns(double rate) { return rope_turns(rate); }
extern "C" float ragged_most() { return Ragged<8, 7, true, true>::MOST; }
extern "C" int ragged_units(int kind, int lgG, int T, int L, int pfx, int group) {
    return kind == 0   ? units<Ragged<8, 7, true, true>>(lgG, T, L, pfx, group)
           : kind == 1 ? units<Ragged<6, 6, false, true>>(lgG, T, L, pfx, group)
                       : units<Ragged<6, 5, false, true>>(lgG, T, L, pfx, group);
}
"""
KINDS = [(8, 7, True), (6, 6, False), (6, 5, False)]  # log2 of a tile's rows and keys; classes


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    at = tmp_path_factory.mktemp("split")
    (at / "split.cu").write_text(SOURCE)
    subprocess.run(["nvcc", *build.ARCH, *build.FLAGS, "-I", build.CSRC, "-shared", "-cudart", "static", "-o",
                    str(at / "split.so"), str(at / "split.cu")], check=True, capture_output=True)
    so = ctypes.CDLL(str(at / "split.so"))
    so.turns.argtypes, so.turns.restype = [ctypes.c_double], ctypes.c_uint64
    so.ragged_about.restype = so.ragged_most.restype = ctypes.c_float
    return so


def _exact(kind, lgG, T, L, pfx, group):
    """Units of one KV head of an entry: its streams one by one."""
    lrt, lkt, pairs = KINDS[kind]
    tile = 2 if pairs else 1
    start = 1 if not pairs else 6 if T << lgG > 64 else 3
    TQ, n, streams = 1 << (lrt - lgG), 0, -(-T // (1 << (lrt - lgG)))
    for k in range(streams):
        last = pfx if group else L - T - pfx + min((k + 1) * TQ, T)
        n += (last + (1 << lkt) - 1) >> lkt
    return n * tile + streams * start


@pytest.mark.parametrize("kind", range(3))
def test_units_of_entries_near_and_far(lib, kind):
    rng = random.Random(kind)
    top = 2 ** 31 - 16  # the most positions a paged cache holds
    cases = [(5, 1, top, 0, 0), (0, 1, top, 0, 0), (0, 1000, top, 0, 0), (0, 7, top, top, 1), (2, 900, top, top - 1000, 0),
             (5, 3, 2 ** 30, 0, 0), (0, 1, 1, 0, 0), (3, 4096, 4096, 0, 0)]
    for _ in range(600):
        T = rng.choice([1, 2, rng.randint(1, 70), rng.randint(1, 3000)])
        L = min(top, T + int(2 ** rng.uniform(0, 31)))
        pfx = rng.choice([0, rng.randint(0, (L - T) // 16) * 16])
        cases.append((rng.randint(0, 5), T, L, pfx, int(rng.random() < 0.2 and pfx > 0)))
    tried = 0
    for c in cases:
        want = _exact(kind, *c)
        if want < 2 ** 31:
            tried += 1
            assert lib.ragged_units(kind, *c) == want, c
    assert tried > 400


@pytest.mark.parametrize("kind", range(3))
def test_estimates_refuse_what_32_bits_do_not_hold_and_little_else(lib, kind):
    # the estimate is no less than the cost (up to fp32's rounding, 2^-20 for its few steps) and more by at most
    # 2.5 tiles a stream (a rounded-up tile, and for the last, partial stream up to 256 keys' tiles of difference)
    lrt, lkt, pairs = KINDS[kind]
    rng = random.Random(10 + kind)
    top, tile = 2 ** 31 - 16, 2 if pairs else 1
    assert lib.ragged_most() * (1 + 2.0 ** -20) < 2 ** 31
    for _ in range(400):
        lgG, T = rng.randint(0, 5), rng.choice([1, rng.randint(1, 100), int(2 ** rng.uniform(0, 16))])
        L = min(top, T + int(2 ** rng.uniform(0, 31)))
        pfx = rng.choice([0, rng.randint(0, (L - T) // 16) * 16])
        c = (lgG, T, L, pfx, int(rng.random() < 0.2 and pfx > 0))
        want, est, streams = _exact(kind, *c), lib.ragged_about(kind, *c), -(-T // (1 << (lrt - lgG)))
        assert want * (1 - 2.0 ** -20) <= est <= want * (1 + 2.0 ** -20) + tile * (streams + 1.5 * (256 >> lkt)), (c, want, est)


def test_long_prompts_are_within_the_limit(lib):
    # 64 heads on 8: a prompt of 800,000 tokens is 1.25 10^9 units, one of 1,000,000 1.95 10^9; 1,100,000 are too many
    for T, fits in ((500000, True), (733000, True), (800000, True), (1000000, True), (1100000, False)):
        c = (0, 3, T, T, 0, 0)
        assert (8 * lib.ragged_about(*c) <= lib.ragged_most()) == fits, T
        assert (8 * _exact(*c) < 2 ** 31) == fits, T


def test_frequencies_as_fractions_of_a_turn(lib):
    # 80 digits of 1 / (2 pi); the fraction is within 2^-62 of a turn, 4 units, for rates of up to 2^44 of either sign
    with decimal.localcontext() as ctx:
        ctx.prec = 80
        pi = decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")
        rng = random.Random(5)
        rates = [0.0, 1.0, 0.5, 2.0 ** 44, 6.283185307179586, 3.141592653589793, 1e-6, 1e-19, 1e-300, 5e-324]
        rates += [10000.0 ** (-i / 64) for i in range(64)] + [2 ** rng.uniform(-70, 44) for _ in range(3000)]
        for f in rates:
            want = decimal.Decimal(f) / (2 * pi) * 2 ** 64
            for sign in (1, -1):
                off = (decimal.Decimal(lib.turns(sign * f)) - sign * want) % 2 ** 64
                assert min(abs(off), abs(2 ** 64 - abs(off))) <= 4, (sign * f, off)
        for f in (2.0 ** 60, 1e30, 1e308, -1e308):  # whatever the fraction, no overflow
            assert 0 <= lib.turns(f) < 2 ** 64

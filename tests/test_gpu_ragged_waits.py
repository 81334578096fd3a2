"""Waits of the ragged attention kernel that last as long as the work they wait for: no limit runs out."""
import ctypes
import subprocess

import pytest
import torch

from kv_cache_decode_kvc_gb300 import build, kvc

from ragged_util import Batch, attention64, check_attention

pytestmark = pytest.mark.gpu

# One block that lets the kernel behind it start at once and ends by itself after ms milliseconds.
LINGER = r"""
#include <cuda_runtime.h>
#include <stdint.h>
__global__ void linger(uint64_t ns) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    uint64_t t0, t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t0));
    for (int i = 0; i < 100000; ++i) {  // 100,000 naps of 50 us: 5 s at most
        __nanosleep(50000);
        asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
        if (t - t0 > ns) break;
    }
}
extern "C" int launch_linger(int ms, void* stream) {
    linger<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>((uint64_t)ms * 1000000ull);
    return (int)cudaGetLastError();
}
"""


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.fixture(scope="module")
def linger(tmp_path_factory):
    at = tmp_path_factory.mktemp("linger")
    (at / "linger.cu").write_text(LINGER)
    subprocess.run(["nvcc", *build.ARCH, "-shared", "-Xcompiler", "-fPIC", "-cudart", "static", "-o",
                    str(at / "linger.so"), str(at / "linger.cu")], check=True, capture_output=True)
    fn = ctypes.CDLL(str(at / "linger.so")).launch_linger
    fn.argtypes, fn.restype = [ctypes.c_int, ctypes.c_void_p], ctypes.c_int
    return fn


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("shared", [False, True])
def test_behind_a_kernel_that_releases_its_dependents_and_runs_on(linger, D, shared):
    bt = Batch([3, 90, 1], [200, 130, 129], 32, 4, 2, D, "bf16", [0, 3], [128], seed=40)
    c, d = bt.cache(kvc), bt.dev()
    out = torch.full((bt.rows, 4, D), float("nan"), dtype=bt.dtype, device="cuda")
    ws = torch.empty(c.attn_workspace_bytes(bt.rows, 1), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert linger(2300, torch.cuda.current_stream().cuda_stream) == 0  # a wait's limit is 2 s
    if shared:
        c.attn_shared(0, d["q"], out, d["table"], d["cu"], d["lens"], d["groups"], d["prefix"], workspace=ws)
    else:
        c.attn_ragged(0, d["q"], out, d["table"], d["cu"], d["lens"], workspace=ws)
    assert c.last_error() == (kvc.KVC_OK, 0)
    check_attention(out, bt, attention64(bt), True)


def test_single_tokens_behind_seconds_of_prompts():
    # one worker takes in a prompt of 131,072 tokens (more than 2 s, a wait's limit), then single tokens of two
    # other sequences: their hand-over begins when the prompt is done
    T, H, D, bs, long = 131072, 8, 128, 256, 700
    new, hist = [T, 1, 1], [0, long, 130]
    lens = [n + h for n, h in zip(new, hist)]
    blocks = [-(-L // bs) for L in lens]
    c = kvc.PagedKVCache(1, sum(blocks), bs, 3, blocks[0], H, H, D)
    K, V = c.layer_views(0)
    g = torch.Generator("cuda").manual_seed(41)
    for x in (K, V):
        x.copy_(torch.randn(x.shape, dtype=x.dtype, device="cuda", generator=g))
    table = torch.zeros(3, blocks[0], dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(blocks):
        table[b, :n] = torch.arange(at, at + n)
        at += n
    i32 = dict(dtype=torch.int32, device="cuda")
    cu, ln = torch.tensor([0, T, T + 1, T + 2], **i32), torch.tensor(lens, **i32)
    q = torch.randn(T + 2, H, D, dtype=torch.bfloat16, device="cuda", generator=g)
    out = torch.full_like(q, float("nan"))
    ws = torch.empty(c.attn_workspace_bytes(T + 2), dtype=torch.uint8, device="cuda")
    c.set_ctas(1)
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    ev[0].record()
    c.attn_ragged(0, q, out, table, cu, ln, workspace=ws)
    ev[1].record()
    assert c.last_error() == (kvc.KVC_OK, 0)
    assert ev[0].elapsed_time(ev[1]) > 2100  # else the sizes no longer make the case
    assert out.isfinite().all()
    for row, b, n in [(0, 0, 1), (1, 0, 2), (300, 0, 301), (T // 2, 0, T // 2 + 1), (T - 1, 0, T), (T, 1, long + 1),
                      (T + 1, 2, 131)]:
        t = torch.arange(n, device="cuda")
        at = table[b, t // bs].long(), t % bs
        for h in (0, 7):
            Kb, Vb = (x[at[0], h, at[1]].cpu().double() for x in (K, V))
            p = torch.softmax(Kb @ q[row, h].cpu().double() / D ** 0.5, 0)
            want, A, got = p @ Vb, p @ Vb.abs(), out[row, h].cpu().double()
            # the weights' and the output's rounding to bf16, and as much again of the first for the fp32 sums
            assert ((got - want).abs() <= 2.0 ** -7 * A + 2.0 ** -8 * want.abs()).all(), (row, h)

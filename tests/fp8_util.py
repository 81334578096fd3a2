"""The paged cache held in 8 bits: its definition in 64 bits, inputs, tolerances.

Values are E4M3 codes times a power of two per block and head, so a double holds them exactly; E4M3
rounding itself is torch's cast of an fp32 value that is exact there (a 4-bit code moved by a power of two)
or, for new values, of the double rounded to fp32 first (off by 2^-25 of it, which moves the result only at a
tie: such values are compared by distance, not by bits)."""
import torch

from ragged_util import Batch, U, rotate64

F8 = torch.float8_e4m3fn
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def exponent(amax):
    """Smallest e >= -64 with amax <= 448 2^e."""
    m, e = torch.frexp(amax.double())
    e = torch.where(amax > 0, e - 9 + (m > 0.875).to(e.dtype), -64)
    return e.clamp(min=-64)


def quantize(x):
    """x [nb, H, bs, D] -> (codes uint8, scales fp32 [nb, H]), every block on its own."""
    x = x.double()
    scale = torch.exp2(exponent(x.abs().amax((2, 3))).double())
    return (x / scale[..., None, None]).float().to(F8).view(torch.uint8), scale.float()


def values(codes, scales):
    return codes.view(F8).double() * scales.double()[..., None, None]


class Cache64:
    """K and V of one layer as codes and scales on the CPU, appended to block by block."""

    def __init__(self, nblocks, H, bs, D):
        self.bs, self.H = bs, H
        self.codes = {x: torch.zeros(nblocks, H, bs, D, dtype=torch.uint8) for x in "KV"}
        self.scales = {x: torch.zeros(nblocks, H) for x in "KV"}
        self.exact = {x: torch.zeros(nblocks, H, bs, D, dtype=torch.float64) for x in "KV"}  # new rows before rounding

    def append(self, table, hist, new, k, v):
        """k, v [new, H, D] in 64 bits of one sequence to positions hist .. (table row: python list)."""
        bs = self.bs
        for j in range(hist // bs, (hist + new - 1) // bs + 1):
            e, lo, hi = int(table[j]), max(hist, j * bs), min(hist + new, (j + 1) * bs)
            held = max(0, hist - j * bs)
            for x, y in (("K", k), ("V", v)):
                y = y[lo - hist:hi - hist].transpose(0, 1).double()  # [H, rows, D]
                fin = torch.where(torch.isfinite(y), y.abs(), 0)
                now = exponent(fin.amax((1, 2)))
                if held:
                    old = torch.log2(self.scales[x][e].double()).clamp(-64, 120).to(now.dtype)
                    now = torch.maximum(now, old)
                    c = self.codes[x][e, :, :held].view(F8).double()
                    self.codes[x][e, :, :held] = (c * torch.exp2((old - now).double())[:, None, None]).float().to(
                        F8).view(torch.uint8)
                s = torch.exp2(now.double())[:, None, None]
                lim = torch.where(now == 120, 240.0, 448.0).double()[:, None, None]
                z = (y / s).clamp(-lim, lim)
                z = torch.where(torch.isfinite(y), z, float("nan"))
                self.codes[x][e, :, lo - j * bs:hi - j * bs] = z.float().to(F8).view(torch.uint8) & torch.where(
                    torch.isnan(z), 0x7F, 0xFF).to(torch.uint8)
                self.exact[x][e, :, lo - j * bs:hi - j * bs] = z
                self.scales[x][e] = torch.exp2(now.double()).float()


def norm64(x, w, eps):
    x = x.double()
    return x if w is None else x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()


def turned(x, w, eps, pos, inv_freq, adjacent, axis=None):
    """Normalised and rotated in 64 bits, and the fp32 kernel's error bound: the norm's factor is off by
    (D / 2 + 8) u (half the D roundings of the sum of squares, its division and sum, rsqrtf's 2 ulp, two
    products), the rotation by 12 u (|y1| + |y2|) (ragged_util)."""
    y = norm64(x, w, eps)
    rel = 0.0 if w is None else (x.shape[-1] / 2 + 8) * U
    if inv_freq is None:
        return y, y.abs() * rel
    z, both = rotate64(y, pos if pos.dim() == 2 else pos[:, None], inv_freq, axis or [0] * len(inv_freq), adjacent)
    still = both == 0  # not rotated (or both 0)
    return z, torch.where(still, z.abs() * rel, both * (12 * U + rel))


class Batch8(Batch):
    """A Batch whose pools are quantized: K8, V8 codes, Ks, Vs scales, and K, V their values."""

    def __init__(self, *a, mag=None, **kw):
        super().__init__(*a, **kw)
        if mag is not None:
            g = torch.Generator().manual_seed(kw.get("seed", 0) + 1)
            for n in "KV":
                x = getattr(self, n).float()
                setattr(self, n, x * torch.exp2(torch.rand(x.shape[:2], generator=g) * 2 * mag - mag)[..., None, None])
        self.requantize()

    def requantize(self):
        self.K8, self.Ks = quantize(self.K)
        self.V8, self.Vs = quantize(self.V)
        self.K, self.V = values(self.K8, self.Ks), values(self.V8, self.Vs)

    def cache(self, kvc, layers=1, layer=0):
        c = kvc.PagedFP8KVCache(layers, self.nblocks, self.bs, self.B, self.max_blocks, self.H_q, self.H_kv, self.D,
                                self.name)
        for view, x in zip(c.layer_views(layer), (self.K8, self.V8, self.Ks, self.Vs)):
            view.copy_(x)
        torch.cuda.synchronize()
        return c


def smallest_weights(bt):
    """What the outputs may be off by where weights are small: a weight times its block's scale of V, scaled so that a row's largest
    is above 2^3, is cut into f16, off by half of 2^-24 there, and its third term, 1/64 of an E5M2 value, by half of 2^-16 / 64:
    2^-23 + 2^-25 together, at most (2^-26 + 2^-28) of the row's largest.  It meets the code."""
    out = torch.zeros(bt.rows, bt.H_q, bt.D, dtype=torch.float64)
    G = bt.H_q // bt.H_kv
    for b in range(bt.B):
        for h in range(bt.H_kv):
            t = torch.arange(bt.lens[b])
            e = bt.table[b, t // bt.bs].long()
            K, V, s = bt.K[e, h, t % bt.bs], bt.V[e, h, t % bt.bs], bt.Vs[e, h].double().clamp(min=2.0 ** -64)
            for i in range(bt.new[b]):
                n, r = bt.hist[b] + i + 1, bt.cu[b] + i
                p = torch.softmax(bt.q[r, h * G:(h + 1) * G].double() @ K[:n].T / bt.D ** 0.5, -1)
                codes = (V[:n].abs() / s[:n, None]).sum(0)
                out[r, h * G:(h + 1) * G] = (2.0 ** -26 + 2.0 ** -28) * (p * s[:n]).amax(-1, keepdim=True) * codes
    return out

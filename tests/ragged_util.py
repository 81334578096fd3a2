"""Ragged batches over a paged cache: inputs, the 64-bit plain implementations the GPU tests compare
with, and the tolerances.

Tolerances are bounds, term by term (u = 2^-24 for fp32, ub = 2^-8 for bf16: half a step relative to
the value):
  rotation: y = x1 c - x2 s.  c and s come from an angle in half-turns x in [-1, 1) that is cut to 32
    bits (2^-31) and rounded to fp32 (u), so the angle is off by pi (2^-31 + u) < 3.3 u; sincospif
    adds at most 2 ulp of a value up to 1 (4 u), a scale and two products and a sum 4 u:
    |dy| <= (|x1| + |x2|) scale 12 u + (the cache dtype's rounding of y).
  attention: a score is a sum of D products: |ds| <= (D + 3) u X with X = sum |q k| / sqrt(D) (the
    three more: q's scale, the product with log2 e, the subtraction of the maximum, which is at most
    X in size), at most ds_max over the row; a weight is off by 2 ds_max (its own score's error and
    the maximum's) plus 2^-22 of ex2.approx; the two sums over T positions add T u each, the final
    division 2 u.  With A = sum p |v| / sum p:
    |do| <= A (4 ds_max + 2^-21 + 2 T u + 4 u) + rounding of the output (its dtype's half step).
    Weights rounded to bf16 (tensor cores) add ub A.  Both weights and sums count twice: once in the
    numerator, once in the denominator."""
import math

import torch

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
U = 2.0 ** -24


class Batch:
    """new[b] tokens behind hist[b] positions (the shared prefix included), block tables in a random
    order of a pool with spare blocks; sequences of a group [start[g], start[g + 1]) name the same
    blocks for the whole blocks of prefix[g]."""

    def __init__(self, new, hist, bs, H_q, H_kv, D, dtype="bf16", start=None, prefix=None, pad=0, seed=0,
                 spare=3, q_scale=1.0):
        self.new, self.hist, self.bs, self.H_q, self.H_kv, self.D = list(new), list(hist), bs, H_q, H_kv, D
        self.dtype, self.name, self.B = DT[dtype], dtype, len(new)
        self.start = list(start) if start else [0, self.B]
        self.prefix = list(prefix) if prefix else [0] * (len(self.start) - 1)
        self.lens = [n + h for n, h in zip(new, hist)]
        self.max_blocks = max(1, -(-max(self.lens) // bs)) + 1
        g = torch.Generator().manual_seed(seed)
        self.nblocks = self.B * self.max_blocks + spare
        self.table = torch.randperm(self.nblocks, generator=g)[:self.B * self.max_blocks].view(
            self.B, self.max_blocks).to(torch.int32)
        for a, b, p in zip(self.start, self.start[1:], self.prefix):
            for s in range(a + 1, b):
                self.table[s, :p // bs] = self.table[a, :p // bs]
        self.cu = [0]
        for n in self.new:
            self.cu.append(self.cu[-1] + n)
        self.n, self.rows = self.cu[-1], self.cu[-1] + pad
        self.K = torch.randn(self.nblocks, H_kv, bs, D, generator=g).to(self.dtype)
        self.V = torch.randn(self.nblocks, H_kv, bs, D, generator=g).to(self.dtype)
        self.q = (torch.randn(self.rows, H_q, D, generator=g) * q_scale).to(self.dtype)
        self.k = torch.randn(self.rows, H_kv, D, generator=g).to(self.dtype)
        self.v = torch.randn(self.rows, H_kv, D, generator=g).to(self.dtype)

    def seen(self):
        """Pool rows that some sequence holds: bool [nblocks, bs]."""
        s = torch.zeros(self.nblocks, self.bs, dtype=torch.bool)
        for b, L in enumerate(self.lens):
            t = torch.arange(L)
            s[self.table[b, t // self.bs].long(), t % self.bs] = True
        return s

    def cache(self, kvc, layers=1, layer=0):
        c = kvc.PagedKVCache(layers, self.nblocks, self.bs, self.B, self.max_blocks, self.H_q, self.H_kv, self.D,
                             self.name)
        Kv, Vv = c.layer_views(layer)
        Kv.copy_(self.K)
        Vv.copy_(self.V)
        torch.cuda.synchronize()
        return c

    def dev(self):
        i32 = dict(dtype=torch.int32, device="cuda")
        return dict(table=self.table.cuda(), cu=torch.tensor(self.cu, **i32), lens=torch.tensor(self.lens, **i32),
                    groups=torch.tensor(self.start, **i32), prefix=torch.tensor(self.prefix, **i32), q=self.q.cuda(),
                    k=self.k.cuda(), v=self.v.cuda())


def attention64(bt, q=None, K=None, V=None):
    """(out, bound): the definition in 64 bits and the tolerance without the weights' rounding, plus A;
    float64 [rows, H_q, D] each (rows of padding stay 0).  Masked positions are left out, not weighted."""
    q = (bt.q if q is None else q).double()
    K = (bt.K if K is None else K).double()
    V = (bt.V if V is None else V).double()
    D, G = bt.D, bt.H_q // bt.H_kv
    out, tol, A = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(q)
    for b in range(bt.B):
        for h in range(bt.H_kv):
            t = torch.arange(bt.lens[b])
            blocks = bt.table[b, t // bt.bs].long()
            Kb, Vb = K[blocks, h, t % bt.bs], V[blocks, h, t % bt.bs]
            for i in range(bt.new[b]):
                n, r = bt.hist[b] + i + 1, bt.cu[b] + i
                qr = q[r, h * G:(h + 1) * G]
                s = qr @ Kb[:n].T / math.sqrt(D)
                p = torch.softmax(s, -1)
                X = (qr.abs() @ Kb[:n].abs().T / math.sqrt(D)).amax(-1, keepdim=True)
                o, a = p @ Vb[:n], p @ Vb[:n].abs()
                out[r, h * G:(h + 1) * G], A[r, h * G:(h + 1) * G] = o, a
                tol[r, h * G:(h + 1) * G] = (a * (4 * (D + 3) * U * X + 2.0 ** -21 + (2 * n + 4) * U)
                                             + HALF_STEP[bt.dtype] * o.abs())
    return out, tol, A


def check_attention(got, bt, ref, tensor_cores=False, rows=None):
    """Every output within its bound; rows: the packed rows to look at (default all real ones)."""
    out, tol, A = ref
    rows = torch.arange(bt.n) if rows is None else torch.as_tensor(rows)
    tol = tol + (2.0 ** -8 * A if tensor_cores else 0)
    err = (got.cpu().double() - out)[rows].abs()
    bad = ~(err <= tol[rows])  # NaN is bad
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} outputs off, first {bad.nonzero()[0].tolist()}, "
                           f"worst {float(torch.nan_to_num(err / tol[rows], nan=1e9).max()):.2f} of the bound")


def rotate64(x, pos, inv_freq, axis, adjacent, scale=1.0):
    """x [n, H, D]; pos [n, axes] -> (rotated in 64 bits, |x1| + |x2| per element)."""
    x = x.double()
    pairs = len(inv_freq)
    i = torch.arange(pairs)
    i1 = 2 * i if adjacent else i
    i2 = 2 * i + 1 if adjacent else i + pairs
    ang = pos.double()[:, torch.as_tensor(axis)] * torch.tensor(inv_freq, dtype=torch.float64)
    c, s = scale * ang.cos()[:, None], scale * ang.sin()[:, None]
    y, w = x.clone(), torch.zeros_like(x)
    y[..., i1] = x[..., i1] * c - x[..., i2] * s
    y[..., i2] = x[..., i2] * c + x[..., i1] * s
    w[..., i1] = w[..., i2] = (x[..., i1].abs() + x[..., i2].abs()) * abs(scale)
    return y, w

"""Cases, plain forms and exact values of the operators around the 8-bit paged cache.

Four calls of a serving step:

- ``norm``: append with the norm of every query and key head and the rotation by its position in one
  pass, to a plain paged cache.
- ``write``: the same append (with or without the norms) to a paged cache held in 8 bits: E4M3 codes
  with a power-of-two scale for each block of tokens and KV head.  A block that already holds tokens
  keeps its scale unless a new token needs a larger one; then its codes are scaled down.
- ``read``: positions of that cache read back as packed rows.
- ``attn``: attention of packed new tokens over that cache: single tokens, drafts, chunks of prompts,
  sequences behind a shared prefix.

``own`` picks the side: false computes the plain form (elementary torch operations in 32 bits,
rotation angles in 64), true makes the calls of kv_cache_decode_kvc_gb300.  Lengths are drawn from
the case alone (``mix``), values and block numbers from the seed.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
F8 = torch.float8_e4m3fn
EPS = 1e-6


def _case(op, name, **kw):
    c = dict(op=op, name=name, dtype="bf16", D=128, bs=64, rot=128, adjacent=False, norm=True, pad=0, groups=0,
             prefix_lo=0, prefix_hi=0, mix=1)
    c.update(kw)
    return c


def listed():
    return [
        # one decode step of the 8B serving batch: 24 tokens, the smallest call (latency)
        _case("norm", "norm_decode_8b", B=24, Hq=32, Hkv=8, bs=16, new_lo=1, new_hi=1, hist_lo=1000, hist_hi=2000),
        # prompts of a model with 70B-shaped heads
        _case("norm", "norm_prompts_70b", B=4, Hq=64, Hkv=8, bs=128, new_lo=2500, new_hi=4500, hist_lo=0, hist_hi=700),
        # single precision, small heads, half of them rotated in adjacent pairs, odd lengths
        _case("norm", "norm_f32", dtype="f32", B=7, Hq=8, Hkv=8, D=64, rot=32, adjacent=True, bs=32, new_lo=1,
              new_hi=601, hist_lo=0, hist_hi=999),
        # a decode step into the 8-bit cache: blocks that hold tokens and may need a larger scale
        _case("write", "write_decode_8b", B=24, Hq=32, Hkv=8, bs=16, new_lo=1, new_hi=1, hist_lo=1000, hist_hi=2000,
              norm=False),
        # a step that takes in prompts, beside empty slots of the batch and padded rows
        _case("write", "write_prompts_8b", B=8, Hq=32, Hkv=8, new_lo=0, new_hi=2048, hist_lo=0, hist_hi=2000, pad=37),
        # a prefix taken out of the 8-bit cache, for a cache of another format
        _case("read", "read_prefix_8b", B=8, Hq=32, Hkv=8, new_lo=3000, new_hi=6000, hist_lo=0, hist_hi=0),
        # the last few tokens of every sequence
        _case("read", "read_recent_8b", B=24, Hq=32, Hkv=8, bs=16, new_lo=1, new_hi=100, hist_lo=500, hist_hi=900),
        # the 8B serving batch, one token each: bound by the cache's bytes
        _case("attn", "attn_decode_8b", B=24, Hq=32, Hkv=8, bs=16, new_lo=1, new_hi=1, hist_lo=3000, hist_hi=6000),
        # continuous batching: most sequences decode one token, some bring a chunk
        _case("attn", "attn_mixed_8b", B=24, Hq=32, Hkv=8, bs=32, new_lo=1, new_hi=300, ones=20, hist_lo=3000,
              hist_hi=6000),
        # one chunk of a long prompt, 70B-shaped heads: the largest case
        _case("attn", "attn_chunk_70b", B=1, Hq=64, Hkv=8, bs=128, new_lo=2048, new_hi=2048, hist_lo=12288,
              hist_hi=12288),
        # the 8B serving batch behind one system prompt
        _case("attn", "attn_shared_8b", B=24, Hq=32, Hkv=8, new_lo=1, new_hi=1, groups=1, prefix_lo=2048,
              prefix_hi=2048, hist_lo=900, hist_hi=3900),
        # one KV head, a few drafted tokens to verify per sequence, heads of 64
        _case("attn", "attn_drafts_mqa", B=64, Hq=32, Hkv=1, D=64, rot=64, bs=32, new_lo=1, new_hi=5, hist_lo=2000,
              hist_hi=9000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "write", "read", "attn", "attn"])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 8, 16, 32]) if Hkv <= 2 else rng.choice([1, 2, 4, 8])
    D = rng.choice([64, 128, 128])
    kw = dict(Hkv=Hkv, Hq=Hkv * G, D=D, rot=D, bs=rng.choice([16, 32, 64, 128, 256]), mix=rng.randrange(1 << 30))
    if op != "attn":
        kw.update(dtype=rng.choice(["bf16", "bf16", "f32"]), B=_log(rng, 1, 32), rot=rng.choice([D, D, D // 2]),
                  adjacent=rng.random() < 0.4, pad=rng.choice([0, 0, 13]), norm=op == "norm" or rng.random() < 0.5,
                  new_lo=rng.choice([0, 1]), new_hi=_log(rng, 1, 1500), hist_lo=0, hist_hi=_log(rng, 10, 2000))
        return _case(op, "", **kw)
    f32 = rng.random() < 0.1
    B, new = _log(rng, 1, 8 if f32 else 48), rng.choice([1, 1, 4, _log(rng, 1, 300 if f32 else 2000)])
    kw.update(dtype="f32" if f32 else "bf16", B=B, new_lo=1, new_hi=new, hist_lo=0,
              hist_hi=_log(rng, 10, 1000 if f32 else 8000), pad=rng.choice([0, 5]))
    # the plain form holds [B, Hq, new, history] scores: keep them below the largest listed case's
    while kw["B"] > 1 and kw["B"] * kw["Hq"] * new * (new + kw["hist_hi"]) > 4e8:
        kw["B"] = (kw["B"] + 1) // 2
    if kw["B"] > 1 and new <= 4 and rng.random() < 0.4:
        P = _log(rng, 64, 1000 if f32 else 8000)
        kw.update(groups=rng.choice([1, 1, 2]), prefix_lo=max(1, P // 2), prefix_hi=P)
    return _case("attn", "", **kw)


def _shape(case):
    """Lengths of a case: new tokens, history (the shared prefix included) of each sequence, the first
    sequence of each group and its prefix."""
    r = random.Random(case["mix"] * 7919 + case["B"])
    B, NG, bs = case["B"], max(1, case["groups"]), case["bs"]
    start = [g * B // NG for g in range(NG)] + [B]
    prefix = [r.randint(case["prefix_lo"], case["prefix_hi"]) // bs * bs for _ in range(NG)]
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(B)]
    for b in range(case.get("ones", 0)):
        new[b] = 1
    if sum(new) == 0:
        new[0] = 1
    hist = [r.randint(case["hist_lo"], case["hist_hi"]) for _ in range(B)]
    group = [g for g in range(NG) for _ in range(start[g], start[g + 1])]
    return new, [h + prefix[g] for h, g in zip(hist, group)], start, prefix, group


def _exponent(amax):
    """The smallest e >= -64 with amax <= 448 2^e (448 = 0.875 2^9), of finite amax >= 0."""
    m, e = torch.frexp(amax)
    e = torch.where(amax > 0, e - 9 + (m > 0.875).to(e.dtype), -64)
    return e.clamp(min=-64)


def _pow2(e):
    return torch.ldexp(torch.ones((), device=e.device), e)


def prepare(case, seed):
    new, hist, start, prefix, group = _shape(case)
    B, Hq, Hkv, D, bs, op = case["B"], case["Hq"], case["Hkv"], case["D"], case["bs"], case["op"]
    dt, dev = DTYPES[case["dtype"]], torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    lens = [n + h for n, h in zip(new, hist)]
    max_blocks, n = max(1, -(-max(lens) // bs)), sum(new)
    rows = n + case["pad"]
    # block tables: the pool's blocks in a random order, as many as the batch needs and a few more; the
    # sequences of a group name the same blocks for their prefix
    j = torch.arange(max_blocks)
    first = torch.tensor([start[g] for g in group])
    shared = torch.tensor([prefix[g] // bs for g in group])[:, None]
    needed = (j < torch.tensor([-(-L // bs) for L in lens])[:, None]) & ((j >= shared) | (first == torch.arange(B))[:, None])
    number = (needed.flatten().cumsum(0) - 1).clamp(min=0).view(B, max_blocks) * needed
    number = torch.where(j < shared, number[first], number).to(dev)
    blocks = int(needed.sum()) + 8
    table = torch.randperm(blocks, device=dev, generator=gen).to(torch.int32)[number].contiguous()
    cu = [0]
    for x in new:
        cu.append(cu[-1] + x)
    i32 = dict(dtype=torch.int32, device=dev)
    s = dict(case=case, n=n, max_new=max(new), max_len=max(lens), max_prefix=max(prefix),
             max_own=max(L - prefix[g] for L, g in zip(lens, group)),
             max_group=max(b - a for a, b in zip(start, start[1:])), table=table, cu=torch.tensor(cu, **i32),
             lens=torch.tensor(lens, **i32), groups=torch.tensor(start, **i32), prefix=torch.tensor(prefix, **i32))
    # the cache: a handle of the framework, which owns its block pools, or tensors of the same shape
    shape, names = (blocks, Hkv, bs, D), ("K", "V")
    if own:
        from kv_cache_decode_kvc_gb300 import kvc
        if op == "norm":
            s["cache"] = kvc.PagedKVCache(1, blocks, bs, B, max_blocks, Hq, Hkv, D, case["dtype"])
            s["K"], s["V"] = s["cache"].layer_views(0)
        else:
            s["cache"] = kvc.PagedFP8KVCache(1, blocks, bs, B, max_blocks, Hq, Hkv, D, case["dtype"])
            K, V, s["Ks"], s["Vs"] = s["cache"].layer_views(0)
            s["K"], s["V"] = K.view(F8), V.view(F8)
    elif op == "norm":
        s["K"], s["V"] = torch.empty(shape, dtype=dt, device=dev), torch.empty(shape, dtype=dt, device=dev)
    else:
        s["K"], s["V"] = torch.empty(shape, dtype=F8, device=dev), torch.empty(shape, dtype=F8, device=dev)
        s["Ks"], s["Vs"] = torch.empty(blocks, Hkv, device=dev), torch.empty(blocks, Hkv, device=dev)
    for x in names:
        if op == "norm":
            s[x].copy_(torch.randn(shape, dtype=dt, device=dev, generator=gen))
            continue
        # values about 1, heads and blocks between half and twice that; quantised as the cache holds them
        mag = torch.exp2(torch.rand(blocks, Hkv, 1, 1, device=dev, generator=gen) * 2 - 1)
        y = torch.randn(shape, dtype=torch.bfloat16, device=dev, generator=gen).float() * mag
        scale = _pow2(_exponent(y.abs().amax((2, 3))))
        s[x].view(torch.uint8).copy_((y / scale[..., None, None]).to(F8).view(torch.uint8))
        s[x + "s"].copy_(scale)
    if op in ("norm", "write"):
        # the projections' joint output, [token, (Hq + 2 Hkv) D]: q, k, v are strided views of it
        qkv = torch.randn(rows, (Hq + 2 * Hkv) * D, dtype=dt, device=dev, generator=gen)
        s["q"] = qkv[:, :Hq * D].unflatten(1, (Hq, D))
        s["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
        s["v"] = qkv[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D))
        s["q_out"] = torch.zeros(rows, Hq, D, dtype=dt, device=dev)
        for x in ("q_norm", "k_norm"):
            s[x] = (1 + 0.2 * torch.randn(D, device=dev, generator=gen)).to(dt) if case["norm"] else None
        pairs = case["rot"] // 2
        s["inv_freq"] = [500000.0 ** (-i / pairs) for i in range(pairs)]
        s["freq"] = torch.tensor(s["inv_freq"], dtype=torch.float64, device=dev)
        if own:
            s["rope"] = kvc.Rope(s["inv_freq"], layout="adjacent" if case["adjacent"] else "half")
        # the blocks that the new tokens go to: their sequence and place, and each row's among them
        seq, place, rank = [], [], []
        for b, (T, H) in enumerate(zip(new, hist)):
            if T:
                at = len(seq) - H // bs
                rank += [at + (H + i) // bs for i in range(T)]
                for k in range(H // bs, (H + T - 1) // bs + 1):
                    seq.append(b)
                    place.append(k)
        s["rank"] = torch.tensor(rank, device=dev)
        s["touched"] = table[torch.tensor(seq, device=dev), torch.tensor(place, device=dev)].long()
        s["held"] = torch.tensor([max(0, hist[b] - k * bs) for b, k in zip(seq, place)], device=dev)
    elif op == "read":
        s["k_out"] = torch.zeros(rows, Hkv, D, dtype=dt, device=dev)
        s["v_out"] = torch.zeros(rows, Hkv, D, dtype=dt, device=dev)
    else:
        # queries whose scores spread as trained heads' do (standard deviation about 2)
        s["q"] = torch.randn(rows, Hq, D, dtype=dt, device=dev, generator=gen) * 2
        s["out"] = torch.zeros(rows, Hq, D, dtype=dt, device=dev)
        if own:
            s["ws"] = torch.empty(s["cache"].attn_workspace_bytes(rows, case["groups"]), dtype=torch.uint8, device=dev)
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        c = s["cache"]
        if op in ("norm", "write"):
            c.append_rope(0, s["rope"], s["q"], s["k"], s["v"], s["table"], s["cu"], s["lens"], q_out=s["q_out"],
                          q_norm=s["q_norm"], k_norm=s["k_norm"], norm_eps=EPS)
            return _updated(s)
        if op == "read":
            c.read(0, s["k_out"], s["v_out"], s["table"], s["cu"], s["lens"])
            return {"k": s["k_out"], "v": s["v_out"]}
        if s["case"]["groups"]:
            c.attn_shared(0, s["q"], s["out"], s["table"], s["cu"], s["lens"], s["groups"], s["prefix"],
                          workspace=s["ws"])
        else:
            c.attn_ragged(0, s["q"], s["out"], s["table"], s["cu"], s["lens"], workspace=s["ws"])
        return s["out"]
    if op in ("norm", "write"):
        return _plain_append(s)
    if op == "read":
        return _plain_read(s)
    return _plain_shared(s) if s["case"]["groups"] else _plain_ragged(s)


def _updated(s):
    out = {"q": s["q_out"], "K": s["K"], "V": s["V"]}
    if s["case"]["op"] == "write":
        out.update(Ks=s["Ks"], Vs=s["Vs"])
    return out


# ----------------------------------------------------------------------------- plain forms
def _norm_rotate(x, weight, cos, sin, rot, adjacent):
    """x [n, H, D] (any type) normalised and rotated in 32 bits; cos, sin [n, 1, rot / 2] fp32."""
    y = x.float()
    if weight is not None:
        y = y / (y * y).mean(-1, keepdim=True).add(EPS).sqrt() * weight.float()
    a = y[..., 0:rot:2] if adjacent else y[..., :rot // 2]
    b = y[..., 1:rot:2] if adjacent else y[..., rot // 2:rot]
    ra, rb = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([ra, rb], -1).flatten(-2) if adjacent else torch.cat([ra, rb], -1)
    return torch.cat([r, y[..., rot:]], -1)


def _places(s):
    """Block, offset and slot of every row."""
    cu, n, bs = s["cu"].long(), s["n"], s["case"]["bs"]
    r = torch.arange(n, device=cu.device)
    b = torch.searchsorted(cu[1:], r, right=True)
    slot = s["lens"][b].long() - cu[b + 1] + r
    return s["table"][b, slot // bs].long(), slot % bs, slot


def _plain_append(s):
    case, n = s["case"], s["n"]
    block, off, slot = _places(s)
    ang = slot[:, None].double() * s["freq"]  # angles of far positions: 64 bits
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]
    q = _norm_rotate(s["q"][:n], s["q_norm"], cos, sin, case["rot"], case["adjacent"])
    k = _norm_rotate(s["k"][:n], s["k_norm"], cos, sin, case["rot"], case["adjacent"])
    s["q_out"][:n] = q.to(s["q_out"].dtype)
    if case["op"] == "norm":
        s["K"][block, :, off] = k.to(s["K"].dtype)
        s["V"][block, :, off] = s["v"][:n]
    else:
        _quantise(s, "K", k, block, off)
        _quantise(s, "V", s["v"][:n].float(), block, off)
    return _updated(s)


def _quantise(s, name, x, block, off):
    """x [n, Hkv, D] fp32 into the blocks: the larger scale of what they hold and what comes, the held
    codes scaled down to it, then the new ones."""
    codes, scales, touched, held = s[name].view(torch.uint8), s[name + "s"], s["touched"], s["held"]
    amax = torch.zeros(len(touched), x.shape[1], device=x.device)
    amax.index_reduce_(0, s["rank"], x.abs().amax(-1), "amax")
    before = torch.frexp(scales[touched])[1] - 1
    e = _exponent(amax)
    e = torch.where(held[:, None] > 0, torch.maximum(e, before), e)
    old = codes[touched]
    down = (old.view(F8).float() * _pow2(before - e)[..., None, None]).to(F8).view(torch.uint8)
    keep = torch.arange(old.shape[2], device=x.device) < held[:, None]
    codes[touched] = torch.where(keep[:, None, :, None], down, old)
    scales[touched] = _pow2(e)
    codes[block, :, off] = (x * _pow2(-e)[s["rank"]][..., None]).to(F8).view(torch.uint8)


def _plain_read(s):
    n = s["n"]
    block, off, _ = _places(s)
    for x, out in (("K", s["k_out"]), ("V", s["v_out"])):
        out[:n] = (s[x].view(torch.uint8)[block, :, off].view(F8).float() * s[x + "s"][block][..., None]).to(out.dtype)
    return {"k": s["k_out"], "v": s["v_out"]}


def _rows_of(s):
    """Packed rows of the batch padded to [B, max_new]: row numbers (clamped) and which are real."""
    cu = s["cu"].long()
    i = torch.arange(s["max_new"], device=cu.device)
    rows = cu[:-1, None] + i
    return rows.clamp(max=s["n"] - 1), rows < cu[1:, None]


def _gather(s, name, blocks):
    """The values of blocks [X, nb] of a pool [*, H, bs, D]: fp32 [X, H, nb * bs, D]."""
    v = s[name].view(torch.uint8)[blocks.long()].view(F8).float() * s[name + "s"][blocks.long()][..., None, None]
    return v.transpose(1, 2).flatten(2, 3)


def _plain_ragged(s):
    case, q = s["case"], s["q"]
    B, Hq, Hkv, D, bs = case["B"], case["Hq"], case["Hkv"], case["D"], case["bs"]
    rows, real = _rows_of(s)
    Tm, G = s["max_new"], Hq // Hkv
    blocks = s["table"][:, :-(-s["max_len"] // bs)]
    K, V = _gather(s, "K", blocks), _gather(s, "V", blocks)
    S = K.shape[2]
    qg = q[rows].float().view(B, Tm, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, Tm * G, D)
    lens, new = s["lens"].long(), (s["cu"][1:] - s["cu"][:-1]).long()
    t = torch.arange(S, device=q.device)
    last = (lens - new)[:, None] + torch.arange(Tm, device=q.device)  # [B, Tm] the row's own position
    hidden = (t > last[..., None])[:, None, :, None]  # [B, 1, Tm, 1, S]
    p = ((qg @ K.transpose(-1, -2)) / math.sqrt(D)).view(B, Hkv, Tm, G, S).masked_fill_(hidden, -math.inf)
    p = p.sub_(p.amax(-1, keepdim=True)).exp_()
    z = p.sum(-1).view(B, Hkv, Tm * G, 1)
    V = V * (t < lens[:, None])[:, None, :, None]
    o = (p.view(B, Hkv, Tm * G, S) @ V) / z
    o = o.view(B, Hkv, Tm, G, D).permute(0, 2, 1, 3, 4).reshape(B, Tm, Hq, D)
    s["out"][rows[real]] = o[real].to(q.dtype)
    return s["out"]


def _plain_shared(s):
    case, q = s["case"], s["q"]
    B, Hq, Hkv, D, bs, NG = case["B"], case["Hq"], case["Hkv"], case["D"], case["bs"], case["groups"]
    dev, G, Tm, M = q.device, Hq // Hkv, s["max_new"], s["max_group"]
    rows, real = _rows_of(s)
    start, prefix = s["groups"].long(), s["prefix"].long()
    lens, new = s["lens"].long(), (s["cu"][1:] - s["cu"][:-1]).long()
    b = torch.arange(B, device=dev)
    g = torch.searchsorted(start[1:], b, right=True)
    member = (start[:-1, None] + torch.arange(M, device=dev)).clamp(max=B - 1)  # [NG, M] sequences
    place = b - start[g]
    qb = q[rows].float().view(B, Tm, Hkv, G, D).permute(0, 2, 1, 3, 4) / math.sqrt(D)  # [B, Hkv, Tm, G, D]
    # the group's rows against its prefix, gathered once per group: [NG, Hkv, M Tm G, P]
    np_ = max(1, -(-s["max_prefix"] // bs))
    head = s["table"][start[:-1], :np_]
    Kp, Vp = _gather(s, "K", head), _gather(s, "V", head)
    P = Kp.shape[2]
    seen = (torch.arange(P, device=dev) < prefix[:, None])[:, None, :, None]  # [NG, 1, P, 1]
    qp = qb[member].permute(0, 2, 1, 3, 4, 5).reshape(NG, Hkv, M * Tm * G, D)
    sp = (qp @ Kp.transpose(-1, -2)).masked_fill_(~seen.transpose(-1, -2), -math.inf)
    # each sequence's rows against its own part: [B, Hkv, Tm G, S]
    nb = -(-s["max_own"] // bs)
    cols = ((prefix[g] // bs)[:, None] + torch.arange(nb, device=dev)).clamp(max=s["table"].shape[1] - 1)
    own_blocks = s["table"].gather(1, cols)
    Ks, Vs = _gather(s, "K", own_blocks), _gather(s, "V", own_blocks)
    S = Ks.shape[2]
    t = prefix[g][:, None] + torch.arange(S, device=dev)  # [B, S] positions
    last = (lens - new)[:, None] + torch.arange(Tm, device=dev)
    hidden = (t[:, None] > last[..., None])[:, None, :, None]  # [B, 1, Tm, 1, S]
    ss = (qb.reshape(B, Hkv, Tm * G, D) @ Ks.transpose(-1, -2)).view(B, Hkv, Tm, G, S).masked_fill_(hidden, -math.inf)
    ss = ss.view(B, Hkv, Tm * G, S)
    # one softmax over both: the common maximum, then the two sums
    mp = sp.amax(-1).view(NG, Hkv, M, Tm * G)[g, :, place]  # [B, Hkv, Tm G]
    m = torch.maximum(mp, ss.amax(-1))
    mg = m[member].transpose(1, 2).reshape(NG, Hkv, M * Tm * G)
    pp, ps = (sp - mg[..., None]).exp_(), (ss - m[..., None]).exp_()
    op = (pp @ (Vp * seen)).view(NG, Hkv, M, Tm * G, D)[g, :, place]
    zp = pp.sum(-1).view(NG, Hkv, M, Tm * G)[g, :, place]
    o = op + ps @ (Vs * (t < lens[:, None])[:, None, :, None])
    o = o / (zp + ps.sum(-1))[..., None]
    o = o.view(B, Hkv, Tm, G, D).permute(0, 2, 1, 3, 4).reshape(B, Tm, Hq, D)
    s["out"][rows[real]] = o[real].to(q.dtype)
    return s["out"]


# ----------------------------------------------------------------------------- exact values
def exact(case, seed):
    """The definition in 64 bits, sequence by sequence.  Codes are given before their rounding: a new
    token's value over its block's scale, a held one's over the scale's growth."""
    s = prepare(case, seed)
    new, hist, _, _, _ = _shape(case)
    Hq, Hkv, D, bs, op = case["Hq"], case["Hkv"], case["D"], case["bs"], case["op"]
    G, table = Hq // Hkv, s["table"].cpu()
    pool = {x: s[x].double() for x in ("K", "V")}
    if op in ("norm", "write"):
        q_out = s["q_out"].double()
        pairs = case["rot"] // 2
        freq = torch.tensor(s["inv_freq"], dtype=torch.float64)
        i1 = (torch.arange(pairs) * (2 if case["adjacent"] else 1)).cuda()
        i2 = i1 + (1 if case["adjacent"] else pairs)
        scale = {x: s[x + "s"].double() for x in ("K", "V")} if op == "write" else {}

        def turned(x, w, turn):
            x = x.double()
            if w is not None:
                x = x * torch.rsqrt(x.square().sum(-1, keepdim=True) / D + EPS) * w.double()
            y = x.clone()
            c = torch.complex(x[..., i1], x[..., i2]) * turn
            y[..., i1], y[..., i2] = c.real, c.imag
            return y

        r = 0
        for b, (T, H) in enumerate(zip(new, hist)):
            if T == 0:
                continue
            slots = torch.arange(H, H + T)
            at = slots[:, None].double() * freq
            turn = torch.polar(torch.ones_like(at), at).cuda()[:, None]  # e^{i angle}
            q_out[r:r + T] = turned(s["q"][r:r + T], s["q_norm"], turn)
            vals = {"K": turned(s["k"][r:r + T], s["k_norm"], turn), "V": s["v"][r:r + T].double()}
            r += T
            if op == "norm":
                blocks, off = table[b][slots // bs].long().cuda(), (slots % bs).cuda()
                for x in vals:
                    pool[x][blocks, :, off] = vals[x]
                continue
            for k in range(H // bs, (H + T - 1) // bs + 1):
                lo, hi = max(H, k * bs), min(H + T, (k + 1) * bs)
                e, held = int(table[b, k]), max(0, H - k * bs)
                for x, y in vals.items():
                    y = y[lo - H:hi - H].transpose(0, 1)  # [Hkv, tokens, D]
                    need = torch.exp2(torch.ceil(torch.log2(y.abs().amax((1, 2)).clamp(min=448 * 2.0 ** -64) / 448)))
                    old = scale[x][e].clone()
                    now = torch.maximum(old, need) if held else need
                    pool[x][e, :, :held] *= (old / now)[:, None, None]
                    pool[x][e, :, lo - k * bs:hi - k * bs] = y / now[:, None, None]
                    scale[x][e] = now
        out = {"q": q_out, "K": pool["K"], "V": pool["V"]}
        if op == "write":
            out.update(Ks=scale["K"], Vs=scale["V"])
        return out
    for x in pool:
        pool[x] *= s[x + "s"].double()[..., None, None]
    if op == "read":
        out = {"k": s["k_out"].double(), "v": s["v_out"].double()}
        r = 0
        for b, (T, H) in enumerate(zip(new, hist)):
            slots = torch.arange(H, H + T)
            blocks, off = table[b][slots // bs].long().cuda(), (slots % bs).cuda()
            out["k"][r:r + T], out["v"][r:r + T] = pool["K"][blocks, :, off], pool["V"][blocks, :, off]
            r += T
        return out
    out, r = s["out"].double(), 0
    for b, (T, H) in enumerate(zip(new, hist)):
        L = H + T
        blocks = table[b, :-(-L // bs)].long().cuda()
        for h in range(Hkv):
            K = pool["K"][blocks, h].reshape(-1, D)[:L]
            V = pool["V"][blocks, h].reshape(-1, D)[:L]
            for i in range(0, T, 512):
                m = min(512, T - i)
                q = s["q"][r + i:r + i + m, h * G:(h + 1) * G].double()
                score = torch.einsum("igd,td->igt", q, K) / math.sqrt(D)
                far = torch.arange(L, device=q.device)[None] > H + i + torch.arange(m, device=q.device)[:, None]
                score = score.masked_fill(far[:, None], -math.inf)
                out[r + i:r + i + m, h * G:(h + 1) * G] = torch.softmax(score, -1) @ V
        r += T
    return out


def work(case):
    """Bytes (each input once, each output once) and operations of one pass."""
    new, hist, start, prefix, _ = _shape(case)
    Hq, Hkv, D, bs, op = case["Hq"], case["Hkv"], case["D"], case["bs"], case["op"]
    es, n = DTYPES[case["dtype"]].itemsize, sum(new)
    touched = sum((h + t - 1) // bs - h // bs + 1 for h, t in zip(hist, new) if t)
    if op in ("norm", "write"):
        kv = es if op == "norm" else 1
        flops = n * (Hq + Hkv) * (3 * case["rot"] + (4 * D if case["norm"] else 0))
        return {"bytes": n * D * (Hq * 2 * es + 2 * Hkv * (es + kv)) + (0 if op == "norm" else touched * Hkv * 8),
                "flops": flops}
    if op == "read":
        return {"bytes": 2 * n * Hkv * D * (1 + es) + touched * Hkv * 8, "flops": 2 * n * Hkv * D}
    # a shared prefix is read once for its group; a sequence without new tokens reads nothing
    kv = sum(h + t for h, t in zip(hist, new) if t)
    for a, b, p in zip(start, start[1:], prefix):
        kv -= p * max(0, sum(1 for x in new[a:b] if x) - 1)
    seen = sum(t * h + t * (t + 1) // 2 for h, t in zip(hist, new))
    return {"bytes": 2 * kv * Hkv * D + 8 * Hkv * (kv // bs) + 2 * n * Hq * D * es, "flops": 4 * seen * Hq * D}

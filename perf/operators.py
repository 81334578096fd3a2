"""Cases, plain forms and exact values of the operators on ragged batches over the paged cache.

Three operators, which follow one another in a serving step:

- ``append``: the new tokens' keys (rotated by their positions) and values go to their slots of
  the paged cache, the queries are rotated on the way.  Positions have one axis, or several
  (time, height, width) where each pair of dimensions belongs to an axis.
- ``ragged``: attention of each sequence's new tokens (a prompt, a chunk of one, or one token)
  over its history in the paged cache, causal among the new tokens.
- ``shared``: the same for a batch in groups, whose sequences start with the same blocks: the
  common prefix is attended once for all the query rows of its group.

``own`` picks the side: false computes the plain form (elementary torch operations in 32 bits,
rotation angles in 64), true makes the calls of kv_cache_decode_kvc_gb300.  Lengths are drawn
from the case alone (``mix``), values and block numbers from the seed.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _case(op, name, **kw):
    c = dict(op=op, name=name, dtype="bf16", D=128, bs=64, axes=1, rot=128, adjacent=False, pad=0,
             groups=1, prefix_lo=0, prefix_hi=0, mix=1)
    c.update(kw)
    return c


def listed():
    return [
        # one decode step of the 8B serving batch: 24 tokens, the smallest call (latency)
        _case("append", "append_decode_8b", B=24, Hq=32, Hkv=8, bs=16, new_lo=1, new_hi=1, hist_lo=3000, hist_hi=6000),
        # a step that takes in prompts, beside empty slots of the batch and padded rows
        _case("append", "append_prompts_8b", B=8, Hq=32, Hkv=8, new_lo=0, new_hi=2048, hist_lo=0, hist_hi=4000, pad=37),
        # image and video tokens with (time, height, width) positions, 70B-shaped heads
        _case("append", "append_video_70b", B=4, Hq=64, Hkv=8, bs=128, new_lo=3500, new_hi=4500, hist_lo=0, hist_hi=700,
              axes=3),
        # single precision, a rotation of half the head in adjacent pairs, odd lengths
        _case("append", "append_f32", dtype="f32", B=7, Hq=8, Hkv=8, D=64, rot=32, adjacent=True, bs=32, new_lo=1,
              new_hi=601, hist_lo=0, hist_hi=999),
        # continuous batching: most sequences decode one token, some bring a chunk
        _case("ragged", "ragged_mixed_8b", B=24, Hq=32, Hkv=8, bs=16, new_lo=1, new_hi=300, ones=20, hist_lo=3000,
              hist_hi=6000),
        # prompts from their first token on
        _case("ragged", "ragged_prompts_8b", B=6, Hq=32, Hkv=8, new_lo=700, new_hi=4096, hist_lo=0, hist_hi=0),
        # one chunk of a long prompt, 70B-shaped heads: the largest case
        _case("ragged", "ragged_chunk_70b", B=1, Hq=64, Hkv=8, bs=128, new_lo=4096, new_hi=4096, hist_lo=12288,
              hist_hi=12288),
        # single precision, small heads
        _case("ragged", "ragged_f32", dtype="f32", B=5, Hq=8, Hkv=2, D=64, bs=32, new_lo=1, new_hi=333, hist_lo=100,
              hist_hi=1500),
        # the 8B serving batch behind one system prompt, one token each
        _case("shared", "shared_chat_8b", B=24, Hq=32, Hkv=8, new_lo=1, new_hi=1, prefix_lo=2048, prefix_hi=2048,
              hist_lo=900, hist_hi=3900),
        # many short answers to one long document
        _case("shared", "shared_document_8b", B=256, Hq=32, Hkv=8, bs=16, new_lo=1, new_hi=1, prefix_lo=16384,
              prefix_hi=16384, hist_lo=0, hist_hi=500),
        # 70B-shaped heads, a longer document, fewer sequences
        _case("shared", "shared_document_70b", B=32, Hq=64, Hkv=8, bs=128, new_lo=1, new_hi=1, prefix_lo=32768,
              prefix_hi=32768, hist_lo=0, hist_hi=900),
        # several prompts' groups, one KV head, a few drafted tokens to verify per sequence
        _case("shared", "shared_drafts_mqa", B=64, Hq=32, Hkv=1, new_lo=1, new_hi=5, groups=3, prefix_lo=2000,
              prefix_hi=9000, hist_lo=50, hist_hi=1200),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "ragged", "shared"])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 8, 16, 32]) if Hkv <= 2 else rng.choice([1, 2, 4, 8])
    kw = dict(Hkv=Hkv, Hq=Hkv * G, D=rng.choice([64, 128, 128]), bs=rng.choice([16, 32, 64, 128, 256]),
              mix=rng.randrange(1 << 30))
    if op == "append":
        D = kw["D"]
        kw.update(dtype=rng.choice(["bf16", "bf16", "f32"]), B=_log(rng, 1, 32), axes=rng.choice([1, 3]),
                  rot=rng.choice([D, D, D // 2]), adjacent=rng.random() < 0.4, pad=rng.choice([0, 0, 13]),
                  new_lo=rng.choice([0, 1]), new_hi=_log(rng, 1, 1500), hist_lo=0, hist_hi=_log(rng, 10, 4000))
        return _case("append", "", **kw)
    if op == "ragged":
        f32 = rng.random() < 0.2
        B = _log(rng, 1, 8 if f32 else 24)
        new = _log(rng, 1, 300 if f32 else 2500)
        kw.update(dtype="f32" if f32 else "bf16", B=B, new_lo=1, new_hi=new, hist_lo=0,
                  hist_hi=_log(rng, 10, 1000 if f32 else 6000), pad=rng.choice([0, 5]))
        # the plain form holds [B, Hq, new, history] scores: keep them below the largest listed case's
        while kw["B"] > 1 and kw["B"] * kw["Hq"] * new * (new + kw["hist_hi"]) > 4e8:
            kw["B"] = (kw["B"] + 1) // 2
        return _case("ragged", "", **kw)
    f32 = rng.random() < 0.15
    P = _log(rng, 64, 2048 if f32 else 16384)
    kw.update(dtype="f32" if f32 else "bf16", B=_log(rng, 2, 24 if f32 else 128), groups=rng.choice([1, 1, 2, 3]), new_lo=1, new_hi=rng.choice([1, 1, 4]),
              prefix_lo=max(1, P // 2), prefix_hi=P, hist_lo=0, hist_hi=_log(rng, 10, 1500))
    kw["groups"] = min(kw["groups"], kw["B"])
    return _case("shared", "", **kw)


def _shape(case):
    """Lengths of a case: new tokens, history (the shared prefix included) of each sequence, the
    first sequence of each group and its prefix."""
    r = random.Random(case["mix"] * 7919 + case["B"])
    B, NG, bs = case["B"], case["groups"], case["bs"]
    start = [g * B // NG for g in range(NG)] + [B]
    prefix = [r.randint(case["prefix_lo"], case["prefix_hi"]) // bs * bs for _ in range(NG)]
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(B)]
    for b in range(case.get("ones", 0)):
        new[b] = 1
    if sum(new) == 0:
        new[0] = 1
    hist = [r.randint(case["hist_lo"], case["hist_hi"]) for _ in range(B)]
    group = [g for g in range(NG) for _ in range(start[g], start[g + 1])]
    hist = [h + prefix[g] for h, g in zip(hist, group)]
    return new, hist, start, prefix, group


def prepare(case, seed):
    new, hist, start, prefix, group = _shape(case)
    B, Hq, Hkv, D, bs = case["B"], case["Hq"], case["Hkv"], case["D"], case["bs"]
    dt, dev = DTYPES[case["dtype"]], torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    lens = [n + h for n, h in zip(new, hist)]
    max_blocks = -(-max(lens) // bs)
    n = sum(new)
    # block tables: the pool's blocks in a random order, as many as the batch needs and a few more;
    # the sequences of a group name the same blocks for their prefix
    j = torch.arange(max_blocks)
    first = torch.tensor([start[g] for g in group])
    shared = torch.tensor([prefix[g] // bs for g in group])[:, None]
    needed = (j < torch.tensor([-(-L // bs) for L in lens])[:, None]) & ((j >= shared) | (first == torch.arange(B))[:, None])
    number = (needed.flatten().cumsum(0) - 1).view(B, max_blocks) * needed
    number = torch.where(j < shared, number[first], number).to(dev)
    blocks = int(needed.sum()) + 8
    table = torch.randperm(blocks, device=dev, generator=gen).to(torch.int32)[number].contiguous()
    cu = [0]
    for x in new:
        cu.append(cu[-1] + x)
    s = dict(case=case, n=n, max_new=max(new), max_len=max(lens), max_prefix=max(prefix),
             max_own=max(L - prefix[g] for L, g in zip(lens, group)),
             max_group=max(b - a for a, b in zip(start, start[1:])),
             table=table, cu=torch.tensor(cu, dtype=torch.int32, device=dev),
             lens=torch.tensor(lens, dtype=torch.int32, device=dev),
             groups=torch.tensor(start, dtype=torch.int32, device=dev),
             prefix=torch.tensor(prefix, dtype=torch.int32, device=dev))
    # the cache: a handle of the framework, which owns its block pools, or tensors of the same shape
    shape = (blocks, Hkv, bs, D)
    if own:
        from kv_cache_decode_kvc_gb300 import kvc
        s["cache"] = kvc.PagedKVCache(1, shape[0], bs, B, max_blocks, Hq, Hkv, D, case["dtype"])
        s["K"], s["V"] = s["cache"].layer_views(0)
    else:
        s["K"], s["V"] = torch.empty(shape, dtype=dt, device=dev), torch.empty(shape, dtype=dt, device=dev)
    s["K"].copy_(torch.randn(shape, dtype=dt, device=dev, generator=gen))
    s["V"].copy_(torch.randn(shape, dtype=dt, device=dev, generator=gen))
    rows = n + case["pad"]
    if case["op"] == "append":
        # the projections' joint output, [token, (Hq + 2 Hkv) D]: q, k, v are strided views of it
        qkv = torch.randn(rows, (Hq + 2 * Hkv) * D, dtype=dt, device=dev, generator=gen)
        s["q"] = qkv[:, :Hq * D].unflatten(1, (Hq, D))
        s["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
        s["v"] = qkv[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D))
        s["q_out"] = torch.zeros(rows, Hq, D, dtype=dt, device=dev)
        pairs = case["rot"] // 2
        s["inv_freq"] = [500000.0 ** (-i / pairs) for i in range(pairs)]
        s["axis"] = [0] * pairs if case["axes"] == 1 else [0 if i < pairs // 4 else 1 + (i - pairs // 4) % 2
                                                            for i in range(pairs)]
        if case["axes"] > 1:
            # (time, height, width): the history's text positions, then frames of 24 x 24 patches
            r = torch.arange(rows, device=dev)
            t0 = torch.randint(0, 30000, (1,), device=dev, generator=gen)
            s["positions"] = torch.stack([t0 + r // 576, t0 + r // 24 % 24, t0 + r % 24]).to(torch.int32)
        else:
            s["positions"] = None  # the slot in the sequence
        s["freq"] = torch.tensor(s["inv_freq"], dtype=torch.float64, device=dev)
        s["axis_of"] = torch.tensor(s["axis"], device=dev)
        if own:
            s["rope"] = kvc.Rope(s["inv_freq"], layout="adjacent" if case["adjacent"] else "half", axis=s["axis"])
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
        if op == "append":
            c.append_rope(0, s["rope"], s["q"], s["k"], s["v"], s["table"], s["cu"], s["lens"], q_out=s["q_out"],
                          positions=s["positions"])
            return {"q": s["q_out"], "K": s["K"], "V": s["V"]}
        if op == "ragged":
            c.attn_ragged(0, s["q"], s["out"], s["table"], s["cu"], s["lens"], workspace=s["ws"])
        else:
            c.attn_shared(0, s["q"], s["out"], s["table"], s["cu"], s["lens"], s["groups"], s["prefix"],
                          workspace=s["ws"])
        return s["out"]
    if op == "append":
        return _plain_append(s)
    if op == "ragged":
        return _plain_ragged(s)
    return _plain_shared(s)


# ----------------------------------------------------------------------------- plain forms
def _rotate(x, cos, sin, rot, adjacent):
    """x [n, H, D] (any type) rotated in 32 bits; cos, sin [n, 1, rot / 2] fp32."""
    y = x.float()
    a = y[..., 0:rot:2] if adjacent else y[..., :rot // 2]
    b = y[..., 1:rot:2] if adjacent else y[..., rot // 2:rot]
    ra, rb = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([ra, rb], -1).flatten(-2) if adjacent else torch.cat([ra, rb], -1)
    return torch.cat([r, y[..., rot:]], -1).to(x.dtype)


def _plain_append(s):
    case, n, cu = s["case"], s["n"], s["cu"].long()
    dev, bs = cu.device, case["bs"]
    r = torch.arange(n, device=dev)
    b = torch.searchsorted(cu[1:], r, right=True)
    slot = s["lens"][b].long() - cu[b + 1] + r
    pos = slot[None] if s["positions"] is None else s["positions"][:, :n].long()
    ang = pos[s["axis_of"]].T.double() * s["freq"]  # angles of far positions: 64 bits
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]
    block, off = s["table"][b, slot // bs].long(), slot % bs
    s["q_out"][:n] = _rotate(s["q"][:n], cos, sin, case["rot"], case["adjacent"])
    s["K"][block, :, off] = _rotate(s["k"][:n], cos, sin, case["rot"], case["adjacent"])
    s["V"][block, :, off] = s["v"][:n]
    return {"q": s["q_out"], "K": s["K"], "V": s["V"]}


def _rows_of(s):
    """Packed rows of the batch padded to [B, max_new]: row numbers (clamped) and which are real."""
    cu = s["cu"].long()
    i = torch.arange(s["max_new"], device=cu.device)
    rows = cu[:-1, None] + i
    return rows.clamp(max=s["n"] - 1), rows < cu[1:, None]


def _gather(pool, blocks):
    """Blocks [X, nb] of a pool [*, H, bs, D] as fp32 [X, H, nb * bs, D]."""
    return pool[blocks.long()].transpose(1, 2).flatten(2, 3).float()


def _plain_ragged(s):
    case, q = s["case"], s["q"]
    B, Hq, Hkv, D, bs = case["B"], case["Hq"], case["Hkv"], case["D"], case["bs"]
    rows, real = _rows_of(s)
    Tm, G = s["max_new"], Hq // Hkv
    K = _gather(s["K"], s["table"][:, :-(-s["max_len"] // bs)])
    V = _gather(s["V"], s["table"][:, :-(-s["max_len"] // bs)])
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
    Kp, Vp = _gather(s["K"], s["table"][start[:-1], :np_]), _gather(s["V"], s["table"][start[:-1], :np_])
    P = Kp.shape[2]
    seen = (torch.arange(P, device=dev) < prefix[:, None])[:, None, :, None]  # [NG, 1, P, 1]
    qp = qb[member].permute(0, 2, 1, 3, 4, 5).reshape(NG, Hkv, M * Tm * G, D)
    sp = (qp @ Kp.transpose(-1, -2)).masked_fill_(~seen.transpose(-1, -2), -math.inf)
    # each sequence's rows against its own part: [B, Hkv, Tm G, S]
    nb = -(-s["max_own"] // bs)
    cols = ((prefix[g] // bs)[:, None] + torch.arange(nb, device=dev)).clamp(max=s["table"].shape[1] - 1)
    own_blocks = s["table"].gather(1, cols)
    Ks, Vs = _gather(s["K"], own_blocks), _gather(s["V"], own_blocks)
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
    """The definition in 64 bits, token by token (append) or sequence by sequence (attention)."""
    s = prepare(case, seed)
    new, hist, _, _, _ = _shape(case)
    Hq, Hkv, D, bs = case["Hq"], case["Hkv"], case["D"], case["bs"]
    G = Hq // Hkv
    table = s["table"].cpu()
    if case["op"] == "append":
        K, V = s["K"].double(), s["V"].double()
        q_out = s["q_out"].double()
        freq = torch.tensor(s["inv_freq"], dtype=torch.float64)
        pairs, r = len(s["inv_freq"]), 0
        i1 = torch.arange(pairs) * (2 if case["adjacent"] else 1)
        i2 = i1 + (1 if case["adjacent"] else pairs)
        pos = None if s["positions"] is None else s["positions"].cpu()
        for b, (T, H) in enumerate(zip(new, hist)):
            if T == 0:
                continue
            slots = torch.arange(H, H + T)
            at = torch.stack([slots if pos is None else pos[a, r:r + T] for a in s["axis"]], 1).double()
            turn = torch.polar(torch.ones_like(at), at * freq).cuda()[:, None]  # e^{i angle}
            blocks, off = table[b][slots // bs].long().cuda(), (slots % bs).cuda()
            for src, dst in ((s["q"], q_out), (s["k"], None)):
                x = src[r:r + T].double()
                y = x.clone()
                c = torch.complex(x[..., i1.cuda()], x[..., i2.cuda()]) * turn
                y[..., i1.cuda()], y[..., i2.cuda()] = c.real, c.imag
                if dst is None:
                    K[blocks, :, off] = y
                else:
                    dst[r:r + T] = y
            V[blocks, :, off] = s["v"][r:r + T].double()
            r += T
        return {"q": q_out, "K": K, "V": V}
    out, r = s["out"].double(), 0
    for b, (T, H) in enumerate(zip(new, hist)):
        L = H + T
        blocks = table[b, :-(-L // bs)].long().cuda()
        for h in range(Hkv):
            K = s["K"][blocks, h].reshape(-1, D)[:L].double()
            V = s["V"][blocks, h].reshape(-1, D)[:L].double()
            for i in range(0, T, 512):
                n = min(512, T - i)
                q = s["q"][r + i:r + i + n, h * G:(h + 1) * G].double()
                score = torch.einsum("igd,td->igt", q, K) / math.sqrt(D)
                far = torch.arange(L, device=q.device)[None] > H + i + torch.arange(n, device=q.device)[:, None]
                score = score.masked_fill(far[:, None], -math.inf)
                out[r + i:r + i + n, h * G:(h + 1) * G] = torch.softmax(score, -1) @ V
        r += T
    return out


def work(case):
    """Bytes (each input once, each output once) and operations of one pass."""
    new, hist, start, prefix, _ = _shape(case)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    es = DTYPES[case["dtype"]].itemsize
    n = sum(new)
    if case["op"] == "append":
        return {"bytes": 2 * n * (Hq + 2 * Hkv) * D * es, "flops": 3 * n * (Hq + Hkv) * case["rot"]}
    # a shared prefix is read once for its group; a sequence without new tokens reads nothing
    kv = sum(h + t for h, t in zip(hist, new) if t)
    for a, b, p in zip(start, start[1:], prefix):
        kv -= p * max(0, sum(1 for x in new[a:b] if x) - 1)
    seen = sum(t * h + t * (t + 1) // 2 for h, t in zip(hist, new))
    return {"bytes": 2 * kv * Hkv * D * es + 2 * n * Hq * D * es, "flops": 4 * seen * Hq * D}

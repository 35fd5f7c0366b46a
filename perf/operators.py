"""The serving operators around the attention kernels, as cases to be measured:
rotary positions with several axes (and their gradient), appending tokens to a
paged key/value cache, attention of one new token over that cache, and
eviction from the cache by accumulated attention weight.

With ``own`` false ``run`` computes each operator from elementary torch
operations in 32 bits (angles in 64); with ``own`` true it makes the calls a
user makes of this package.  ``exact`` computes the same in 64 bits.

A paged cache is a pool ``[pages, Hkv, page, d]`` for K and one for V; row b of
``block_table`` names the pages of sequence b in order, ``seq_lens[b]`` its
length.  ``scores [pages, Hkv, page]`` holds the attention weight each cached
key has received so far, summed over the query heads of its group.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # q and k of the standard training workload, video positions (time, height, width).
        dict(name="rope_train", op="rope", backward=False, dtype="bf16", batch=4, hq=16, hkv=16, n=2048, d=128, rot=128,
             axes=3, interleaved=False, start=0),
        # The gradient on the grouped-query training workload.
        dict(name="rope_grad_gqa", op="rope", backward=True, dtype="bf16", batch=2, hq=32, hkv=8, n=8192, d=128, rot=128,
             axes=3, interleaved=False, start=0),
        # An image of odd size, half the head rotated, adjacent pairs, far into a long document.
        dict(name="rope_image_odd", op="rope", backward=False, dtype="fp16", batch=1, hq=8, hkv=2, n=513, d=64, rot=32,
             axes=2, interleaved=True, start=1000003),
        # One decoding step of 64 sequences: q and k rotated, k and v stored.
        dict(name="append_token", op="append", dtype="bf16", batch=64, hq=32, hkv=8, d=128, page=16, tokens=1, length=4096,
             ragged=True, axes=3, start=0),
        # A chunk of prompts of different lengths, 8192 tokens in all.
        dict(name="append_prompt", op="append", dtype="bf16", batch=5, hq=32, hkv=8, d=128, page=64, tokens=2600,
             length=2600, ragged=True, axes=3, start=0),
        # One sequence, short cache: latency.
        dict(name="decode_one", op="decode", dtype="bf16", batch=1, hq=8, hkv=2, d=128, page=16, length=1000, ragged=False,
             window=0, scores=False),
        # The decode workload: 8 sequences with 32768 keys.
        dict(name="decode_long", op="decode", dtype="bf16", batch=8, hq=32, hkv=8, d=128, page=64, length=32768,
             ragged=False, window=0, scores=False),
        # Many sequences of very different lengths (some slots of the batch empty), no grouping, d = 64.
        dict(name="decode_ragged", op="decode", dtype="fp16", batch=64, hq=16, hkv=16, d=64, page=32, length=8192,
             ragged=True, window=0, scores=False),
        # A step that also adds each key's attention weight to its score.
        dict(name="decode_scores", op="decode", dtype="bf16", batch=16, hq=32, hkv=8, d=128, page=16, length=8192,
             ragged=True, window=0, scores=True),
        # One conversation cut to half its length.
        dict(name="evict_one", op="evict", dtype="bf16", batch=1, hkv=2, d=128, page=16, length=1000, ragged=False,
             budget=500, recent=64, sinks=4),
        # A batch cut to 2048 keys a sequence.
        dict(name="evict_batch", op="evict", dtype="bf16", batch=16, hkv=8, d=128, page=16, length=8192, ragged=True,
             budget=2048, recent=256, sinks=4),
        # Two long documents cut to a quarter.
        dict(name="evict_long", op="evict", dtype="fp16", batch=2, hkv=8, d=128, page=64, length=131072, ragged=False,
             budget=32768, recent=1024, sinks=16),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "decode", "decode", "evict"])
    dtype = rng.choice(["bf16", "fp16"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8, 16])
    hq = hkv * rng.choice([1, 2, 3, 4, 8, 16] if hkv <= 2 else [1, 2, 4])
    page = rng.choice([16, 32, 48, 64, 128])
    if op == "rope":
        c = dict(op=op, backward=rng.random() < 0.5, dtype=dtype, hq=hq, hkv=hkv, d=d, rot=rng.choice([d, d, d // 2]),
                 axes=rng.choice([1, 2, 3]), interleaved=rng.random() < 0.3, start=rng.choice([0, 0, _log(rng, 1, 10 ** 7)]))
        c["batch"] = rng.randint(1, 4)
        c["n"] = _log(rng, 1, max(1, 2 * 40 * 8192 * 128 // (c["batch"] * (hq + hkv) * d)))
        return c
    if op == "append":
        c = dict(op=op, dtype=dtype, hq=hq, hkv=hkv, d=d, page=page, ragged=rng.random() < 0.7, axes=rng.choice([0, 1, 3]),
                 start=rng.choice([0, _log(rng, 1, 10 ** 6)]))
        if rng.random() < 0.5:
            c["batch"], c["tokens"] = _log(rng, 1, 256), 1
            c["length"] = _log(rng, 1, 4096)
        else:
            c["batch"] = rng.randint(1, 8)
            c["tokens"] = _log(rng, 2, 8192 // c["batch"])
            c["length"] = c["tokens"] + rng.choice([0, rng.randint(1, 2000)])
        return c
    if op == "decode":
        c = dict(op=op, dtype=dtype, batch=_log(rng, 1, 128), hq=hq, hkv=hkv, d=d, page=page, ragged=rng.random() < 0.6,
                 scores=rng.random() < 0.3)
        # No more key/value elements than 8 sequences x 8 heads x 32768 keys x 128.
        c["length"] = _log(rng, 1, min(131072, 8 * 8 * 32768 * 128 // (c["batch"] * hkv * d)))
        c["window"] = rng.choice([0, 0, 0, _log(rng, 1, 4096)])
        return c
    c = dict(op=op, dtype=dtype, batch=_log(rng, 1, 32), hkv=hkv, d=d, page=page, ragged=rng.random() < 0.6)
    c["length"] = _log(rng, 1, min(131072, 2 * 8 * 131072 * 128 // (c["batch"] * hkv * d)))
    c["budget"] = max(1, int(c["length"] * rng.uniform(0.1, 0.9)))
    c["sinks"] = min(c["budget"] // 4, rng.choice([0, 1, 4, 16]))
    c["recent"] = min(c["budget"] // 2, rng.choice([0, 1, 64, 1000]))
    return c


def _lens(c):
    """Cache lengths of the batch: all equal, or spread from none to the case's length (the last one has it)."""
    if not c["ragged"]:
        return [c["length"]] * c["batch"]
    r = random.Random(c["batch"] * 1000003 + c["length"])
    low = c["tokens"] if c["op"] == "append" and c["tokens"] == 1 else 0
    out = [r.randint(low, c["length"]) if r.random() < 0.9 else low for _ in range(c["batch"] - 1)]
    return out + [c["length"]]


def _new_tokens(c):
    """Tokens each sequence appends: one, or a prompt's worth, never more than the sequence then holds."""
    return [min(c["tokens"], n) for n in _lens(c)]


def work(c):
    e = 2
    if c["op"] == "rope":
        x = c["batch"] * (c["hq"] + c["hkv"]) * c["n"] * c["d"]
        return {"bytes": 2 * e * x + 4 * c["axes"] * c["batch"] * c["n"], "flops": 3 * x * c["rot"] // c["d"]}
    if c["op"] == "append":
        t = sum(_new_tokens(c))
        x = t * (c["hq"] + 2 * c["hkv"]) * c["d"] if c["axes"] else t * 2 * c["hkv"] * c["d"]
        return {"bytes": 2 * e * x + 4 * t * (c["axes"] + c["hkv"]),
                "flops": 3 * t * (c["hq"] + c["hkv"]) * c["d"] if c["axes"] else 0}
    lens = _lens(c)
    if c["op"] == "decode":
        keys = sum(min(n, c["window"]) if c["window"] else n for n in lens)
        b = keys * c["hkv"] * 2 * c["d"] * e + c["batch"] * c["hq"] * (2 * c["d"] * e + 4)
        if c["scores"]:
            b += 8 * keys * c["hkv"]
        return {"bytes": b, "flops": 4 * keys * c["hq"] * c["d"]}
    kept = sum(min(n, c["budget"]) for n in lens)
    return {"bytes": 4 * sum(lens) * c["hkv"] + kept * c["hkv"] * (4 * c["d"] * e + 8), "flops": 0}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _positions(shape, axes, start, dev):
    """Positions of frames of 24 x 32 patches, in order: (time, height, width), the last `axes` of them; text has one axis."""
    t = torch.arange(start, start + shape[-1], device=dev, dtype=torch.int64)
    if axes == 1:
        p = t[None]
    else:
        p = torch.stack([start + (t - start) // 768, (t - start) // 32 % 24 + start, (t - start) % 32 + start])[3 - axes:]
    return p.reshape((axes,) + (1,) * (len(shape) - 1) + shape[-1:]).expand((axes,) + tuple(shape)).to(torch.int32).contiguous()


def _frequencies(rot, axes, dev):
    """One frequency and one axis for each pair: the pairs are dealt to the axes in contiguous runs."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    return (10000.0 ** (-2.0 * i / rot)).to(dev), (torch.arange(rot // 2) * axes // (rot // 2)).to(torch.int32).to(dev)


def _pool(c, g, dev, lens, more_pages=0):
    """Pools with their pages in random order, as an allocator leaves them after a while."""
    page, pages_of = c["page"], [-(-n // c["page"]) for n in lens]
    total = sum(pages_of) + more_pages + 3
    shape = (total, c["hkv"], page, c["d"])
    dt = DTYPES[c["dtype"]]
    k = torch.empty(shape, dtype=dt, device=dev).normal_(generator=g)
    v = torch.empty(shape, dtype=dt, device=dev).normal_(generator=g)
    order = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    table = torch.zeros((c["batch"], max(1, max(pages_of))), dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(pages_of):
        table[b, :n] = order[at:at + n]
        at += n
    return k, v, table, torch.tensor(lens, dtype=torch.int32, device=dev), order[at:]


def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    dt = DTYPES[c["dtype"]]
    if c["op"] == "rope":
        q = torch.empty((c["batch"], c["hq"], c["n"], c["d"]), dtype=dt, device=dev).normal_(generator=g)
        k = torch.empty((c["batch"], c["hkv"], c["n"], c["d"]), dtype=dt, device=dev).normal_(generator=g)
        w, axes = _frequencies(c["rot"], c["axes"], dev)
        return dict(c=c, q=q, k=k, pos=_positions((c["batch"], c["n"]), c["axes"], c["start"], dev), w=w, axes=axes)
    lens = _lens(c)
    if c["op"] == "append":
        kc, vc, table, sl, _ = _pool(c, g, dev, lens)
        new = _new_tokens(c)
        cu = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], dtype=torch.int32, device=dev)
        t = sum(new)
        # The output of one projection, split into q, k and v.
        qkv = torch.empty((t, c["hq"] + 2 * c["hkv"], c["d"]), dtype=dt, device=dev).normal_(generator=g)
        q, k, v = qkv.split([c["hq"], c["hkv"], c["hkv"]], dim=1)
        s = dict(c=c, kc=kc, vc=vc, table=table, lens=sl, cu=cu, k=k, v=v, q=q,
                 scores=torch.rand(kc.shape[:3], generator=g, device=dev))
        if c["axes"]:
            s["w"], s["axes"] = _frequencies(c["d"], c["axes"], dev)
            s["pos"] = _positions((t,), c["axes"], c["start"], dev)
        return s
    if c["op"] == "decode":
        kc, vc, table, sl, _ = _pool(c, g, dev, lens)
        q = torch.empty((c["batch"], c["hq"], c["d"]), dtype=torch.float32, device=dev).normal_(generator=g).mul_(1.5).to(dt)
        s = dict(c=c, q=q, kc=kc, vc=vc, table=table, lens=sl)
        if c["scores"]:
            s["scores"] = torch.rand(kc.shape[:3], generator=g, device=dev)
            s["after"] = torch.empty_like(s["scores"])
        return s
    # Eviction: scores are sums of softmax weights, heavy-tailed, with keys that never received any.
    dst = [-(-min(n, c["budget"]) // c["page"]) for n in lens]
    kc, vc, table, sl, spare = _pool(c, g, dev, lens, more_pages=sum(dst))
    scores = torch.empty(kc.shape[:3], device=dev).normal_(generator=g).mul_(2.0).exp_()
    scores.mul_(torch.rand(kc.shape[:3], generator=g, device=dev) > 0.2)
    to = torch.zeros((c["batch"], -(-c["budget"] // c["page"])), dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(dst):
        to[b, :n] = spare[at:at + n]
        at += n
    return dict(c=c, kc=kc, vc=vc, table=table, lens=sl, scores=scores, to=to)


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(s):
    c = s["c"]
    if own:
        import exact_io_aware_flashattention_gb300 as fa
        if c["op"] == "rope":
            turn = fa.rope_backward if c["backward"] else fa.rope
            return turn(s["q"], s["k"], s["pos"], s["w"], s["axes"], interleaved=c["interleaved"])
        if c["op"] == "append":
            cu = None if c["tokens"] == 1 else s["cu"]
            if not c["axes"]:
                fa.paged_append(s["kc"], s["vc"], s["table"], s["lens"], s["k"], s["v"], cu_seqlens=cu, scores=s["scores"])
                return s["kc"], s["vc"], s["scores"]
            q = fa.paged_append(s["kc"], s["vc"], s["table"], s["lens"], s["k"], s["v"], cu_seqlens=cu, scores=s["scores"],
                                q=s["q"], positions=s["pos"], inv_freq=s["w"], axes=s["axes"])
            return s["kc"], s["vc"], s["scores"], q
        if c["op"] == "decode":
            if not c["scores"]:
                return fa.paged_decode(s["q"], s["kc"], s["vc"], s["table"], s["lens"], window=c["window"])
            s["after"].copy_(s["scores"])    # a step that may be taken back keeps the scores before it
            o, lse = fa.paged_decode(s["q"], s["kc"], s["vc"], s["table"], s["lens"], window=c["window"], scores=s["after"])
            return o, lse, s["after"]
        new, kept = fa.paged_evict(s["kc"], s["vc"], s["scores"], s["table"], s["lens"], s["to"], c["budget"],
                                   recent=c["recent"], sinks=c["sinks"])
        return s["kc"], s["vc"], s["scores"], new, kept
    return {"rope": _plain_rope, "append": _plain_append, "decode": _plain_decode, "evict": _plain_evict}[c["op"]](s)


def _turn(x, cos, sin, rot, interleaved):
    """x [..., d] with its first `rot` elements turned; cos, sin [..., rot / 2]."""
    y = x.float()
    if interleaved:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([turned, y[..., rot:]], dim=-1).to(x.dtype)


def _cos_sin(pos, w, axes):
    """Angles pos[axis of the pair] * frequency in 64 bits: at a position of a million, 32 bits leave 2^-4 of a radian."""
    angle = pos[axes.long()].double().movedim(0, -1) * w
    return angle.cos().float(), angle.sin().float()


def _plain_rope(s):
    c = s["c"]
    cos, sin = _cos_sin(s["pos"], s["w"], s["axes"])
    cos, sin = cos[:, None], sin[:, None]
    if c["backward"]:
        sin = -sin
    return (_turn(s["q"], cos, sin, c["rot"], c["interleaved"]), _turn(s["k"], cos, sin, c["rot"], c["interleaved"]))


def _plain_append(s):
    c, page = s["c"], s["c"]["page"]
    t = s["k"].shape[0]
    token = torch.arange(t, device=s["k"].device)
    cu = s["cu"].long()
    seq = torch.searchsorted(cu[1:], token, right=True)
    at = s["lens"].long()[seq] - (cu[seq + 1] - token)
    where = s["table"][seq, at // page].long()
    k, q = s["k"], None
    if c["axes"]:
        cos, sin = _cos_sin(s["pos"], s["w"], s["axes"])
        cos, sin = cos[:, None], sin[:, None]
        k = _turn(k, cos, sin, c["d"], False)
        q = _turn(s["q"], cos, sin, c["d"], False)
    s["kc"][where, :, at % page] = k
    s["vc"][where, :, at % page] = s["v"]
    s["scores"][where, :, at % page] = 0.0
    return (s["kc"], s["vc"], s["scores"]) if q is None else (s["kc"], s["vc"], s["scores"], q)


def _plain_decode(s):
    c = s["c"]
    B, Hkv, d, G = c["batch"], c["hkv"], c["d"], c["hq"] // c["hkv"]
    L = s["table"].shape[1] * c["page"]
    k = s["kc"][s["table"].long()].transpose(1, 2).reshape(B, Hkv, L, d).float()
    v = s["vc"][s["table"].long()].transpose(1, 2).reshape(B, Hkv, L, d).float()
    j = torch.arange(L, device=k.device)
    n = s["lens"].long()[:, None]
    seen = (j < n) & (j >= n - c["window"]) if c["window"] else j < n
    x = torch.matmul(s["q"].float().view(B, Hkv, G, d) * d ** -0.5, k.transpose(-1, -2))
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top.isinf(), 0.0, top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, 1.0)
    o = torch.matmul(p, v.masked_fill(~seen[:, None, :, None], 0.0)).view(B, c["hq"], d).to(s["q"].dtype)
    lse = (torch.where(top.isinf(), 0.0, top) + total.log()).view(B, c["hq"])
    if not c["scores"]:
        return o, lse
    s["after"].copy_(s["scores"])
    add = p.sum(2).view(B, Hkv, -1, c["page"]).transpose(1, 2)       # [B, pages, Hkv, page]
    s["after"].index_put_((s["table"].long(),), add, accumulate=True)
    return o, lse, s["after"]


def _plain_evict(s):
    c, page = s["c"], s["c"]["page"]
    B, Hkv, budget = c["batch"], c["hkv"], c["budget"]
    L = s["table"].shape[1] * page
    x = s["scores"][s["table"].long()].transpose(1, 2).reshape(B, Hkv, L)
    j = torch.arange(max(L, budget), device=x.device)
    x = torch.nn.functional.pad(x, (0, j.numel() - L))
    n = s["lens"].long()[:, None, None]
    x = torch.where((j < c["sinks"]) | (j >= n - c["recent"]), math.inf, x)
    x = torch.where(j < n, x, -math.inf).expand(B, Hkv, -1)
    first = torch.sort(x, dim=-1, descending=True, stable=True)[1][..., :budget]
    i = torch.arange(budget, device=x.device)
    new = n.clamp(max=budget)
    kept = torch.sort(torch.where(i < new, first, j.numel()), dim=-1)[0]
    b, h, r = (torch.arange(B, device=x.device)[:, None, None].expand_as(kept),
               torch.arange(Hkv, device=x.device)[:, None].expand_as(kept), i.expand_as(kept))
    have = (i < new).expand_as(kept)
    b, h, r, src = b[have], h[have], r[have], kept[have]
    old_page, new_page = s["table"][b, src // page].long(), s["to"][b, r // page].long()
    s["kc"][new_page, h, r % page] = s["kc"][old_page, h, src % page]
    s["vc"][new_page, h, r % page] = s["vc"][old_page, h, src % page]
    s["scores"][new_page, h, r % page] = s["scores"][old_page, h, src % page]
    return (s["kc"], s["vc"], s["scores"], new.reshape(B).to(torch.int32), torch.where(have, kept, -1).to(torch.int32))


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------
def _exact_rotation(x, pos, w, axes, rot, interleaved, sign):
    """x [..., tokens.., d] as complex numbers times e^{i sign angle}; pos [axes, ...] broadcast against x[..., 0]."""
    y = x.double().clone()
    for i in range(rot // 2):
        lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        z = torch.complex(y[..., lo].clone(), y[..., hi].clone())
        angle = sign * pos[int(axes[i])].double() * float(w[i])
        z = z * torch.complex(angle.cos(), angle.sin())
        y[..., lo], y[..., hi] = z.real, z.imag
    return y


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "rope":
        sign = -1.0 if c["backward"] else 1.0
        return tuple(_exact_rotation(x, s["pos"][:, :, None], s["w"], s["axes"], c["rot"], c["interleaved"], sign)
                     for x in (s["q"], s["k"]))
    lens, page = _lens(c), c["page"]
    if c["op"] == "append":
        k, v, q = s["k"].double(), s["v"].double(), None
        if c["axes"]:
            k = _exact_rotation(k, s["pos"][:, :, None], s["w"], s["axes"], c["d"], False, 1.0)
            q = _exact_rotation(s["q"], s["pos"][:, :, None], s["w"], s["axes"], c["d"], False, 1.0)
        kc, vc, sc = s["kc"].double(), s["vc"].double(), s["scores"].double()
        at = 0
        for b, new in enumerate(_new_tokens(c)):
            i = torch.arange(lens[b] - new, lens[b], device=kc.device)
            pages = s["table"][b].long()[i // page]
            kc[pages, :, i % page] = k[at:at + new]
            vc[pages, :, i % page] = v[at:at + new]
            sc[pages, :, i % page] = 0.0
            at += new
        return (kc, vc, sc) if q is None else (kc, vc, sc, q)
    if c["op"] == "decode":
        G = c["hq"] // c["hkv"]
        o = torch.zeros((c["batch"], c["hq"], c["d"]), dtype=torch.float64, device=s["q"].device)
        lse = torch.full((c["batch"], c["hq"]), -math.inf, dtype=torch.float64, device=o.device)
        sc = s["scores"].double() if c["scores"] else None
        for b, n in enumerate(lens):
            i = torch.arange(max(0, n - c["window"]) if c["window"] else 0, n, device=o.device)
            if i.numel() == 0:
                continue
            pages = s["table"][b].long()[i // page]
            for g in range(c["hkv"]):
                k, v = s["kc"][pages, g, i % page].double(), s["vc"][pages, g, i % page].double()
                x = (s["q"][b, g * G:(g + 1) * G].double() @ k.T) / math.sqrt(c["d"])
                z = torch.logsumexp(x, dim=-1)
                p = torch.exp(x - z[:, None])
                o[b, g * G:(g + 1) * G] = p @ v
                lse[b, g * G:(g + 1) * G] = z
                if sc is not None:
                    sc[pages, g, i % page] += p.sum(0)
        return (o, lse) if sc is None else (o, lse, sc)
    B, Hkv = c["batch"], c["hkv"]
    kc, vc, sc = s["kc"].double(), s["vc"].double(), s["scores"].double()
    kept = torch.full((B, Hkv, c["budget"]), -1, dtype=torch.int32, device=kc.device)
    for b, n in enumerate(lens):
        m = min(n, c["budget"])
        if m == 0:
            continue
        i = torch.arange(n, device=kc.device)
        pages = s["table"][b].long()[i // page]
        r = torch.arange(m, device=kc.device)
        to = s["to"][b].long()[r // page]
        for h in range(Hkv):
            x = s["scores"][pages, h, i % page].double()
            safe = (i < c["sinks"]) | (i >= n - c["recent"])
            if m < n:
                free = i[~safe]
                order = torch.argsort(-x[free], stable=True)[:m - int(safe.sum())]
                mine = torch.cat([i[safe], free[order]]).sort()[0]
            else:
                mine = i
            kept[b, h, :m] = mine.to(torch.int32)
            kc[to, h, r % page] = s["kc"][pages[mine], h, mine % page].double()
            vc[to, h, r % page] = s["vc"][pages[mine], h, mine % page].double()
            sc[to, h, r % page] = s["scores"][pages[mine], h, mine % page].double()
    return kc, vc, sc, torch.tensor([min(n, c["budget"]) for n in lens], dtype=torch.int32, device=kc.device), kept

"""Operators for models that norm their queries and keys, and for serving from
a key/value cache held in 4 bits, as cases to be measured: the norm of each
head's rows with the position rotation in the same pass (and its gradient),
appending tokens to the 4-bit cache (normed and turned on the way), reading
keys and values back from it as 16-bit rows, and attention of one new token
over it.

With ``own`` false ``run`` computes each operator from elementary torch
operations in 32 bits (angles and long sums in 64); with ``own`` true it makes
the calls a user makes of this package.  ``exact`` computes the same in 64 bits.

Norm and rotation of a row x of d elements: x times (mean x^2 + eps)^-1/2 times
the weights, then pair i turned by position[axis_i] * frequency_i.

The 4-bit cache: a row is first rounded to the tensors' type T; each group of 64
of its elements has z = its smallest and s = T((largest - z) / 15), both in T,
and holds x as the whole number c = (x - z) / s, rounded to nearest (ties to
even), between 0 and 15 (0 where s is 0); it stands for z + s c.  Cached rows
are returned as these values, in T where a call returns them so.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
GROUP = 64
EPS = 1e-6


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # q and k of the standard training workload, video positions (time, height, width).
        dict(name="norm_rope_train", op="norm", backward=False, dtype="bf16", batch=4, hq=16, hkv=16, n=2048, d=128, rot=128,
             axes=3, interleaved=False, start=0, weights="bf16"),
        # An image of odd size, half the head rotated, adjacent pairs, far into a long document.
        dict(name="norm_rope_image_odd", op="norm", backward=False, dtype="fp16", batch=1, hq=8, hkv=2, n=513, d=64, rot=32,
             axes=2, interleaved=True, start=1000003, weights="fp32"),
        # The gradient on the grouped-query training workload.
        dict(name="norm_rope_grad_gqa", op="norm", backward=True, dtype="bf16", batch=2, hq=32, hkv=8, n=8192, d=128, rot=128,
             axes=3, interleaved=False, start=0, weights="bf16"),
        # The gradient of a short, odd sequence.
        dict(name="norm_rope_grad_odd", op="norm", backward=True, dtype="fp16", batch=1, hq=8, hkv=2, n=513, d=64, rot=64,
             axes=1, interleaved=False, start=0, weights="fp32"),
        # One decoding step of 64 sequences: q and k normed and turned, k and v stored; the new rows read back.
        dict(name="append4_token", op="append", dtype="bf16", batch=64, hq=32, hkv=8, d=128, page=16, tokens=1, length=4096,
             ragged=True, axes=3, norm=True, start=0, weights="bf16"),
        # A chunk of prompts of different lengths, then read back for the attention over it.
        dict(name="append4_prompt", op="append", dtype="bf16", batch=5, hq=32, hkv=8, d=128, page=64, tokens=2600,
             length=2600, ragged=True, axes=3, norm=True, start=0, weights="bf16"),
        # The prefix of a long prompt read back, for the attention of its next chunk.
        dict(name="read4_prefix", op="read", dtype="bf16", batch=1, hkv=8, d=128, page=64, length=32768, ragged=False,
             n=32768),
        # The last 1000 keys of sequences of very different lengths, some shorter (or empty).
        dict(name="read4_window", op="read", dtype="fp16", batch=16, hkv=4, d=64, page=16, length=4096, ragged=True, n=1000),
        # One sequence, short cache: latency.
        dict(name="decode4_one", op="decode", dtype="bf16", batch=1, hq=8, hkv=2, d=128, page=16, length=1000, ragged=False,
             window=0),
        # 16 long sequences.
        dict(name="decode4_long", op="decode", dtype="bf16", batch=16, hq=32, hkv=8, d=128, page=64, length=32768,
             ragged=False, window=0),
        # Many sequences of very different lengths (some slots of the batch empty), no grouping, d = 64.
        dict(name="decode4_ragged", op="decode", dtype="fp16", batch=64, hq=16, hkv=16, d=64, page=32, length=8192,
             ragged=True, window=0),
        # Sixteen query heads a group and a sliding window.
        dict(name="decode4_window", op="decode", dtype="bf16", batch=32, hq=32, hkv=2, d=128, page=16, length=16384,
             ragged=True, window=4096),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


# No drawn case has more elements than these (the largest listed ones have them).
_MOST_ROWS = 2 * 40 * 8192 * 128
_MOST_CACHED = 16 * 8 * 32768 * 128


def draw(rng):
    op = rng.choice(["norm", "norm", "append", "read", "decode", "decode"])
    dtype = rng.choice(["bf16", "fp16"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8, 16])
    hq = hkv * rng.choice([1, 2, 3, 4, 8, 16] if hkv <= 2 else [1, 2, 4])
    page = rng.choice([16, 32, 48, 64, 128])
    if op == "norm":
        c = dict(op=op, backward=rng.random() < 0.5, dtype=dtype, hq=hq, hkv=hkv, d=d, rot=rng.choice([d, d, d // 2]),
                 axes=rng.choice([0, 1, 2, 3]), interleaved=rng.random() < 0.3,
                 start=rng.choice([0, 0, _log(rng, 1, 10 ** 7)]), weights=rng.choice([dtype, "fp32"]))
        c["batch"] = rng.randint(1, 4)
        c["n"] = _log(rng, 1, max(1, _MOST_ROWS // (c["batch"] * (hq + hkv) * d)))
        return c
    if op == "append":
        c = dict(op=op, dtype=dtype, hq=hq, hkv=hkv, d=d, page=page, ragged=rng.random() < 0.7, axes=rng.choice([0, 1, 3]),
                 norm=rng.random() < 0.6, start=rng.choice([0, _log(rng, 1, 10 ** 6)]), weights=rng.choice([dtype, "fp32"]))
        if rng.random() < 0.5:
            c["batch"], c["tokens"] = _log(rng, 1, 256), 1
            c["length"] = _log(rng, 1, 4096)
        else:
            c["batch"] = rng.randint(1, 8)
            c["tokens"] = _log(rng, 2, 8192 // c["batch"])
            c["length"] = c["tokens"] + rng.choice([0, rng.randint(1, 2000)])
        return c
    c = dict(op=op, dtype=dtype, hkv=hkv, d=d, page=page, ragged=rng.random() < 0.6)
    if op == "read":
        c["batch"] = _log(rng, 1, 32)
        c["length"] = _log(rng, 1, min(131072, _MOST_CACHED // 8 // (c["batch"] * hkv * d)))
        c["n"] = c["length"] if rng.random() < 0.5 else _log(rng, 1, c["length"])
        return c
    c["hq"], c["batch"] = hq, _log(rng, 1, 128)
    c["length"] = _log(rng, 1, min(131072, _MOST_CACHED // (c["batch"] * hkv * d)))
    c["window"] = rng.choice([0, 0, 0, _log(rng, 1, 4096)])
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


def _cached_row(d):
    """Bytes of one key's row: codes, and s and z of each group."""
    return d // 2 + d // GROUP * 4


def work(c):
    e, d = 2, c["d"]
    if c["op"] == "norm":
        x = c["batch"] * (c["hq"] + c["hkv"]) * c["n"] * d
        turned = 3 * x * c["rot"] // d if c["axes"] else 0
        w = 2 * d * (4 if c["weights"] == "fp32" else 2)
        if c["backward"]:
            return {"bytes": 3 * e * x + 4 * c["axes"] * c["batch"] * c["n"] + w + 8 * d, "flops": turned + 11 * x}
        return {"bytes": 2 * e * x + 4 * c["axes"] * c["batch"] * c["n"] + w, "flops": turned + 4 * x}
    if c["op"] == "append":
        new = _new_tokens(c)
        t, back = sum(new), max(new) * c["batch"]
        q = t * c["hq"] * d if c["axes"] or c["norm"] else 0
        kv = 2 * t * c["hkv"]
        return {"bytes": 2 * e * q + kv * (e * d + 2 * _cached_row(d)) + 2 * back * c["hkv"] * e * d + 4 * t * c["axes"],
                "flops": 8 * q + 10 * kv * d}
    lens = _lens(c)
    if c["op"] == "read":
        keys = sum(min(n, c["n"]) for n in lens)
        return {"bytes": 2 * c["hkv"] * (keys * _cached_row(d) + c["batch"] * c["n"] * e * d), "flops": 4 * keys * c["hkv"] * d}
    keys = sum(min(n, c["window"]) if c["window"] else n for n in lens)
    return {"bytes": 2 * keys * c["hkv"] * _cached_row(d) + c["batch"] * c["hq"] * (2 * d * e + 4),
            "flops": 4 * keys * c["hq"] * d}


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


def _rows(g, dev, shape, dt):
    """Rows of a projection: channels of different size, as trained ones have."""
    size = torch.empty(shape[-1], device=dev).normal_(generator=g).mul_(0.5).exp_()
    return torch.empty(shape, dtype=dt, device=dev).normal_(generator=g).mul_(size.to(dt))


def _norm_weights(g, dev, c):
    dt = torch.float32 if c["weights"] == "fp32" else DTYPES[c["dtype"]]
    return [(1 + 0.2 * torch.empty(c["d"], device=dev).normal_(generator=g)).to(dt) for _ in range(2)]


def _pages(c, g, dev, lens):
    """Block table with the pages in random order, as an allocator leaves them after a while."""
    pages_of = [-(-n // c["page"]) for n in lens]
    total = sum(pages_of) + 3
    order = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    table = torch.zeros((c["batch"], max(1, max(pages_of))), dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(pages_of):
        table[b, :n] = order[at:at + n]
        at += n
    return total, table, torch.tensor(lens, dtype=torch.int32, device=dev)


def _offsets(counts, dev):
    return torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=torch.int32, device=dev)


def _plain_pool(c, total, dev):
    """Codes two to a byte (the even element in the low half), s and z, of K and of V."""
    dt, rows = DTYPES[c["dtype"]], (total, c["hkv"], c["page"])
    return {x: dict(codes=torch.zeros(rows + (c["d"] // 2,), dtype=torch.uint8, device=dev),
                    s=torch.zeros(rows + (c["d"] // GROUP,), dtype=dt, device=dev),
                    z=torch.zeros(rows + (c["d"] // GROUP,), dtype=dt, device=dev)) for x in "kv"}


def _cached(c, g, dev, rows):
    """A cache full of keys and values; or, if `rows`, their rows [T, Hkv, d] alone, sequence after sequence."""
    lens = _lens(c)
    total, table, sl = _pages(c, g, dev, lens)
    k, v = (_rows(g, dev, (sum(lens), c["hkv"], c["d"]), DTYPES[c["dtype"]]) for _ in range(2))
    s = dict(c=c, table=table, lens=sl)
    cu = _offsets(lens, dev)
    if rows:
        s["k"], s["v"] = k, v
    elif own:
        import exact_io_aware_flashattention_gb300 as fa
        s["cache"] = fa.paged4_cache(total, c["hkv"], c["page"], c["d"], device=dev)
        fa.paged4_append(s["cache"], table, sl, k, v, cu_seqlens=cu)
    else:
        s["pool"] = _plain_pool(c, total, dev)
        _store(s["pool"], table, sl, cu, c["page"], k, v)
    return s


def prepare(c, seed):
    return _prepare(c, seed, False)


def _prepare(c, seed, rows):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    dt = DTYPES[c["dtype"]]
    if c["op"] == "norm":
        heads = {"q": c["hq"], "k": c["hkv"]}
        s = dict(c=c, **{x: _rows(g, dev, (c["batch"], h, c["n"], c["d"]), dt) for x, h in heads.items()})
        s["wq"], s["wk"] = _norm_weights(g, dev, c)
        if c["axes"]:
            s["w"], s["axes"] = _frequencies(c["rot"], c["axes"], dev)
            s["pos"] = _positions((c["batch"], c["n"]), c["axes"], c["start"], dev)
        if c["backward"]:
            for x in heads:
                s["d" + x] = torch.empty_like(s[x]).normal_(generator=g)
        return s
    if c["op"] == "append":
        lens, new = _lens(c), _new_tokens(c)
        total, table, sl = _pages(c, g, dev, lens)
        t = sum(new)
        # The output of one projection, split into q, k and v.
        q, k, v = _rows(g, dev, (t, c["hq"] + 2 * c["hkv"], c["d"]), dt).split([c["hq"], c["hkv"], c["hkv"]], dim=1)
        s = dict(c=c, table=table, lens=sl, cu=_offsets(new, dev), q=q, k=k, v=v, n=max(new))
        s["wq"], s["wk"] = _norm_weights(g, dev, c)
        if c["axes"]:
            s["w"], s["axes"] = _frequencies(c["d"], c["axes"], dev)
            s["pos"] = _positions((t,), c["axes"], c["start"], dev)
        if rows:
            pass
        elif own:
            import exact_io_aware_flashattention_gb300 as fa
            s["cache"] = fa.paged4_cache(total, c["hkv"], c["page"], c["d"], device=dev)
        else:
            s["pool"] = _plain_pool(c, total, dev)
        return s
    s = _cached(c, g, dev, rows)
    if c["op"] == "decode":
        s["q"] = torch.empty((c["batch"], c["hq"], c["d"]), dtype=torch.float32, device=dev).normal_(generator=g).to(dt)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(s):
    c = s["c"]
    if own:
        import exact_io_aware_flashattention_gb300 as fa
        turn = dict(positions=s["pos"], inv_freq=s["w"], axes=s["axes"]) if c.get("axes") else {}
        if c["op"] == "norm":
            if turn:
                turn["interleaved"] = c["interleaved"]
            if c["backward"]:
                return fa.qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["wq"], s["wk"], eps=EPS, **turn)
            return fa.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], eps=EPS, **turn)
        if c["op"] == "append":
            cu = None if c["tokens"] == 1 else s["cu"]
            norm = dict(q_weight=s["wq"], k_weight=s["wk"], eps=EPS) if c["norm"] else {}
            q = s["q"] if norm or turn else None
            q = fa.paged4_append(s["cache"], s["table"], s["lens"], s["k"], s["v"], cu_seqlens=cu, q=q, **norm, **turn)
            k, v = fa.paged4_read(s["cache"], s["table"], s["lens"], s["n"], DTYPES[c["dtype"]])
            return (k, v) if q is None else (k, v, q)
        if c["op"] == "read":
            return fa.paged4_read(s["cache"], s["table"], s["lens"], c["n"], DTYPES[c["dtype"]])
        return fa.paged4_decode(s["q"], s["cache"], s["table"], s["lens"], window=c["window"])
    return {"norm": _plain_norm, "append": _plain_append, "read": _plain_read, "decode": _plain_decode}[c["op"]](s)


def _turn(y, cos, sin, rot, interleaved):
    """y [..., d] in 32 bits with its first `rot` elements turned; cos, sin [..., rot / 2]."""
    if interleaved:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([turned, y[..., rot:]], dim=-1)


def _cos_sin(s):
    """Angles pos[axis of the pair] * frequency in 64 bits: at a position of a million, 32 bits leave 2^-4 of a radian."""
    angle = s["pos"][s["axes"].long()].double().movedim(0, -1) * s["w"]
    return angle.cos().float()[..., None, :, :], angle.sin().float()[..., None, :, :]


def _inverse_size(x):
    return torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)


def _plain_norm(s):
    c, out, weights = s["c"], [], []
    if c["axes"]:
        cos, sin = _cos_sin(s)
    for name in "qk":
        x, w = s[name].float(), s["w" + name].float()
        r = _inverse_size(x)
        if not c["backward"]:
            y = x * r * w
            if c["axes"]:
                y = _turn(y, cos, sin, c["rot"], c["interleaved"])
            out.append(y.to(s[name].dtype))
            continue
        g = s["d" + name].float()
        if c["axes"]:
            g = _turn(g, cos, -sin, c["rot"], c["interleaved"])
        xr, gw = x * r, g * w
        out.append((r * (gw - xr * (gw * xr).mean(-1, keepdim=True))).to(s[name].dtype))
        weights.append((g * xr).sum((0, 1, 2), dtype=torch.float64).float())
    return tuple(out + weights)


def _quantised(x):
    """Codes (0 to 15, 32 bits), s and z of rows [..., d] of 16-bit values."""
    y = x.float().unflatten(-1, (-1, GROUP))
    lo, hi = y.amin(-1, keepdim=True), y.amax(-1, keepdim=True)
    s = ((hi - lo) / 15.0).to(x.dtype)
    c = ((y - lo) / s.float()).round().clamp(0, 15)
    c = torch.where(s.float() == 0, 0.0, c)
    return c.flatten(-2), s.squeeze(-1), lo.squeeze(-1).to(x.dtype)


def _values(codes, s, z):
    """What packed codes [..., d / 2] stand for, in 32 bits."""
    c = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).float()
    return (z.float()[..., None] + s.float()[..., None] * c.unflatten(-1, (-1, GROUP))).flatten(-2)


def _slots(table, lens, cu, page, t):
    """Page and slot of each of t tokens, which are the last of their sequences."""
    token = torch.arange(t, device=table.device)
    cu = cu.long()
    seq = torch.searchsorted(cu[1:], token, right=True)
    at = lens.long()[seq] - (cu[seq + 1] - token)
    return table[seq, at // page].long(), at % page


def _store(pool, table, lens, cu, page, k, v):
    where, slot = _slots(table, lens, cu, page, k.shape[0])
    step = max(1, 2 ** 27 // max(1, k[:1].numel()))           # tokens at a time: the 32-bit rows are large
    for x, rows in (("k", k), ("v", v)):
        for a in range(0, k.shape[0], step):
            c, s, z = _quantised(rows[a:a + step])
            c = c.to(torch.uint8)
            p, i = where[a:a + step], slot[a:a + step]
            pool[x]["codes"][p, :, i] = c[..., 0::2] | (c[..., 1::2] << 4)
            pool[x]["s"][p, :, i] = s
            pool[x]["z"][p, :, i] = z


def _last(s, n):
    """The last n keys of each sequence: K and V rows [B, Hkv, n, d], zero where a sequence has fewer."""
    c = s["c"]
    j = s["lens"].long()[:, None] - n + torch.arange(n, device=s["lens"].device)
    at = j.clamp(min=0)
    page = torch.gather(s["table"].long(), 1, at // c["page"])
    out = []
    for x in "kv":
        rows = _values(*(s["pool"][x][y][page, :, at % c["page"]] for y in ("codes", "s", "z")))     # [B, n, Hkv, d]
        rows = torch.where((j >= 0)[..., None, None], rows, 0.0)
        out.append(rows.transpose(1, 2).to(DTYPES[c["dtype"]]).contiguous())
    return tuple(out)


def _plain_append(s):
    c, k, q = s["c"], s["k"], s["q"]
    if c["norm"] or c["axes"]:
        y = {}
        for name in "qk":
            x = s[name].float()
            if c["norm"]:
                x = x * _inverse_size(x) * s["w" + name].float()
            if c["axes"]:
                cos, sin = (t[0, :, None] for t in _cos_sin(s))
                x = _turn(x, cos, sin, c["d"], False)
            y[name] = x.to(s[name].dtype)
        q, k = y["q"], y["k"]
    else:
        q = None
    _store(s["pool"], s["table"], s["lens"], s["cu"], c["page"], k, s["v"])
    back = _last(s, s["n"])
    return back if q is None else back + (q,)


def _plain_read(s):
    return _last(s, s["c"]["n"])


def _plain_decode(s):
    c = s["c"]
    B, Hkv, d, G = c["batch"], c["hkv"], c["d"], c["hq"] // c["hkv"]
    L, table = s["table"].shape[1] * c["page"], s["table"].long()
    j = torch.arange(L, device=table.device)
    n = s["lens"].long()[:, None]
    seen = (j < n) & (j >= n - c["window"]) if c["window"] else j < n
    k, v = (_values(*(s["pool"][x][y][table].transpose(1, 2).reshape(B, Hkv, L, -1) for y in ("codes", "s", "z")))
            for x in "kv")
    x = torch.matmul(s["q"].float().view(B, Hkv, G, d) * d ** -0.5, k.transpose(-1, -2))
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top.isinf(), 0.0, top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, 1.0)
    o = torch.matmul(p, v.masked_fill(~seen[:, None, :, None], 0.0)).view(B, c["hq"], d).to(s["q"].dtype)
    lse = (torch.where(top.isinf(), 0.0, top) + total.log()).view(B, c["hq"])
    return o, lse


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------
def _exact_row(x, w, pos, freq, axes, interleaved):
    """Normed (w not None) and turned (pos not None) rows x [..., d] in 64 bits, pairs as complex numbers; pos
    [axes, ...] broadcast against x[..., 0].  Differentiable."""
    if w is not None:
        x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS) * w
    if pos is None:
        return x
    rot = 2 * freq.numel()
    head = x[..., :rot].unflatten(-1, (rot // 2, 2) if interleaved else (2, rot // 2))
    z = torch.complex(head[..., 0], head[..., 1]) if interleaved else torch.complex(head[..., 0, :], head[..., 1, :])
    angle = pos.double()[axes.long()].movedim(0, -1) * freq
    z = z * torch.polar(torch.ones_like(angle), angle)
    head = torch.stack([z.real, z.imag], -1 if interleaved else -2).flatten(-2)
    return torch.cat([head, x[..., rot:]], -1)


def _exact_values(x, dt):
    """The values that the cache holds for rows x [..., d], which are rounded to dt first."""
    y = x.to(dt).double().unflatten(-1, (-1, GROUP))
    z, top = y.min(-1, keepdim=True)[0], y.max(-1, keepdim=True)[0]
    s = ((top - z) / 15).to(dt).double()
    steps = torch.round((y - z) / torch.where(s > 0, s, 1.0))
    return (z + s * torch.minimum(steps, torch.full_like(steps, 15.0))).flatten(-2)


def _exact_norm(c, s):
    out, weights = [], []
    pos = s["pos"][:, :, None] if c["axes"] else None
    turn = (s["w"], s["axes"], c["interleaved"]) if c["axes"] else (None, None, False)
    for name in "qk":
        w = s["w" + name].double()
        y, dw = torch.empty(s[name].shape, dtype=torch.float64, device=w.device), torch.zeros_like(w)
        for b in range(c["batch"]):
            p = pos[:, b:b + 1] if c["axes"] else None
            x = s[name][b:b + 1].double()
            if not c["backward"]:
                y[b:b + 1] = _exact_row(x, w, p, *turn)
                continue
            for h in range(x.shape[1]):        # by the derivative of the definition, a head at a time
                xh, wh = x[:, h:h + 1].clone().requires_grad_(), w.clone().requires_grad_()
                dx, d = torch.autograd.grad(_exact_row(xh, wh, p, *turn), (xh, wh), s["d" + name][b:b + 1, h:h + 1].double())
                y[b:b + 1, h:h + 1] = dx
                dw += d
        out.append(y)
        weights.append(dw)
    return tuple(out + weights) if c["backward"] else tuple(out)


def exact(c, seed):
    s = _prepare(c, seed, True)
    if c["op"] == "norm":
        return _exact_norm(c, s)
    lens, dt, dev = _lens(c), DTYPES[c["dtype"]], s["lens"].device
    if c["op"] == "append":
        turn = (s["pos"][:, :, None], s["w"], s["axes"], False) if c["axes"] else (None, None, None, False)
        rows = [_exact_row(s[x].double(), s["w" + x].double() if c["norm"] else None, *turn) for x in "qk"]
        q, k, v = rows[0], _exact_values(rows[1], dt), _exact_values(s["v"], dt)
        out = [torch.zeros((c["batch"], c["hkv"], s["n"], c["d"]), dtype=torch.float64, device=dev) for _ in range(2)]
        at = 0
        for b, new in enumerate(_new_tokens(c)):
            for o, x in zip(out, (k, v)):
                o[b, :, s["n"] - new:] = x[at:at + new].transpose(0, 1)
            at += new
        return tuple(out) + ((q,) if c["norm"] or c["axes"] else ())
    k, v = s["k"], s["v"]
    if c["op"] == "read":
        out = [torch.zeros((c["batch"], c["hkv"], c["n"], c["d"]), dtype=torch.float64, device=dev) for _ in range(2)]
        at = 0
        for b, n in enumerate(lens):
            m = min(n, c["n"])
            for o, x in zip(out, (k, v)):
                o[b, :, c["n"] - m:] = _exact_values(x[at + n - m:at + n], dt).transpose(0, 1)
            at += n
        return tuple(out)
    G = c["hq"] // c["hkv"]
    o = torch.zeros((c["batch"], c["hq"], c["d"]), dtype=torch.float64, device=dev)
    lse = torch.full((c["batch"], c["hq"]), -math.inf, dtype=torch.float64, device=dev)
    at = 0
    for b, n in enumerate(lens):
        first = max(0, n - c["window"]) if c["window"] else 0
        if n > 0:
            kb, vb = (_exact_values(x[at + first:at + n], dt).transpose(0, 1) for x in (k, v))
            x = torch.einsum("hgd,hnd->hgn", s["q"][b].double().view(c["hkv"], G, -1), kb) / math.sqrt(c["d"])
            top = torch.logsumexp(x, dim=-1)
            o[b] = torch.einsum("hgn,hnd->hgd", torch.exp(x - top[..., None]), vb).reshape(c["hq"], -1)
            lse[b] = top.reshape(-1)
        at += n
    return o, lse

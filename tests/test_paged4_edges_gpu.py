"""Where the 4-bit cache's calls and the normed rows could lose a last place or
a range (GPU).  Tolerances as in test_paged4_gpu (u = half a step of the
tensors' type), but for what a test states itself.
"""
import math

import numpy as np
import pytest
import torch

import exact_io_aware_flashattention_gb300 as fa
from oracle import paged4
from tests.test_paged4_gpu import (BF, DEV, F32, HF, TINY, U, assert_decoded, assert_normed, assert_read, f64, filled, last_rows,
                                   new_cache, offsets, ok, rounder, tables, turned, weights)

pytestmark = pytest.mark.gpu


def widened(table, wide):
    """The same table, or with as many columns more as make the parts equal instead of clusters."""
    if not wide:
        return table
    t = torch.full((table.shape[0], 4000), 2 ** 30, dtype=torch.int32, device=DEV)
    t[:, :table.shape[1]] = table
    return t


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (4, 1), (8, 2), (6, 1), (16, 2), (32, 2), (20, 1)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dt", [BF, HF])
def test_weights_whose_products_cancel(cuda_lib, dt, d, Hq, Hkv, wide):
    # Two keys of opposite values and nearly equal weights, 1 and exp(-delta): o is their difference, and a weight rounded
    # to 11 bits would show in it.  Rows of one value are held exactly (s = 0), odd numbers -15 .. 15 too (s = 2).
    # K is 0 and -kappa, q one value t a head, so a score is off by its own roundings, X (d + 8) 2^-23 with X = delta; its
    # exponential by 2^-21 (a factor 2); a weight by 2^-22; the sums of two keys' products, of codes from 0 and their start,
    # by 16 2^-23: all relative to A = sum p (|z| + 32 s).
    B, kappa = 8, 2.0 ** -12
    k = torch.zeros((2 * B, Hkv, d))
    k[1::2] = -kappa
    g = torch.Generator().manual_seed(Hq * d)
    v = torch.randint(0, 16, (B, Hkv, d), generator=g).float() * 2 - 15
    v[..., 0::64], v[..., 1::64] = -15.0, 15.0
    v = torch.stack([v, -v], dim=1).reshape(2 * B, Hkv, d)
    q = (1 + torch.randint(0, 64, (B, Hq, 1), generator=g) / 64).expand(B, Hq, d)
    k, v, q = (t.to(dt).to(DEV).contiguous() for t in (k, v, q))
    cache, table, ln, _, _ = filled([2] * B, Hkv, 16, d, dt, seed=7, rows=[k, v])
    o, _ = fa.paged4_decode(q, cache, widened(table, wide), ln)
    ok()
    for b in range(B):
        kb, vb = (f64(t)[2 * b:2 * b + 2].swapaxes(0, 1) for t in (k, v))
        want, _, x, a = paged4.decode(f64(q)[b], kb, vb, d ** -0.5, 0, rounder(dt))
        e = (x * (d + 8) * 2.0 ** -23 + 2.0 ** -21)[:, None]
        bound = U[dt] * np.abs(want) + (2.1 * e + 2.0 ** -22 + 16 * 2.0 ** -23) * a + TINY[dt]
        err = np.abs(f64(o)[b] - want)
        assert (err <= bound).all(), f"sequence {b}: {(err > bound).sum()} values, {(err / bound).max()} of the bound"


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("Hq,d", [(4, 64), (4, 128), (8, 128), (16, 64), (32, 128)])
@pytest.mark.parametrize("top", [100, 111, 114, 118])
def test_values_near_the_top_of_the_range(cuda_lib, top, Hq, d, wide):
    # Steps of V up to 2^117: at a unit's end the sums of codes go back to units of V by way of factors past fp32's range.
    lens = [12, 1, 30]
    g = torch.Generator().manual_seed(top)
    k = torch.randn((sum(lens), 2, d), generator=g).to(BF).to(DEV)
    v = (torch.randn((sum(lens), 2, d), generator=g) * 2.0 ** top).to(BF).to(DEV)
    cache, table, ln, _, _ = filled(lens, 2, 16, d, BF, seed=8, rows=[k, v])
    q = torch.randn((3, Hq, d), generator=g).to(BF).to(DEV)
    o, lse = fa.paged4_decode(q, cache, widened(table, wide), ln)
    ok()
    assert o.isfinite().all()
    assert_decoded(o, lse, q, k, v, lens, d ** -0.5, 0, f"values of 2^{top}")


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("Hq", [4, 16, 32])
@pytest.mark.parametrize("scale", [1e-20, 1e-30, 0.125])
@pytest.mark.parametrize("dt", [BF, HF])
def test_queries_of_zero_and_tiny_scales(cuda_lib, dt, scale, Hq, wide):
    # Weights all alike, beside keys that are masked: o is the mean of the values.
    lens = [70, 1, 33]
    cache, table, ln, k, v = filled(lens, 2, 16, 64, dt, seed=10)
    q = torch.zeros((3, Hq, 64), dtype=dt, device=DEV)
    o, lse = fa.paged4_decode(q, cache, widened(table, wide), ln, scale=scale)
    ok()
    assert_decoded(o, lse, q, k, v, lens, scale, 0)


def outlier(dt, d, Hq, Hkv, n, at, times, seed):
    """A sequence whose key `at` nobody attends to (its score is 200 below the others') and whose value is `times` larger."""
    g = torch.Generator().manual_seed(seed)
    u = torch.randint(0, 2, (d,), generator=g).float() * 2 - 1
    k = 0.01 * torch.randn((n, Hkv, d), generator=g)
    v = torch.randn((n, Hkv, d), generator=g)
    k[at] = -200.0 / math.sqrt(d) * u
    v[at] *= times
    q = u + 0.1 * torch.randn((1, Hq, d), generator=g)
    return [t.to(dt).to(DEV) for t in (q, k, v)]


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("Hq", [4, 16, 32])
@pytest.mark.parametrize("dt,times", [(BF, 2.0 ** 8), (BF, 2.0 ** 14), (BF, 2.0 ** 22), (BF, 2.0 ** 115), (HF, 2.0 ** 8), (HF, 2.0 ** 13)])
@pytest.mark.parametrize("at", [0, 70])
def test_a_key_of_large_steps_that_nobody_attends_to(cuda_lib, at, dt, times, Hq, wide):
    # Weights times steps are held to 2^-22 of themselves or 2^-31 S, S the largest visible step: those of the other keys
    # lose that much and no more, min(p s, 2^-31 S) each, times 7.5 at most.
    d, n, Hkv = 128, 100, 2
    q, k, v = outlier(dt, d, Hq, Hkv, n, at, times, seed=int(math.log2(times)) + at)
    cache, table, ln, _, _ = filled([n], Hkv, 16, d, dt, seed=9, rows=[k, v])
    o, lse = fa.paged4_decode(q, cache, widened(table, wide), ln)
    ok()
    r = rounder(dt)
    kn, vn = (f64(t).swapaxes(0, 1) for t in (k, v))
    want, _, _, a = paged4.decode(f64(q)[0], kn, vn, d ** -0.5, 0, r)
    others = np.delete(kn, at, axis=1)
    x = paged4.decode(f64(q)[0], others, others, d ** -0.5, 0, r)[2]    # the bound of their scores
    s = np.repeat(paged4.quantise(vn, r)[1], 64, -1)                   # [Hkv, n, d]
    kv, G = paged4.values(kn, r), Hq // Hkv
    e = (x * (d + 8) * 2.0 ** -23 + 2.0 ** -21 + n * 2.0 ** -24)[:, None]
    lost = np.zeros_like(want)
    for h in range(Hq):
        y = d ** -0.5 * (kv[h // G] @ f64(q)[0, h])
        p = np.exp(y - y.max())
        p /= p.sum()
        lost[h] = 7.5 * np.minimum(p[:, None] * s[h // G], 2.0 ** -31 * s[h // G].max(0)).sum(0)
    bound = U[dt] * np.abs(want) + (2.1 * e + 2.0 ** -22 * 7.5 / 32 + (d + n) * 2.0 ** -23) * a + lost + TINY[dt]
    err = np.abs(f64(o)[0] - want)
    assert (err <= bound).all(), f"{(err > bound).sum()} values, {(err / np.maximum(bound, 1e-30)).max()} of the bound"
    assert lse.isfinite().all()


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("Hq,Hkv,d,sections,interleaved", [(8, 2, 128, (64,), False), (12, 4, 64, (32,), False), (8, 1, 128, (16, 16), False),
                                                           (16, 8, 128, (64,), True), (5, 5, 64, None, False)])
def test_rows_do_not_depend_on_how_many_are_appended_with_them(cuda_lib, Hq, Hkv, d, sections, interleaved, dt):
    # One token a call, a few, and all in one: q and the pool's bytes are the same.
    n = 6000
    g = torch.Generator().manual_seed(d + Hq)
    q, k, v = torch.randn((n, Hq + 2 * Hkv, d), generator=g).to(dt).to(DEV).split([Hq, Hkv, Hkv], dim=1)
    rot, kw = turned(g, sections, interleaved, 100, 1, n)
    pos = None if rot is None else rot[0][:, 0]
    norm = dict(q_weight=weights(g, d, F32), k_weight=weights(g, d, F32), eps=1e-6)
    total, table, ln = tables([n], 16, seed=12)
    whole, parts = new_cache(total, Hkv, 16, d, fill=0), new_cache(total, Hkv, 16, d, fill=0)

    def append(cache, at, end):
        ln.fill_(end)
        turn = {} if rot is None else dict(kw, positions=pos[:, at:end])
        return fa.paged4_append(cache, table, ln, k[at:end], v[at:end], cu_seqlens=offsets([end - at]), q=q[at:end], **norm, **turn)
    want = append(whole, 0, n)
    got, at = [], 0
    for c in [1] * 40 + [3, 17, 64, 100, 400, 1500, n]:
        end = min(at + c, n)
        got.append(append(parts, at, end))
        at = end
    ok()
    got = torch.cat(got)
    assert torch.equal(got, want), f"{(got != want).sum().item()} values of q"
    assert torch.equal(parts, whole)


def elementary_rows(x, w, eps, pos, freq, axes, interleaved):
    """Rows x [T, H, d] normed and turned by elementary fp32 operations, each rounded as it is: squares of elements 32
    columns apart are added first, then neighbours; angles are formed in 64 bits and their sines and cosines rounded."""
    dt, d = x.dtype, x.shape[-1]
    y = x.float()
    if eps is not None:
        p = y * y
        s = p[..., :32] + p[..., 32:64]
        for i in range(64, d, 32):
            s = s + p[..., i:i + 32]
        while s.shape[-1] > 1:
            s = s[..., 0::2] + s[..., 1::2]
        y = y * torch.rsqrt(s / d + eps)
        if w is not None:
            y = y * w.float()
    if pos is not None:
        rot = 2 * freq.numel()
        angle = (pos[axes.long()].double().movedim(0, -1) * freq)[:, None]
        c, s = angle.cos().float(), angle.sin().float()
        a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:rot])
        u, v = a * c - b * s, b * c + a * s
        head = torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)
        y = torch.cat([head, y[..., rot:]], -1)
    return y.to(dt)


def held(x):
    """What the cache holds for 16-bit rows x [T, H, d], in x's type."""
    y = x.float().unflatten(-1, (-1, 64))
    lo, hi = y.amin(-1, keepdim=True), y.amax(-1, keepdim=True)
    s = ((hi - lo) / 15.0).to(x.dtype).float()
    c = torch.where(s == 0, 0.0, ((y - lo) / s).round().clamp(0, 15))
    return (lo.double() + s.double() * c.double()).float().to(x.dtype).flatten(-2)


@pytest.mark.parametrize("d,sections,interleaved", [(128, None, False), (128, (64,), False), (128, (64,), True), (128, (32,), False),
                                                    (128, (16, 24), False), (128, (16,), True), (64, (32,), False), (64, (32,), True),
                                                    (64, (8, 8), False)])
def test_rows_of_k_are_those_of_elementary_operations(cuda_lib, d, sections, interleaved):
    # A last place of a 16-bit value can move a code by a whole step, and a row's sum that is off by a last place shows as
    # often.  What remains is the angles, within 2^-29.5: a value of fp16 moves by a last place, 2^-11 of itself at least, in
    # 2^-17.5 of the cases (their error is 2^-28.5 (|a| + |b|) wide), and shows where it is its group's smallest or largest or
    # a code's border is in that place (3e-3 of the others): 2.2 values of 64.  2^20 groups, so 13 are expected at most; 24
    # are three deviations more.  A sum off by 2^-24 in half of the rows would show in some 90.
    T, H = 2 ** 22 // d, 16
    g = torch.Generator().manual_seed(d + len(sections or ()))
    k = torch.randn((T, H, d), generator=g).to(HF).to(DEV)
    w = weights(g, d, F32)
    rot, kw = turned(g, sections, interleaved, 0, 1, T)
    pos = None
    if rot is not None:
        pos = kw["positions"] = rot[0][:, 0].contiguous()
    total, table, ln = tables([T], 64, seed=13)
    cache = new_cache(total, H, 64, d)
    fa.paged4_append(cache, table, ln, k, k, cu_seqlens=offsets([T]), k_weight=w, eps=1e-6, **kw)
    got, raw = fa.paged4_read(cache, table, ln, T, HF)
    want = held(elementary_rows(k, w, 1e-6, pos, kw.get("inv_freq"), kw.get("axes"), interleaved)).transpose(0, 1)[None]
    ok()
    assert torch.equal(raw, held(k).transpose(0, 1)[None])
    off = (got != want).unflatten(-1, (-1, 64)).any(-1)
    assert off.sum().item() <= 24, f"{off.sum().item()} of {off.numel()} groups"


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("Hq,Hkv,d,sections,interleaved", [(8, 2, 128, (64,), False), (8, 2, 128, (16, 16), True), (6, 2, 64, (32,), False),
                                                           (32, 2, 128, (64,), False)])
def test_serving_run_step_by_step(cuda_lib, Hq, Hkv, d, sections, interleaved, dt):
    # Prompts, then steps of one token: what the cache holds and the attention over it, compared at every step.  (Of some
    # 30000 values of K, those that the angles' last places move, 1e-6 of them: none.)
    lens = [70, 0, 33]
    g = torch.Generator().manual_seed(71)
    total, table, _ = tables([n + 8 for n in lens], 16, seed=72)
    cache = new_cache(total, Hkv, 16, d)
    wq, wk = weights(g, d, dt), weights(g, d, dt)
    freq, axes = fa.rope_frequencies(sections, device=DEV)
    turn = dict(inv_freq=freq, axes=axes, interleaved=interleaved)
    rows = [[[], []] for _ in lens]
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    for step in range(8):
        counts = [1, 1, 1] if step else list(lens)
        if step:
            lens = [n + 1 for n in lens]
        ln.copy_(torch.tensor(lens, dtype=torch.int32))
        q, k, v = torch.randn((sum(counts), Hq + 2 * Hkv, d), generator=g).to(dt).to(DEV).split([Hq, Hkv, Hkv], dim=1)
        one = torch.tensor([n - c + i for n, c in zip(lens, counts) for i in range(c)], dtype=torch.int32, device=DEV)
        pos = torch.stack([one + 5 * i for i in range(len(sections))])
        qn = fa.paged4_append(cache, table, ln, k, v, cu_seqlens=None if step else offsets(counts), q=q, q_weight=wq, k_weight=wk,
                              eps=1e-6, positions=pos, **turn)
        kn, at = elementary_rows(k, wk, 1e-6, pos, freq, axes, interleaved), 0
        for b, c in enumerate(counts):
            rows[b][0].append(kn[at:at + c])
            rows[b][1].append(v[at:at + c])
            at += c
        ok()
        assert_normed(qn.transpose(0, 1)[None], q.transpose(0, 1)[None], wq, 1e-6, (pos[:, None], freq, axes, interleaved), "q")
        kall, vall = (torch.cat([t for r in rows for t in r[i]]) for i in range(2))
        got = fa.paged4_read(cache, table, ln, max(lens), dt)
        assert_read(got[0], last_rows(kall, lens, max(lens), dt), dt, "k")
        assert_read(got[1], last_rows(vall, lens, max(lens), dt), dt, "v")
        if step:
            window = 0 if step % 2 else 50
            o, lse = fa.paged4_decode(qn, cache, table, ln, window=window)
            ok()
            assert_decoded(o, lse, qn, kall, vall, lens, d ** -0.5, window, f"step {step}")


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("Hq,Hkv", [(4, 1), (8, 1), (32, 2), (20, 1)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_query_that_is_not_finite_spoils_its_head_alone(cuda_lib, bad, Hq, Hkv, wide):
    lens = [300, 0, 41]
    cache, table, ln, k, v = filled(lens, Hkv, 16, 128, BF, seed=14)
    table = widened(table, wide)
    q = torch.randn((3, Hq, 128), generator=torch.Generator().manual_seed(15)).to(BF).to(DEV)
    want, wl = fa.paged4_decode(q, cache, table, ln)
    spoilt = q.clone()
    spoilt[0, Hq - 1, 77] = bad
    spoilt[1, 0] = bad                                              # of a sequence without keys
    got, gl = fa.paged4_decode(spoilt, cache, table, ln)
    ok()
    assert not got[0, Hq - 1].isfinite().any()
    assert torch.equal(got[0, :Hq - 1], want[0, :Hq - 1]) and torch.equal(got[1:], want[1:])
    assert torch.equal(gl[0, :Hq - 1], wl[0, :Hq - 1]) and torch.equal(gl[1:], wl[1:])


@pytest.mark.parametrize("dt", [BF, HF])
def test_inputs_that_are_broadcast(cuda_lib, dt):
    # One row for many heads, tokens or sequences (stride 0) gives what its copies give, gradients too.
    d, g = 128, torch.Generator().manual_seed(16)
    x = torch.randn((1, 1, 37, d), generator=g).to(dt).to(DEV)
    dy = torch.randn((3, 1, 1, d), generator=g).to(dt).to(DEV)
    w = weights(g, d, F32)
    freq, axes = fa.rope_frequencies((64,), device=DEV)
    pos = torch.arange(37, dtype=torch.int32, device=DEV).expand(1, 3, 37)
    q, k, dq, dk = x.expand(3, 8, 37, d), x.expand(3, 2, 37, d), dy.expand(3, 8, 37, d), dy.expand(3, 2, 37, d)
    for a, b in ((q, q.contiguous()), (k, k.contiguous())):
        assert torch.equal(fa.qk_norm_rope(a, None, w, None, pos, freq, axes), fa.qk_norm_rope(b, None, w, None, pos, freq, axes))
    got = fa.qk_norm_rope_backward(dq, dk, q, k, w, w, pos, freq, axes)
    want = fa.qk_norm_rope_backward(dq.contiguous(), dk.contiguous(), q.contiguous(), k.contiguous(), w, w, pos.contiguous(), freq, axes)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    total, table, ln = tables([40, 37], 16, seed=17)
    one, all_ = (new_cache(total, 2, 16, d, fill=0) for _ in range(2))
    rows = x[0, 0, :1].expand(40, 2, d)
    cu = offsets([3, 37])
    qs = x[0, :, :1].expand(40, 8, d)
    turn = dict(positions=torch.arange(40, dtype=torch.int32, device=DEV)[None], inv_freq=freq, axes=axes)
    a = fa.paged4_append(one, table, ln, rows, rows, cu_seqlens=cu, q=qs, k_weight=w, eps=1e-6, **turn)
    b = fa.paged4_append(all_, table, ln, rows.contiguous(), rows.contiguous(), cu_seqlens=cu, q=qs.contiguous(), k_weight=w, eps=1e-6, **turn)
    assert torch.equal(a, b) and torch.equal(one, all_)
    query = x[0, :, :1].expand(2, 8, d)
    ln.copy_(torch.tensor([3, 37], dtype=torch.int32))
    assert all(torch.equal(s, t) for s, t in zip(fa.paged4_decode(query, one, table, ln), fa.paged4_decode(query.contiguous(), one, table, ln)))
    with pytest.raises(fa.FAError):
        fa.qk_norm_rope_backward(dq, None, q, None, w, None, pos, freq, axes, dq_out=dq)       # rows that many would write
    ok()


def test_norm_without_eps_and_with_a_whole_number(cuda_lib):
    # eps = 0 (a row of zeros is then 0 times infinity) and numbers that are no floats, by the Python marshalling.
    x = torch.randn((1, 2, 9, 64), generator=torch.Generator().manual_seed(18)).to(HF).to(DEV)
    x[0, 0, 3] = 0
    y = fa.qk_norm_rope(x, None, None, None, eps=0)
    z = fa.qk_norm_rope(x, None, None, None, eps=0.0)
    ok()
    assert torch.equal(y.nan_to_num(7.0), z.nan_to_num(7.0))
    assert y[0, 0, 3].isnan().all() and y[0, 1].isfinite().all()
    rest = [i for i in range(9) if i != 3]
    assert_normed(y[:, :, rest], x[:, :, rest], None, 0.0, None, "eps 0")


def test_two_calls_on_two_streams_share_a_pool(cuda_lib):
    # Two streams append to different sequences of one pool and read them, again and again; then the pool is as if one had.
    lens, d, n = [500, 500], 128, 500
    g = torch.Generator().manual_seed(19)
    total, table, _ = tables(lens, 16, seed=20)
    rows = [torch.randn((n, 2, d), generator=g).to(BF).to(DEV) for _ in range(2)]
    alone, both = (new_cache(total, 2, 16, d, fill=0) for _ in range(2))
    lengths = torch.arange(n + 1, dtype=torch.int32, device=DEV)
    for b in range(2):
        fa.paged4_append(alone, table[b:b + 1], lengths[n:], rows[b], rows[b], cu_seqlens=offsets([n]))
    q = torch.randn((1, 8, d), generator=g).to(BF).to(DEV)
    want = [fa.paged4_decode(q, alone, table[b:b + 1], lengths[n:]) for b in range(2)]
    ok()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    cu = offsets([1])
    for at in range(n):
        for b in range(2):
            fa.paged4_append(both, table[b:b + 1], lengths[at + 1:at + 2], rows[b][at:at + 1], rows[b][at:at + 1], cu_seqlens=cu,
                             stream=streams[b])
            got[b] = fa.paged4_decode(q, both, table[b:b + 1], lengths[at + 1:at + 2], stream=streams[b])
    ok()
    assert torch.equal(both, alone)
    for b in range(2):
        assert all(torch.equal(x, y) for x, y in zip(got[b], want[b]))


def test_groups_wider_than_fp32_read_as_nan(cuda_lib):
    # 3e38 and -3e38 are bf16 numbers, their difference is no fp32 one; half as far apart they are held.
    x = torch.randn((3, 1, 64), generator=torch.Generator().manual_seed(21))
    x[1, 0, 5], x[1, 0, 60] = 3e38, -3e38
    x[2, 0, 5], x[2, 0, 60] = 1.5e38, -1.5e38
    x = x.to(BF).to(DEV)
    total, table, ln = tables([3], 16, seed=22)
    cache = new_cache(total, 1, 16, 64)
    fa.paged4_append(cache, table, ln, x, x, cu_seqlens=offsets([3]))
    for got in fa.paged4_read(cache, table, ln, 3, BF):
        assert got[0, 0, 1].isnan().all()
        assert_read(got[:, :, [0, 2]], last_rows(x[[0, 2]], [2], 2, BF), BF)
    ok()

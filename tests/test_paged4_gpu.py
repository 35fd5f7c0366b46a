"""GPU parity of the normed rotary positions and of the 4-bit cache (append,
read back, one-token attention) against the fp64 oracle, through the Python
binding.

Tolerances (u = half a step of the tensors' type: bf16 2^-8, fp16 2^-11).

Norm and rotation: the sum of d squares is off by d 2^-24 of itself at most,
its inverse root by half of that, the root's own 2^-22 and the division's
2^-24; two products round by 2^-23: y = x r w is off by N = (d / 2 + 8) 2^-24 of
itself.  The rotation adds 2e-6 (|a| + |b|) of the pair's normed values (see
test_paged_gpu: there with sines off by 4.2e-7, here they are finer), and the
rounding u |ref|.

Its gradient: dx = r (g w - x r m), m = mean(g w x r).  g is off by 2e-6 of its
pair's |a| + |b| =: G, r by N; m, a sum of d products, by (2 N + d 2^-24) M + 2e-6
mean(G |w x r|) with M = mean |g w x r|; so dx by r [2e-6 G |w| + |x r| 2e-6 mean(G
|w x r|) + 4 N (|g w| + |x r| M)], and the rounding.  dw, a sum over R rows, by sum
[2e-6 G + 2 N |g|] |x r| + R 2^-24 sum |g x r|.

4 bits: without norm and rotation the codes are those of the oracle (its
quotients tie exactly where the kernel's do); the value z + s c, rounded to
fp32 and to the type, is off by u + 2^-23 of itself.  With them the 16-bit row is
off by e (above), its group's ends too, and so the value is within s / 2 + 15 u s
(s rounded, codes cut at 15) of the row's, s <= ((range + 2 e) / 15)(1 + u).

Attention: products of q with z + s c are formed as s times sums of q c, and z
times sums of q, each in fp32: the parts are bounded by |q| (|z| + 32 s), and X =
scale sum |q| (|z| + 32 s); a score is off by X (d + 8) 2^-23 (adders may truncate: a
factor 2), its exponential by 2^-22, sums over n keys by n 2^-24 together e; lse is
off by e.  (q enters in fp16 times a power of two of its head, which brings the
largest element Q to 2^10: one of fp16's subnormal steps is 2^-34 Q, so a score is off
by scale 15 s d 2^-35 Q at most, 2^-36 d X, which the 8 above holds.)  The weights s p
enter as fp16 values W off by 2^-11 of themselves (bf16; half a step of ten bits) or,
two values, by 2^-22 (fp16), or by half a subnormal step, 2^-25, where the group's
largest s so far counts 2^6 at least: 2^-31 S; each times |c - 7.5| <= 7.5.  The sum of the p that
these are relative to is 1 at least, so with A = sum p (|z| + 32 s) >= 32 sum p s and S
the group's largest visible s, o is off by (2.1 e + W 7.5 / 32 + (d + n) 2^-23) A + n
2^-28 S and its rounding.
"""
import math
import threading

import numpy as np
import pytest
import torch

import exact_io_aware_flashattention_gb300 as fa
from oracle import paged, paged4, ref
from tests.parity import GRAD_REL_L2, GuardedBuffers, assert_fwd, rel_l2

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
WEIGHT = {torch.bfloat16: 2.0 ** -11, torch.float16: 2.0 ** -22}          # the decode kernel's weights
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -24}       # fp16's subnormal step
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def f64(t):
    return t.detach().double().cpu().numpy()


def ok():
    torch.cuda.synchronize()
    fa.check_device_status()


def rounder(dt):
    return lambda x: torch.from_numpy(np.asarray(x, dtype=np.float64)).to(dt).double().numpy()


def rotary_of(rot):
    """(positions, inv_freq, axes, interleaved) as numpy, or None."""
    return None if rot is None else (rot[0].cpu().numpy(), rot[1].cpu().numpy(), rot[2].cpu().numpy(), rot[3])


def pair_sums(x, rot):
    """|a| + |b| of the pair that each element belongs to, 0 where nothing is turned."""
    out = np.zeros_like(x)
    if rot is None:
        return out
    r, a = len(rot[1]), np.abs(x)
    lo, hi = (np.arange(0, 2 * r, 2), np.arange(1, 2 * r, 2)) if rot[3] else (np.arange(r), np.arange(r, 2 * r))
    out[..., lo] = out[..., hi] = a[..., lo] + a[..., hi]
    return out


def norm_error(x, w, eps, rot):
    """(the normed and turned rows, a bound of their error before rounding)."""
    y = paged4.norm(x, w, eps)
    n = (x.shape[-1] / 2 + 8) * 2.0 ** -24
    e = (2e-6 + n) * pair_sums(y, rot) + n * np.abs(y)
    return y if rot is None else paged.rotate(y, *rot), e


def assert_normed(out, x, w, eps, rot, what):
    want, e = norm_error(f64(x), None if w is None else f64(w), eps, rotary_of(rot))
    err = np.abs(f64(out) - want)
    bound = U[out.dtype] * np.abs(want) + 1.01 * e + TINY[out.dtype]
    assert (err <= bound).all(), f"{what}: {(err > bound).sum()} values, {(err / np.maximum(bound, 1e-30)).max()} of the bound"


def weights(g, d, dt):
    return None if dt is None else (1 + 0.3 * torch.randn((d,), generator=g)).to(dt).to(DEV)


def turned(g, sections, interleaved, start, B, N):
    if sections is None:
        return None, {}
    pos = (start + torch.randint(0, 60, (len(sections), B, N), generator=g)).to(torch.int32).to(DEV)
    w, axes = fa.rope_frequencies(sections, device=DEV)
    return (pos, w, axes, interleaved), dict(positions=pos, inv_freq=w, axes=axes, interleaved=interleaved)


@pytest.fixture(params=["native", "python"])
def marshalling(request, monkeypatch, cuda_lib):
    if request.param == "native":
        assert fa.native_marshalling()
    else:
        monkeypatch.setattr(fa, "_native", fa._NotBuilt)
    return request.param


# ---------------------------------------------------------------------------
# Norm and rotation
# ---------------------------------------------------------------------------
NORM = [
    # B, Hq, Hk, N, d, sections (None: no rotation), interleaved, first position, dtype, weights' dtype (None: ones)
    (1, 1, 0, 1, 64, (32,), False, 0, BF, BF),
    (2, 4, 2, 33, 128, (16, 24, 24), False, 0, BF, BF),
    (1, 3, 1, 257, 128, (20, 12), True, 5, HF, F32),
    (3, 5, 5, 7, 64, (8,), False, 10 ** 6, HF, HF),
    (1, 2, 1, 40, 64, (8, 0, 8), True, 2 ** 31 - 100, BF, F32),
    (1, 2, 2, 65, 256, (64, 64), False, -30, BF, None),
    (2, 9, 3, 19, 16, (8,), False, 3, HF, F32),
    (1, 32, 8, 300, 80, (40,), False, 3, BF, BF),             # d not a power of two
    (1, 6, 6, 50, 96, (16,), True, 77, BF, F32),
    (2, 3, 1, 21, 48, None, False, 0, HF, HF),                # the norm alone
    (1, 8, 8, 130, 128, None, False, 0, BF, None),
    (1, 20000, 3, 5, 16, (8,), False, 0, BF, F32),            # more heads than blocks for eight each
    (1, 3000, 1000, 9, 32, (16,), True, 4, HF, F32),
    (2, 1, 700, 3, 64, (32,), False, 0, BF, BF),
    (1, 40, 1, 1000, 128, (64,), False, 0, BF, F32),          # k's few rows and many angles
    (1, 1, 1, 1, 112, (56,), False, 9, BF, BF),
    (4, 32, 32, 1, 128, (64,), False, 4000, BF, BF),          # one token a sequence
    (1, 40, 8, 5000, 64, (32,), False, 0, HF, F32),           # several items a block
]


@pytest.mark.parametrize("B,Hq,Hk,N,d,sections,interleaved,start,dt,wdt", NORM)
def test_norm(cuda_lib, B, Hq, Hk, N, d, sections, interleaved, start, dt, wdt):
    g = torch.Generator().manual_seed(N * d + Hq)
    q = (2.0 * torch.randn((B, Hq, N, d), generator=g)).to(dt).to(DEV)
    k = (0.1 * torch.randn((B, Hk, N, d), generator=g)).to(dt).to(DEV) if Hk else None
    wq, wk = weights(g, d, wdt), weights(g, d, wdt) if Hk else None
    rot, kw = turned(g, sections, interleaved, start, B, N)
    gb = GuardedBuffers(DEV)
    qo = gb.empty((B, Hq, N, d), dt)
    if k is None:
        assert fa.qk_norm_rope(q, None, wq, None, eps=1e-5, q_out=qo, **kw) is qo
    else:
        ko = gb.empty((B, Hk, N, d), dt)
        fa.qk_norm_rope(q, k, wq, wk, eps=1e-5, q_out=qo, k_out=ko, **kw)
    ok()
    gb.check()
    assert_normed(qo, q, wq, 1e-5, rot, "q")
    if k is not None:
        assert_normed(ko, k, wk, 1e-5, rot, "k")


def assert_norm_gradient(dx, dw, dy, x, w, eps, rot, what):
    xn, gn, wn = f64(x), f64(dy), None if w is None else f64(w)
    rn = rotary_of(rot)
    want, want_w = paged4.norm_rope_backward(gn, xn, wn, eps, rn)
    d, R = xn.shape[-1], xn.size // xn.shape[-1]
    n = (d / 2 + 8) * 2.0 ** -24
    one = np.ones(d) if wn is None else np.abs(wn)
    gt = np.abs(gn if rn is None else paged.rotate(gn, *rn, inverse=True))
    G = pair_sums(gn, rn)
    r = 1.0 / np.sqrt((xn * xn).mean(-1, keepdims=True) + eps)
    xr = np.abs(xn) * r
    M = (gt * one * xr).mean(-1, keepdims=True)
    e = r * (2e-6 * G * one + xr * 2e-6 * (G * one * xr).mean(-1, keepdims=True) + (4 * n + d * 2.0 ** -24) * (gt * one + xr * M))
    bound = U[dx.dtype] * np.abs(want) + 1.01 * e + TINY[dx.dtype]
    err = np.abs(f64(dx) - want)
    assert (err <= bound).all(), f"{what}: {(err > bound).sum()} values, {(err / np.maximum(bound, 1e-30)).max()} of the bound"
    if dw is not None:
        bound = ((2e-6 * G + 2 * n * gt) * xr).reshape(-1, d).sum(0) + R * 2.0 ** -24 * (gt * xr).reshape(-1, d).sum(0)
        err = np.abs(f64(dw) - want_w)
        assert (err <= bound).all(), f"{what} weights: {(err / bound).max()} of the bound"


@pytest.mark.parametrize("B,Hq,Hk,N,d,sections,interleaved,start,dt,wdt", NORM)
def test_norm_gradient(cuda_lib, B, Hq, Hk, N, d, sections, interleaved, start, dt, wdt):
    g = torch.Generator().manual_seed(N * d + Hq + 1)
    q, dq = ((s * torch.randn((B, Hq, N, d), generator=g)).to(dt).to(DEV) for s in (2.0, 1.0))
    k, dk = ((s * torch.randn((B, Hk, N, d), generator=g)).to(dt).to(DEV) if Hk else None for s in (0.3, 1.0))
    wq, wk = weights(g, d, wdt), weights(g, d, wdt) if Hk else None
    rot, kw = turned(g, sections, interleaved, start, B, N)
    gb = GuardedBuffers(DEV)
    out = dict(dq_out=gb.empty((B, Hq, N, d), dt))
    if Hk:
        out["dk_out"] = gb.empty((B, Hk, N, d), dt)
    if wdt is not None:
        out["dq_weight"] = gb.empty((d,), F32)
        if Hk:
            out["dk_weight"] = gb.empty((d,), F32)
        out["workspace"] = gb.empty((fa.qk_norm_rope_backward_workspace(d).numel(),), torch.uint8)
    r = fa.qk_norm_rope_backward(dq, dk, q, k, wq, wk, eps=1e-5, **out, **kw)
    ok()
    gb.check()
    assert len(r) == (4 if Hk else 2) and r[0] is out["dq_out"]
    assert_norm_gradient(r[0], r[2 if Hk else 1], dq, q, wq, 1e-5, rot, "q")
    if Hk:
        assert_norm_gradient(r[1], r[3], dk, k, wk, 1e-5, rot, "k")


@pytest.mark.parametrize("layout", ["token-major", "head-major"])
def test_norm_in_place_on_a_projection(cuda_lib, layout):
    B, Hq, Hk, N, d = 2, 4, 2, 37, 64
    g = torch.Generator().manual_seed(3)
    x, y = (torch.randn((B, Hq + 2 * Hk, N, d), generator=g).to(BF).to(DEV) for _ in range(2))
    if layout == "token-major":
        x, y = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (x, y))      # [B, N, H, d] in memory
    before, after = x.clone(), y.clone()
    wq, wk = weights(g, d, F32), weights(g, d, F32)
    rot, kw = turned(g, (32,), False, 0, B, N)
    (q, k, v), (dq, dk, dv) = (t.split([Hq, Hk, Hk], dim=1) for t in (x, y))
    (q0, k0, v0), (dq0, dk0, dv0) = (t.split([Hq, Hk, Hk], dim=1) for t in (before, after))
    _, _, dwq, dwk = fa.qk_norm_rope_backward(dq, dk, q, k, wq, wk, dq_out=dq, dk_out=dk, **kw)
    fa.qk_norm_rope(q, k, wq, wk, q_out=q, k_out=k, **kw)
    ok()
    assert_normed(q, q0, wq, 1e-6, rot, "q")
    assert_normed(k, k0, wk, 1e-6, rot, "k")
    assert_norm_gradient(dq, dwq, dq0, q0, wq, 1e-6, rot, "dq")
    assert_norm_gradient(dk, dwk, dk0, k0, wk, 1e-6, rot, "dk")
    assert torch.equal(v, v0) and torch.equal(dv, dv0)


def test_norm_of_odd_rows(cuda_lib):
    # Rows of zeros, of one huge element, and rows with NaN or infinities, which stay theirs.
    x = torch.randn((1, 1, 6, 128), generator=torch.Generator().manual_seed(5)).to(BF).to(DEV)
    x[0, 0, 1] = 0
    x[0, 0, 2, 7] = 1e10
    x[0, 0, 3, 100] = float("nan")
    x[0, 0, 4, 0] = float("inf")
    y = fa.qk_norm_rope(x, None, None, None)
    dx, dw = fa.qk_norm_rope_backward(torch.ones_like(x), None, x, None, torch.ones(128, device=DEV), None)
    ok()
    fine = [0, 1, 2, 5]
    assert_normed(y[:, :, fine], x[:, :, fine], None, 1e-6, None, "fine rows")
    assert not y[0, 0, 1].any()
    assert y[0, 0, 3].isnan().all() and dx[0, 0, 3].isnan().all()
    assert y[0, 0, 4, 0].isnan() and not y[0, 0, 4, 1:].any()
    assert_norm_gradient(dx[:, :, fine], None, torch.ones_like(x)[:, :, fine], x[:, :, fine], None, 1e-6, None, "fine rows")
    assert dw.isnan().any()


def test_norm_gradient_is_reproducible_and_takes_what_is_asked(cuda_lib):
    g = torch.Generator().manual_seed(8)
    q, dq = (torch.randn((2, 8, 777, 128), generator=g).to(BF).to(DEV) for _ in range(2))
    k, dk = (torch.randn((2, 2, 777, 128), generator=g).to(BF).to(DEV) for _ in range(2))
    wq, wk = weights(g, 128, BF), weights(g, 128, BF)
    _, kw = turned(g, (64,), False, 0, 2, 777)
    first = fa.qk_norm_rope_backward(dq, dk, q, k, wq, wk, **kw)
    again = fa.qk_norm_rope_backward(dq, dk, q, k, wq, wk, **kw)
    some = fa.qk_norm_rope_backward(dq, dk, q, k, wq, None, **kw)
    ok()
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    assert some[3] is None and torch.equal(some[0], first[0]) and torch.equal(some[2], first[2])
    none = fa.qk_norm_rope_backward(dq, None, q, None, None, None, **kw)
    ok()
    assert none[1] is None and len(none) == 2


@pytest.mark.parametrize("deterministic", [False, True])
def test_norm_in_a_training_step(cuda_lib, deterministic):
    # norm and rotation, attention, its backward, and back: gradients of the
    # inputs and weights against the oracle from the same normed tensors.
    B, Hq, Hk, N, d = 1, 4, 2, 300, 64
    g = torch.Generator().manual_seed(11)
    q, k, v, do = (torch.randn((B, h, N, d), generator=g).to(BF).to(DEV) for h in (Hq, Hk, Hk, Hq))
    wq, wk = weights(g, d, F32), weights(g, d, F32)
    rot, kw = turned(g, (8, 12, 12), False, 0, B, N)
    qr, kr = fa.qk_norm_rope(q, k, wq, wk, **kw)
    o, lse = fa.forward(qr, kr, v, causal=True)
    dqr, dkr, dv = fa.backward(qr, kr, v, o, lse, do, causal=True, deterministic=deterministic)
    dq, dk, dwq, dwk = fa.qk_norm_rope_backward(dqr, dkr, q, k, wq, wk, **kw)
    ok()
    rq, rk, _ = ref.attention_backward(f64(qr), f64(kr), f64(v), f64(do), True, d ** -0.5)
    rn = rotary_of(rot)
    for got, dw, dy, x, w, name in ((dq, dwq, rq, q, wq, "q"), (dk, dwk, rk, k, wk, "k")):
        want, want_w = paged4.norm_rope_backward(dy, f64(x), f64(w), 1e-6, rn)
        # dx is dy through a linear map per row of norm at most r max w; the attention's relative error passes it.
        r = 1.0 / np.sqrt((f64(x) ** 2).mean(-1, keepdims=True) + 1e-6)
        grow = (r.max() * np.abs(f64(w)).max()) * np.linalg.norm(dy) / np.linalg.norm(want)
        assert rel_l2(f64(got), want) <= GRAD_REL_L2 * grow + 2 * U[BF], name
        size = np.sqrt(((dy ** 2).sum() * ((f64(x) * r) ** 2).max()))
        assert np.abs(f64(dw) - want_w).max() <= (GRAD_REL_L2 + U[BF]) * size * math.sqrt(dy.size // d), name


def test_norm_bad_axis_is_recorded(cuda_lib):
    q = torch.randn((1, 1, 4, 64), device=DEV).to(BF)
    w, axes = fa.rope_frequencies((32,), device=DEV)
    axes[5] = 1
    fa.qk_norm_rope(q, None, None, None, torch.zeros((1, 1, 4), dtype=torch.int32, device=DEV), w, axes)
    assert fa.fa_last_device_status()[0] == fa.FA_ERR_BAD_INDEX
    ok()


def test_norm_offsets_past_32_bits(cuda_lib):
    N, d = 2 ** 24 + 40, 128                    # 2^31 elements and a few rows
    x = torch.zeros((1, 1, N, d), dtype=BF, device=DEV)
    x[:, :, :64].normal_()
    x[:, :, -64:].normal_()
    head, tail = x[:, :, :64].clone(), x[:, :, -64:].clone()
    pos = torch.arange(N, dtype=torch.int32, device=DEV).view(1, 1, N)
    w, axes = fa.rope_frequencies((64,), device=DEV)
    wt = weights(torch.Generator().manual_seed(1), d, F32)
    kw = dict(inv_freq=w, axes=axes)
    dy = torch.zeros_like(x)
    dy[:, :, :64].normal_()
    dy[:, :, -64:].normal_()
    h2, t2 = dy[:, :, :64].clone(), dy[:, :, -64:].clone()
    _, dw = fa.qk_norm_rope_backward(dy, None, x, None, wt, None, pos, dq_out=dy, **kw)
    fa.qk_norm_rope(x, None, wt, None, pos, q_out=x, **kw)
    ok()
    for at, x0, y0, what in ((slice(0, 64), head, h2, "first rows"), (slice(N - 64, N), tail, t2, "last rows")):
        rot = (pos[:, :, at], w, axes, False)
        assert_normed(x[:, :, at], x0, wt, 1e-6, rot, what)
        assert_norm_gradient(dy[:, :, at], None, y0, x0, wt, 1e-6, rot, what)
    both = torch.cat([h2, t2], 2), torch.cat([head, tail], 2)
    rot = (torch.cat([pos[:, :, :64], pos[:, :, -64:]], 2), w, axes, False)
    _, want = paged4.norm_rope_backward(f64(both[0]), f64(both[1]), f64(wt), 1e-6, rotary_of(rot))
    assert np.abs(f64(dw) - want).max() <= 128 * 4 * 2e-5          # 128 rows, values of about 4, far above their errors


# ---------------------------------------------------------------------------
# 4-bit cache
# ---------------------------------------------------------------------------
def new_cache(pages, Hkv, ps, d, layout="hnd", fill=0xFF):
    """A pool in one of several memory orders; 0xFF bytes are NaN s and z, and codes of 15."""
    row = d + d // 8
    if layout == "hnd":
        return torch.full((pages, Hkv, ps, row), fill, dtype=torch.uint8, device=DEV)
    if layout == "hpd":                                             # heads outside
        return torch.full((Hkv, pages, ps, row), fill, dtype=torch.uint8, device=DEV).transpose(0, 1)
    return torch.full((pages, 2, Hkv + 1, ps, row), fill, dtype=torch.uint8, device=DEV)[:, 1, 1:]     # layers side by side


def tables(lens, ps, seed, extra=2):
    """Block table with pages in random order; columns past a sequence's pages are far out of range."""
    g = torch.Generator().manual_seed(seed)
    n = [-(-x // ps) for x in lens]
    total = sum(n) + extra
    order = torch.randperm(total, generator=g).tolist()
    table = torch.full((len(lens), max(1, max(n)) + 1), 2 ** 30, dtype=torch.int32)
    at = 0
    for b, m in enumerate(n):
        table[b, :m] = torch.tensor(order[at:at + m], dtype=torch.int32)
        at += m
    return total, table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)


def offsets(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=DEV)


def filled(lens, Hkv, ps, d, dt, seed, layout="hnd", sigma=1.0, rows=None):
    """A cache holding sequences of these lengths, and their 16-bit rows k, v [T, Hkv, d]."""
    total, table, ln = tables(lens, ps, seed)
    g = torch.Generator().manual_seed(seed + 1)
    if rows is None:
        size = torch.exp(0.5 * torch.randn((d,), generator=g))
        rows = [(sigma * size * torch.randn((sum(lens), Hkv, d), generator=g)).to(dt).to(DEV) for _ in range(2)]
    cache = new_cache(total, Hkv, ps, d, layout)
    if sum(lens):
        assert fa.paged4_append(cache, table, ln, *rows, cu_seqlens=offsets(lens)) is None
    return cache, table, ln, rows[0], rows[1]


def assert_decoded(o, lse, q, k, v, lens, scale, window, what=""):
    """k, v [T, Hkv, d]: the 16-bit rows of the sequences, one after another."""
    dt, d, at = o.dtype, q.shape[-1], 0
    kn, vn, qn, on, ln = f64(k), f64(v), f64(q), f64(o), f64(lse)
    for b, n in enumerate(lens):
        r = rounder(dt)
        ro, rl, x, a = paged4.decode(qn[b], kn[at:at + n].swapaxes(0, 1), vn[at:at + n].swapaxes(0, 1), scale, window, r)
        at += n
        e = (x * (d + 8) * 2.0 ** -23 + 2.0 ** -21 + n * 2.0 ** -24)
        most = np.zeros_like(a)
        if n:
            s = paged4.quantise(vn[at - min(n, window or n):at], r)[1].max(0)            # [Hkv, d / 64]
            most = np.repeat(np.repeat(s, 64, 1), qn.shape[1] // s.shape[0], 0)
        bound = (U[dt] * np.abs(ro) + (2.1 * e[:, None] + WEIGHT[dt] * 7.5 / 32 + (d + n) * 2.0 ** -23) * a
                 + n * 2.0 ** -28 * most + TINY[dt])
        err = np.abs(on[b] - ro)
        assert (err <= bound).all(), f"{what} sequence {b}: o off by {(err / np.maximum(bound, 1e-30)).max()} of the bound"
        if n == 0:
            assert np.isneginf(ln[b]).all(), what
        else:
            assert (np.abs(ln[b] - rl) <= e + 2.0 ** -22 * np.abs(rl)).all(), f"{what} sequence {b}: lse"


def last_rows(x, lens, n, dt):
    """The oracle's read: [B, Hkv, n, d] of rows [T, Hkv, d]."""
    v = paged4.values(f64(x), rounder(dt))
    out, at = np.zeros((len(lens), x.shape[1], n, x.shape[2])), 0
    for b, m in enumerate(lens):
        take = min(m, n)
        if take:
            out[b, :, n - take:] = v[at + m - take:at + m].swapaxes(0, 1)
        at += m
    return out


def assert_read(got, want, dt, what=""):
    err, bound = np.abs(f64(got) - want), (U[dt] + 2.0 ** -23) * np.abs(want) + TINY[dt]
    assert np.array_equal(np.isnan(err), np.isnan(want)), what
    off = err > bound
    assert not off.any(), f"{what}: {off.sum()} values"


APPEND = [
    # lens, new (None: one each), padding tokens, Hq, Hkv, d, page, sections, weights (False: no norm), dtype, layout
    ([1], None, 0, 1, 1, 64, 16, (32,), BF, BF, "hnd"),
    ([5, 0, 17, 64], None, 0, 8, 2, 128, 16, (16, 24, 24), BF, BF, "hpd"),
    ([100, 33, 0, 64], [37, 0, 0, 64], 5, 6, 3, 64, 48, (32,), F32, HF, "layers"),
    ([300, 7], [300, 7], 0, 4, 4, 128, 64, (40,), False, BF, "hnd"),
    ([40, 40], [3, 1], 2, 0, 2, 64, 16, None, False, HF, "hnd"),
    ([130], [129], 0, 9, 1, 128, 32, None, F32, BF, "layers"),
    ([64, 70], [20, 70], 0, 0, 5, 128, 16, (64,), None, HF, "hpd"),
    ([1000, 600], [1000, 600], 0, 16, 8, 128, 128, (64,), HF, HF, "hnd"),
    ([40, 9], [40, 9], 0, 3, 2, 128, 16, (8,), F32, BF, "hnd"),           # vectors of both groups in a thread
    ([40, 9], [40, 9], 0, 3, 2, 128, 16, (8, 16), None, HF, "hnd"),
    ([40, 9], [40, 9], 0, 3, 2, 128, 16, (16, 32), F32, BF, "hnd"),
    ([40, 9], None, 0, 3, 2, 128, 16, (56,), False, HF, "hnd"),
    ([40, 9], [40, 9], 0, 2, 2, 64, 16, (8,), F32, BF, "hnd"),
]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("lens,new,pad,Hq,Hkv,d,page,sections,wdt,dt,layout", APPEND)
def test_append_and_read(cuda_lib, lens, new, pad, Hq, Hkv, d, page, sections, wdt, dt, layout, interleaved):
    total, table, ln = tables(lens, page, seed=Hq + d)
    counts = new or [min(1, n) for n in lens]
    T = (sum(new) if new else len(lens)) + pad
    g = torch.Generator().manual_seed(T)
    x = torch.randn((T, Hq + 2 * Hkv, d), generator=g).to(dt).to(DEV)
    q, k, v = x.split([Hq, Hkv, Hkv], dim=1)
    rot, kw = turned(g, sections, interleaved, 3, 1, T)
    if rot is not None:
        rot = (rot[0], rot[1], rot[2], rot[3])
        kw["positions"] = rot[0][:, 0]
    if wdt is not False:
        kw.update(eps=1e-5, q_weight=weights(g, d, wdt), k_weight=weights(g, d, wdt))
    cache = new_cache(total, Hkv, page, d, layout, fill=0x5A)
    gb = GuardedBuffers(DEV)
    qo = None
    if Hq:
        qo = gb.empty((T, Hq, d), dt)
        qo.fill_(7.0)
        kw.update(q=q, q_out=qo)
    fa.paged4_append(cache, table, ln, k, v, cu_seqlens=offsets(new) if new else None, **kw)
    n = max(max(counts), 1)
    ko, vo = gb.empty((len(lens), Hkv, n, d), dt), gb.empty((len(lens), Hkv, n, d), dt)
    fa.paged4_read(cache, table, ln, n, dt, ko, vo)
    ok()
    gb.check()
    places = paged.token_places(lens, None if new is None else [0] + list(np.cumsum(new)), T)
    eps, wq, wk = kw.get("eps"), kw.get("q_weight"), kw.get("k_weight")
    rn = rotary_of(rot)

    def expected(rows, w):
        """(rows [T, H, d], bound of their error) as [1, H, T, d] in fp64."""
        y = f64(rows).swapaxes(0, 1)[None]
        if eps is not None:
            return norm_error(y, None if w is None else f64(w), eps, rn)
        e = 2e-6 * pair_sums(y, rn)
        return (y if rn is None else paged.rotate(y, *rn)), e
    if Hq:
        want, e = expected(q, wq)
        got = f64(qo).swapaxes(0, 1)[None]
        for t, pl in enumerate(places):
            if pl is None:
                assert (got[:, :, t] == 7.0).all(), "a padding row was written"
            else:
                bound = U[dt] * np.abs(want[:, :, t]) + 1.01 * e[:, :, t] + TINY[dt]
                assert (np.abs(got[:, :, t] - want[:, :, t]) <= bound).all(), f"q of token {t}"
    exact = eps is None and rot is None
    wk_rows, ek = expected(k, wk)
    u = U[dt]
    for t, pl in enumerate(places):
        if pl is None:
            continue
        b, row = pl[0], n - (lens[pl[0]] - pl[1])
        assert_read(vo[b, :, row], paged4.values(f64(v[t]), rounder(dt)), dt, f"v of token {t}")
        if exact:
            assert_read(ko[b, :, row], paged4.values(f64(k[t]), rounder(dt)), dt, f"k of token {t}")
        else:
            y = wk_rows[0, :, t]
            e = (ek[0, :, t] + u * np.abs(y) + TINY[dt]).reshape(Hkv, -1, 64)
            yg = y.reshape(Hkv, -1, 64)
            most = e.max(-1, keepdims=True)
            s = (yg.max(-1, keepdims=True) - yg.min(-1, keepdims=True) + 2 * most) / 15 * (1 + u)
            bound = s * (0.5 + 15 * u) + e + most + u * (np.abs(yg) + s) + TINY[dt]
            assert (np.abs(f64(ko[b, :, row]).reshape(yg.shape) - yg) <= bound).all(), f"k of token {t}"
    # Nothing else was written: with every stored token's bytes put back the pool is as it was.
    probe = cache.clone()
    other = torch.zeros_like(k)
    fa.paged4_append(probe, table, ln, other, other, cu_seqlens=offsets(new) if new else None)
    blank = new_cache(total, Hkv, page, d, layout, fill=0x5A)
    fa.paged4_append(blank, table, ln, other, other, cu_seqlens=offsets(new) if new else None)
    ok()
    assert torch.equal(probe, blank)


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("d", [64, 128])
def test_codes_of_odd_groups(cuda_lib, d, dt):
    r = np.random.default_rng(7)
    fi = torch.finfo(dt)
    x = r.normal(size=(24, 1, d))
    x[0] = 0.0
    x[1] = -3.25
    x[2] = np.where(r.random(d) < 0.5, 1.0, -1.0)
    x[3] = r.integers(0, 16, size=d) * 0.5                    # many values on a code or between two
    x[4] = r.integers(0, 31, size=d) * 0.25
    x[5] = 1000.0 + r.integers(0, 3, size=d) * 8              # a small range far from zero
    x[6] = r.normal(size=d) * float(fi.tiny) * 4              # subnormal steps
    x[7, 0, 5] = float("nan")
    x[8, 0, 63] = float("inf")
    x[9, 0, 0] = -float("inf")
    x[10] = float("nan")
    x[11] = float("inf")
    x[12] = np.where(np.arange(d) % 2, 3e4, -3e4)
    x[13, 0, 7] = 900.0                                       # one large value
    x[14] = -0.0
    x[15] = r.normal(size=d) * 1e-3 + 0.5
    x[16] = float(fi.max) / 4 * r.random(d)
    rows = torch.from_numpy(x).to(dt).to(DEV)
    cache, table, ln, _, _ = filled([24], 1, 16, d, dt, seed=3, rows=[rows, rows.flip(0).contiguous()])
    k, v = fa.paged4_read(cache, table, ln, 24, dt)
    ok()
    assert_read(k, last_rows(rows, [24], 24, dt), dt, "k")
    assert torch.equal(torch.nan_to_num(v.flip(2)), torch.nan_to_num(k))
    assert (k[0, 0, 1] == -3.25).all() and not k[0, 0, 0].any()


READ = [
    # lens, n, Hkv, d, page, dtype, layout
    ([1], 1, 1, 64, 16, BF, "hnd"),
    ([0], 3, 2, 128, 16, HF, "hnd"),
    ([100, 0, 17, 1], 17, 3, 128, 16, BF, "layers"),
    ([100, 0, 17, 1], 129, 2, 64, 48, HF, "hpd"),
    ([1000], 1000, 8, 128, 64, BF, "hnd"),
    ([333, 222], 300, 1, 64, 32, BF, "hpd"),
]


@pytest.mark.parametrize("lens,n,Hkv,d,page,dt,layout", READ)
def test_read(cuda_lib, lens, n, Hkv, d, page, dt, layout):
    cache, table, ln, k, v = filled(lens, Hkv, page, d, dt, seed=n, layout=layout)
    ko, vo = fa.paged4_read(cache, table, ln, n, dt)
    # Token-major parts of one buffer as outputs.
    gb = GuardedBuffers(DEV)
    both = gb.empty((len(lens), n, 2 * Hkv + 1, d), dt)
    both.fill_(7.0)
    k2, v2 = both[:, :, :Hkv].transpose(1, 2), both[:, :, Hkv + 1:].transpose(1, 2)
    fa.paged4_read(cache, table, ln, n, dt, k2, v2)
    ok()
    gb.check()
    assert_read(ko, last_rows(k, lens, n, dt), dt, "k")
    assert_read(vo, last_rows(v, lens, n, dt), dt, "v")
    assert torch.equal(k2, ko) and torch.equal(v2, vo) and (both[:, :, Hkv] == 7.0).all()


DECODE = [
    # lens, Hq, Hkv, d, page, window, dtype, layout
    ([1], 1, 1, 64, 16, 0, BF, "hnd"),
    ([0], 4, 2, 128, 16, 0, BF, "hnd"),
    ([15, 16, 17, 0, 31, 33], 8, 2, 128, 16, 0, BF, "hnd"),
    ([127, 128, 129, 255, 256, 257], 4, 4, 64, 32, 0, HF, "hpd"),
    ([1000, 1, 0, 777], 6, 2, 128, 48, 0, BF, "layers"),
    ([2500, 300], 8, 1, 64, 64, 0, HF, "hnd"),
    ([700, 130, 50], 9, 1, 128, 16, 0, BF, "hpd"),            # nine heads a group
    ([500, 90], 32, 2, 64, 128, 0, BF, "hnd"),                # sixteen
    ([333, 64], 17, 1, 128, 16, 0, HF, "layers"),
    ([260, 65], 33, 1, 64, 16, 0, BF, "hnd"),
    ([150], 72, 1, 128, 32, 0, BF, "hnd"),
    ([1000, 5, 0, 64], 8, 2, 128, 16, 1, BF, "hnd"),
    ([1000, 100, 65], 8, 4, 64, 16, 64, HF, "hnd"),
    ([1000, 257, 3], 4, 2, 128, 80, 250, BF, "hpd"),
    ([400, 60], 4, 2, 128, 16, 10 ** 9, BF, "hnd"),
    ([10000], 2, 1, 128, 256, 0, BF, "hnd"),
    ([5000, 4999], 16, 1, 128, 64, 0, HF, "hnd"),
]


@pytest.mark.parametrize("lens,Hq,Hkv,d,page,window,dt,layout", DECODE)
def test_decode(cuda_lib, lens, Hq, Hkv, d, page, window, dt, layout):
    cache, table, ln, k, v = filled(lens, Hkv, page, d, dt, seed=Hq * 100 + d, layout=layout)
    B = len(lens)
    g = torch.Generator().manual_seed(9)
    q = torch.randn((B, Hq + 3, d), generator=g).to(dt).to(DEV)[:, 1:Hq + 1]     # strided rows
    gb = GuardedBuffers(DEV)
    o, lse = gb.empty((B, Hq, d), dt), gb.empty((B, Hq), F32)
    ws = gb.empty((fa.paged4_decode_workspace(B, Hq, cache).numel(),), torch.uint8)
    fa.paged4_decode(q, cache, table, ln, scale=0.11, window=window, out=o, lse=lse, workspace=ws)
    ok()
    gb.check()
    assert_decoded(o, lse, q, k, v, lens, 0.11, window, f"{lens}")


def spread(B, longest, seed):
    """Lengths of a batch: some empty, some of one key, the rest anything."""
    g = torch.Generator().manual_seed(seed)
    return [[0, 1, int(x)][int(p)] if p < 2 else int(x)
            for x, p in zip(torch.randint(1, longest + 1, (B,), generator=g), torch.randint(0, 12, (B,), generator=g))]


@pytest.mark.parametrize("B,longest,Hq,Hkv,d,page,window,dt", [
    (40, 1800, 8, 4, 128, 16, 0, BF),        # several tiles a CTA, units cut in two
    (24, 1800, 16, 8, 64, 32, 0, HF),
    (30, 1400, 16, 1, 128, 48, 0, BF),       # sixteen heads a group
    (16, 1800, 40, 2, 64, 16, 400, BF),      # two head chunks and more, a window
    (300, 60, 2, 1, 64, 16, 0, BF),          # more sequences than a block has threads
    (700, 140, 2, 2, 64, 16, 0, HF),
    (400, 50, 16, 8, 128, 16, 0, HF),        # many units of one tile
    (90, 700, 8, 8, 128, 32, 0, HF),         # units of one to three tiles: parts that begin at a unit's end
    (90, 700, 16, 4, 64, 16, 0, HF),
    (120, 600, 16, 2, 64, 48, 300, HF),
    (280, 600, 32, 2, 64, 32, 0, BF),        # and more sequences than threads
    (90, 1100, 5, 5, 128, 16, 0, BF),
])
def test_decode_batches(cuda_lib, B, longest, Hq, Hkv, d, page, window, dt):
    lens = spread(B, longest, seed=B)
    cache, table, ln, k, v = filled(lens, Hkv, page, d, dt, seed=B + 1)
    q = torch.randn((B, Hq, d), generator=torch.Generator().manual_seed(B + 2)).to(dt).to(DEV)
    o, lse = fa.paged4_decode(q, cache, table, ln, window=window)
    ok()
    assert_decoded(o, lse, q, k, v, lens, d ** -0.5, window, f"batch of {B}")


@pytest.mark.parametrize("sigma,scale", [(4.0, 0.3), (0.0, 1.0)])
@pytest.mark.parametrize("dt", [BF, HF])
def test_decode_peaked_and_flat(cuda_lib, sigma, scale, dt):
    # Scores of +-50 and more: single keys dominate and the running maximum keeps moving; and all scores equal.
    cache, table, ln, k, v = filled([1900, 64, 300], 2, 16, 64, dt, seed=5, sigma=sigma)
    q = (4.0 * torch.randn((3, 8, 64), generator=torch.Generator().manual_seed(6))).to(dt).to(DEV)
    o, lse = fa.paged4_decode(q, cache, table, ln, scale=scale)
    ok()
    assert_decoded(o, lse, q, k, v, [1900, 64, 300], scale, 0, f"sigma {sigma}")


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("lens,Hq,Hkv,d", [([900], 8, 1, 128), ([1300] * 40, 16, 2, 64), ([1300] * 20, 32, 2, 128)])
def test_decode_heads_of_very_different_size(cuda_lib, lens, Hq, Hkv, d, dt):
    # Each head's q in its own range, and elements of one head far apart.
    cache, table, ln, k, v = filled(lens, Hkv, 16, d, dt, seed=61)
    g = torch.Generator().manual_seed(62)
    q = torch.randn((len(lens), Hq, d), generator=g)
    lo = -10 if dt is HF else -60
    q *= 2.0 ** torch.randint(lo, 4, (len(lens), Hq, 1), generator=g)
    q[:, ::3, ::2] *= 2.0 ** -9
    q = q.to(dt).to(DEV)
    o, lse = fa.paged4_decode(q, cache, table, ln, scale=0.3)
    ok()
    assert_decoded(o, lse, q, k, v, lens, 0.3, 0, "heads")


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("down", [False, True])
@pytest.mark.parametrize("lens,Hq,Hkv,d", [([900], 8, 1, 128), ([900] * 48, 4, 2, 64), ([900] * 40, 16, 1, 128)])
def test_decode_steps_of_very_different_size(cuda_lib, lens, Hq, Hkv, d, down, dt):
    # The steps of V grow (or shrink) by 2^20 along a sequence, one group's much faster than the other's, some are 0; and
    # the keys with the largest steps may weigh nothing.
    g = torch.Generator().manual_seed(63)
    T, n = sum(lens), lens[0]
    up = torch.arange(T) % n / n
    size = 2.0 ** torch.stack([20 * up - 12, 3 * up], 1)[:, :d // 64]
    v = torch.randn((T, Hkv, d // 64, 64), generator=g) * (size.flip(0) if down else size)[:, None, :, None]
    v[::7] = 0.25
    k = torch.randn((T, Hkv, d), generator=g)
    k[:, :, 0] = 8 * up[:, None] - 4
    k, v = k.to(dt).to(DEV), v.reshape(T, Hkv, d).to(dt).to(DEV)
    cache, table, ln, _, _ = filled(lens, Hkv, 32, d, dt, seed=64, rows=[k, v])
    q = torch.randn((len(lens), Hq, d), generator=g)
    q[:, ::2, 0] = -6
    q = q.to(dt).to(DEV)
    o, lse = fa.paged4_decode(q, cache, table, ln, scale=0.5)
    ok()
    assert_decoded(o, lse, q, k, v, lens, 0.5, 0, "steps")


@pytest.mark.parametrize("d", [64, 128])
def test_last_keys_of_the_longest_sequences(cuda_lib, d):
    # Lengths up to 2^30, the most a table may hold, over one page that it names again and again: the last keys.
    ps, n = 65536, 500
    lens = [2 ** 30, 2 ** 30 - 15, 2 ** 30 - 300]
    g = torch.Generator().manual_seed(67)
    k, v = (torch.randn((ps, 1, d), generator=g).to(BF).to(DEV) for _ in range(2))
    cache = new_cache(1, 1, ps, d)
    one = torch.zeros((1, 1), dtype=torch.int32, device=DEV)
    fa.paged4_append(cache, one, torch.tensor([ps], dtype=torch.int32, device=DEV), k, v, cu_seqlens=offsets([ps]))
    table = torch.zeros((3, 16384), dtype=torch.int32, device=DEV)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    at = torch.tensor([[(m - n + i) % ps for i in range(n)] for m in lens]).reshape(-1).to(DEV)
    q = torch.randn((3, 4, d), generator=g).to(BF).to(DEV)
    for window in (1, 15, n):
        o, lse = fa.paged4_decode(q, cache, table, ln, window=window)
        ok()
        assert_decoded(o, lse, q, k[at], v[at], [n] * 3, d ** -0.5, window, f"window {window}")
    kr, vr = fa.paged4_read(cache, table, ln, n, BF)
    ok()
    assert_read(kr, last_rows(k[at], [n] * 3, n, BF), BF, "k")
    assert_read(vr, last_rows(v[at], [n] * 3, n, BF), BF, "v")


@pytest.mark.parametrize("backwards", [False, True])
def test_decode_of_pages_side_by_side(cuda_lib, backwards):
    # One kv head and pages in order: the records of a tile follow one another in memory, across pages too.
    lens, d = [2000, 1999, 15, 300], 128
    _, _, _, k, v = filled(lens, 1, 16, d, BF, seed=65)
    n = [-(-x // 16) for x in lens]
    first = np.concatenate([[0], np.cumsum(n)])
    table = torch.stack([torch.arange(max(n)) + int(first[b]) for b in range(4)]).to(torch.int32)
    if backwards:
        table = int(first[-1]) - 1 - table
    table, ln = table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    cache = new_cache(int(first[-1]), 1, 16, d)
    fa.paged4_append(cache, table, ln, k, v, cu_seqlens=offsets(lens))
    q = torch.randn((4, 6, d), generator=torch.Generator().manual_seed(66)).to(BF).to(DEV)
    o, lse = fa.paged4_decode(q, cache, table, ln)
    ok()
    assert_decoded(o, lse, q, k, v, lens, d ** -0.5, 0, "side by side")


@pytest.mark.parametrize("down", [False, True])
def test_decode_rising_and_falling_scores(cuda_lib, down):
    # Key j's score is about j times a step: the maximum moves with every key, by little and by much.
    n, d = 700, 128
    g = torch.Generator().manual_seed(21)
    k = 0.05 * torch.randn((n, 1, d), generator=g)
    k[:, 0, 0] += torch.arange(n) * 0.11 * (-1 if down else 1)
    k, v = k.to(BF).to(DEV), torch.randn((n, 1, d), generator=g).to(BF).to(DEV)
    cache, table, ln, _, _ = filled([n], 1, 16, d, BF, seed=22, rows=[k, v])
    q = torch.randn((1, 3, d), generator=g)
    q[:, :, 0] = torch.tensor([1.0, 10.0, 100.0])
    q = q.to(BF).to(DEV)
    o, lse = fa.paged4_decode(q, cache, table, ln, scale=0.1)
    ok()
    assert_decoded(o, lse, q, k, v, [n], 0.1, 0)


@pytest.mark.parametrize("dt", [BF, HF])
def test_decode_with_rows_that_are_not_finite(cuda_lib, dt):
    # A NaN in a visible row of K spoils its sequence and kv head, one in V the 64 elements of its group; a window that
    # hides the row silences it.
    lens = [200, 100]
    _, _, _, k, v = filled(lens, 2, 16, 128, dt, seed=31)
    k[20, 0, 3] = float("nan")
    v[220, 1, 100] = float("inf")
    cache, table, ln, _, _ = filled(lens, 2, 16, 128, dt, seed=31, rows=[k, v])
    q = torch.randn((2, 8, 128), generator=torch.Generator().manual_seed(32)).to(dt).to(DEV)
    o, lse = fa.paged4_decode(q, cache, table, ln)
    ow, lw = fa.paged4_decode(q, cache, table, ln, window=60)
    ok()
    assert o[0, :4].isnan().all() and lse[0, :4].isnan().all()
    assert o[0, 4:].isfinite().all() and o[1, :4].isfinite().all() and lse[1].isfinite().all()
    assert o[1, 4:, 64:].isnan().all() and o[1, 4:, :64].isfinite().all()
    assert_decoded(ow[:1], lw[:1], q[:1], k[:200].nan_to_num(), v[:200], [200], 128 ** -0.5, 60)


def test_decode_pages_shared_by_sequences(cuda_lib):
    cache, table, ln, k, v = filled([300, 0], 2, 16, 64, BF, seed=41)
    table[1] = table[0]
    ln[1] = 100
    q = torch.randn((2, 4, 64), generator=torch.Generator().manual_seed(42)).to(BF).to(DEV)
    o, lse = fa.paged4_decode(q, cache, table, ln)
    ok()
    assert_decoded(o, lse, q, torch.cat([k, k[:100]]), torch.cat([v, v[:100]]), [300, 100], 0.125, 0)


def test_decode_is_reproducible(cuda_lib):
    lens = [3000, 17, 0, 900]
    cache, table, ln, _, _ = filled(lens, 2, 16, 128, BF, seed=43)
    q = torch.randn((4, 16, 128), generator=torch.Generator().manual_seed(44)).to(BF).to(DEV)
    first = fa.paged4_decode(q, cache, table, ln)
    for _ in range(5):
        again = fa.paged4_decode(q, cache, table, ln)
        ok()
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


SHORT = [
    # lens, Hq, Hkv, d, page, window, dtype: few units of few tiles, and behind a wide table
    ([1], 8, 2, 128, 16, 0, BF),
    ([1000], 8, 2, 128, 16, 0, BF),
    ([130, 0, 5, 1200], 4, 1, 64, 32, 0, HF),
    ([600, 601], 32, 2, 128, 16, 0, BF),
    ([900, 30], 40, 2, 64, 16, 100, BF),
    ([700] * 8, 32, 8, 128, 16, 0, HF),
]


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("lens,Hq,Hkv,d,page,window,dt", SHORT)
def test_decode_short_sequences_behind_any_table(cuda_lib, lens, Hq, Hkv, d, page, window, dt, wide):
    cache, table, ln, k, v = filled(lens, Hkv, page, d, dt, seed=51)
    if wide:
        t = torch.full((len(lens), 2 ** 30 // page), 2 ** 30, dtype=torch.int32, device=DEV)
        t[:, :table.shape[1]] = table
        table = t
    q = torch.randn((len(lens), Hq, d), generator=torch.Generator().manual_seed(52)).to(dt).to(DEV)
    o, lse = fa.paged4_decode(q, cache, table, ln, window=window)
    ok()
    assert_decoded(o, lse, q, k, v, lens, d ** -0.5, window)


def status_and_clear():
    s = fa.fa_last_device_status()[0]
    ok()
    return s


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("bad", ["page", "negative page", "length", "negative length"])
def test_bad_indices_are_recorded(cuda_lib, bad, wide):
    # The other sequence's outputs are right all the same.
    lens = [300, 200]
    cache, table, ln, k, v = filled(lens, 2, 16, 64, BF, seed=61)
    if wide:
        t = torch.full((2, 4000), 2 ** 30, dtype=torch.int32, device=DEV)
        t[:, :table.shape[1]] = table
        table = t
    q = torch.randn((2, 8, 64), generator=torch.Generator().manual_seed(62)).to(BF).to(DEV)
    good = table.clone()
    if "page" in bad:
        table[0, 3] = cache.shape[0] if bad == "page" else -1
    else:
        ln[0] = table.shape[1] * 16 + 1 if bad == "length" else -5
    o, lse = fa.paged4_decode(q, cache, table, ln)
    assert status_and_clear() == fa.FA_ERR_BAD_INDEX
    assert_decoded(o[1:], lse[1:], q[1:], k[300:], v[300:], [200], 0.125, 0)
    kr, _ = fa.paged4_read(cache, table, ln, 300, BF)
    assert status_and_clear() == fa.FA_ERR_BAD_INDEX
    assert_read(kr[1:], last_rows(k[300:], [200], 300, BF), BF)
    # An append to the bad place is skipped, and nothing else is touched.
    if "page" in bad:
        ln[0] = 3 * 16 + 5
    before = cache.clone()
    fa.paged4_append(cache, table, ln, k[[0, 300]], v[[0, 300]])
    assert status_and_clear() == fa.FA_ERR_BAD_INDEX
    changed = (cache != before).flatten(1).any(1).nonzero().flatten().tolist()
    assert set(changed) <= {good[1, 199 // 16].item()}


@pytest.mark.parametrize("cu", [[1, 2, 4], [0, 3, 2], [0, 2, 5]])
def test_append_bad_offsets_are_recorded(cuda_lib, cu):
    total, table, ln = tables([30, 40], 16, seed=63)
    cache = new_cache(total, 2, 16, 64, fill=0)
    k = torch.randn((4, 2, 64), device=DEV).to(BF)
    fa.paged4_append(cache, table, ln, k, k, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV))
    assert status_and_clear() == fa.FA_ERR_BAD_INDEX


def test_append_without_tokens_and_in_place(cuda_lib):
    total, table, ln = tables([30, 40], 16, seed=64)
    cache = new_cache(total, 2, 16, 64)
    x = torch.zeros((0, 2, 64), dtype=BF, device=DEV)
    assert fa.paged4_append(cache, table, ln, x, x, cu_seqlens=offsets([0, 0])) is None
    g = torch.Generator().manual_seed(65)
    q, k = torch.randn((2, 4, 64), generator=g).to(BF).to(DEV), torch.randn((2, 2, 64), generator=g).to(BF).to(DEV)
    w = weights(g, 64, BF)
    apart = fa.paged4_append(cache, table, ln, k, k, q=q, q_weight=w, k_weight=w, eps=1e-6)
    same = fa.paged4_append(cache, table, ln, k, k, q=q, q_weight=w, k_weight=w, eps=1e-6, q_out=q)
    ok()
    assert same is q and torch.equal(same, apart)


def test_cache_offsets_past_32_bits(cuda_lib):
    Hkv, ps, d = 8, 64, 128
    pages = 2 ** 32 // (Hkv * ps * 144) + 40
    cache = torch.empty((pages, Hkv, ps, 144), dtype=torch.uint8, device=DEV)
    use = [pages - 1, 3, pages - 20, pages // 2 + 7]
    table = torch.tensor([use], dtype=torch.int32, device=DEV)
    ln = torch.tensor([250], dtype=torch.int32, device=DEV)
    g = torch.Generator().manual_seed(15)
    k, v = (torch.randn((250, Hkv, d), generator=g).to(BF).to(DEV) for _ in range(2))
    fa.paged4_append(cache, table, ln, k, v, cu_seqlens=offsets([250]))
    q = torch.randn((1, 16, d), generator=g).to(BF).to(DEV)
    o, lse = fa.paged4_decode(q, cache, table, ln)
    kr, vr = fa.paged4_read(cache, table, ln, 250, BF)
    ok()
    assert_decoded(o, lse, q, k, v, [250], d ** -0.5, 0, "far pages")
    assert_read(kr, last_rows(k, [250], 250, BF), BF)
    assert_read(vr, last_rows(v, [250], 250, BF), BF)


# ---------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dt", [BF, HF])
def test_serving_run(cuda_lib, dt):
    # Prompts appended, then steps of one token: each step's attention against the oracle over the 16-bit rows that
    # qk_norm_rope gives for the same tokens.
    Hq, Hkv, d, ps = 8, 2, 128, 16
    lens = [70, 0, 33]
    g = torch.Generator().manual_seed(71)
    total, table, _ = tables([n + 8 for n in lens], ps, seed=72)
    cache = new_cache(total, Hkv, ps, d)
    wq, wk = weights(g, d, dt), weights(g, d, dt)
    w, axes = fa.rope_frequencies((64,), device=DEV)
    norm = dict(q_weight=wq, k_weight=wk, eps=1e-6, inv_freq=w, axes=axes)
    rows = [[[], []] for _ in lens]

    def tokens(counts):
        T = sum(counts)
        x = torch.randn((T, Hq + 2 * Hkv, d), generator=g).to(dt).to(DEV)
        pos = torch.tensor([n - c + i for n, c in zip(lens, counts) for i in range(c)], dtype=torch.int32, device=DEV)[None]
        return (*x.split([Hq, Hkv, Hkv], dim=1), pos)

    def remember(k, v, pos, counts):
        kn = fa.qk_norm_rope(k.transpose(0, 1)[None], None, wk, None, pos[:, None], w, axes)[0].transpose(0, 1)
        at = 0
        for b, c in enumerate(counts):
            rows[b][0].append(kn[at:at + c])
            rows[b][1].append(v[at:at + c])
            at += c
    q, k, v, pos = tokens(lens)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    fa.paged4_append(cache, table, ln, k, v, cu_seqlens=offsets(lens), q=q, positions=pos, **norm)
    remember(k, v, pos, lens)
    for step in range(6):
        lens = [n + 1 for n in lens]
        ln.copy_(torch.tensor(lens, dtype=torch.int32))
        q, k, v, pos = tokens([1, 1, 1])
        qn = fa.paged4_append(cache, table, ln, k, v, q=q, positions=pos, **norm)
        o, lse = fa.paged4_decode(qn, cache, table, ln, window=0 if step % 2 else 50)
        remember(k, v, pos, [1, 1, 1])
        ok()
        assert_normed(qn.transpose(0, 1)[None], q.transpose(0, 1)[None], wq, 1e-6, (pos[:, None], w, axes, False), "q")
        kall, vall = (torch.cat([t for r in rows for t in r[i]]) for i in range(2))
        # The fused kernel may round a key's 16-bit value the other way and so move a code by a step; the read shows the
        # values that the attention has to use.
        got, _ = fa.paged4_read(cache, table, ln, max(lens), dt)
        want = last_rows(kall, lens, max(lens), dt)
        same = np.abs(f64(got) - want) <= (U[dt] + 2.0 ** -23) * np.abs(want)
        assert same.mean() > 0.99
        if same.all():
            assert_decoded(o, lse, qn, kall, vall, lens, d ** -0.5, 0 if step % 2 else 50, f"step {step}")


@pytest.mark.parametrize("chunk", [100, 37])
def test_prompt_in_chunks(cuda_lib, chunk):
    # Each chunk is appended, the sequence read back, and the chunk's queries attend to it: forward_ex on what the cache
    # holds against the oracle on the same values.
    Hq, Hkv, d, n = 4, 2, 128, 230
    g = torch.Generator().manual_seed(81)
    total, table, ln = tables([n], 16, seed=82)
    cache = new_cache(total, Hkv, 16, d)
    q, k, v = (torch.randn((n, h, d), generator=g).to(BF).to(DEV) for h in (Hq, Hkv, Hkv))
    for at in range(0, n, chunk):
        end = min(at + chunk, n)
        ln.fill_(end)
        fa.paged4_append(cache, table, ln, k[at:end], v[at:end], cu_seqlens=offsets([end - at]))
        kc, vc = fa.paged4_read(cache, table, ln, end, BF)
        qc = q[at:end].transpose(0, 1)[None].contiguous()
        o, lse = fa.forward_ex(qc, kc, vc, causal=True)
        ok()
        assert_read(kc, last_rows(k[:end], [end], end, BF), BF)
        ro, rl = ref.attention_forward(f64(qc), f64(kc), f64(vc), True, d ** -0.5)
        assert_fwd(o, lse, ro, rl, f"chunk at {at}")


def test_one_token_agrees_with_the_16_bit_path_over_the_values_read(cuda_lib):
    # paged_decode over a 16-bit cache that holds the values the 4-bit one stands for.
    lens, Hkv, d, ps = [200, 64], 2, 64, 16
    g = torch.Generator().manual_seed(83)
    rows = [(torch.randint(0, 16, (sum(lens), Hkv, d), generator=g) * 0.25 - 2).to(BF).to(DEV) for _ in range(2)]
    for x in rows:
        x[..., 0], x[..., 1] = -2.0, 1.75                         # every row is held exactly
    cache, table, ln, k, v = filled(lens, Hkv, ps, d, BF, seed=84, rows=rows)
    kc = torch.zeros((cache.shape[0], Hkv, ps, d), dtype=BF, device=DEV)
    vc = torch.zeros_like(kc)
    fa.paged_append(kc, vc, table, ln, k, v, cu_seqlens=offsets(lens))
    q = torch.randn((2, 8, d), generator=g).to(BF).to(DEV)
    o, lse = fa.paged4_decode(q, cache, table, ln)
    o16, l16 = fa.paged_decode(q, kc, vc, table, ln)
    ok()
    assert_decoded(o, lse, q, k, v, lens, 0.125, 0)
    assert (o.float() - o16.float()).abs().max().item() <= 2 * U[BF] * o16.float().abs().max().item()
    assert (lse - l16).abs().max().item() <= 1e-3


def one_step(dt=BF, lens=(300, 0, 41, 900)):
    """A step's calls on fixed buffers: step(stream) -> outputs; the inputs to change between replays."""
    lens = list(lens)
    Hq, Hkv, d = 8, 2, 64
    cache, table, ln, _, _ = filled(lens, Hkv, 16, d, dt, seed=91)
    g = torch.Generator().manual_seed(92)
    x = torch.randn((4, Hq + 2 * Hkv, d), generator=g).to(dt).to(DEV)
    q, k, v = x.split([Hq, Hkv, Hkv], dim=1)
    wq, wk = weights(g, d, dt), weights(g, d, dt)
    w, axes = fa.rope_frequencies((32,), device=DEV)
    pos = torch.tensor([[max(n - 1, 0) for n in lens]], dtype=torch.int32, device=DEV)
    y = torch.randn((1, Hq + 2 * Hkv, 50, d), generator=g).to(dt).to(DEV)
    py = torch.arange(50, dtype=torch.int32, device=DEV).view(1, 1, 50)

    def step(stream=None):
        qn = fa.paged4_append(cache, table, ln, k, v, q=q, q_weight=wq, k_weight=wk, eps=1e-6, positions=pos, inv_freq=w,
                              axes=axes, stream=stream)
        o, lse = fa.paged4_decode(qn, cache, table, ln, stream=stream)
        kr, vr = fa.paged4_read(cache, table, ln, 20, dt, stream=stream)
        yq, yk = fa.qk_norm_rope(y[:, :Hq], y[:, Hq:Hq + Hkv], wq, wk, py, w, axes, stream=stream)
        grads = fa.qk_norm_rope_backward(yq, yk, y[:, :Hq], y[:, Hq:Hq + Hkv], wq, wk, py, w, axes, stream=stream)
        live = [b for b, n in enumerate(lens) if n]
        return [o, lse, kr, vr, yq, yk, *grads], qn, live
    return step, x, y


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def live_rows(r):
    """Outputs of a step without the query rows of empty sequences, whose inputs were never written."""
    out, _, live = r
    return [out[0][live], *out[1:]]


def test_step_in_a_captured_graph(cuda_lib):
    step, x, y = one_step()
    want = live_rows(step())
    ok()
    want = [t.clone() for t in want]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for gr in graphs:
        with torch.cuda.graph(gr):
            outs.append(step())
    for i in (0, 1, 0):
        for t in outs[i][0]:
            t.zero_()
        graphs[i].replay()
        ok()
        assert same(live_rows(outs[i]), want)
    x.mul_(0.5)
    y.add_(0.25)
    graphs[0].replay()
    ok()
    got = [t.clone() for t in live_rows(outs[0])]
    again = live_rows(step())
    ok()
    assert same(got, again) and not torch.equal(got[4], want[4])


def test_captured_decode_follows_lengths_and_tables(cuda_lib):
    lens = [300, 40, 0, 129]
    cache, table, ln, k, v = filled(lens, 2, 16, 64, BF, seed=95)
    at = np.concatenate([[0], np.cumsum(lens)])
    g = torch.Generator().manual_seed(96)
    q = torch.randn((4, 8, 64), generator=g).to(BF).to(DEV)
    fa.paged4_decode(q, cache, table, ln)
    ok()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = fa.paged4_decode(q, cache, table, ln)
        kr, _ = fa.paged4_read(cache, table, ln, 64, BF)
    t0 = table.clone()
    for order, n in (([0, 1, 2, 3], [300, 40, 0, 129]), ([3, 0, 1, 2], [100, 299, 33, 0]), ([1, 1, 0, 3], [7, 40, 16, 1])):
        table.copy_(t0[order])
        ln.copy_(torch.tensor(n, dtype=torch.int32))
        q.copy_(torch.randn((4, 8, 64), generator=g))
        graph.replay()
        ok()
        kk, vv = (torch.cat([x[at[s]:at[s] + m] for s, m in zip(order, n)]) for x in (k, v))
        assert_decoded(o, lse, q, kk, vv, n, 0.125, 0, f"{n}")
        assert_read(kr, last_rows(kk, n, 64, BF), BF)


def test_steps_on_two_streams_and_threads(cuda_lib):
    steps = [one_step(), one_step(dt=HF, lens=(700, 64, 0, 9))]
    want = [[t.clone() for t in live_rows(s[0]())] for s in steps]
    ok()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(10):
        for i in range(2):
            got[i].append(steps[i][0](stream=streams[i]))
    ok()
    for i in range(2):
        assert all(same(live_rows(r), want[i]) for r in got[i])
    got, errors = [None, None], []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            stream.wait_stream(torch.cuda.default_stream())
            with torch.cuda.stream(stream):
                got[i] = [steps[i][0]() for _ in range(20)]
            stream.synchronize()
        except Exception as e:          # reported by the test's thread
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    ok()
    assert not errors, errors
    for i in range(2):
        assert all(same(live_rows(r), want[i]) for r in got[i])


def test_calls_between_other_kernels_on_one_stream(cuda_lib):
    # Inputs written right before a call and outputs overwritten right after it, with nothing that waits in between.
    cache, table, ln, _, _ = filled([900, 5, 300, 64], 2, 16, 64, BF, seed=101)
    g = torch.Generator().manual_seed(102)
    qs = [torch.randn((4, 8, 64), generator=g).to(BF).to(DEV) for _ in range(6)]
    ws = fa.paged4_decode_workspace(4, 8, cache)
    nws = fa.qk_norm_rope_backward_workspace(64)
    w = torch.ones(64, device=DEV)

    def norm(x):
        return x.transpose(0, 1)[None].contiguous()
    want = [fa.paged4_decode(q, cache, table, ln)[0].clone() for q in qs]
    grads = [[t.clone() for t in fa.qk_norm_rope_backward(norm(q), None, norm(q * 2), None, w, None)] for q in qs]
    ok()
    buf, out, lse = torch.empty_like(qs[0]), torch.empty_like(qs[0]), torch.empty((4, 8), device=DEV)
    xin, gin, gout, dw = (torch.empty_like(norm(qs[0])) for _ in range(3)), None, None, torch.empty(64, device=DEV)
    xin, gin, gout = xin
    for _ in range(10):
        got, got_grads = [], []
        for q in qs:
            buf.copy_(q)
            fa.paged4_decode(buf, cache, table, ln, out=out, lse=lse, workspace=ws)
            got.append(out.clone())
            buf.fill_(float("nan"))
            out.fill_(float("nan"))
            gin.copy_(norm(q))
            xin.copy_(norm(q * 2))
            fa.qk_norm_rope_backward(gin, None, xin, None, w, None, dq_out=gout, dq_weight=dw, workspace=nws)
            got_grads.append([gout.clone(), dw.clone()])
            for t in (gin, xin, gout, dw):
                t.fill_(float("nan"))
        ok()
        assert same(got, want)
        assert all(same(a, b) for a, b in zip(got_grads, grads))


@pytest.mark.parametrize("seed", range(40))
def test_random_cases(cuda_lib, seed):
    r = np.random.default_rng(1000 + seed)
    dt = [BF, HF][r.integers(2)]
    d, ps = int(r.choice([64, 128])), int(r.choice([16, 32, 48, 64, 256]))
    Hkv = int(r.integers(1, 5))
    Hq = Hkv * int(r.choice([1, 2, 3, 5, 8, 9, 16, 20]))
    B = int(r.integers(1, 9))
    lens = [int(x) if r.random() > 0.15 else 0 for x in r.integers(1, int(r.choice([20, 300, 2500])), size=B)]
    layout = str(r.choice(["hnd", "hpd", "layers"]))
    cache, table, ln, k, v = filled(lens, Hkv, ps, d, dt, seed=seed, layout=layout, sigma=float(r.choice([0.1, 1.0, 3.0])))
    window = int(r.choice([0, 0, r.integers(1, 600)]))
    q = torch.from_numpy(r.normal(size=(B, Hq, d))).to(dt).to(DEV)
    o, lse = fa.paged4_decode(q, cache, table, ln, window=window)
    n = int(r.integers(1, max(lens + [1]) + 10))
    kr, vr = fa.paged4_read(cache, table, ln, n, dt)
    ok()
    assert_decoded(o, lse, q, k, v, lens, d ** -0.5, window, f"seed {seed}")
    assert_read(kr, last_rows(k, lens, n, dt), dt, "k")
    assert_read(vr, last_rows(v, lens, n, dt), dt, "v")


# ---------------------------------------------------------------------------
# Binding
# ---------------------------------------------------------------------------
def test_both_marshallings_make_the_same_calls(cuda_lib, monkeypatch):
    def calls():
        out = []
        for dt in (BF, HF):
            step, _, _ = one_step(dt)
            out += live_rows(step())
            cache, table, ln, k, v = filled([50, 0, 33], 2, 16, 128, dt, seed=111, layout="layers")
            g = torch.Generator().manual_seed(112)
            q = torch.randn((3, 8, 128), generator=g).to(dt).to(DEV)
            out += fa.paged4_decode(q, cache, table, ln, 0.2, 20, torch.empty_like(q), torch.empty((3, 8), device=DEV),
                                    fa.paged4_decode_workspace(3, 8, cache))
            out += fa.paged4_read(cache, table, ln, 7, dt, torch.empty((3, 2, 7, 128), dtype=dt, device=DEV))
            w = weights(g, 128, F32)
            x = q[None]
            out.append(fa.qk_norm_rope(x, None, w, None))
            out.append(fa.qk_norm_rope(x, None, None, None, q_out=torch.empty_like(x)))
            out += fa.qk_norm_rope_backward(x, None, x, None, w, None)
            out += fa.qk_norm_rope_backward(x, x, x, x, w, w, dk_out=torch.empty_like(x), dq_weight=torch.empty_like(w))
            out.append(fa.paged4_append(cache, table, ln, q[:, :2], q[:, 2:4], q=q, eps=1e-6)[[0, 2]])
            out.append(cache)
        ok()
        return out
    assert fa.native_marshalling()
    native = calls()
    monkeypatch.setattr(fa, "_native", fa._NotBuilt)
    python = calls()
    for a, b in zip(native, python):
        assert a.shape == b.shape and a.dtype == b.dtype and torch.equal(a, b)


def test_binding_refusals(marshalling):
    cache, table, ln, k, v = filled([20], 2, 16, 64, BF, seed=121)
    q = torch.zeros((1, 4, 64), dtype=BF, device=DEV)
    w = torch.ones(64, device=DEV)
    x = q[None]
    for error, call in [
        (TypeError, lambda: fa.paged4_decode(q.float(), cache, table, ln)),
        (TypeError, lambda: fa.paged4_decode(q, cache, table.long(), ln)),
        (TypeError, lambda: fa.paged4_decode(q, cache.view(torch.int8), table, ln)),
        (ValueError, lambda: fa.paged4_decode(q, cache, table, ln.expand(2))),
        (ValueError, lambda: fa.paged4_decode(q, cache[..., :64], table, ln)),
        (ValueError, lambda: fa.paged4_decode(q, cache[:, :, ::2], table, ln)),
        (ValueError, lambda: fa.paged4_decode(q.expand(2, 4, 64), cache, table, ln)),
        (fa.FAError, lambda: fa.paged4_decode(q[:, :3], cache, table, ln)),
        (fa.FAError, lambda: fa.paged4_decode(q, cache, table, ln, window=-1)),
        (fa.FAError, lambda: fa.paged4_decode(q, cache, table, ln, out=q)),
        (fa.FAError, lambda: fa.paged4_decode(q, cache, table, ln, scale=-1.0)),
        (fa.FAError, lambda: fa.paged4_decode(q, cache, table, ln, workspace=torch.empty(8, dtype=torch.uint8, device=DEV))),
        (ValueError, lambda: fa.paged4_append(cache, table, ln, q[:, :2].expand(3, 2, 64), q[:, :2].expand(3, 2, 64))),
        (ValueError, lambda: fa.paged4_append(cache, table, ln, q[:, :2], q[:, :2], q=q)),
        (ValueError, lambda: fa.paged4_append(cache, table, ln, q[:, :2], q[:, :2], q=q, q_weight=w)),
        (TypeError, lambda: fa.paged4_append(cache, table, ln, q[:, :2], q[:, :2].half())),
        (fa.FAError, lambda: fa.paged4_append(cache, table, ln, q[:, :2], q[:, :2], q=q, eps=-1.0)),
        (TypeError, lambda: fa.paged4_read(cache, table, ln, 5, torch.float32)),
        (ValueError, lambda: fa.paged4_read(cache, table, ln, 0, BF)),
        (TypeError, lambda: fa.paged4_read(cache, table, ln, 5, BF, torch.empty((1, 2, 5, 64), dtype=HF, device=DEV))),
        (TypeError, lambda: fa.qk_norm_rope(x, None, w.half(), None)),
        (TypeError, lambda: fa.qk_norm_rope(x, x, w, w.to(BF))),
        (ValueError, lambda: fa.qk_norm_rope(x, None, w[:32], None)),
        (ValueError, lambda: fa.qk_norm_rope(x, None, w, w)),
        (ValueError, lambda: fa.qk_norm_rope(x, None, w, None, positions=torch.zeros((1, 1, 4), dtype=torch.int32, device=DEV))),
        (fa.FAError, lambda: fa.qk_norm_rope(x, None, w, None, eps=float("nan"))),
        (fa.FAError, lambda: fa.qk_norm_rope(x, x, w, w, q_out=x, k_out=x)),
        (ValueError, lambda: fa.qk_norm_rope_backward(x, x, x, None, w, None)),
        (ValueError, lambda: fa.qk_norm_rope_backward(x, None, x, None, None, None, dq_weight=torch.empty_like(w))),
        (ValueError, lambda: fa.qk_norm_rope_backward(x[:, :, :2], None, x, None, w, None)),
        (fa.FAError, lambda: fa.qk_norm_rope_backward(x, None, x.clone(), None, w, None, dq_weight=w)),
    ]:
        with pytest.raises(error):
            call()
    ok()


def test_one_key_and_odd_scale_types(marshalling):
    cache, table, ln, k, v = filled([1], 1, 16, 64, HF, seed=131)
    q = torch.randn((1, 2, 64), device=DEV).to(HF)
    a = fa.paged4_decode(q, cache, table, ln, scale=1)
    b = fa.paged4_decode(q, cache, table, ln, scale=np.float32(1.0))
    ok()
    assert same(a, b)
    assert_decoded(*a, q, k, v, [1], 1.0, 0)

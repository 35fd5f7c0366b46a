"""GPU parity of rotary positions, paged append, paged one-token attention and
eviction against the fp64 oracle, through the Python binding.

Tolerances (u = half a step of the tensors' type: bf16 2^-8, fp16 2^-11).

Rotation: |out - ref| <= u |ref| + c (|x| + |y|) + tiny, where c bounds the fp32
part: the angle, at most pi, is rounded by its conversion, its scaling and the
scale's constant (3 pi 2^-24 = 5.6e-7), its sine or cosine is off by 2^-21.2 =
4.2e-7, and two products and a sum round by 3 2^-24 = 1.8e-7: 1.2e-6.  The
rounding of a value that is off by e is off by at most u (|ref| + e) + e <
u |ref| + 1.01 e, so c = 2e-6 holds; tiny is the fp16 subnormal step.

Attention: with A = sum p |v| (from the oracle) the weights are applied
rounded to the tensors' type (u A), o is rounded once (u |o|), and a relative
error e of each weight moves o by at most 2 e A (numerator and denominator).
e: a score is a sum of d products in fp32 (d 2^-23 relative to scale sum |q k|,
the factor 2 for adders that truncate), rounded by its scaling (2^-23), its
exponential by 2^-22, and sums over n keys by n 2^-24.  lse is off by e, the
accumulated weights by 2 e of themselves; an fp32 weight below 2^-126 is a
subnormal or 0, so each of the G weights of a key is off by at most 2^-126
more.  scale sum |q k| <= X = scale |q|_2
max |k|_2.
"""
import math

import numpy as np
import pytest
import torch

import exact_io_aware_flashattention_gb300 as fa
from oracle import paged, ref
from tests.parity import GRAD_REL_L2, GuardedBuffers, rel_l2

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
BF, HF = torch.bfloat16, torch.float16


def f64(t):
    return t.detach().double().cpu().numpy()


def ok():
    torch.cuda.synchronize()
    fa.check_device_status()


# ---------------------------------------------------------------------------
# Rotary positions
# ---------------------------------------------------------------------------
def rotation_bound(x, ref, r, interleaved, dt):
    pair = np.abs(f64(x))
    size = np.zeros_like(ref)
    lo, hi = (np.arange(0, 2 * r, 2), np.arange(1, 2 * r, 2)) if interleaved else (np.arange(r), np.arange(r, 2 * r))
    s = pair[..., lo] + pair[..., hi]
    size[..., lo], size[..., hi] = s, s
    return U[dt] * np.abs(ref) + 2e-6 * size + (2.0 ** -24 if dt == HF else 0.0)


def assert_rotated(out, x, pos, w, axes, interleaved, inverse, what):
    ref = paged.rotate(f64(x), pos.cpu().numpy(), w.cpu().numpy(), axes.cpu().numpy(), interleaved, inverse)
    err = np.abs(f64(out) - ref)
    off = err > rotation_bound(x, ref, w.numel(), interleaved, out.dtype)
    assert not off.any(), f"{what}: {off.sum()} values, {err.max()}"


ROPE = [
    # B, Hq, Hk, N, d, sections, interleaved, first position, dtype
    (1, 1, 0, 1, 64, (32,), False, 0, BF),
    (2, 4, 2, 33, 128, (16, 24, 24), False, 0, BF),
    (1, 3, 1, 257, 128, (20, 12), True, 5, HF),
    (3, 5, 5, 7, 64, (8,), False, 10 ** 6, HF),            # partial, far
    (1, 2, 1, 40, 64, (8, 0, 8), True, 2 ** 31 - 100, BF), # an axis without pairs, the last positions
    (1, 2, 2, 65, 256, (64, 64), False, -30, BF),          # negative positions
    (2, 9, 3, 19, 16, (8,), False, 3, HF),
    (1, 32, 8, 300, 80, (40,), False, 3, BF),              # d not a power of two
    (1, 6, 6, 50, 96, (16,), True, 77, BF),
]


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("B,Hq,Hk,N,d,sections,interleaved,start,dt", ROPE)
def test_rope(cuda_lib, B, Hq, Hk, N, d, sections, interleaved, start, dt, inverse):
    g = torch.Generator().manual_seed(N * d + Hq)
    q = torch.randn((B, Hq, N, d), generator=g).to(dt).to(DEV)
    k = torch.randn((B, Hk, N, d), generator=g).to(dt).to(DEV) if Hk else None
    A = len(sections)
    pos = (start + torch.randint(0, 60, (A, B, N), generator=g)).to(torch.int32).to(DEV)
    w, axes = fa.rope_frequencies(sections, device=DEV)
    gb = GuardedBuffers(DEV)
    turn = fa.rope_backward if inverse else fa.rope
    qo = gb.empty((B, Hq, N, d), dt)
    if k is None:
        assert turn(q, None, pos, w, axes, interleaved, qo) is qo
    else:
        ko = gb.empty((B, Hk, N, d), dt)
        turn(q, k, pos, w, axes, interleaved, qo, ko)
    ok()
    gb.check()
    assert_rotated(qo, q, pos, w, axes, interleaved, inverse, "q")
    r = 2 * w.numel()
    assert torch.equal(qo[..., r:], q[..., r:])
    if k is not None:
        assert_rotated(ko, k, pos, w, axes, interleaved, inverse, "k")


@pytest.mark.parametrize("layout", ["token-major", "head-major"])
def test_rope_in_place_on_a_projection(cuda_lib, layout):
    B, Hq, Hk, N, d = 2, 4, 2, 37, 64
    g = torch.Generator().manual_seed(3)
    x = torch.randn((B, Hq + 2 * Hk, N, d), generator=g).to(BF).to(DEV)
    if layout == "token-major":
        x = x.transpose(1, 2).contiguous().transpose(1, 2)      # [B, N, H, d] in memory
    before = x.clone()
    q, k, v = x.split([Hq, Hk, Hk], dim=1)
    pos = torch.arange(N, dtype=torch.int32, device=DEV).expand(1, B, N)
    w, axes = fa.rope_frequencies((32,), device=DEV)
    fa.rope(q, k, pos, w, axes, q_out=q, k_out=k)
    ok()
    q0, k0, v0 = before.split([Hq, Hk, Hk], dim=1)
    assert_rotated(q, q0, pos, w, axes, False, False, "q")
    assert_rotated(k, k0, pos, w, axes, False, False, "k")
    assert torch.equal(v, v0)


def test_rope_gradient_is_the_transpose(cuda_lib):
    # <g, R x> = <R^T g, x> with R x and R^T g from the kernels, and the
    # backward of the forward gives x back.
    g = torch.Generator().manual_seed(4)
    x, y = (torch.randn((1, 3, 50, 128), generator=g).to(HF).to(DEV) for _ in range(2))
    pos = torch.randint(0, 10 ** 6, (3, 1, 50), generator=g).to(torch.int32).to(DEV)
    w, axes = fa.rope_frequencies((16, 24, 24), device=DEV)
    fx, by = fa.rope(x, None, pos, w, axes), fa.rope_backward(y, None, pos, w, axes)
    ok()
    lhs, rhs = float((f64(y) * f64(fx)).sum()), float((f64(by) * f64(x)).sum())
    size = float(np.abs(f64(y) * f64(fx)).sum() + np.abs(f64(by) * f64(x)).sum())
    assert abs(lhs - rhs) <= (U[HF] + 4e-6) * size
    back = fa.rope_backward(fx, None, pos, w, axes)
    ok()
    # Two roundings of values at most |x| + |y| each.
    assert (back.float() - x.float()).abs().max().item() <= 4 * U[HF] * 2 * x.float().abs().max().item()


@pytest.mark.parametrize("deterministic", [False, True])
def test_rope_in_a_training_step(cuda_lib, deterministic):
    # rope, attention, its backward, rope_backward: gradients of the unturned q
    # and k against the oracle from the same turned tensors.
    B, Hq, Hk, N, d = 1, 4, 2, 300, 64
    g = torch.Generator().manual_seed(11)
    q, k, v, do = (torch.randn((B, h, N, d), generator=g).to(BF).to(DEV) for h in (Hq, Hk, Hk, Hq))
    pos = torch.stack([torch.arange(N) // 100, torch.arange(N) // 10 % 10, torch.arange(N) % 10]).to(torch.int32)
    pos = pos[:, None].expand(3, B, N).to(DEV)
    w, axes = fa.rope_frequencies((8, 12, 12), device=DEV)
    qr, kr = fa.rope(q, k, pos, w, axes)
    o, lse = fa.forward(qr, kr, v, causal=True)
    dqr, dkr, dv = fa.backward(qr, kr, v, o, lse, do, causal=True, deterministic=deterministic)
    dq, dk = fa.rope_backward(dqr, dkr, pos, w, axes)
    ok()
    rq, rk, rv = ref.attention_backward(f64(qr), f64(kr), f64(v), f64(do), True, d ** -0.5)
    turn_back = lambda x: paged.rotate(x, pos.cpu().numpy(), w.cpu().numpy(), axes.cpu().numpy(), inverse=True)  # noqa: E731
    # A rotation keeps norms, so the attention's tolerance carries over; the
    # rotated gradients are rounded once more.
    for got, want, name in ((dq, turn_back(rq), "dq"), (dk, turn_back(rk), "dk"), (dv, rv, "dv")):
        assert rel_l2(f64(got), want) <= GRAD_REL_L2 + U[BF], name


def test_rope_bad_axis_is_recorded(cuda_lib):
    q = torch.randn((1, 1, 4, 64), device=DEV).to(BF)
    w, axes = fa.rope_frequencies((32,), device=DEV)
    axes[5] = 1
    fa.rope(q, None, torch.zeros((1, 1, 4), dtype=torch.int32, device=DEV), w, axes)
    s, _ = fa.fa_last_device_status()
    assert s == fa.FA_ERR_BAD_INDEX
    ok()


# ---------------------------------------------------------------------------
# Paged cache
# ---------------------------------------------------------------------------
def new_pool(pages, Hkv, ps, d, dt, layout="hnd", fill=float("nan")):
    """k and v caches [pages, Hkv, ps, d] in one of several memory orders."""
    if layout == "hnd":
        k, v = (torch.full((pages, Hkv, ps, d), fill, dtype=dt, device=DEV) for _ in range(2))
    elif layout == "nhd":
        k, v = (torch.full((pages, ps, Hkv, d), fill, dtype=dt, device=DEV).transpose(1, 2) for _ in range(2))
    else:                                                        # k and v page by page
        x = torch.full((pages, 2, Hkv, ps, d), fill, dtype=dt, device=DEV)
        k, v = x[:, 0], x[:, 1]
    return k, v


def filled(lens, Hkv, ps, d, dt, seed, layout="hnd", extra=2, sigma=1.0, share=False):
    """A cache holding sequences of these lengths; every other slot is NaN, and
    block table columns past a sequence's pages are far out of range."""
    g = torch.Generator().manual_seed(seed)
    n = [-(-x // ps) for x in lens]
    total = sum(n) + extra
    k, v = new_pool(total, Hkv, ps, d, dt, layout)
    order = torch.randperm(total, generator=g).tolist()
    table = torch.full((len(lens), max(1, max(n)) + 1), 2 ** 30, dtype=torch.int32)
    at = 0
    for b, x in enumerate(lens):
        table[b, :n[b]] = torch.tensor(order[at:at + n[b]], dtype=torch.int32)
        at += n[b]
        for j in range(n[b]):
            m = min(ps, x - j * ps)
            k[table[b, j].item(), :, :m] = (sigma * torch.randn((Hkv, m, d), generator=g)).to(dt).to(DEV)
            v[table[b, j].item(), :, :m] = torch.randn((Hkv, m, d), generator=g).to(dt).to(DEV)
    return k, v, table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)


def assert_decoded(o, lse, q, k, v, table, lens, scale, window, scores=None, before=None, what=""):
    dt, d = o.dtype, q.shape[-1]
    kn, vn, tb, ln = f64(k), f64(v), table.cpu().numpy(), lens.cpu().numpy()
    ro, rl, rw, a = paged.decode(f64(q), kn, vn, tb, ln, scale, window)
    seen = max(1, int(ln.max()))
    big = np.sqrt(np.nanmax((np.where(np.isnan(kn), 0, kn) ** 2).sum(-1))) * np.sqrt((f64(q) ** 2).sum(-1).max())
    e = scale * big * (d * 2.0 ** -23 + 2.0 ** -23) + 2.0 ** -21 + seen * 2.0 ** -24
    err = np.abs(f64(o) - ro)
    bound = U[dt] * (a + np.abs(ro)) + 2.1 * e * a + (2.0 ** -24 if dt == HF else 0.0)
    if dt == HF:
        bound = bound + 2.0 ** -25 * seen * np.nanmax(np.abs(vn))      # weights below fp16's normal range
    worst = (err / np.maximum(bound, 1e-30)).max()
    assert worst <= 1, f"{what}: o off by {worst} of the bound"
    fine = np.isfinite(rl)
    gl = f64(lse)
    assert np.array_equal(np.isneginf(gl), ~fine), what
    far = np.abs(gl[fine] - rl[fine]) > e + 2.0 ** -23 * np.abs(rl[fine])
    assert not far.any(), f"{what}: {far.sum()} lse"
    if scores is not None:
        ps = k.shape[2]
        want = f64(before)
        for b, n in enumerate(ln):
            for j in range(n):
                want[tb[b, j // ps], :, j % ps] += rw[b][:, j]
        got = f64(scores)
        grown = np.abs(want - f64(before))
        least = q.shape[1] // k.shape[1] * 2.0 ** -126
        off = np.abs(got - want) > 2.1 * e * grown + 2.0 ** -23 * np.abs(want) + least
        assert not off.any(), f"{what}: {off.sum()} scores"


DECODE = [
    # lens, Hq, Hkv, d, page, window, dtype, layout
    ([1], 1, 1, 64, 16, 0, BF, "hnd"),
    ([0], 4, 2, 128, 16, 0, BF, "hnd"),
    ([15, 16, 17, 0, 31, 33], 8, 2, 128, 16, 0, BF, "hnd"),
    ([63, 64, 65, 127, 128, 129], 4, 4, 64, 32, 0, HF, "nhd"),
    ([1000, 1, 0, 777], 6, 2, 128, 48, 0, BF, "pair"),        # page 48, three heads a group
    ([2500, 300], 8, 1, 64, 64, 0, HF, "hnd"),
    ([700, 130, 50], 9, 1, 128, 16, 0, BF, "nhd"),            # nine heads a group
    ([500, 90], 32, 2, 64, 128, 0, BF, "hnd"),                # sixteen
    ([333, 64], 17, 1, 128, 16, 0, HF, "pair"),
    ([260, 65], 33, 1, 64, 16, 0, BF, "hnd"),
    ([150], 72, 1, 128, 32, 0, BF, "hnd"),
    ([1000, 5, 0, 64], 8, 2, 128, 16, 1, BF, "hnd"),
    ([1000, 100, 65], 8, 4, 64, 16, 64, HF, "hnd"),
    ([1000, 257, 3], 4, 2, 128, 80, 250, BF, "nhd"),
    ([400, 60], 4, 2, 128, 16, 10 ** 9, BF, "hnd"),
    ([10000], 2, 1, 128, 256, 0, BF, "hnd"),
]


@pytest.mark.parametrize("with_scores", [False, True])
@pytest.mark.parametrize("lens,Hq,Hkv,d,page,window,dt,layout", DECODE)
def test_decode(cuda_lib, lens, Hq, Hkv, d, page, window, dt, layout, with_scores):
    k, v, table, ln = filled(lens, Hkv, page, d, dt, seed=Hq * 100 + d, layout=layout)
    B = len(lens)
    g = torch.Generator().manual_seed(9)
    proj = torch.randn((B, Hq + 3, d), generator=g).to(dt).to(DEV)
    q = proj[:, 1:Hq + 1]                                            # strided rows
    gb = GuardedBuffers(DEV)
    o, lse = gb.empty((B, Hq, d), dt), gb.empty((B, Hq), torch.float32)
    ws = gb.empty((fa.paged_decode_workspace(B, Hq, k, table, with_scores).numel(),), torch.uint8)
    scores = before = None
    if with_scores:
        scores = gb.empty(tuple(k.shape[:3]), torch.float32)
        scores.copy_(torch.rand(k.shape[:3], generator=g))
        before = scores.clone()
    scale = 0.11
    fa.paged_decode(q, k, v, table, ln, scale=scale, window=window, scores=scores, out=o, lse=lse, workspace=ws)
    ok()
    gb.check()
    assert_decoded(o, lse, q, k, v, table, ln, scale, window, scores, before, f"{lens}")


def spread(B, longest, seed):
    """Lengths of a batch: some empty, some of one key, the rest anything."""
    g = torch.Generator().manual_seed(seed)
    return [[0, 1, int(x)][int(p)] if p < 2 else int(x)
            for x, p in zip(torch.randint(1, longest + 1, (B,), generator=g), torch.randint(0, 12, (B,), generator=g))]


@pytest.mark.parametrize("with_scores", [False, True])
@pytest.mark.parametrize("B,longest,Hq,Hkv,d,page,window,dt", [
    (40, 900, 8, 4, 128, 16, 0, BF),        # several tiles a CTA, units cut in two
    (24, 900, 16, 8, 64, 32, 0, HF),
    (30, 700, 16, 1, 128, 48, 0, BF),       # sixteen heads a group
    (16, 900, 40, 2, 64, 16, 200, BF),      # two head chunks, a window
    (161, 60, 2, 1, 64, 16, 0, BF),         # one sequence more than a block has threads
    (700, 70, 2, 2, 64, 16, 0, HF),
])
def test_decode_batches(cuda_lib, B, longest, Hq, Hkv, d, page, window, dt, with_scores):
    lens = spread(B, longest, seed=B)
    k, v, table, ln = filled(lens, Hkv, page, d, dt, seed=B + 1)
    g = torch.Generator().manual_seed(B + 2)
    q = torch.randn((B, Hq, d), generator=g).to(dt).to(DEV)
    scores = torch.rand(k.shape[:3], generator=g).to(DEV) if with_scores else None
    before = scores.clone() if with_scores else None
    o, lse = fa.paged_decode(q, k, v, table, ln, window=window, scores=scores)
    ok()
    assert_decoded(o, lse, q, k, v, table, ln, d ** -0.5, window, scores, before, f"batch of {B}")


@pytest.mark.parametrize("sigma,scale", [(4.0, 0.3), (0.0, 1.0)])
def test_decode_peaked_and_flat(cuda_lib, sigma, scale):
    # Scores of +-50 and more: single keys dominate and the running maximum
    # keeps moving; and all scores equal.
    k, v, table, ln = filled([900, 64, 300], 2, 16, 64, HF, seed=5, sigma=sigma)
    q = (4.0 * torch.randn((3, 8, 64), generator=torch.Generator().manual_seed(6))).to(HF).to(DEV)
    scores = torch.zeros(k.shape[:3], device=DEV)
    o, lse = fa.paged_decode(q, k, v, table, ln, scale=scale, scores=scores)
    ok()
    assert_decoded(o, lse, q, k, v, table, ln, scale, 0, scores, torch.zeros_like(scores), f"sigma {sigma}")


def test_decode_rising_scores(cuda_lib):
    # Each tile's scores exceed the last one's by far, then fall again: the
    # running maximum moves at every step.
    n, d = 640, 64
    k, v, table, ln = filled([n], 1, 16, d, BF, seed=8)
    step = torch.cat([torch.arange(20), torch.arange(20).flip(0)]) * 2.0
    for j in range(n // 16):
        k[table[0, j].item(), 0, :, 0] = step[j].item()
    q = torch.randn((1, 4, d), generator=torch.Generator().manual_seed(7))
    q[:, :, 0] = torch.tensor([8.0, -8.0, 4.0, 16.0])
    q = q.to(BF).to(DEV)
    scores = torch.zeros(k.shape[:3], device=DEV)
    o, lse = fa.paged_decode(q, k, v, table, ln, scale=0.5, scores=scores)
    ok()
    assert_decoded(o, lse, q, k, v, table, ln, 0.5, 0, scores, torch.zeros_like(scores), "rising")


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("gap", [12.0, 17.5, 20.0])
def test_decode_many_small_weights(cuda_lib, dt, gap):
    # One key of score `gap` and value 1, all others of score 0 and value 3000:
    # weights of e^-17.5 = 2^-25.2 are below what fp16 holds next to 1, and yet
    # 4000 of them carry a quarter of the result.
    n, d = 4000, 64
    k, v, table, ln = filled([n], 1, 64, d, dt, seed=18)
    k.zero_()
    v.fill_(3000.0)
    p, s = table[0, 20].item(), 7
    k[p, 0, s, 0] = gap
    v[p, 0, s] = 1.0
    q = torch.zeros((1, 2, d), dtype=dt, device=DEV)
    q[:, :, 0] = 1.0
    o, lse = fa.paged_decode(q, k, v, table, ln, scale=1.0)
    ok()
    w = n * math.exp(-gap)
    want = (1.0 + (w - math.exp(-gap)) * 3000.0) / (1.0 + w - math.exp(-gap))
    # The weights' and the result's rounding, and fp32 sums of n terms.
    assert (o.double() / want - 1).abs().max().item() <= 2.1 * U[dt] + n * 2.0 ** -23
    assert abs(lse[0, 0].item() - math.log(math.exp(gap) + n - 1)) <= n * 2.0 ** -24 + 2.0 ** -20


@pytest.mark.parametrize("B,Hq,Hkv,d,longest,dt", [
    (3000, 8, 8, 128, 16, BF),
    (1500, 16, 4, 128, 40, HF),
    (1200, 32, 2, 128, 16, BF),             # sixteen heads a group
    (2000, 8, 4, 64, 16, HF),
    (1000, 20, 2, 64, 30, BF),
])
def test_decode_many_units_of_one_tile(cuda_lib, B, Hq, Hkv, d, longest, dt):
    # Dozens of units in a row for each CTA, most of them of one 16-key slice,
    # so that three of its four warps have nothing to do between one unit's sums
    # and the next's: each unit's statistics stay apart, in every run alike.
    lens = torch.randint(0, longest + 1, (B,), generator=torch.Generator().manual_seed(B)).tolist()
    k, v, table, ln = filled(lens, Hkv, 16, d, dt, seed=B + 1, sigma=3.0)
    q = torch.randn((B, Hq, d), generator=torch.Generator().manual_seed(B + 2)).to(dt).to(DEV)
    o, lse = fa.paged_decode(q, k, v, table, ln, scale=0.2)
    again = [fa.paged_decode(q, k, v, table, ln, scale=0.2) for _ in range(30)]
    ok()
    assert_decoded(o, lse, q, k, v, table, ln, 0.2, 0, what=f"{B} short sequences")
    for o2, l2 in again:
        assert torch.equal(o, o2) and torch.equal(lse, l2)


# Weights at more than the tensors' precision.  q and k are small integers, so
# the scores are exact in fp32 whatever the order of the sums, and with n keys
# of scores |x| <= X (log2 units) what is left of the error of o, relative to A =
# sum p |v|, is:
#   the weights as two values of the tensors' type, the first rounded down (off
#     by up to 2 u), the second to nearest: 2 u^2 (fp16: and half a subnormal
#     step, 2^-25, next to a largest weight of 2^12, so 2^-37 of max |v| for
#     each key);
#   x: two roundings of at most X 2^-24 in its scaling and one of 2 X 2^-24 in
#     its difference to the maximum; 2^x to 2^-22, again for each of R
#     rescalings of a key's weight on its way to the sum; each twice (numerator
#     and denominator);
#   sums of n terms in fp32 that truncate, of O and l: n 2^-23 each; the last
#     product and quotient 2^-22.
@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("lens,Hq,Hkv,d,wide", [
    ([50, 64, 37], 8, 2, 128, False),                     # in clusters
    ([50, 64, 37], 8, 2, 128, True),                      # in equal parts
    ([60, 33], 4, 4, 64, True),
    ([64, 3, 41], 16, 1, 128, True),                      # sixteen heads a group
    ([64, 17], 12, 1, 64, False),
])
def test_decode_weights_are_finer_than_the_tensors_type(cuda_lib, lens, Hq, Hkv, d, wide, dt):
    n, scale = max(lens), 2.0 ** -5
    k, v, table, ln = filled(lens, Hkv, 16, d, dt, seed=41)
    g = torch.Generator().manual_seed(42)
    k.copy_(torch.where(k.isnan().cpu(), torch.nan, torch.randint(-2, 3, k.shape, generator=g).float()))
    q = torch.randint(-2, 3, (len(lens), Hq, d), generator=g).to(dt).to(DEV)
    o, _ = fa.paged_decode(q, k, v, widened(table, 1 << 15, 16) if wide else table, ln, scale=scale)
    ok()
    kn, vn = f64(k), f64(v)
    ro, _, _, a = paged.decode(f64(q), kn, vn, table.cpu().numpy(), ln.cpu().numpy(), scale, 0)
    X = 1.4427 * scale * d * 4
    R = 8                                                 # tiles of a warp, its warps, CTAs: few keys, so few
    e = math.log(2) * X * 2.0 ** -22 + (1 + R) * 2.0 ** -22
    rel = 2 * U[dt] ** 2 + 2 * e + 2 * n * 2.0 ** -23 + 2.0 ** -22
    floor = 2.0 ** -37 * n * np.nanmax(np.abs(vn)) + 2.0 ** -25 if dt == HF else 0.0
    bound = U[dt] * np.abs(ro) + 1.01 * rel * a + floor
    worst = (np.abs(f64(o) - ro) / bound).max()
    assert worst <= 1, f"off by {worst} of the bound"


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("wide", [False, True])
def test_decode_infinite_values(cuda_lib, wide, dt):
    # An infinite v under a positive weight, be it a power of two (the largest)
    # or any other, gives an infinite o; two of opposite sign, or a NaN, NaN.
    k, v, table, ln = filled([70, 33], 2, 16, 64, dt, seed=43)
    flat = lambda b, j: (table[b, j // 16].item(), slice(None), j % 16)  # noqa: E731
    q = torch.randn((2, 4, 64), generator=torch.Generator().manual_seed(44)).to(dt).to(DEV)
    for j in range(70):
        v[flat(0, j)][:, j % 64] = (math.inf, -math.inf)[j // 32 % 2]      # 64 .. 69 meet 0 .. 5, of the same sign
    v[flat(1, 5)][:, 7] = math.inf
    v[flat(1, 6)][:, 7] = -math.inf
    v[flat(1, 7)][:, 9] = math.nan
    o, lse = fa.paged_decode(q, k, v, widened(table, 1 << 15, 16) if wide else table, ln)
    ok()
    assert bool((o[0, :, :32] == math.inf).all()) and bool((o[0, :, 32:] == -math.inf).all())
    assert bool(o[1, :, [7, 9]].isnan().all())
    rest = [i for i in range(64) if i not in (7, 9)]
    assert bool(o[1, :, rest].isfinite().all()) and bool(lse.isfinite().all())


def test_decode_pages_shared_by_sequences(cuda_lib):
    # Two sequences with a common prefix: the weights of both add up.
    k, v, table, ln = filled([200, 200], 2, 16, 64, BF, seed=12)
    table[1, :6] = table[0, :6]
    ln[1] = 150
    q = torch.randn((2, 4, 64), generator=torch.Generator().manual_seed(1)).to(BF).to(DEV)
    scores = torch.zeros(k.shape[:3], device=DEV)
    o, lse = fa.paged_decode(q, k, v, table, ln, scores=scores)
    ok()
    assert_decoded(o, lse, q, k, v, table, ln, 0.125, 0, scores, torch.zeros_like(scores), "shared")


def test_decode_is_reproducible_and_independent_of_the_rest_of_the_batch(cuda_lib):
    k, v, table, ln = filled([3000, 70, 1200, 0, 16], 2, 16, 128, BF, seed=13)
    q = torch.randn((5, 8, 128), generator=torch.Generator().manual_seed(2)).to(BF).to(DEV)
    o1, l1 = fa.paged_decode(q, k, v, table, ln)
    o2, l2 = fa.paged_decode(q, k, v, table, ln)
    ok()
    assert torch.equal(o1, o2) and torch.equal(l1, l2)


@pytest.mark.parametrize("dt", [BF, HF])
def test_decode_alone_and_within_a_batch(cuda_lib, dt):
    # Another batch cuts a sequence's keys elsewhere, so the sums have another
    # order: equal within twice the bound of one of them, not bit by bit.
    lens = [3000, 70, 1200, 0, 16, 900]
    k, v, table, ln = filled(lens, 2, 16, 128, dt, seed=46)
    q = torch.randn((len(lens), 8, 128), generator=torch.Generator().manual_seed(47)).to(dt).to(DEV)
    o, lse = fa.paged_decode(q, k, v, table, ln)
    ok()
    assert_decoded(o, lse, q, k, v, table, ln, 128 ** -0.5, 0, what="together")
    for b in range(len(lens)):
        i = slice(b, b + 1)
        o1, l1 = fa.paged_decode(q[i], k, v, table[i], ln[i])
        ok()
        assert_decoded(o1, l1, q[i], k, v, table[i], ln[i], 128 ** -0.5, 0, what=f"sequence {b} alone")
        # The scores are the same ones. On either side o is rounded once, the
        # weights are off by 2 u^2, and the sums of n terms of O and l by n 2^-23
        # of sum p |v| <= max |v| each; rescalings, one for 16 keys or more, by
        # 2^-22 each: less than the sums.
        n, top = lens[b], float(torch.nan_to_num(v.float()).abs().max())
        far = (o1.float() - o[i].float()).abs()
        assert bool((far <= 2 * U[dt] * o[i].float().abs() + 4 * (n * 2.0 ** -23 + 2 * U[dt] ** 2) * top).all())
        assert torch.equal(torch.isneginf(l1), torch.isneginf(lse[i]))


def widened(table, keys, page):
    """The table with columns, far out of range, for this many keys a sequence."""
    wide = torch.full((table.shape[0], -(-keys // page)), 2 ** 30, dtype=torch.int32, device=table.device)
    wide[:, :table.shape[1]] = table
    return wide


SHORT = [
    # lens, Hq, Hkv, d, page, window, dtype: units a cluster takes, shared by 8, 4, 2 or 1 CTAs
    ([0], 2, 1, 64, 16, 0, BF),
    ([1], 3, 1, 128, 16, 0, HF),
    ([640], 8, 2, 128, 16, 0, BF),                            # more tiles than CTAs
    ([511, 3, 0, 129, 64], 8, 2, 128, 16, 0, HF),             # CTAs without a tile, and whole clusters
    ([900, 0, 257, 128], 16, 1, 64, 48, 0, BF),               # sixteen heads a group
    ([700, 65], 40, 2, 128, 16, 0, HF),                       # two chunks, the second not full
    ([1500, 1000, 100], 13, 1, 64, 64, 300, BF),              # a window, so other tiles than the first
    ([2000, 10], 4, 4, 128, 256, 1, HF),
    (list(range(0, 800, 37)), 8, 2, 64, 16, 0, HF),           # 44 units: four CTAs
    (list(range(0, 600, 15)), 8, 2, 128, 16, 0, BF),          # 80 units: two
    (list(range(0, 400, 4)), 6, 2, 64, 32, 0, BF),            # 200 units: one
    (list(range(0, 170)), 4, 2, 128, 16, 0, HF),              # 340 units: more than run at a time
]


@pytest.mark.parametrize("lens,Hq,Hkv,d,page,window,dt", SHORT)
def test_decode_by_clusters_and_by_equal_parts(cuda_lib, lens, Hq, Hkv, d, page, window, dt):
    k, v, table, ln = filled(lens, Hkv, page, d, dt, seed=len(lens) + Hq, layout="nhd" if page > 32 else "hnd")
    q = torch.randn((len(lens), Hq, d), generator=torch.Generator().manual_seed(4)).to(dt).to(DEV)
    gb = GuardedBuffers(DEV)
    o, lse = gb.empty((len(lens), Hq, d), dt), gb.empty((len(lens), Hq), torch.float32)
    for t in (table, widened(table, 1 << 15, page)):
        o.fill_(float("nan"))
        lse.fill_(float("nan"))
        fa.paged_decode(q, k, v, t, ln, window=window, out=o, lse=lse)
        ok()
        gb.check()
        assert_decoded(o, lse, q, k, v, t, ln, d ** -0.5, window, what=f"{t.shape[1]} columns")
        o2, l2 = fa.paged_decode(q, k, v, t, ln, window=window)
        assert torch.equal(o, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("lens,Hq,Hkv,d,page,window,dt", SHORT)
def test_scores_by_clusters_and_by_equal_parts(cuda_lib, lens, Hq, Hkv, d, page, window, dt):
    k, v, table, ln = filled(lens, Hkv, page, d, dt, seed=len(lens) + Hq + 1, layout="nhd" if page > 32 else "hnd")
    g = torch.Generator().manual_seed(5)
    q = torch.randn((len(lens), Hq, d), generator=g).to(dt).to(DEV)
    before = torch.rand(k.shape[:3], generator=g).to(DEV)
    gb = GuardedBuffers(DEV)
    scores = gb.empty(tuple(k.shape[:3]), torch.float32)
    for t in (table, widened(table, 1 << 15, page)):
        ws = gb.empty((fa.paged_decode_workspace(len(lens), Hq, k, t, True).numel(),), torch.uint8)
        scores.copy_(before)
        o, lse = fa.paged_decode(q, k, v, t, ln, window=window, scores=scores, workspace=ws)
        ok()
        gb.check()
        assert_decoded(o, lse, q, k, v, t, ln, d ** -0.5, window, scores, before, f"{t.shape[1]} columns")
        again = before.clone()
        o2, l2 = fa.paged_decode(q, k, v, t, ln, window=window, scores=again, workspace=ws)
        assert torch.equal(o, o2) and torch.equal(lse, l2) and torch.equal(scores, again)


@pytest.mark.parametrize("bad", ["page", "negative page", "length", "negative length"])
def test_decode_by_clusters_records_bad_indices(cuda_lib, bad):
    lens = [400, 300, 50]
    k, v, table, ln = filled(lens, 2, 16, 128, HF, seed=15)
    q = torch.randn((3, 4, 128), generator=torch.Generator().manual_seed(3)).to(HF).to(DEV)
    good_o, good_l = fa.paged_decode(q, k, v, table, ln)
    ok()
    t2, n2 = table.clone(), ln.clone()
    if bad.endswith("page"):
        t2[1, 3] = -1 if bad.startswith("neg") else k.shape[0]
    else:
        n2[1] = -5 if bad.startswith("neg") else table.shape[1] * 16 + 1
    o, l = fa.paged_decode(q, k, v, t2, n2)
    s, _ = fa.fa_last_device_status()
    assert s == fa.FA_ERR_BAD_INDEX
    for b in (0, 2):                                      # a cluster does not see the other sequences
        assert torch.equal(o[b], good_o[b]) and torch.equal(l[b], good_l[b])
    ok()


@pytest.mark.parametrize("bad", ["page", "negative page", "length", "negative length"])
def test_decode_bad_indices_are_recorded(cuda_lib, bad):
    lens = [100, 200, 50]
    k, v, table, ln = filled(lens, 2, 16, 64, BF, seed=14)
    q = torch.randn((3, 4, 64), generator=torch.Generator().manual_seed(3)).to(BF).to(DEV)
    good_o, good_l = fa.paged_decode(q, k, v, table, ln)
    ok()
    t2, n2 = table.clone(), ln.clone()
    if bad.endswith("page"):
        t2[1, 3] = -1 if bad.startswith("neg") else k.shape[0]
    else:
        n2[1] = -5 if bad.startswith("neg") else table.shape[1] * 16 + 1
    scores = torch.zeros(k.shape[:3], device=DEV)
    o, l = fa.paged_decode(q, k, v, t2, n2, scores=scores)
    s, _ = fa.fa_last_device_status()
    assert s == fa.FA_ERR_BAD_INDEX
    for b in (0, 2):                                      # the other sequences are as before, up to the split's rounding
        assert (o[b].float() - good_o[b].float()).abs().max().item() <= 0.05
        assert (l[b] - good_l[b]).abs().max().item() <= 1e-3
    ok()


def test_decode_offsets_past_32_bits(cuda_lib):
    # Element offsets past 2^31 in the pool, and past 2^32 bytes.
    Hkv, ps, d = 8, 64, 128
    pages = 2 ** 31 // (Hkv * ps * d) + 40
    k = torch.empty((pages, Hkv, ps, d), dtype=BF, device=DEV)
    v = torch.empty_like(k)
    g = torch.Generator().manual_seed(15)
    use = [pages - 1, 3, pages - 20, pages // 2 + 7]
    for p in use:
        k[p] = torch.randn((Hkv, ps, d), generator=g).to(BF).to(DEV)
        v[p] = torch.randn((Hkv, ps, d), generator=g).to(BF).to(DEV)
    table = torch.tensor([use], dtype=torch.int32, device=DEV)
    ln = torch.tensor([250], dtype=torch.int32, device=DEV)
    q = torch.randn((1, 16, d), generator=g).to(BF).to(DEV)
    scores = torch.zeros((pages, Hkv, ps), device=DEV)
    # The new token's row lands at the far end too.
    kn, vn = (torch.randn((1, Hkv, d), generator=g).to(BF).to(DEV) for _ in range(2))
    use2 = torch.tensor([use[::-1]], dtype=torch.int32, device=DEV)
    fa.paged_append(k, v, use2, ln, kn, vn, scores=scores)
    o, lse = fa.paged_decode(q, k, v, use2, ln, scores=scores)
    dst = torch.tensor([[pages - 2, pages - 3]], dtype=torch.int32, device=DEV)
    nl, kept = fa.paged_evict(k, v, scores, use2, ln, dst, 100, recent=10, sinks=1)
    ok()
    small = torch.tensor(use[::-1] + [pages - 2, pages - 3], device=DEV)
    ks, vs, ss = k[small], v[small], scores[small]
    t = torch.arange(4, dtype=torch.int32, device=DEV)[None]
    assert torch.equal(ks[3, :, 249 % 64], kn[0]) and torch.equal(vs[3, :, 249 % 64], vn[0])
    assert_decoded(o, lse, q, ks, vs, t, ln, d ** -0.5, 0, what="far pages")
    for h in range(Hkv):
        row = ss[:4, h].reshape(-1)[:250].cpu().tolist()
        want = paged.kept_keys(row, 100, 10, 1)
        assert kept[0, h].tolist() == want
        assert torch.equal(ks[4:, h].reshape(-1, d)[:100], ks[:4, h].reshape(-1, d)[want])
        assert torch.equal(vs[4:, h].reshape(-1, d)[:100], vs[:4, h].reshape(-1, d)[want])


def test_decode_workspace_past_32_bits(cuda_lib):
    # Block tables with room for 2^20 keys a sequence: the stashed scores of the
    # last sequences lie more than 2^32 elements into the workspace.
    B, Hq, Hkv, d = 66, 64, 2, 64
    k, v, table, ln = filled([20 + b % 7 for b in range(B)], Hkv, 16, d, BF, seed=16)
    wide = torch.full((B, 2 ** 16), 2 ** 30, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = table
    g = torch.Generator().manual_seed(17)
    q = torch.randn((B, Hq, d), generator=g).to(BF).to(DEV)
    scores = torch.zeros(k.shape[:3], device=DEV)
    assert fa.fa_paged_decode_workspace_bytes(B, Hq, Hkv, d, 16, 2 ** 16, 1) > 2 ** 34
    o, lse = fa.paged_decode(q, k, v, wide, ln, scores=scores)
    ok()
    assert_decoded(o, lse, q, k, v, table, ln, 0.125, 0, scores, torch.zeros_like(scores), "wide table")


def test_rope_offsets_past_32_bits(cuda_lib):
    N, d = 2 ** 24 + 40, 128                    # 2^31 elements and a few rows
    x = torch.empty((1, 1, N, d), dtype=BF, device=DEV)
    x[:, :, :64].normal_()
    x[:, :, -64:].normal_()
    head, tail = x[:, :, :64].clone(), x[:, :, -64:].clone()
    pos = torch.arange(N, dtype=torch.int32, device=DEV).view(1, 1, N)
    w, axes = fa.rope_frequencies((64,), device=DEV)
    fa.rope(x, None, pos, w, axes, q_out=x)
    ok()
    assert_rotated(x[:, :, :64], head, pos[:, :, :64], w, axes, False, False, "first rows")
    assert_rotated(x[:, :, -64:], tail, pos[:, :, -64:], w, axes, False, False, "last rows")


# ---------------------------------------------------------------------------
# Append
# ---------------------------------------------------------------------------
def check_append(k0, v0, s0, kc, vc, sc, table, lens, cu, k, v, q, qo, q0, rot):
    """Every slot of the pools and every row of q_out, bit by bit where nothing is turned."""
    T, ps = k.shape[0], kc.shape[2]
    places = paged.token_places(lens, cu, T)
    want_k, want_v, want_s = k0.clone(), v0.clone(), s0.clone()
    for t, pl in enumerate(places):
        if pl is None:
            if qo is not None:
                assert torch.equal(qo[t], q0[t]), "a padding row was written"
            continue
        p, s = table[pl[0], pl[1] // ps].item(), pl[1] % ps
        if rot is None:
            want_k[p, :, s] = k[t]
        else:
            pos, w, axes, inter = rot
            got = kc[p, :, s][None, :, None]
            assert_rotated(got, k[t][None, :, None], pos[:, t].view(-1, 1, 1), w, axes, inter, False, "k")
            want_k[p, :, s] = kc[p, :, s]
            if qo is not None:
                assert_rotated(qo[t][None, :, None], q[t][None, :, None], pos[:, t].view(-1, 1, 1), w, axes, inter, False, "q")
        want_v[p, :, s] = v[t]
        want_s[p, :, s] = 0
    bits = lambda x: x.contiguous().view(torch.int16)  # noqa: E731
    assert torch.equal(bits(kc), bits(want_k)) and torch.equal(bits(vc), bits(want_v)) and torch.equal(sc, want_s)


APPEND = [
    # lens, new (None: one each), padding tokens, Hq, Hkv, d, page, sections, interleaved, dtype, layout
    ([5, 0, 16, 17, 1], None, 0, 4, 2, 64, 16, (32,), False, BF, "hnd"),
    ([100, 33, 0, 64], [100, 1, 0, 30], 3, 8, 2, 128, 32, (16, 24, 24), False, BF, "pair"),
    ([40, 50], [40, 0], 0, 0, 3, 128, 48, None, False, HF, "nhd"),
    ([1], [1], 0, 1, 1, 64, 16, (16,), True, HF, "hnd"),
    ([0, 0], [0, 0], 2, 2, 2, 64, 16, (32,), False, BF, "hnd"),
    ([300, 7], [290, 7], 1, 5, 1, 128, 16, (20, 12), True, BF, "nhd"),
]


@pytest.mark.parametrize("lens,new,pad,Hq,Hkv,d,page,sections,inter,dt,layout", APPEND)
def test_append(cuda_lib, lens, new, pad, Hq, Hkv, d, page, sections, inter, dt, layout):
    kc, vc, table, ln = filled(lens, Hkv, page, d, dt, seed=21, layout=layout)
    sc = torch.rand(kc.shape[:3], device=DEV)
    k0, v0, s0 = kc.clone(), vc.clone(), sc.clone()
    cu = None if new is None else [sum(new[:b]) for b in range(len(new) + 1)]
    T = len(lens) if new is None else cu[-1] + pad
    g = torch.Generator().manual_seed(22)
    x = torch.randn((T, Hq + 2 * Hkv, d), generator=g).to(dt).to(DEV)
    q, k, v = x.split([Hq, Hkv, Hkv], dim=1)
    rot, kw, qo, q0 = None, {}, None, None
    if sections:
        w, axes = fa.rope_frequencies(sections, device=DEV)
        pos = torch.randint(-5, 100000, (len(sections), T), generator=g).to(torch.int32).to(DEV)
        rot = (pos, w, axes, inter)
        gb = GuardedBuffers(DEV)
        qo = gb.empty((T, Hq, d), dt)
        qo.fill_(7.0)
        q0 = qo.clone()
        kw = dict(q=q, positions=pos, inv_freq=w, axes=axes, interleaved=inter, q_out=qo)
    cud = None if cu is None else torch.tensor(cu, dtype=torch.int32, device=DEV)
    fa.paged_append(kc, vc, table, ln, k, v, cu_seqlens=cud, scores=sc, **kw)
    ok()
    check_append(k0, v0, s0, kc, vc, sc, table, lens, cu, k, v, q, qo, q0, rot)
    if sections:
        gb.check()


def test_append_in_place_q_and_no_tokens(cuda_lib):
    kc, vc, table, ln = filled([9, 3], 2, 16, 64, BF, seed=23)
    x = torch.randn((2, 8, 64), device=DEV).to(BF)
    q, k, v = x.split([4, 2, 2], dim=1)
    q0 = q.clone()
    w, axes = fa.rope_frequencies((32,), device=DEV)
    pos = torch.tensor([[8, 2]], dtype=torch.int32, device=DEV)
    assert fa.paged_append(kc, vc, table, ln, k, v, q=q, positions=pos, inv_freq=w, axes=axes, q_out=q) is q
    ok()
    assert_rotated(q.transpose(0, 1)[None], q0.transpose(0, 1)[None], pos[:, None], w, axes, False, False, "q")
    before = kc.clone()
    fa.paged_append(kc, vc, table, ln, k[:0], v[:0], cu_seqlens=torch.zeros(3, dtype=torch.int32, device=DEV))
    ok()
    assert torch.equal(kc.view(torch.int16), before.view(torch.int16))


@pytest.mark.parametrize("bad", ["page", "length", "more tokens than keys", "offsets"])
def test_append_bad_indices_are_recorded(cuda_lib, bad):
    kc, vc, table, ln = filled([20, 40], 2, 16, 64, BF, seed=24)
    before = kc.clone()
    x = torch.randn((6, 2, 64), device=DEV).to(BF)
    cu = torch.tensor([0, 3, 6], dtype=torch.int32, device=DEV)
    if bad == "page":
        table[1, 2] = kc.shape[0]
    elif bad == "length":
        ln[1] = table.shape[1] * 16 + 3
    elif bad == "offsets":
        cu = torch.tensor([0, -2, 6], dtype=torch.int32, device=DEV)
    else:
        ln[1] = 2
    fa.paged_append(kc, vc, table, ln, x, x, cu_seqlens=cu)
    s, _ = fa.fa_last_device_status()
    assert s == (fa.FA_OK if bad == "offsets" else fa.FA_ERR_BAD_INDEX) or bad == "offsets"
    if bad != "offsets":
        changed = (kc.view(torch.int16) != before.view(torch.int16)).any(-1).any(1)
        slots = {(table[0, 1].item(), s) for s in (1, 2, 3)}
        if bad == "more tokens than keys":
            slots |= {(table[1, 0].item(), s) for s in (0, 1)}
        assert {tuple(i) for i in changed.nonzero().tolist()} == slots
    ok()


@pytest.mark.parametrize("cu,stored", [
    # offsets for lengths 20, 40, 33 and 9 tokens; (sequence, index) of each token that may be stored
    ([3, 4, 6, 9], [None, None, None, (0, 19), (1, 38), (1, 39), (2, 30), (2, 31), (2, 32)]),    # not from 0
    ([0, -2, 6, 9], [None] * 6 + [(2, 30), (2, 31), (2, 32)]),
    ([-5, 2, 6, 9], [None, None, (1, 36), (1, 37), (1, 38), (1, 39), (2, 30), (2, 31), (2, 32)]),
    ([0, 2, 6, 10], [(0, 18), (0, 19), (1, 36), (1, 37), (1, 38), (1, 39), None, None, None]),   # past the tokens
    ([0, 6, 4, 9], [(0, 14 + t) for t in range(6)] + [(2, 30), (2, 31), (2, 32)]),               # not in order
    ([0, 2, 6, -1], [None] * 9),
    ([1, 1, 1, 1], [None] * 9),
])
def test_append_bad_offsets_are_recorded_and_touch_no_other_slot(cuda_lib, cu, stored):
    lens, T = [20, 40, 33], 9
    kc, vc, table, ln = filled(lens, 2, 16, 64, BF, seed=25, layout="pair")
    sc = torch.rand(kc.shape[:3], device=DEV)
    want_k, want_v, want_s = kc.clone(), vc.clone(), sc.clone()
    g = torch.Generator().manual_seed(26)
    x = torch.randn((T, 8, 64), generator=g).to(BF).to(DEV)
    q, k, v = x.split([4, 2, 2], dim=1)
    w, axes = fa.rope_frequencies((32,), device=DEV)
    pos = torch.zeros((1, T), dtype=torch.int32, device=DEV)          # a turn by 0 keeps every bit
    qo = torch.full_like(q, 7.0)
    want_q = qo.clone()
    fa.paged_append(kc, vc, table, ln, k, v, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV), q=q, positions=pos,
                    inv_freq=w, axes=axes, scores=sc, q_out=qo)
    s, _ = fa.fa_last_device_status()
    assert s == fa.FA_ERR_BAD_INDEX
    for t, at in enumerate(stored):
        if at is None:
            continue
        p, slot = table[at[0], at[1] // 16].item(), at[1] % 16
        want_k[p, :, slot], want_v[p, :, slot], want_s[p, :, slot], want_q[t] = k[t], v[t], 0, q[t]
    bits = lambda x: x.contiguous().view(torch.int16)  # noqa: E731
    assert torch.equal(bits(kc), bits(want_k)) and torch.equal(bits(vc), bits(want_v))
    assert torch.equal(sc, want_s) and torch.equal(qo, want_q)
    ok()


def test_append_bad_offsets_of_many_sequences_are_recorded(cuda_lib):
    # One pair out of order among many more sequences than a block has threads,
    # and every token finds a place in some sequence.
    B = 3000
    lens = [5] * B
    kc, vc, table, ln = filled(lens, 1, 16, 64, HF, seed=27)
    x = torch.randn((B, 1, 64), device=DEV).to(HF)
    cu = torch.arange(B + 1, dtype=torch.int32, device=DEV)
    fa.paged_append(kc, vc, table, ln, x, x, cu_seqlens=cu)
    ok()
    for at in (1, 129, 2600, B - 1):
        bad = cu.clone()
        bad[at] = at - 2
        fa.paged_append(kc, vc, table, ln, x, x, cu_seqlens=bad)
        assert fa.fa_last_device_status()[0] == fa.FA_ERR_BAD_INDEX
    ok()


# ---------------------------------------------------------------------------
# Eviction
# ---------------------------------------------------------------------------
EVICT = [
    # lens, Hkv, d, page, budget, recent, sinks, kind of scores, dtype, layout
    ([40], 1, 64, 16, 20, 0, 0, "normal", BF, "hnd"),
    ([0, 1, 16, 17, 100], 2, 64, 16, 16, 4, 2, "normal", BF, "hnd"),
    ([1000, 500, 2], 2, 128, 48, 333, 100, 4, "heavy", HF, "pair"),
    ([300, 299, 5000], 3, 64, 32, 299, 298, 1, "normal", BF, "nhd"),     # nothing left to choose
    ([700, 31], 2, 128, 16, 128, 0, 0, "ties", BF, "hnd"),
    ([700, 130], 1, 64, 16, 1, 0, 0, "equal", HF, "hnd"),
    ([700, 130], 1, 64, 16, 1, 1, 0, "equal", HF, "hnd"),
    ([2100, 64], 2, 64, 64, 1500, 10, 0, "odd", BF, "hnd"),              # NaN, infinities, -0
    ([40000], 1, 64, 64, 5000, 100, 4, "heavy", BF, "hnd"),
    ([9000, 4097], 2, 64, 128, 8999, 0, 16, "narrow", BF, "hnd"),        # values that share their high bits
    # More keys than shared memory holds: in one block (too many units for a
    # cluster each), and over a whole cluster.
    ([60000] + [40] * 79, 1, 64, 2048, 1000, 10, 4, "heavy", BF, "hnd"),
    ([450001], 1, 64, 4096, 60000, 5, 0, "heavy", BF, "hnd"),
    ([450001], 1, 64, 4096, 300000, 1000, 7, "ties", BF, "hnd"),
]


def make_scores(kind, shape, g):
    x = torch.randn(shape, generator=g)
    if kind == "heavy":
        x = (2 * x).exp() * (torch.rand(shape, generator=g) > 0.3)
    elif kind == "ties":
        x = torch.randint(0, 4, shape, generator=g).float()
    elif kind == "equal":
        x = torch.full(shape, 0.25)
    elif kind == "narrow":
        x = 1.0 + torch.randint(0, 200, shape, generator=g).float() * 2.0 ** -23
    elif kind == "odd":
        pick = torch.randint(0, 8, shape, generator=g)
        for i, value in enumerate((float("nan"), float("inf"), -float("inf"), -0.0, 0.0, -1.5)):
            x = torch.where(pick == i, torch.tensor(value), x)
    return x


@pytest.mark.parametrize("lens,Hkv,d,page,budget,recent,sinks,kind,dt,layout", EVICT)
def test_evict(cuda_lib, lens, Hkv, d, page, budget, recent, sinks, kind, dt, layout):
    cols = -(-budget // page)
    kc, vc, table, ln = filled(lens, Hkv, page, d, dt, seed=31, layout=layout, extra=len(lens) * cols + 2)
    g = torch.Generator().manual_seed(32)
    sc = make_scores(kind, kc.shape[:3], g).to(DEV)
    used = {p for b, n in enumerate(lens) for p in table[b, :-(-n // page)].tolist()}
    spare = [p for p in range(kc.shape[0]) if p not in used]
    dst = torch.tensor(spare[:len(lens) * cols], dtype=torch.int32, device=DEV).view(len(lens), cols)
    k0, v0, s0 = kc.clone(), vc.clone(), sc.clone()
    gb = GuardedBuffers(DEV)
    nl, kept = gb.empty((len(lens),), torch.int32), gb.empty((len(lens), Hkv, budget), torch.int32)
    fa.paged_evict(kc, vc, sc, table, ln, dst, budget, recent, sinks, new_lens=nl, kept=kept)
    ok()
    gb.check()
    want_k, want_v, want_s = k0.clone(), v0.clone(), s0.clone()
    for b, n in enumerate(lens):
        m = min(n, budget)
        assert nl[b].item() == m
        if m == 0:
            assert bool((kept[b] == -1).all())
            continue
        j = torch.arange(n, device=DEV)
        sp = table[b].long()[j // page]
        r = torch.arange(m, device=DEV)
        dp = dst[b].long()[r // page]
        for h in range(Hkv):
            keep = paged.kept_keys(s0[sp, h, j % page].cpu().tolist(), budget, recent, sinks)
            assert kept[b, h].tolist() == keep + [-1] * (budget - m), (b, h)
            i = torch.tensor(keep, device=DEV)
            want_k[dp, h, r % page] = k0[sp[i], h, i % page]
            want_v[dp, h, r % page] = v0[sp[i], h, i % page]
            want_s[dp, h, r % page] = s0[sp[i], h, i % page]
    bits = lambda x, t: x.contiguous().view(t)  # noqa: E731
    assert torch.equal(bits(kc, torch.int16), bits(want_k, torch.int16))
    assert torch.equal(bits(vc, torch.int16), bits(want_v, torch.int16))
    assert torch.equal(bits(sc, torch.int32), bits(want_s, torch.int32))


@pytest.mark.parametrize("bad", ["source page", "target page", "length"])
def test_evict_bad_indices_are_recorded(cuda_lib, bad):
    kc, vc, table, ln = filled([100, 60], 2, 16, 64, BF, seed=33, extra=6)
    used = {p for b, n in enumerate([100, 60]) for p in table[b, :-(-n // 16)].tolist()}
    spare = [p for p in range(kc.shape[0]) if p not in used]
    dst = torch.tensor(spare[:4], dtype=torch.int32, device=DEV).view(2, 2)
    sc = torch.rand(kc.shape[:3], device=DEV)
    s0 = sc.clone()
    if bad == "source page":
        table[0, 1] = -7
    elif bad == "target page":
        dst[0, 1] = kc.shape[0] + 5
    else:
        ln[0] = 10 ** 6
    nl, kept = fa.paged_evict(kc, vc, sc, table, ln, dst, 32)
    s, _ = fa.fa_last_device_status()
    assert s == fa.FA_ERR_BAD_INDEX
    row = s0[table[1].long()[torch.arange(60, device=DEV) // 16], 1, torch.arange(60, device=DEV) % 16]
    assert kept[1, 1].tolist() == paged.kept_keys(row.cpu().tolist(), 32, 0, 0)
    ok()


# ---------------------------------------------------------------------------
# Random sweep
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("seed", range(48))
def test_random_cases(cuda_lib, seed):
    """Append (ragged or one token), decode and evict on one random cache."""
    r = np.random.default_rng(seed)
    pick = lambda *x: x[r.integers(len(x))]  # noqa: E731
    dt, d, layout = pick(BF, HF), pick(64, 128), pick("hnd", "nhd", "pair")
    Hkv = int(r.integers(1, 5))
    Hq = Hkv * int(pick(1, 2, 3, 4, 7, 8, 9, 16, 20))
    page = int(pick(16, 32, 48, 64, 112, 256))
    B = int(r.integers(1, 9))
    lens = [int(x) for x in r.integers(0, pick(20, 200, 900) + 1, B)]
    budget = int(r.integers(1, max(lens) + 2))
    recent = int(r.integers(0, budget + 1))
    sinks = int(r.integers(0, budget - recent + 1))
    cols = -(-budget // page)
    kc, vc, table, ln = filled(lens, Hkv, page, d, dt, seed=seed, layout=layout, extra=B * cols + 1,
                               sigma=float(pick(0.5, 1.0, 2.0)))
    g = torch.Generator().manual_seed(seed + 1000)
    sc = torch.rand(kc.shape[:3], generator=g).to(DEV)
    # Append: the newest tokens once more, with other values.
    one = r.random() < 0.5
    new = None if one else [int(r.integers(0, n + 1)) for n in lens]
    cu = None if one else [sum(new[:b]) for b in range(B + 1)]
    T = B if one else cu[-1] + int(r.integers(0, 3))
    x = torch.randn((T, Hq + 2 * Hkv, d), generator=g).to(dt).to(DEV)
    q, k, v = x.split([Hq, Hkv, Hkv], dim=1)
    rot, kw, qo, q0 = None, {}, None, None
    if r.random() < 0.7 and T:
        n_axes = int(r.integers(1, 4))
        pairs = 8 * int(r.integers(1, d // 16 + 1))
        w = torch.from_numpy(1e4 ** -r.random(pairs)).to(DEV)
        axes = torch.from_numpy(r.integers(0, n_axes, pairs).astype(np.int32)).to(DEV)
        pos = torch.randint(-100, 10 ** 7, (n_axes, T), generator=g).to(torch.int32).to(DEV)
        rot = (pos, w, axes, bool(r.random() < 0.5))
        qo = torch.full((T, Hq, d), 7.0, dtype=dt, device=DEV)
        q0 = qo.clone()
        kw = dict(q=q, positions=pos, inv_freq=w, axes=axes, interleaved=rot[3], q_out=qo)
    k0, v0, s0 = kc.clone(), vc.clone(), sc.clone()
    cud = None if one else torch.tensor(cu, dtype=torch.int32, device=DEV)
    fa.paged_append(kc, vc, table, ln, k, v, cu_seqlens=cud, scores=sc, **kw)
    ok()
    check_append(k0, v0, s0, kc, vc, sc, table, lens, cu, k, v, q, qo, q0, rot)
    # Decode.
    window = int(pick(0, 0, 1, 30, 300))
    scale = float(pick(d ** -0.5, 0.03, 0.4))
    qd = torch.randn((B, Hq, d), generator=g).to(dt).to(DEV)
    before = sc.clone()
    with_scores = r.random() < 0.6
    o, lse = fa.paged_decode(qd, kc, vc, table, ln, scale=scale, window=window, scores=sc if with_scores else None)
    ok()
    assert_decoded(o, lse, qd, kc, vc, table, ln, scale, window, sc if with_scores else None, before, f"seed {seed}")
    # Evict.
    used = {p for b, n in enumerate(lens) for p in table[b, :-(-n // page)].tolist()}
    spare = [p for p in range(kc.shape[0]) if p not in used]
    dst = torch.tensor(spare[:B * cols], dtype=torch.int32, device=DEV).view(B, cols)
    s0 = f64(sc)
    rows = [(paged.gather(f64(kc), table[b].cpu().numpy(), n), paged.gather(f64(vc), table[b].cpu().numpy(), n),
             paged.gather(s0, table[b].cpu().numpy(), n)) for b, n in enumerate(lens)]
    nl, kept = fa.paged_evict(kc, vc, sc, table, ln, dst, budget, recent, sinks)
    ok()
    for b, n in enumerate(lens):
        m = min(n, budget)
        assert nl[b].item() == m
        got = [paged.gather(f64(t), dst[b].cpu().numpy(), m) for t in (kc, vc, sc)]
        for h in range(Hkv):
            keep = paged.kept_keys(rows[b][2][h].tolist(), budget, recent, sinks)
            assert kept[b, h].tolist() == keep + [-1] * (budget - m)
            for t in range(3):
                assert np.array_equal(got[t][h], rows[b][t][h][keep]), (seed, b, h, t)


# ---------------------------------------------------------------------------
# Together, and how calls are made
# ---------------------------------------------------------------------------
class Served:
    """A few decoding steps over a paged cache, mirrored in fp64 on the CPU."""

    def __init__(self, dt, B=3, Hq=8, Hkv=2, d=64, page=16, budget=40):
        self.dt, self.B, self.Hq, self.Hkv, self.d, self.page, self.budget = dt, B, Hq, Hkv, d, page, budget
        self.kc, self.vc = new_pool(64, Hkv, page, d, dt)
        self.sc = torch.full((64, Hkv, page), 1e9, device=DEV)
        self.g = torch.Generator().manual_seed(41)
        self.w, self.axes = fa.rope_frequencies((8, 12, 12), device=DEV)
        self.free = torch.randperm(64, generator=self.g).tolist()

    def pages(self, n):
        out, self.free = self.free[:n], self.free[n:]
        return out


@pytest.mark.parametrize("dt", [BF, HF])
def test_serving_run(cuda_lib, dt):
    """Prompt, decoding steps with scores, eviction, more steps: the cache and
    each step's output against the oracle."""
    s = Served(dt)
    B, Hq, Hkv, d, page = s.B, s.Hq, s.Hkv, s.d, s.page
    lens = [50, 17, 64]
    true_len = list(lens)                                   # positions go on after an eviction
    table = torch.zeros((B, 6), dtype=torch.int32)
    for b in range(B):
        table[b] = torch.tensor(s.pages(6))
    table = table.to(DEV)

    def project(T):
        return torch.randn((T, Hq + 2 * Hkv, d), generator=s.g).to(dt).to(DEV).split([Hq, Hkv, Hkv], dim=1)

    def positions(p):
        p = torch.tensor(p, dtype=torch.int32, device=DEV)
        return torch.stack([p, p // 8, p % 8])

    cu = torch.tensor([0, 50, 67, 131], dtype=torch.int32, device=DEV)
    q, k, v = project(131)
    pos = positions([i for n in lens for i in range(n)])
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    fa.paged_append(s.kc, s.vc, table, ln, k, v, cu_seqlens=cu, q=q, positions=pos, inv_freq=s.w, axes=s.axes, scores=s.sc)
    ok()
    acc = [np.zeros((Hkv, n)) for n in lens]

    def step():
        nonlocal ln
        q, k, v = project(B)
        ln = ln + 1
        pos = positions(true_len)
        qr = fa.paged_append(s.kc, s.vc, table, ln, k, v, q=q, positions=pos, inv_freq=s.w, axes=s.axes, scores=s.sc)
        before = s.sc.clone()
        o, lse = fa.paged_decode(qr, s.kc, s.vc, table, ln, scores=s.sc)
        ok()
        assert_decoded(o, lse, qr, s.kc, s.vc, table, ln, d ** -0.5, 0, s.sc, before, "step")
        # The step from the unturned rows, in 64 bits throughout: the newest
        # key's score against the query, both turned by the same angles, is
        # that of the unturned rows up to their roundings.
        rq, rk = f64(qr), f64(s.kc)
        for b in range(B):
            n = int(ln[b])
            kn = rk[table[b, (n - 1) // page].item(), :, (n - 1) % page]
            for h in range(Hq):
                a, r = f64(q[b, h]), f64(k[b, h // (Hq // Hkv)])
                plain, turned = float(a @ r), float(rq[b, h] @ kn[h // (Hq // Hkv)])
                assert abs(plain - turned) <= (2 * U[dt] + 1e-5) * 2 * np.linalg.norm(a) * np.linalg.norm(r)
            true_len[b] += 1
            w = paged.decode(rq[b:b + 1], rk, f64(s.vc), table[b:b + 1].cpu().numpy(), [n], d ** -0.5)[2][0]
            acc[b] = np.concatenate([acc[b], np.zeros((Hkv, 1))], axis=1) + w

    def check_scores():
        for b in range(B):
            n = int(ln[b])
            got = paged.gather(f64(s.sc), table[b].cpu().numpy(), n)
            assert np.abs(got - acc[b]).max() <= 1e-3 * max(1.0, acc[b].max())

    for _ in range(4):
        step()
    check_scores()
    # Evict into fresh pages; the kept keys by the oracle from the scores.
    new_table = torch.zeros((B, 6), dtype=torch.int32)
    for b in range(B):
        new_table[b] = torch.tensor(s.pages(6))
    new_table = new_table.to(DEV)
    rows = [paged.gather(f64(s.sc), table[b].cpu().numpy(), int(ln[b])) for b in range(B)]
    kv_before = [(paged.gather(f64(s.kc), table[b].cpu().numpy(), int(ln[b])),
                  paged.gather(f64(s.vc), table[b].cpu().numpy(), int(ln[b]))) for b in range(B)]
    new, kept = fa.paged_evict(s.kc, s.vc, s.sc, table, ln, new_table[:, :3], s.budget, recent=8, sinks=2)
    ok()
    table = new_table
    for b in range(B):
        m = int(new[b])
        assert m == min(int(ln[b]), s.budget)
        k2, v2 = (paged.gather(f64(x), table[b].cpu().numpy(), m) for x in (s.kc, s.vc))
        old = acc[b]
        acc[b] = np.zeros((Hkv, m))
        for h in range(Hkv):
            want = paged.kept_keys(rows[b][h].tolist(), s.budget, 8, 2)
            assert kept[b, h, :m].tolist() == want
            assert np.array_equal(k2[h], kv_before[b][0][h][want]) and np.array_equal(v2[h], kv_before[b][1][h][want])
            acc[b][h] = old[h][want]
    ln = new
    for _ in range(3):
        step()
    check_scores()


def one_step(dt=BF, B=4, lens=(100, 0, 37, 512)):
    """Inputs of a decoding step and a function that makes it."""
    k, v, table, ln = filled(list(lens), 2, 16, 128, dt, seed=51)
    g = torch.Generator().manual_seed(52)
    x = torch.randn((B, 12, 128), generator=g).to(dt).to(DEV)
    w, axes = fa.rope_frequencies((64,), device=DEV)
    pos = (ln - 1).clamp(min=0)[None].contiguous()
    scores = torch.zeros(k.shape[:3], device=DEV)
    q, kn, vn = x.split([8, 2, 2], dim=1)

    def step(stream=None):
        qr = fa.paged_append(k, v, table, ln, kn, vn, q=q, positions=pos, inv_freq=w, axes=axes, scores=scores,
                             stream=stream)
        o, lse = fa.paged_decode(qr, k, v, table, ln, scores=scores, stream=stream)
        return o, lse
    return step, x, scores


def test_step_in_a_captured_graph(cuda_lib):
    step, x, scores = one_step()
    o, lse = step()
    ok()
    after_one = scores.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()                                        # warm-up outside the capture
    torch.cuda.current_stream().wait_stream(side)
    graph, graph2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go, gl = step()
    with torch.cuda.graph(graph2):
        go2, gl2 = step()
    rows = torch.tensor([0, 2, 3], device=DEV)        # sequence 1 is padding: its q row is not written
    for gr, a, l in ((graph, go, gl), (graph2, go2, gl2), (graph, go, gl)):
        a.zero_()
        scores.zero_()
        gr.replay()
        ok()
        assert torch.equal(a[rows], o[rows]) and torch.equal(l, lse)
        assert torch.equal(scores, after_one)
    # New inputs in the same buffers.
    x.mul_(0.5)
    graph.replay()
    ok()
    a, l = go.clone(), gl.clone()
    o3, l3 = step()
    ok()
    assert torch.equal(a[rows], o3[rows]) and torch.equal(l, l3)


def test_captured_decode_follows_lengths_and_tables(cuda_lib):
    # A graph captured for one batch replays for others: lengths, pages and
    # queries change in place, as a serving loop changes them.
    k, v, table, ln = filled([300, 40, 0, 129], 2, 16, 64, BF, seed=71)
    g = torch.Generator().manual_seed(72)
    q = torch.randn((4, 8, 64), generator=g).to(BF).to(DEV)
    scores = torch.zeros(k.shape[:3], device=DEV)
    fa.paged_decode(q, k, v, table, ln, scores=scores)
    ok()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = fa.paged_decode(q, k, v, table, ln, scores=scores)
    tables = [table.clone(), table[[3, 0, 1, 2]].clone(), table[[1, 1, 0, 3]].clone()]
    for t, n in zip(tables, ([300, 40, 0, 129], [100, 299, 33, 0], [7, 40, 16, 1])):
        table.copy_(t)
        ln.copy_(torch.tensor(n, dtype=torch.int32))
        q.copy_(torch.randn((4, 8, 64), generator=g))
        scores.zero_()
        graph.replay()
        ok()
        assert_decoded(o, lse, q, k, v, table, ln, 0.125, 0, scores, torch.zeros_like(scores), f"{n}")


def test_capture_with_a_forked_stream(cuda_lib):
    # Two steps on two branches of one graph, other kernels before, between and after.
    a, b = one_step(), one_step(dt=HF, lens=(700, 64, 0, 9))
    want = [a[0](), b[0]()]
    ok()
    side = torch.cuda.Stream()
    x = torch.zeros(1 << 20, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cur = torch.cuda.current_stream()
        x.add_(1.0)
        side.wait_stream(cur)
        with torch.cuda.stream(side):
            got_b = b[0]()
            y = x * 2.0
        got_a = a[0]()
        x.mul_(1.0)
        cur.wait_stream(side)
        again = a[0]()
        z = x + y
    for n in range(1, 4):
        for o, _ in (got_a, got_b, again):
            o.zero_()
        graph.replay()
        ok()
        assert z[0].item() == 3.0 * n
        for (o, l), (wo, wl), skip in ((got_a, want[0], 1), (again, want[0], 1), (got_b, want[1], 2)):
            rows = torch.tensor([r for r in range(4) if r != skip], device=DEV)
            assert torch.equal(o[rows], wo[rows]) and torch.equal(l, wl)


def test_calls_between_other_kernels_on_one_stream(cuda_lib):
    # Inputs written right before a call and outputs overwritten right after it,
    # with nothing that waits in between.
    k, v, table, ln = filled([900, 5, 300, 64], 2, 16, 64, BF, seed=81)
    g = torch.Generator().manual_seed(82)
    qs = [torch.randn((4, 8, 64), generator=g).to(BF).to(DEV) for _ in range(6)]
    want = [fa.paged_decode(q, k, v, table, ln)[0].clone() for q in qs]
    w, axes = fa.rope_frequencies((32,), device=DEV)
    pos = torch.arange(4, dtype=torch.int32, device=DEV).view(1, 1, 4)
    turned = [fa.rope(q.transpose(0, 1)[None].contiguous(), None, pos, w, axes).clone() for q in qs]
    ok()
    buf, out, lse = torch.empty_like(qs[0]), torch.empty_like(qs[0]), torch.empty((4, 8), device=DEV)
    ws = fa.paged_decode_workspace(4, 8, k, table)
    rin, rout = torch.empty_like(turned[0]), torch.empty_like(turned[0])
    got, got_turned = [], []
    for _ in range(20):
        got, got_turned = [], []
        for q in qs:
            buf.copy_(q)
            fa.paged_decode(buf, k, v, table, ln, out=out, lse=lse, workspace=ws)
            got.append(out.clone())
            buf.fill_(float("nan"))
            out.fill_(float("nan"))
            rin.copy_(q.transpose(0, 1)[None])
            fa.rope(rin, None, pos, w, axes, q_out=rout)
            got_turned.append(rout.clone())
            rin.fill_(float("nan"))
            rout.fill_(float("nan"))
        ok()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        assert all(torch.equal(x, y) for x, y in zip(got_turned, turned))


def test_calls_from_two_threads(cuda_lib):
    import threading
    steps = [one_step(), one_step(dt=HF, lens=(700, 64, 0, 9))]
    want = [s[0]() for s in steps]
    ok()
    got, errors = [None, None], []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            stream.wait_stream(torch.cuda.default_stream())
            with torch.cuda.stream(stream):
                got[i] = [steps[i][0]() for _ in range(30)]
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
    for i, skip in enumerate((1, 2)):
        rows = torch.tensor([r for r in range(4) if r != skip], device=DEV)
        for o, l in got[i]:
            assert torch.equal(o[rows], want[i][0][rows]) and torch.equal(l, want[i][1])


def test_steps_on_two_streams(cuda_lib):
    # Two independent steps in flight at once, on streams that are not the
    # current one, many times over.
    a, b = one_step(), one_step(dt=HF, lens=(700, 64, 0, 9))
    want = [s[0]() for s in (a, b)]
    ok()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate((a, b)):
            got[i].append(s[0](stream=streams[i]))
    ok()
    skip = [1, 2]
    for i in range(2):
        rows = torch.tensor([r for r in range(4) if r != skip[i]], device=DEV)
        for o, l in got[i]:
            assert torch.equal(o[rows], want[i][0][rows]) and torch.equal(l, want[i][1])


def test_native_marshalling_is_there(cuda_lib):
    assert fa.native_marshalling(), "see _lib/fa_torch.txt"


@pytest.fixture(params=["native", "python"])
def marshalling(request, monkeypatch, cuda_lib):
    if request.param == "native":
        assert fa.native_marshalling()
    else:
        monkeypatch.setattr(fa, "_native", fa._NotBuilt)
    return request.param


@pytest.mark.parametrize("given", [False, True])
def test_both_marshallings_make_the_same_calls(cuda_lib, monkeypatch, given):
    """Every operator once through each, with and without the optional arguments."""
    def calls():
        g = torch.Generator().manual_seed(91)
        kc, vc, table, ln = filled([50, 0, 33], 2, 16, 64, HF, seed=92, layout="pair", extra=9)
        used = set(table[0, :4].tolist()) | set(table[2, :3].tolist())
        spare = [p for p in range(kc.shape[0]) if p not in used]
        x = torch.randn((3, 12, 64), generator=g).to(HF).to(DEV)
        q, k, v = x.split([8, 2, 2], dim=1)
        w, axes = fa.rope_frequencies((8, 8, 16), device=DEV)
        pos = torch.randint(0, 99, (3, 3), generator=g).to(torch.int32).to(DEV)
        sc = torch.rand(kc.shape[:3], generator=g).to(DEV)
        cu = torch.tensor([0, 2, 2, 3], dtype=torch.int32, device=DEV)
        new = lambda t: torch.full_like(t, 7.0) if given else None  # noqa: E731
        out = [fa.paged_append(kc, vc, table, ln, k, v), sc]
        out[0] is None or pytest.fail("q out of nothing")
        q1 = torch.zeros((3, 8, 64), dtype=HF, device=DEV)
        q1 = fa.paged_append(kc, vc, table, ln, k, v, cu, q, pos, w, axes, given, sc if given else None, q1)
        o, lse = fa.paged_decode(q1, kc, vc, table, ln, 0.2 if given else None, 20 if given else 0, sc if given else None,
                                 new(q1), torch.zeros((3, 8), device=DEV) if given else None,
                                 fa.paged_decode_workspace(3, 8, kc, table, given) if given else None)
        dst = torch.tensor(spare[:6], dtype=torch.int32, device=DEV).view(3, 2)
        nl, kept = fa.paged_evict(kc, vc, sc, table, ln, dst, 20, 3, 1, torch.zeros(3, dtype=torch.int32, device=DEV) if given else None)
        qb = torch.randn((2, 3, 9, 80), generator=g).to(BF).to(DEV).transpose(1, 2).contiguous().transpose(1, 2)
        pb = torch.arange(9, dtype=torch.int32, device=DEV).expand(3, 2, 9)
        r1 = fa.rope(qb, None, pb, w, axes, given, new(qb))
        r2, r3 = fa.rope_backward(qb, qb[:, :1], pb, w, axes, given, new(qb), new(qb[:, :1]))
        ok()
        return [kc, vc, sc, q1, o, lse, nl, kept, r1, r2, r3]
    assert fa.native_marshalling()
    native = calls()
    monkeypatch.setattr(fa, "_native", fa._NotBuilt)
    python = calls()
    for a, b in zip(native, python):
        assert a.shape == b.shape and a.dtype == b.dtype
        assert torch.equal(torch.nan_to_num(a.float(), nan=-3.0), torch.nan_to_num(b.float(), nan=-3.0))


def test_a_failed_allocation_raises(cuda_lib):
    # A block table whose workspace no device has room for.
    k, v, table, ln = filled([20], 2, 16, 64, BF, seed=95)
    q = torch.zeros((1, 512, 64), dtype=BF, device=DEV)
    wide = table.new_zeros((1, 2 ** 26))
    wide[:, :2] = table[:, :2]
    scores = torch.zeros(k.shape[:3], device=DEV)
    with pytest.raises(torch.OutOfMemoryError):
        fa.paged_decode(q, k, v, wide, ln, scores=scores)          # 2 TB
    o, _ = fa.paged_decode(q[:, :4], k, v, table, ln)
    ok()
    assert torch.isfinite(o).all()


def test_binding_refusals(marshalling):
    k, v, table, ln = filled([20], 2, 16, 64, BF, seed=61)
    q = torch.zeros((1, 4, 64), dtype=BF, device=DEV)
    with pytest.raises(TypeError):
        fa.paged_decode(q.half(), k, v, table, ln)
    with pytest.raises(TypeError):
        fa.paged_decode(q, k, v, table.long(), ln)
    with pytest.raises(ValueError):
        fa.paged_decode(q, k, v, table, ln.expand(2))
    with pytest.raises(ValueError):
        fa.paged_decode(q, k, v.transpose(1, 2).contiguous().transpose(1, 2), table, ln)
    with pytest.raises(ValueError):
        fa.paged_decode(q, k, v, table, ln, scores=torch.zeros(k.shape[:2], device=DEV))
    with pytest.raises(fa.FAError):
        fa.paged_decode(q[:, :3], k, v, table, ln)                     # 3 query heads, 2 kv heads
    with pytest.raises(fa.FAError):
        fa.paged_decode(q, k, v, table, ln, window=-1)
    with pytest.raises(fa.FAError):
        fa.paged_decode(q, k, v, table, ln, out=q)
    with pytest.raises(ValueError):
        fa.paged_append(k, v, table, ln, q[:, :2].expand(3, 2, 64), q[:, :2].expand(3, 2, 64))
    with pytest.raises(ValueError):
        fa.paged_evict(k, v, torch.zeros(k.shape[:3], device=DEV), table, ln, table[:, :1], 0)
    with pytest.raises(fa.FAError):
        fa.paged_evict(k, v, torch.zeros(k.shape[:3], device=DEV), table, ln, table, 10)
    ok()

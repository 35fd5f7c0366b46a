"""Norms of queries and keys and the 4-bit cache on the CPU: pins of their fp64
oracle (by hand, differences, the 16-bit oracle) and the refusals of the C
entry points, which come before any CUDA call."""
import ctypes
import math

import numpy as np
import pytest

import exact_io_aware_flashattention_gb300 as fa
from exact_io_aware_flashattention_gb300 import _build
from oracle import paged, paged4


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fa.load_library()


def bf16(x):
    import torch
    return torch.from_numpy(np.asarray(x)).to(torch.bfloat16).double().numpy()


# ---------------------------------------------------------------------------
# Oracle pins
# ---------------------------------------------------------------------------
def test_norm_by_hand():
    assert np.allclose(paged4.norm(np.array([3.0, 4.0]), None, 0.0), np.array([3.0, 4.0]) / math.sqrt(12.5), atol=1e-15)
    assert np.allclose(paged4.norm(np.array([3.0, 4.0]), np.array([2.0, -1.0]), 12.5),
                       np.array([6.0, -4.0]) / 5.0, atol=1e-15)
    assert not paged4.norm(np.zeros(4), None, 1e-6).any()


@pytest.mark.parametrize("turned", [False, True])
@pytest.mark.parametrize("weights", [False, True])
def test_norm_gradient_against_differences(turned, weights):
    r = np.random.default_rng(1)
    x, g = r.normal(size=(1, 2, 3, 24)), r.normal(size=(1, 2, 3, 24))
    w = r.normal(size=24) if weights else None
    rotary = (r.integers(0, 50, size=(2, 1, 3)), 0.5 ** np.arange(8), [0, 0, 1, 1, 0, 1, 0, 1], True) if turned else None
    dx, dw = paged4.norm_rope_backward(g, x, w, 1e-3, rotary)

    def loss(x, w):
        return (g * paged4.norm_rope(x, w, 1e-3, rotary)).sum()
    for _ in range(10):
        e = np.zeros_like(x)
        at = tuple(r.integers(0, n) for n in x.shape)
        e[at] = 1e-6
        assert abs((loss(x + e, w) - loss(x - e, w)) / 2e-6 - dx[at]) < 1e-7
    one = np.ones(24) if w is None else w
    for i in (0, 11, 23):
        e = np.zeros(24)
        e[i] = 1e-6
        assert abs((loss(x, one + e) - loss(x, one - e)) / 2e-6 - dw[i]) < 1e-7


def test_quantised_by_hand():
    x = np.zeros(64)
    x[1], x[2], x[3], x[4] = 15.0, 7.4, 7.5, 8.5
    c, s, z = paged4.quantise(x, bf16)
    assert s.tolist() == [1.0] and z.tolist() == [0.0] and c[:5].tolist() == [0, 15, 7, 8, 8]      # ties to even
    c, s, z = paged4.quantise(np.full(64, -2.5), bf16)
    assert not s.any() and not c.any() and z.tolist() == [-2.5]
    assert np.array_equal(paged4.values(np.full(128, -2.5), bf16), np.full(128, -2.5))
    for bad in (math.nan, math.inf, -math.inf):
        x = np.arange(128.0)
        x[100] = bad
        v = paged4.values(x, bf16)
        assert np.isfinite(v[:64]).all() and np.isnan(v[64:]).all()


def test_values_are_within_half_a_step():
    r = np.random.default_rng(3)
    x = bf16(r.normal(size=(50, 128)))
    c, s, z = paged4.quantise(x, bf16)
    step = np.repeat(s, 64, axis=-1)
    assert c.min() == 0 and c.max() == 15
    # Half a step, and 15 roundings of s (2^-8 of it, half a step of bf16 at most).
    assert (np.abs(paged4.values(x, bf16) - x) <= step * (0.5 + 15 * 2.0 ** -8)).all()


def test_decode_of_exactly_held_rows_is_the_16_bit_one():
    # Rows whose values are z + s c already.
    r = np.random.default_rng(4)
    n, d, Hq, Hkv = 21, 64, 4, 2
    k, v = (r.integers(0, 16, size=(Hkv, n, d)) * 0.25 - 2.0 for _ in range(2))
    k[..., 0], k[..., 1], v[..., 0], v[..., 1] = -2.0, 1.75, -2.0, 1.75
    q = r.normal(size=(Hq, d))
    assert np.array_equal(paged4.values(k, bf16), k)
    pages = np.zeros((2, Hkv, 16, d)), np.zeros((2, Hkv, 16, d))
    for p, x in zip(pages, (k, v)):
        for j in range(n):
            p[j // 16, :, j % 16] = x[:, j]
    for window in (0, 5):
        o, lse, x, a = paged4.decode(q, k, v, 0.3, window, bf16)
        ro, rl, _, ra = paged.decode(q[None], *pages, [[0, 1]], [n], 0.3, window)
        assert np.allclose(o, ro[0], atol=1e-12) and np.allclose(lse, rl[0], atol=1e-12)
        assert (a >= ra[0] - 1e-12).all()


# ---------------------------------------------------------------------------
# Refusals
# ---------------------------------------------------------------------------
A = 1 << 24   # fake, aligned, far apart "device" addresses (never dereferenced)
LL = ctypes.c_longlong
NAN, INF = float("nan"), float("inf")


def arr(*x):
    return (LL * len(x))(*x)


def rotary(**kw):
    a = dict(positions=20 * A, axis_stride=64, batch_stride=0, inv_freq=21 * A, axes=22 * A, n_axes=3, rot=64, interleaved=0)
    a.update(kw)
    return fa.fa_rotary(**a)


def norm(**kw):
    a = dict(q_weight=23 * A, k_weight=24 * A, weights_fp32=0, eps=1e-6)
    a.update(kw)
    return fa.fa_qk_norm(**a)


def valid(call):
    """A valid call passes every check and then fails for want of a GPU; where there is one it is not made."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("fake addresses: only where no kernel can run")
    assert call() in (fa.FA_ERR_CUDA, fa.FA_ERR_UNSUPPORTED_DEVICE, fa.FA_ERR_LAUNCH)


S = (8192, 4096, 64)


def forward(**kw):
    a = dict(q=A, q_strides=arr(*S), q_out=2 * A, q_out_strides=arr(*S), k=3 * A, k_strides=arr(4096, 4096, 64), k_out=4 * A,
             k_out_strides=arr(4096, 4096, 64), B=2, Hq=2, Hk=1, N=64, d=64, dtype=fa.FA_BF16, norm=norm(), rotary=rotary(),
             stream=None)
    a.update(kw)
    return fa.fa_qk_norm_rope(**a)


NORM_ERRORS = [
    (dict(B=0), fa.FA_ERR_BAD_SHAPE),
    (dict(N=0), fa.FA_ERR_BAD_SHAPE),
    (dict(N=1 << 30), fa.FA_ERR_BAD_SHAPE),
    (dict(Hk=-1), fa.FA_ERR_BAD_SHAPE),
    (dict(Hq=70000), fa.FA_ERR_BAD_SHAPE),
    (dict(d=72), fa.FA_ERR_UNSUPPORTED_HEADDIM),
    (dict(d=272), fa.FA_ERR_UNSUPPORTED_HEADDIM),
    (dict(dtype=2), fa.FA_ERR_BAD_ARGUMENT),
    (dict(norm=None), fa.FA_ERR_NULL_PTR),
    (dict(norm=norm(weights_fp32=2)), fa.FA_ERR_BAD_ARGUMENT),
    (dict(norm=norm(eps=-1e-6)), fa.FA_ERR_BAD_ARGUMENT),
    (dict(norm=norm(eps=NAN)), fa.FA_ERR_BAD_ARGUMENT),
    (dict(norm=norm(eps=INF)), fa.FA_ERR_BAD_ARGUMENT),
    (dict(norm=norm(q_weight=23 * A + 8)), fa.FA_ERR_MISALIGNED),
    (dict(norm=norm(k_weight=24 * A + 2, weights_fp32=1)), fa.FA_ERR_MISALIGNED),
    (dict(rotary=rotary(rot=24)), fa.FA_ERR_BAD_ARGUMENT),
    (dict(rotary=rotary(axes=None)), fa.FA_ERR_NULL_PTR),
    (dict(q=None), fa.FA_ERR_NULL_PTR),
    (dict(k=None), fa.FA_ERR_NULL_PTR),
    (dict(q=A + 8), fa.FA_ERR_MISALIGNED),
    (dict(q_strides=arr(8192, 4096, 68)), fa.FA_ERR_MISALIGNED),
    (dict(q_strides=arr(8192, -4096, 64)), fa.FA_ERR_BAD_ARGUMENT),
]


@pytest.mark.parametrize("kw,status", NORM_ERRORS + [
    (dict(Hk=0), fa.FA_ERR_BAD_SHAPE),
    (dict(q_out=A + 256), fa.FA_ERR_ALIASING),                       # partly over its input
    (dict(q_out=A, q_out_strides=arr(4096, 8192, 64)), fa.FA_ERR_ALIASING),   # in place, dimensions exchanged
    (dict(q_out=3 * A), fa.FA_ERR_ALIASING),                         # over the other tensor's input
    (dict(k_out=2 * A), fa.FA_ERR_ALIASING),                         # two outputs
    (dict(q_out_strides=arr(8192, 0, 64)), fa.FA_ERR_ALIASING),      # rows on top of each other
    (dict(q_out=20 * A), fa.FA_ERR_ALIASING),                        # over the positions
    (dict(k_out=24 * A), fa.FA_ERR_ALIASING),                        # over the weights
])
def test_norm_refuses(lib, kw, status):
    assert forward(**kw) == status


def test_norm_accepts(lib):
    valid(forward)
    valid(lambda: forward(rotary=None, norm=norm(q_weight=None, k_weight=None)))
    valid(lambda: forward(q_out=A, k_out=3 * A, norm=norm(weights_fp32=1, q_weight=23 * A + 4)))
    valid(lambda: forward(k=None, k_out=None, Hk=0, k_strides=None, k_out_strides=None))


WS = 1 << 22


def backward(**kw):
    a = dict(dq_out=5 * A, dq_out_strides=arr(*S), q=A, q_strides=arr(*S), dq=2 * A, dq_strides=arr(*S), dk_out=6 * A,
             dk_out_strides=arr(4096, 4096, 64), k=3 * A, k_strides=arr(4096, 4096, 64), dk=4 * A,
             dk_strides=arr(4096, 4096, 64), dq_weight=7 * A, dk_weight=8 * A, B=2, Hq=2, Hk=1, N=64, d=64,
             dtype=fa.FA_BF16, norm=norm(), rotary=rotary(), workspace=9 * A, workspace_bytes=WS, stream=None)
    a.update(kw)
    return fa.fa_qk_norm_rope_bwd(**a)


@pytest.mark.parametrize("kw,status", NORM_ERRORS + [
    (dict(dq_out=None), fa.FA_ERR_NULL_PTR),
    (dict(dk=None), fa.FA_ERR_NULL_PTR),
    (dict(Hk=0), fa.FA_ERR_BAD_SHAPE),
    (dict(workspace=None), fa.FA_ERR_NULL_PTR),
    (dict(workspace_bytes=64), fa.FA_ERR_WORKSPACE_TOO_SMALL),
    (dict(dq_weight=7 * A + 2), fa.FA_ERR_MISALIGNED),
    (dict(dq=A), fa.FA_ERR_ALIASING),                                # over the forward's input
    (dict(dq=5 * A, dq_strides=arr(4096, 8192, 64)), fa.FA_ERR_ALIASING),
    (dict(dq=6 * A), fa.FA_ERR_ALIASING),                            # over the other tensor's gradient
    (dict(dk=2 * A), fa.FA_ERR_ALIASING),
    (dict(dk_weight=7 * A), fa.FA_ERR_ALIASING),
    (dict(dk_weight=24 * A), fa.FA_ERR_ALIASING),                    # over the weights
    (dict(workspace=A), fa.FA_ERR_ALIASING),
    (dict(workspace=7 * A), fa.FA_ERR_ALIASING),
])
def test_norm_gradient_refuses(lib, kw, status):
    assert backward(**kw) == status


def test_norm_gradient_accepts(lib):
    valid(backward)
    valid(lambda: backward(dq=5 * A, dk=6 * A))
    valid(lambda: backward(dq_weight=None, dk_weight=None, workspace=None, workspace_bytes=0))
    valid(lambda: backward(dk_out=None, k=None, dk=None, dk_weight=None, Hk=0, dk_out_strides=None, k_strides=None,
                           dk_strides=None))
    assert 0 < fa.fa_qk_norm_rope_bwd_workspace_bytes(64) <= WS
    assert fa.fa_qk_norm_rope_bwd_workspace_bytes(72) == 0 and fa.fa_qk_norm_rope_bwd_workspace_bytes(0) == 0


def pool(**kw):
    a = dict(data=A, page_stride=2 * 16 * 72, head_stride=16 * 72, num_pages=8, page_size=16, Hkv=2, d=64, dtype=fa.FA_BF16)
    a.update(kw)
    return fa.fa_paged4_kv(**a)


def table(**kw):
    a = dict(pages=5 * A, stride=4, max_pages=4)
    a.update(kw)
    return fa.fa_page_table(**a)


POOL_ERRORS = [
    (dict(data=None), fa.FA_ERR_NULL_PTR),
    (dict(dtype=7), fa.FA_ERR_BAD_ARGUMENT),
    (dict(num_pages=0), fa.FA_ERR_BAD_SHAPE),
    (dict(Hkv=0), fa.FA_ERR_BAD_SHAPE),
    (dict(page_size=8), fa.FA_ERR_BAD_SHAPE),
    (dict(page_size=24), fa.FA_ERR_BAD_SHAPE),
    (dict(page_size=65552), fa.FA_ERR_BAD_SHAPE),
    (dict(d=96), fa.FA_ERR_UNSUPPORTED_HEADDIM),
    (dict(head_stride=16 * 72 + 8), fa.FA_ERR_MISALIGNED),
    (dict(head_stride=0), fa.FA_ERR_BAD_ARGUMENT),           # heads on top of each other
    (dict(head_stride=16 * 71), fa.FA_ERR_BAD_ARGUMENT),     # a page is longer
    (dict(page_stride=-4096), fa.FA_ERR_BAD_ARGUMENT),
    (dict(page_stride=1 << 60), fa.FA_ERR_BAD_ARGUMENT),
    (dict(data=A + 8), fa.FA_ERR_MISALIGNED),
]
TABLE_ERRORS = [
    (dict(kv=None), fa.FA_ERR_NULL_PTR),
    (dict(table=None), fa.FA_ERR_NULL_PTR),
    (dict(table=table(max_pages=0)), fa.FA_ERR_BAD_SHAPE),
    (dict(table=table(max_pages=2 ** 26 + 1)), fa.FA_ERR_BAD_SHAPE),
    (dict(table=table(pages=5 * A + 2)), fa.FA_ERR_MISALIGNED),
    (dict(seq_lens=None), fa.FA_ERR_NULL_PTR),
    (dict(seq_lens=6 * A + 2), fa.FA_ERR_MISALIGNED),
    (dict(B=0), fa.FA_ERR_BAD_SHAPE),
]
CACHE_ERRORS = [(dict(kv=pool(**k)), s) for k, s in POOL_ERRORS] + TABLE_ERRORS


def append(**kw):
    a = dict(kv=pool(), table=table(), seq_lens=6 * A, cu_seqlens=None, B=2, T=2, k=7 * A, k_strides=arr(512, 64),
             v=7 * A + 256, v_strides=arr(512, 64), q=7 * A + 512, q_strides=arr(512, 64), q_out=7 * A + 512,
             q_out_strides=arr(512, 64), Hq=4, norm=norm(), rotary=rotary(), stream=None)
    a.update(kw)
    return fa.fa_paged4_append(**a)


@pytest.mark.parametrize("kw,status", CACHE_ERRORS + [
    (dict(table=table(pages=A)), fa.FA_ERR_ALIASING),
    (dict(T=3), fa.FA_ERR_BAD_SHAPE),                         # one token a sequence
    (dict(T=-1, cu_seqlens=9 * A), fa.FA_ERR_BAD_SHAPE),
    (dict(norm=None, rotary=None), fa.FA_ERR_BAD_ARGUMENT),   # q with nothing to do to it
    (dict(q=None), fa.FA_ERR_NULL_PTR),
    (dict(Hq=0), fa.FA_ERR_BAD_SHAPE),
    (dict(k=A + 4096), fa.FA_ERR_ALIASING),                   # the new rows lie in the pool
    (dict(q_out=A), fa.FA_ERR_ALIASING),
    (dict(q_out=7 * A), fa.FA_ERR_ALIASING),                  # q_out over k
    (dict(q_out=23 * A), fa.FA_ERR_ALIASING),                 # q_out over the weights
    (dict(Hq=2, q_out_strides=arr(64, 512)), fa.FA_ERR_ALIASING),   # in place, dimensions exchanged
    (dict(v_strides=arr(512, 63)), fa.FA_ERR_MISALIGNED),
    (dict(norm=norm(eps=-1.0)), fa.FA_ERR_BAD_ARGUMENT),
    (dict(rotary=rotary(rot=128)), fa.FA_ERR_BAD_ARGUMENT),
])
def test_append_refuses(lib, kw, status):
    assert append(**kw) == status


def test_append_accepts(lib):
    valid(append)
    valid(lambda: append(norm=None))
    valid(lambda: append(rotary=None))
    valid(lambda: append(norm=None, rotary=None, q=None, q_out=None, Hq=0, q_strides=None, q_out_strides=None))
    assert append(T=0, cu_seqlens=9 * A) == fa.FA_OK


def read(**kw):
    a = dict(kv=pool(), table=table(), seq_lens=6 * A, k=7 * A, k_strides=arr(*S), v=8 * A, v_strides=arr(*S), B=2, N=64,
             stream=None)
    a.update(kw)
    return fa.fa_paged4_read(**a)


@pytest.mark.parametrize("kw,status", CACHE_ERRORS + [
    (dict(k=None), fa.FA_ERR_NULL_PTR),
    (dict(N=0), fa.FA_ERR_BAD_SHAPE),
    (dict(N=2 ** 30 + 1), fa.FA_ERR_BAD_SHAPE),
    (dict(v=7 * A), fa.FA_ERR_ALIASING),
    (dict(k=A), fa.FA_ERR_ALIASING),
    (dict(v_strides=arr(8192, 0, 64)), fa.FA_ERR_ALIASING),
    (dict(k=7 * A + 8), fa.FA_ERR_MISALIGNED),
])
def test_read_refuses(lib, kw, status):
    assert read(**kw) == status


def decode(**kw):
    a = dict(q=7 * A, q_strides=arr(256, 64), kv=pool(), table=table(), seq_lens=6 * A, o=9 * A, lse=10 * A, B=2, Hq=4,
             window=0, scale=0.125, workspace=11 * A, workspace_bytes=1 << 24, stream=None)
    a.update(kw)
    return fa.fa_paged4_decode(**a)


@pytest.mark.parametrize("kw,status", CACHE_ERRORS + [
    (dict(q=None), fa.FA_ERR_NULL_PTR),
    (dict(workspace=None), fa.FA_ERR_NULL_PTR),
    (dict(Hq=3), fa.FA_ERR_BAD_SHAPE),
    (dict(window=-1), fa.FA_ERR_BAD_ARGUMENT),
    (dict(scale=0.0), fa.FA_ERR_BAD_ARGUMENT),
    (dict(scale=INF), fa.FA_ERR_BAD_ARGUMENT),
    (dict(workspace_bytes=16), fa.FA_ERR_WORKSPACE_TOO_SMALL),
    (dict(q_strides=arr(256, 60)), fa.FA_ERR_MISALIGNED),
    (dict(lse=10 * A + 4), fa.FA_ERR_MISALIGNED),
    (dict(o=7 * A), fa.FA_ERR_ALIASING),
    (dict(o=A + 64), fa.FA_ERR_ALIASING),
    (dict(lse=9 * A), fa.FA_ERR_ALIASING),
    (dict(workspace=A), fa.FA_ERR_ALIASING),
])
def test_decode_refuses(lib, kw, status):
    assert decode(**kw) == status


def test_read_and_decode_accept(lib):
    valid(read)
    valid(decode)
    f = fa.fa_paged4_decode_workspace_bytes
    assert 0 < f(2, 4, 2, 64) <= 1 << 24
    assert f(2, 4, 3, 64) == 0 and f(2, 4, 2, 96) == 0 and f(0, 4, 2, 64) == 0


def test_binding_refuses_cpu_tensors_and_wrong_types():
    import torch
    cache = fa.paged4_cache(4, 2, 16, 64, device="cpu")
    assert cache.shape == (4, 2, 16, 72) and cache.dtype == torch.uint8
    t, n = torch.zeros((1, 2), dtype=torch.int32), torch.zeros((1,), dtype=torch.int32)
    q = torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.paged4_decode(q, cache, t, n)
    with pytest.raises(TypeError):
        fa.paged4_decode(q.float(), cache, t, n)
    with pytest.raises(ValueError):
        fa.paged4_read(cache, t, n, 4, torch.bfloat16)
    with pytest.raises(TypeError):
        fa.paged4_read(cache, t, n, 4, torch.float32)
    with pytest.raises(ValueError):
        fa.paged4_append(cache, t, n, q, q)
    with pytest.raises(ValueError):
        fa.qk_norm_rope(q[None], None, None, None)
    with pytest.raises(TypeError):
        fa.qk_norm_rope(q[None].float(), None, None, None)
    for bad in (dict(d=96), dict(page_size=8)):
        with pytest.raises(fa.FAError):
            fa.paged4_cache(**dict(dict(pages=4, Hkv=2, page_size=16, d=64, device="cpu"), **bad))

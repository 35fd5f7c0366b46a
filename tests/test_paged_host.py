"""Paged cache and rotary positions on the CPU: pins of their fp64 oracle
(closed forms, the contiguous-attention oracle, differences) and the refusals
of the C entry points, which come before any CUDA call."""
import ctypes
import math
import os

import numpy as np
import pytest

import exact_io_aware_flashattention_gb300 as fa
from exact_io_aware_flashattention_gb300 import _build
from oracle import paged, ref


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fa.load_library()


# ---------------------------------------------------------------------------
# Oracle pins
# ---------------------------------------------------------------------------
def test_rotation_of_one_pair():
    # d = 2, one pair: (1, 0) turns to (cos, sin).
    x = np.array([1.0, 0.0]).reshape(1, 1, 1, 2)
    y = paged.rotate(x, np.array([[[5]]]), [0.25], [0])
    assert np.allclose(y.ravel(), [math.cos(1.25), math.sin(1.25)], atol=1e-15)
    z = paged.rotate(y, np.array([[[5]]]), [0.25], [0], inverse=True)
    assert np.allclose(z, x, atol=1e-15)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_dot_products_of_relative_positions(interleaved):
    # q at position p + s and k at p: the product depends on s alone.
    r = np.random.default_rng(0)
    q, k, w = r.normal(size=(1, 1, 1, 16)), r.normal(size=(1, 1, 1, 16)), 0.3 ** np.arange(8)
    axes = [0, 1, 2, 0, 1, 2, 0, 1]

    def dot(p):
        turn = lambda x, at: paged.rotate(x, np.array(at).reshape(3, 1, 1), w, axes, interleaved)  # noqa: E731
        return float((turn(q, [p + 3, 2 * p + 1, p]) * turn(k, [p, 2 * p, p + 4])).sum())
    assert abs(dot(0) - dot(1234)) < 1e-9


def test_rotation_gradient_against_differences():
    r = np.random.default_rng(1)
    x, g = r.normal(size=(1, 2, 3, 24)), r.normal(size=(1, 2, 3, 24))
    pos, w, axes = r.integers(0, 50, size=(2, 1, 3)), 0.5 ** np.arange(8), [0, 0, 1, 1, 0, 1, 0, 1]
    grad = paged.rotate(g, pos, w, axes, inverse=True)
    for _ in range(10):
        at = tuple(r.integers(0, n) for n in x.shape)
        e = np.zeros_like(x)
        e[at] = 1e-6
        num = (g * (paged.rotate(x + e, pos, w, axes) - paged.rotate(x - e, pos, w, axes))).sum() / 2e-6
        assert abs(num - grad[at]) < 1e-8


@pytest.mark.parametrize("window", [0, 5])
def test_decode_equals_last_row_of_contiguous_attention(window):
    r = np.random.default_rng(2)
    B, Hq, Hkv, n, d, ps = 2, 4, 2, 37, 8, 16
    k, v, q = r.normal(size=(B, Hkv, n, d)), r.normal(size=(B, Hkv, n, d)), r.normal(size=(B, Hq, 1, d))
    table = np.array([[4, 0, 2], [1, 5, 3]])
    kc, vc = np.full((6, Hkv, ps, d), np.nan), np.full((6, Hkv, ps, d), np.nan)
    for b in range(B):
        for j in range(n):
            kc[table[b, j // ps], :, j % ps], vc[table[b, j // ps], :, j % ps] = k[b, :, j], v[b, :, j]
    o, lse, weights, a = paged.decode(q[:, :, 0], kc, vc, table, [n, n], 0.4, window)
    ro, rl = ref.attention_forward(q, k, v, True, 0.4, window=window)
    assert np.allclose(o, ro[:, :, 0], atol=1e-12) and np.allclose(lse, rl[:, :, 0], atol=1e-12)
    assert all(np.allclose(w.sum(1), Hq // Hkv) for w in weights)
    assert np.all(a >= np.abs(o) - 1e-12)


def test_decode_of_an_empty_sequence():
    o, lse, weights, _ = paged.decode(np.ones((1, 2, 4)), np.ones((1, 1, 16, 4)), np.ones((1, 1, 16, 4)), [[0]], [0], 1.0)
    assert not o.any() and np.all(lse == -np.inf) and weights[0].shape == (1, 0)


def test_kept_keys_by_hand():
    s = [5.0, 1.0, 3.0, 3.0, 3.0, 0.0, 9.0, 0.5]
    assert paged.kept_keys(s, 8, 0, 0) == list(range(8))
    assert paged.kept_keys(s, 4, 0, 0) == [0, 2, 3, 6]             # ties: the lowest indices
    assert paged.kept_keys(s, 4, 2, 1) == [0, 2, 6, 7]
    assert paged.kept_keys([0.0, -0.0, math.nan, 0.0], 2, 0, 0) == [0, 1]
    assert paged.kept_keys([math.nan, -1.0, math.nan], 2, 0, 0) == [0, 1]
    assert paged.kept_keys(s, 1, 1, 0) == [7]


def test_token_places():
    assert paged.token_places([3, 0, 1], None, 3) == [(0, 2), None, (2, 0)]
    assert paged.token_places([5, 0, 2], [0, 2, 2, 3], 5) == [(0, 3), (0, 4), (2, 1), None, None]


# ---------------------------------------------------------------------------
# Refusals
# ---------------------------------------------------------------------------
A = 1 << 24   # fake, aligned, far apart "device" addresses (never dereferenced)
LL = ctypes.c_longlong


def arr(*x):
    return (LL * len(x))(*x)


def rotary(**kw):
    a = dict(positions=20 * A, axis_stride=64, batch_stride=0, inv_freq=21 * A, axes=22 * A, n_axes=3, rot=64, interleaved=0)
    a.update(kw)
    return fa.fa_rotary(**a)


def rope(**kw):
    a = dict(q=A, q_strides=arr(8192, 4096, 64), q_out=2 * A, q_out_strides=arr(8192, 4096, 64), k=3 * A,
             k_strides=arr(4096, 4096, 64), k_out=4 * A, k_out_strides=arr(4096, 4096, 64), B=2, Hq=2, Hk=1, N=64, d=64,
             dtype=fa.FA_BF16, rotary=rotary(), inverse=0, stream=None)
    a.update(kw)
    return fa.fa_rope(**a)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), fa.FA_ERR_NULL_PTR),
    (dict(k=None), fa.FA_ERR_NULL_PTR),
    (dict(Hk=0), fa.FA_ERR_BAD_SHAPE),
    (dict(B=0), fa.FA_ERR_BAD_SHAPE),
    (dict(N=0), fa.FA_ERR_BAD_SHAPE),
    (dict(N=1 << 30, B=2), fa.FA_ERR_BAD_SHAPE),
    (dict(d=72), fa.FA_ERR_UNSUPPORTED_HEADDIM),
    (dict(d=272), fa.FA_ERR_UNSUPPORTED_HEADDIM),
    (dict(dtype=2), fa.FA_ERR_BAD_ARGUMENT),
    (dict(inverse=2), fa.FA_ERR_BAD_ARGUMENT),
    (dict(q=A + 8), fa.FA_ERR_MISALIGNED),
    (dict(q_strides=arr(8192, 4096, 68)), fa.FA_ERR_MISALIGNED),
    (dict(q_strides=arr(8192, -4096, 64)), fa.FA_ERR_BAD_ARGUMENT),
    (dict(q_strides=arr(1 << 60, 4096, 64)), fa.FA_ERR_BAD_ARGUMENT),
    (dict(q_out=A + 256), fa.FA_ERR_ALIASING),                       # partly over its input
    (dict(q_out=A, q_out_strides=arr(8192, 64, 128)), fa.FA_ERR_ALIASING),   # in place with other strides
    (dict(q_out=3 * A), fa.FA_ERR_ALIASING),                         # over the other tensor's input
    (dict(k_out=2 * A), fa.FA_ERR_ALIASING),                         # two outputs
    (dict(q_out_strides=arr(8192, 0, 64)), fa.FA_ERR_ALIASING),      # rows on top of each other
    (dict(q_out=20 * A), fa.FA_ERR_ALIASING),                        # over the positions
    (dict(rotary=rotary(rot=24)), fa.FA_ERR_BAD_ARGUMENT),
    (dict(rotary=rotary(rot=128)), fa.FA_ERR_BAD_ARGUMENT),
    (dict(rotary=rotary(n_axes=0)), fa.FA_ERR_BAD_ARGUMENT),
    (dict(rotary=rotary(interleaved=2)), fa.FA_ERR_BAD_ARGUMENT),
    (dict(rotary=rotary(axes=None)), fa.FA_ERR_NULL_PTR),
    (dict(rotary=rotary(inv_freq=21 * A + 4)), fa.FA_ERR_MISALIGNED),
    (dict(rotary=None), fa.FA_ERR_NULL_PTR),
])
def test_rope_refuses(lib, kw, status):
    assert rope(**kw) == status


OK_OR_NO_GPU = (fa.FA_OK, fa.FA_ERR_CUDA, fa.FA_ERR_UNSUPPORTED_DEVICE, fa.FA_ERR_LAUNCH)


def valid(call):
    """A valid call passes every check and then fails for want of a GPU; where there is one it is not made."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("fake addresses: only where no kernel can run")
    assert call() in OK_OR_NO_GPU[1:]


def test_rope_accepts_in_place_on_parts_of_one_projection(lib):
    # [B, N, Hq + Hk, d]: q and k are interleaved row by row; turned in place.
    s = arr(64 * 192, 64, 192)
    valid(lambda: rope(q=A, q_strides=s, q_out=A, q_out_strides=s, k=A + 256, k_strides=s, k_out=A + 256, k_out_strides=s))
    # [B, Hq + Hk, N, d]: q and k are interleaved batch by batch.
    s = arr(3 * 4096, 4096, 64)
    valid(lambda: rope(q=A, q_strides=s, q_out=A, q_out_strides=s, k=A + 2 * 8192, k_strides=s, k_out=A + 2 * 8192,
                       k_out_strides=s))
    # The same with k one head too early.
    assert rope(q=A, q_strides=s, q_out=A, q_out_strides=s, k=A + 8192, k_strides=s, k_out=A + 8192,
                k_out_strides=s) == fa.FA_ERR_ALIASING


def pool(**kw):
    # [pages, 2, Hkv, page, d]: k and v interleaved page by page.
    a = dict(k=A, v=A + 2 * 16 * 64 * 2, page_stride=2 * 2 * 16 * 64, head_stride=16 * 64, slot_stride=64, num_pages=8,
             page_size=16, Hkv=2, d=64, dtype=fa.FA_BF16)
    a.update(kw)
    return fa.fa_paged_kv(**a)


def table(**kw):
    a = dict(pages=5 * A, stride=4, max_pages=4)
    a.update(kw)
    return fa.fa_page_table(**a)


def append(**kw):
    a = dict(kv=pool(), table=table(), seq_lens=6 * A, cu_seqlens=None, B=2, T=2, k=7 * A, k_strides=arr(512, 64),
             v=7 * A + 256, v_strides=arr(512, 64), q=7 * A + 512, q_strides=arr(512, 64), q_out=7 * A + 512,
             q_out_strides=arr(512, 64), Hq=4, rotary=rotary(), scores=8 * A, stream=None)
    a.update(kw)
    return fa.fa_paged_append(**a)


POOL_ERRORS = [
    (dict(k=None), fa.FA_ERR_NULL_PTR),
    (dict(dtype=7), fa.FA_ERR_BAD_ARGUMENT),
    (dict(num_pages=0), fa.FA_ERR_BAD_SHAPE),
    (dict(page_size=8), fa.FA_ERR_BAD_SHAPE),
    (dict(page_size=24), fa.FA_ERR_BAD_SHAPE),
    (dict(d=96), fa.FA_ERR_UNSUPPORTED_HEADDIM),
    (dict(slot_stride=60), fa.FA_ERR_MISALIGNED),
    (dict(head_stride=0), fa.FA_ERR_BAD_ARGUMENT),           # heads on top of each other
    (dict(page_stride=-4096), fa.FA_ERR_BAD_ARGUMENT),
    (dict(v=A + 8), fa.FA_ERR_MISALIGNED),
]


@pytest.mark.parametrize("kw,status", [(dict(kv=pool(**k)), s) for k, s in POOL_ERRORS] + [
    (dict(kv=None), fa.FA_ERR_NULL_PTR),
    (dict(kv=pool(v=A + 1024)), fa.FA_ERR_ALIASING),          # k's and v's pages overlap
    (dict(table=None), fa.FA_ERR_NULL_PTR),
    (dict(table=table(max_pages=0)), fa.FA_ERR_BAD_SHAPE),
    (dict(table=table(max_pages=2 ** 26 + 1)), fa.FA_ERR_BAD_SHAPE),       # more than 2^30 keys a sequence
    (dict(table=table(pages=5 * A + 2)), fa.FA_ERR_MISALIGNED),
    (dict(table=table(pages=A)), fa.FA_ERR_ALIASING),
    (dict(seq_lens=None), fa.FA_ERR_NULL_PTR),
    (dict(T=3), fa.FA_ERR_BAD_SHAPE),                         # one token a sequence
    (dict(T=-1, cu_seqlens=9 * A), fa.FA_ERR_BAD_SHAPE),
    (dict(B=0), fa.FA_ERR_BAD_SHAPE),
    (dict(rotary=None), fa.FA_ERR_BAD_ARGUMENT),              # q without rotary
    (dict(q=None), fa.FA_ERR_NULL_PTR),
    (dict(Hq=0), fa.FA_ERR_BAD_SHAPE),
    (dict(k=A + 4096), fa.FA_ERR_ALIASING),                   # the new rows lie in the pool
    (dict(q_out=A), fa.FA_ERR_ALIASING),
    (dict(q_out=7 * A), fa.FA_ERR_ALIASING),                  # q_out over k
    (dict(scores=A), fa.FA_ERR_ALIASING),
    (dict(scores=8 * A + 4), fa.FA_ERR_MISALIGNED),
    (dict(v_strides=arr(512, 63)), fa.FA_ERR_MISALIGNED),
])
def test_append_refuses(lib, kw, status):
    assert append(**kw) == status


def test_in_place_with_two_dimensions_exchanged_is_refused(lib):
    # The rows are the same ones, but each is written where another is read:
    # batch and head of q, head and token of k, token and head of appended q.
    s = arr(8192, 4096, 64)
    assert rope(q_out=A, q_out_strides=arr(4096, 8192, 64)) == fa.FA_ERR_ALIASING
    assert rope(q_strides=s, q_out=A, q_out_strides=s, k=3 * A, k_strides=arr(1 << 20, 4096, 64), Hk=64, k_out=3 * A,
                k_out_strides=arr(1 << 20, 64, 4096)) == fa.FA_ERR_ALIASING
    assert append(Hq=2, q_strides=arr(512, 64), q_out_strides=arr(64, 512)) == fa.FA_ERR_ALIASING
    # A stride that is never stepped does not matter.
    valid(lambda: rope(B=1, q_out=A, q_out_strides=arr(64, 4096, 64)))


def test_append_accepts_a_projection_and_an_interleaved_pool(lib):
    valid(append)
    assert append(T=0, cu_seqlens=9 * A) == fa.FA_OK


WS = 1 << 26


def decode(**kw):
    a = dict(q=7 * A, q_strides=arr(256, 64), kv=pool(), table=table(), seq_lens=6 * A, o=9 * A, lse=10 * A, scores=8 * A,
             B=2, Hq=4, window=0, scale=0.125, workspace=11 * A, workspace_bytes=WS, stream=None)
    a.update(kw)
    return fa.fa_paged_decode(**a)


@pytest.mark.parametrize("kw,status", [(dict(kv=pool(**k)), s) for k, s in POOL_ERRORS] + [
    (dict(q=None), fa.FA_ERR_NULL_PTR),
    (dict(workspace=None), fa.FA_ERR_NULL_PTR),
    (dict(Hq=3), fa.FA_ERR_BAD_SHAPE),
    (dict(B=0), fa.FA_ERR_BAD_SHAPE),
    (dict(window=-1), fa.FA_ERR_BAD_ARGUMENT),
    (dict(scale=0.0), fa.FA_ERR_BAD_ARGUMENT),
    (dict(scale=float("inf")), fa.FA_ERR_BAD_ARGUMENT),
    (dict(workspace_bytes=16), fa.FA_ERR_WORKSPACE_TOO_SMALL),
    (dict(q_strides=arr(256, 60)), fa.FA_ERR_MISALIGNED),
    (dict(lse=10 * A + 4), fa.FA_ERR_MISALIGNED),
    (dict(o=7 * A), fa.FA_ERR_ALIASING),
    (dict(o=A + 64), fa.FA_ERR_ALIASING),
    (dict(lse=9 * A), fa.FA_ERR_ALIASING),
    (dict(workspace=A), fa.FA_ERR_ALIASING),
    (dict(scores=9 * A), fa.FA_ERR_ALIASING),
])
def test_decode_refuses(lib, kw, status):
    assert decode(**kw) == status


def test_decode_workspace(lib):
    f = fa.fa_paged_decode_workspace_bytes
    assert 0 < f(2, 4, 2, 64, 16, 4, 0) <= f(2, 4, 2, 64, 16, 4, 1) <= WS
    assert f(2, 4, 3, 64, 16, 4, 0) == 0 and f(2, 4, 2, 96, 16, 4, 0) == 0 and f(0, 4, 2, 64, 16, 4, 0) == 0
    assert f(2, 4, 2, 64, 20, 4, 0) == 0 and f(2, 4, 2, 64, 16, 0, 0) == 0
    assert f(1, 1, 1, 64, 16, 2 ** 26, 0) > 0 and f(1, 1, 1, 64, 16, 2 ** 26 + 1, 0) == 0
    valid(decode)


def evict(**kw):
    a = dict(kv=pool(), scores=8 * A, table=table(), seq_lens=6 * A, dst=table(pages=5 * A + 4096), new_lens=12 * A,
             kept=13 * A, B=2, budget=20, recent=4, sinks=2, stream=None)
    a.update(kw)
    return fa.fa_paged_evict(**a)


@pytest.mark.parametrize("kw,status", [(dict(kv=pool(**k)), s) for k, s in POOL_ERRORS] + [
    (dict(scores=None), fa.FA_ERR_NULL_PTR),
    (dict(kept=None), fa.FA_ERR_NULL_PTR),
    (dict(dst=None), fa.FA_ERR_NULL_PTR),
    (dict(budget=0), fa.FA_ERR_BAD_ARGUMENT),
    (dict(budget=65), fa.FA_ERR_BAD_ARGUMENT),                # more than dst's pages hold
    (dict(dst=table(pages=5 * A + 4096, max_pages=2 ** 26 + 1)), fa.FA_ERR_BAD_SHAPE),
    (dict(recent=-1), fa.FA_ERR_BAD_ARGUMENT),
    (dict(recent=10, sinks=11), fa.FA_ERR_BAD_ARGUMENT),
    (dict(recent=2 ** 31 - 1, sinks=2 ** 31 - 1), fa.FA_ERR_BAD_ARGUMENT),
    (dict(dst=table()), fa.FA_ERR_ALIASING),                  # onto the source pages
    (dict(kept=12 * A), fa.FA_ERR_ALIASING),
    (dict(new_lens=6 * A), fa.FA_ERR_ALIASING),
    (dict(kv=pool(v=A + 1024)), fa.FA_ERR_ALIASING),
])
def test_evict_refuses(lib, kw, status):
    assert evict(**kw) == status


def test_evict_accepts(lib):
    valid(evict)


def test_bad_index_has_a_text(lib):
    assert "out of range" in fa.fa_strerror(fa.FA_ERR_BAD_INDEX)


def test_rope_frequencies():
    w, ax = fa.rope_frequencies((2, 3, 3), base=100.0, device="cpu")
    assert ax.tolist() == [0, 0, 1, 1, 1, 2, 2, 2]
    assert np.allclose(w.numpy(), 100.0 ** (-np.arange(8) / 8))
    with pytest.raises(ValueError):
        fa.rope_frequencies((0, 0))


def test_binding_refuses_cpu_tensors_and_wrong_types():
    import torch
    kc = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)
    t, n = torch.zeros((1, 2), dtype=torch.int32), torch.zeros((1,), dtype=torch.int32)
    w, ax = fa.rope_frequencies((32,), device="cpu")
    with pytest.raises(ValueError):
        fa.paged_decode(torch.zeros((1, 2, 64), dtype=torch.bfloat16), kc, kc.clone(), t, n)
    with pytest.raises(TypeError):
        fa.rope(torch.zeros((1, 2, 4, 64)), None, torch.zeros((1, 1, 4), dtype=torch.int32), w, ax)
    with pytest.raises(ValueError):
        fa.rope(kc[0], None, torch.zeros((1, 1, 4), dtype=torch.int32), w, ax)


# ---------------------------------------------------------------------------
# The native marshalling's build
# ---------------------------------------------------------------------------
@pytest.fixture
def fresh_native(lib, monkeypatch):
    """The native marshalling as a new process finds it."""
    pytest.importorskip("torch")
    monkeypatch.setattr(fa, "_native", None)
    if not fa.native_marshalling():
        pytest.skip("not built here (see _lib/fa_torch.txt)")
    monkeypatch.setattr(fa, "_native", None)


@pytest.mark.parametrize("what", ["torch", "fa.h"])
def test_native_marshalling_of_another_torch_or_header_is_not_loaded(fresh_native, monkeypatch, tmp_path, what):
    if what == "torch":
        import torch
        monkeypatch.setattr(torch, "__version__", torch.__version__ + "1")
    else:
        text = open(os.path.join(_build.INCLUDE, "fa.h")).read()
        (tmp_path / "fa.h").write_text(text.replace("int n_axes;", "int n_axes, more;"))
        monkeypatch.setattr(_build, "INCLUDE", str(tmp_path))
    assert not fa.native_marshalling()
    assert not _build.native_up_to_date()


def test_native_marshalling_is_compiled_again_for_another_torch(fresh_native, monkeypatch):
    # The library's sources are as they were: only the module is built.
    import torch
    made = []
    monkeypatch.setattr(_build, "_compile_torch", lambda: made.append(1))
    monkeypatch.setattr(_build, "_compile", lambda src: pytest.fail("the library was compiled"))
    _build.build()
    assert not made
    monkeypatch.setattr(torch, "__version__", torch.__version__ + "1")
    _build.build()
    assert made


@pytest.mark.parametrize("failure", ["compiler", "no compiler"])
def test_a_failed_build_leaves_no_native_marshalling(monkeypatch, tmp_path, failure):
    so, log = tmp_path / "fa_torch.so", tmp_path / "fa_torch.txt"
    so.write_bytes(b"of an earlier build")
    monkeypatch.setattr(_build, "TORCH_PATH", str(so))
    monkeypatch.setattr(_build, "TORCH_LOG", str(log))

    def run(cmd, **kw):
        if failure == "no compiler":
            raise FileNotFoundError("g++")
        return _build.subprocess.CompletedProcess(cmd, 1, "", "an error")
    monkeypatch.setattr(_build.subprocess, "run", run)
    _build._compile_torch()
    assert not so.exists()
    assert ("an error" if failure == "compiler" else "FileNotFoundError") in log.read_text()
    assert _build.native_up_to_date()              # not tried again with the same torch, Python and header

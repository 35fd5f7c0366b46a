"""fp64 NumPy definitions of the norms of queries and keys and of the cache
held in 4 bits.

Test infrastructure only, like the rest of this package: written from the
formulas, sharing nothing with the CUDA path.
"""
import math

import numpy as np

from oracle import paged

GROUP = 64


def norm(x, w, eps):
    """Rows x [..., d] times (mean of squares + eps)^-1/2 times w (None: ones)."""
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return x * r * (1.0 if w is None else w)


def norm_rope(x, w, eps, rotary=None):
    """x [B, H, N, d]; rotary (positions, inv_freq, axes, interleaved) or None."""
    y = norm(x, w, eps)
    return y if rotary is None else paged.rotate(y, *rotary)


def norm_rope_backward(dy, x, w, eps, rotary=None):
    """Gradients of x and of the weights (those of ones where w is None)."""
    g = dy if rotary is None else paged.rotate(dy, *rotary, inverse=True)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xr, gw = x * r, g * (1.0 if w is None else w)
    return r * (gw - xr * (gw * xr).mean(-1, keepdims=True)), (g * xr).reshape(-1, x.shape[-1]).sum(0)


def quantise(x, round16):
    """Codes [..., d], and s and z [..., d / 64], of rows of 16-bit values x [..., d]; round16 rounds to their type."""
    y = x.reshape(x.shape[:-1] + (x.shape[-1] // GROUP, GROUP))
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        lo, hi = y.min(-1), y.max(-1)               # NaN where there is one
        s = round16((hi - lo) / 15.0)
        c = np.where(s[..., None] == 0, 0.0, np.rint((y - lo[..., None]) / s[..., None]))
        c = np.clip(c, 0, 15)
    return c.reshape(x.shape), s, lo


def values(x, round16):
    """What the cache's codes of 16-bit rows x stand for."""
    c, s, z = quantise(x, round16)
    c = c.reshape(s.shape + (GROUP,))
    with np.errstate(invalid="ignore"):
        return (z[..., None] + s[..., None] * c).reshape(x.shape)


def sizes(x, round16):
    """|z| + 32 s of each element's group: what the sums of a product with such a row are made of, at most."""
    _, s, z = quantise(x, round16)
    return np.repeat(np.abs(z) + 32 * s, GROUP, axis=-1)


def decode(q, k, v, scale, window, round16):
    """q [Hq, d] against one sequence's 16-bit rows k, v [Hkv, n, d] as held in 4 bits.  Returns o, lse, and what
    bounds their errors: x [Hq], the largest scale * sum |q| (|z| + 32 s) of a visible key, and a [Hq, d], the sums of
    p (|z| + 32 s) of V."""
    Hq, d = q.shape
    G, n = Hq // k.shape[0], k.shape[1]
    first = max(0, n - window) if window else 0
    o, a, lse, x = np.zeros((Hq, d)), np.zeros((Hq, d)), np.full(Hq, -math.inf), np.zeros(Hq)
    kv, vv, ks, vs = values(k, round16), values(v, round16), sizes(k, round16), sizes(v, round16)
    for h in range(Hq if n > 0 else 0):
        g = h // G
        s = scale * (kv[g, first:] @ q[h])
        m = s.max()
        lse[h] = m + math.log(np.exp(s - m).sum())
        p = np.exp(s - lse[h])
        o[h], a[h] = p @ vv[g, first:], p @ vs[g, first:]
        x[h] = scale * (ks[g, first:] @ np.abs(q[h])).max()
    return o, lse, x, a

"""fp64 NumPy definitions of the rotary positions and the paged-cache operators.

Test infrastructure only, like the rest of this package: written from the
formulas with plain loops, sharing nothing with the CUDA path.
"""
import math

import numpy as np


def rotate(x, positions, inv_freq, axes, interleaved=False, inverse=False):
    """x [B, H, N, d], positions [n_axes, B, N]: pair i of the first 2 * len(inv_freq)
    elements turned by positions[axes[i]] * inv_freq[i] (negated when inverse)."""
    y = np.array(x, dtype=np.float64)
    r = len(inv_freq)
    for i in range(r):
        lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + r)
        angle = positions[axes[i]].astype(np.float64) * float(inv_freq[i])
        if inverse:
            angle = -angle
        c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
        a, b = np.array(y[..., lo]), np.array(y[..., hi])
        y[..., lo], y[..., hi] = a * c - b * s, b * c + a * s
    return y


def token_places(seq_lens, cu_seqlens, T):
    """(sequence, index) of each of T new tokens, None for padding."""
    out = []
    for t in range(T):
        if cu_seqlens is None:
            out.append((t, seq_lens[t] - 1) if seq_lens[t] > 0 else None)
            continue
        b = [b for b in range(len(seq_lens)) if cu_seqlens[b] <= t < cu_seqlens[b + 1]]
        out.append((b[0], seq_lens[b[0]] - (cu_seqlens[b[0] + 1] - t)) if b else None)
    return out


def gather(cache, pages, n):
    """Rows 0 .. n-1 of a sequence: [Hkv, n, ...] from cache [pages, Hkv, page_size, ...]."""
    ps = cache.shape[2]
    out = np.zeros((cache.shape[1], n) + cache.shape[3:], dtype=cache.dtype)
    for j in range(n):
        out[:, j] = cache[pages[j // ps], :, j % ps]
    return out


def decode(q, k_cache, v_cache, block_table, seq_lens, scale, window=0):
    """q [B, Hq, d].  Returns o [B, Hq, d], lse [B, Hq], the list of per-sequence
    weights [Hkv, len] summed over each group's heads (0 for keys a window hides),
    and a [B, Hq, d], the sums of p |v| that bound how far rounding p moves o."""
    B, Hq, d = q.shape
    G = Hq // k_cache.shape[1]
    o, a = np.zeros((B, Hq, d)), np.zeros((B, Hq, d))
    lse = np.full((B, Hq), -math.inf)
    weights = []
    for b in range(B):
        n = int(seq_lens[b])
        first = max(0, n - window) if window else 0
        k, v = gather(k_cache, block_table[b], n), gather(v_cache, block_table[b], n)
        w = np.zeros((k_cache.shape[1], n))
        for h in range(Hq if n > 0 else 0):
            s = scale * (k[h // G, first:] @ q[b, h])
            m = s.max()
            lse[b, h] = m + math.log(np.exp(s - m).sum())
            p = np.exp(s - lse[b, h])
            o[b, h] = p @ v[h // G, first:]
            a[b, h] = p @ np.abs(v[h // G, first:])
            w[h // G, first:] += p
        weights.append(w)
    return o, lse, weights, a


def kept_keys(scores, budget, recent, sinks):
    """Indices, ascending, of the keys that stay of a sequence's scores [len]."""
    n = len(scores)
    if n <= budget:
        return list(range(n))
    safe = set(range(sinks)) | set(range(n - recent, n))
    value = [-math.inf if math.isnan(x) else float(x) for x in scores]
    rest = sorted((j for j in range(n) if j not in safe),
                  key=lambda j: (1 if math.isnan(scores[j]) else 0, -value[j], j))
    return sorted(list(safe) + rest[:budget - len(safe)])

"""fp64 oracle of the attention layer's operators -- test infrastructure only, numpy, row by row.

* :func:`attn_prep`          -- zero-centred RMSNorm and rotation of query or key heads.
* :func:`attn_prep_backward` -- its gradients.
* :func:`attn_decode`        -- softmax attention of one token per row over a paged cache.
* :func:`page_mean`          -- mean keys of cache pages.
* :func:`attn_select`        -- the pages with the highest score of their mean key.

The pins (hand-worked values, norms kept by the rotation, differences, brute force) are in
``tests/test_attn_oracle.py``.
"""
from __future__ import annotations

import numpy as np


def _f64(x):
    if hasattr(x, "detach"):
        import torch  # only to read a caller's tensor
        x = x.detach().to("cpu", torch.float64).numpy()
    return np.asarray(x, dtype=np.float64)


def _whole(x):
    return np.asarray(x.detach().cpu().numpy() if hasattr(x, "detach") else x, dtype=np.int64)


def _turn(y, positions, inv_freq, sign):
    """Channels i and i + R of each row, i < R, turned by sign * position * inv_freq[i]."""
    R = len(inv_freq)
    angle = sign * positions[:, None, None] * inv_freq  # [N, 1, R]
    a, b = y[..., :R], y[..., R:2 * R]
    out = y.copy()
    out[..., :R] = a * np.cos(angle) - b * np.sin(angle)
    out[..., R:2 * R] = a * np.sin(angle) + b * np.cos(angle)
    return out


def attn_prep(x, w, positions, inv_freq, eps=1e-6):
    """x [N, H, d], w [d], positions [N], inv_freq [R] (radians per position) -> [N, H, d]."""
    x, w, inv_freq, positions = _f64(x), _f64(w), _f64(inv_freq), _f64(positions)
    n = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * (1.0 + w)
    return _turn(n, positions, inv_freq, 1.0)


def attn_prep_backward(dy, x, w, positions, inv_freq, eps=1e-6):
    """(dx [N, H, d], dw [d]) for dL/dy = dy."""
    dy, x, w, inv_freq, positions = _f64(dy), _f64(x), _f64(w), _f64(inv_freq), _f64(positions)
    dn = _turn(dy, positions, inv_freq, -1.0)
    r = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    dw = np.sum(dn * x * r, axis=(0, 1))
    dn = dn * (1.0 + w)
    dx = r * dn - x * r ** 3 * np.mean(dn * x, axis=-1, keepdims=True)
    return dx, dw


def _row_keys(cache, table_row, hk, positions):
    """Cache rows [len(positions), d] of key head hk."""
    ps = cache.shape[2]
    return np.stack([cache[table_row[p // ps], hk, p % ps] for p in positions]) if len(positions) else \
        np.zeros((0, cache.shape[3]))


def attn_decode(q, k_cache, v_cache, page_table, lens, pages=None, scale=None):
    """q [B, Hq, d], caches [num_pages, Hkv, page_size, d] -> y [B, Hq, d]; rows without a key give zeros.
    pages [B, Hkv, n_sel]: logical pages per key head (negative: skipped)."""
    q, k_cache, v_cache, page_table, lens = _f64(q), _f64(k_cache), _f64(v_cache), _whole(page_table), _whole(lens)
    pages = None if pages is None else _whole(pages)
    B, Hq, d = q.shape
    _, Hkv, ps, _ = k_cache.shape
    G = Hq // Hkv
    scale = d ** -0.5 if scale is None else scale
    y = np.zeros((B, Hq, d))
    for b in range(B):
        for hk in range(Hkv):
            if pages is None:
                at = np.arange(lens[b])
            else:
                at = np.concatenate([np.arange(p * ps, min((p + 1) * ps, lens[b])) for p in pages[b, hk] if p >= 0]
                                    + [np.zeros(0, np.int64)]).astype(np.int64)
            if len(at) == 0:
                continue
            k, v = (_row_keys(c, page_table[b], hk, at) for c in (k_cache, v_cache))
            s = scale * q[b, hk * G:(hk + 1) * G] @ k.T
            e = np.exp(s - s.max(axis=1, keepdims=True))
            y[b, hk * G:(hk + 1) * G] = e @ v / e.sum(axis=1, keepdims=True)
    return y


def page_mean(k_cache, page_table, lens, mean, starts=None):
    """A copy of ``mean`` [num_pages, Hkv, d] with the touched pages' rows replaced."""
    k_cache, page_table, lens, mean = _f64(k_cache), _whole(page_table), _whole(lens), _f64(mean).copy()
    starts = np.zeros(len(lens), np.int64) if starts is None else _whole(starts)
    ps = k_cache.shape[2]
    for b in range(len(lens)):
        for page in sorted({p // ps for p in range(starts[b], lens[b])}):
            count = min(ps, lens[b] - page * ps)
            mean[page_table[b, page]] = k_cache[page_table[b, page], :, :count].sum(axis=1) / count
    return mean


def attn_select(q, mean, page_table, lens, page_size, n_sel, n_first=0, n_last=1):
    """pages [B, Hkv, n_sel], ascending, -1 behind the last."""
    q, mean, page_table, lens = _f64(q), _f64(mean), _whole(page_table), _whole(lens)
    B, Hq, _ = q.shape
    Hkv = mean.shape[1]
    G = Hq // Hkv
    out = np.full((B, Hkv, n_sel), -1, np.int64)
    for b in range(B):
        n = -(-lens[b] // page_size)
        for hk in range(Hkv):
            score = [max(float(q[b, hk * G + j] @ mean[page_table[b, p], hk]) for j in range(G)) for p in range(n)]
            kept = [p < n_first or p >= n - n_last for p in range(n)]
            order = sorted(range(n), key=lambda p: (not kept[p], 0.0 if kept[p] else -score[p], p))
            chosen = sorted(order[:n_sel])
            out[b, hk, :len(chosen)] = chosen
    return out

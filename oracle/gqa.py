"""Grouped-query attention over a paged cache (oracle).

TEST INFRASTRUCTURE. Only ``tests/``, ``__graft_entry__.smoke()`` and the CPU
baseline leg of ``bench.py`` may import anything under ``oracle/``.

The textbook definitions in float64: rotation of interleaved pairs of a
head's last r dims, a row's FP8 scale, and softmax attention of grouped
query heads with a causal mask, a sliding window and a sink that counts in
the denominator alone.  A masked key takes no part in any sum, whatever it
holds.
"""

from __future__ import annotations

import math

import numpy as np


def rotate(x, pos, r: int, theta: float):
    """Rows x [n, heads, d] at positions pos [n]: pair j of the last r dims
    (dims d-r+2j, d-r+2j+1) turned by pos * theta^(-2j/r)."""
    y = np.array(x, dtype=np.float64)
    d = y.shape[-1]
    for j in range(r // 2):
        a = np.asarray(pos, np.float64)[:, None] * theta ** (-2.0 * j / r)
        c, s = np.cos(a), np.sin(a)
        u, w = y[..., d - r + 2 * j].copy(), y[..., d - r + 2 * j + 1].copy()
        y[..., d - r + 2 * j] = u * c - w * s
        y[..., d - r + 2 * j + 1] = u * s + w * c
    return y


def row_scale(x):
    """FP8 scale of rows [..., d]: amax / 448, 1 for rows of zeros."""
    a = np.abs(np.asarray(x, np.float64)).max(-1) / 448.0
    return np.where(a == 0, 1.0, a)


def attend(q, k, v, t, scale: float, window: int = 0, sink=None, live=None):
    """Queries q [n, H, d] at positions t [n] over keys and values [m, G, d]
    (query head h reads head h // (H // G)); live [m]: keys that may be seen
    at all.  Returns the outputs, sum_j p_j |v_j| (what the error of rounded
    probabilities is bounded by) and the largest scale * sum_i |q_i k_i| of a
    seen key (what the error of a logit is bounded by)."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    n, H, d = q.shape
    m, G = k.shape[:2]
    pos, t = np.arange(m), np.asarray(t)
    seen = pos[None] <= t[:, None]
    if window:
        seen &= pos[None] > t[:, None] - window
    if live is not None:
        seen &= np.asarray(live, bool)[None]
    out, mag, zmag = np.zeros((n, H, d)), np.zeros((n, H, d)), 0.0
    if not m:
        return out, mag, zmag
    odd = ~np.isfinite(v)
    for h in range(H):
        kh, vh = k[:, h // (H // G)], v[:, h // (H // G)]
        any_seen = seen.any(0)
        z = np.where(seen, (q[:, h] @ np.where(any_seen[:, None], kh, 0).T) * scale, -math.inf)
        if any_seen.any():
            zmag = max(zmag, scale * float((np.abs(q[:, h]) @ np.abs(kh[any_seen]).T).max()))
        top = z.max(1)
        if sink is not None:
            top = np.maximum(top, sink[h])
        top = np.where(top == -math.inf, 0, top)
        p = np.exp(z - top[:, None])
        below = p.sum(1) + (0 if sink is None else np.exp(sink[h] - top))
        p /= np.where(below == 0, 1, below)[:, None]
        o = odd[:, h // (H // G)]
        out[:, h] = p @ np.where(o, 0, vh)
        mag[:, h] = p @ np.abs(np.where(o, 0, vh))
        for j in np.nonzero(o.any(1))[0]:  # infinities and NaN reach the queries that see them
            rows = seen[:, j]
            out[rows, h] += np.where(o[j], vh[j], 0)
    return out, mag, zmag

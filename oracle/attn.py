"""fp64 reference of the operators of a softmax-attention layer beside the delta rule: cache pages
given to requests, the norm of query and key heads with the rotation by position (forward, backward,
into a paged cache), and the attention of one new token over that cache.

Written from the definitions with numpy, row by row where that is the plainest; it shares no code
with the CUDA library.  Test infrastructure only.
"""
from __future__ import annotations

import numpy as np

EPS = 1e-6


def ceil_div(a, b):
    return -(-a // b)


# ------------------------------------------------------------------------------------ pages
def pages(cached, fresh, free_pages, n_free, table, page, tokens):
    """(lens, cu_new, positions, slots, n_left, table) of one step; the inputs are not changed."""
    table = np.array(table, dtype=np.int64, copy=True)
    R, width = table.shape
    top = min(max(int(n_free), 0), len(free_pages))
    lens, cu_new, positions, slots = [], [0], [], []
    left = top
    for r in range(R):
        a, f = max(int(cached[r]), 0), max(int(fresh[r]), 0)
        for j in range(min(ceil_div(a, page), width), min(ceil_div(a + f, page), width)):
            left -= 1
            table[r, j] = free_pages[left] if left >= 0 else -1
        for p in range(a, a + f):
            ok = p // page < width and table[r, p // page] >= 0
            positions.append(p)
            slots.append(table[r, p // page] * page + p % page if ok else -1)
        lens.append(a + f)
        cu_new.append(cu_new[-1] + f)
    pad = max(0, tokens - len(positions))
    return (np.array(lens, dtype=np.int64), np.array(cu_new), np.array((positions + [0] * pad)[:tokens], dtype=np.int64),
            np.array((slots + [-1] * pad)[:tokens], dtype=np.int64), left, table)


# ------------------------------------------------------------------------------------ norm and rotation
def _pair_index(rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def _turn(y, positions, inv_freq, interleaved, sign):
    """y [N, H, d] with its pairs turned by sign * position * inv_freq."""
    out = np.array(y, dtype=np.float64, copy=True)
    rot = 2 * len(inv_freq)
    if rot == 0:
        return out
    ia, ib = _pair_index(rot, interleaved)
    ang = np.asarray(positions, np.float64)[:, None, None] * np.asarray(inv_freq, np.float64)
    c, s = np.cos(ang), sign * np.sin(ang)
    a, b = y[..., ia], y[..., ib]
    out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
    return out


def qkrope(x, w, positions, inv_freq, interleaved=False):
    """x [N, H, d] -> rmsnorm(x) w, turned by position."""
    x = np.asarray(x, np.float64)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + EPS)
    return _turn(y if w is None else y * w, positions, inv_freq, interleaved, 1.0)


def qkrope_bwd(x, w, positions, inv_freq, dy, interleaved=False):
    """(dx, dw) of <dy, qkrope(x)>."""
    x = np.asarray(x, np.float64)
    g = _turn(np.asarray(dy, np.float64), positions, inv_freq, interleaved, -1.0)
    rms = np.sqrt((x * x).mean(-1, keepdims=True) + EPS)
    n = x / rms
    gn = g if w is None else g * w
    return (gn - n * (gn * n).mean(-1, keepdims=True)) / rms, (g * n).sum((0, 1))


# ------------------------------------------------------------------------------------ attention
def attn_decode(q, k_cache, v_cache, table, lens, scale=None, window=0):
    """(o [R, Hq, d], lse [R, Hq]) token by token from the pages."""
    q, k_cache, v_cache = (np.asarray(x, np.float64) for x in (q, k_cache, v_cache))
    R, Hq, d = q.shape
    n_pages, page, Hk, _ = k_cache.shape
    G = Hq // Hk
    scale = d ** -0.5 if scale is None else scale
    o, lse = np.zeros((R, Hq, d)), np.full((R, Hq), -np.inf)
    for r in range(R):
        # the window counts back from the length; beyond room + window it sees nothing of the table
        room = table.shape[1] * page
        n = min(max(int(lens[r]), 0), room + window)
        t = np.arange(max(0, n - window) if window else 0, n)
        t = t[t < room]
        pg = np.asarray(table[r])[t // page] if n else t
        ok = (pg >= 0) & (pg < n_pages)
        t, pg = t[ok], pg[ok]
        if len(t) == 0:
            continue
        k, v = k_cache[pg, t % page], v_cache[pg, t % page]  # [n, Hk, d]
        for h in range(Hq):
            s = scale * (k[:, h // G] @ q[r, h])
            m = s.max()
            p = np.exp(s - m)
            o[r, h] = (p @ v[:, h // G]) / p.sum()
            lse[r, h] = m + np.log(p.sum())
    return o, lse

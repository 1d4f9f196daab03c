"""Plain 64-bit forms of the paged-cache operators -- TEST INFRASTRUCTURE ONLY.

One sequence, head and row after the other, in numpy fp64, from the
definitions; shares no code with the product.  A cache is a dict of numpy
arrays: k, v [P, page_rows, H, D] fp64 (or int8 codes), k_scale, v_scale
[P, H, page_rows] or None, mass, order [P, H, page_rows], table [S, max_pages],
lens [S].
"""
from __future__ import annotations

import numpy as np


def slots(c, s, n=None):
    """(pages, rows) of the first n rows of sequence s."""
    page_rows = c["k"].shape[1]
    i = np.arange(int(c["lens"][s]) if n is None else n)
    return c["table"][s][i // page_rows], i % page_rows


def rows(c, name, s, h):
    """The rows [n, D] of sequence s and KV head h as the numbers they stand for."""
    pg, r = slots(c, s)
    x = c[name][pg, r, h].astype(np.float64)
    if c.get(name + "_scale") is not None:
        x = x * c[name + "_scale"][pg, h, r].astype(np.float64)[:, None]
    return x


def decode(q, c, scale):
    """(out [S, H_q, D], lse [S, H_q], weight of each row [S][H][n], logits' sizes [S, H_q], sum_j w_j |v_j|).

    The sizes are max_j sum_d |q_d k_jd| scale, which bounds the rounding of a
    dot product in lower precision; the last one bounds that of the weights."""
    S, h_q, d = q.shape
    h = c["k"].shape[2]
    g = h_q // h
    out, lse = np.zeros((S, h_q, d)), np.full((S, h_q), -np.inf)
    spread = np.zeros((S, h_q, d))
    size = np.zeros((S, h_q))
    w_all = []
    for s in range(S):
        n = int(c["lens"][s])
        w_s = np.zeros((h, n))
        for j in range(h_q if n else 0):
            k, v = rows(c, "k", s, j // g), rows(c, "v", s, j // g)
            x = (k @ q[s, j]) * scale
            size[s, j] = (np.abs(k) @ np.abs(q[s, j])).max() * scale
            e = np.exp(x - x.max())
            lse[s, j] = x.max() + np.log(e.sum())
            w = e / e.sum()
            out[s, j] = w @ v
            spread[s, j] = w @ np.abs(v)
            w_s[j // g] += w
        w_all.append(w_s)
    return out, lse, w_all, size, spread


def largest_weighted_scale(q, c, scale):
    """int8 values: max_j w_j s_j of each sequence and query head [S, H_q], s_j the value's scale."""
    S, h_q, _ = q.shape
    g = h_q // c["k"].shape[2]
    out = np.zeros((S, h_q))
    for s in range(S):
        pg, r = slots(c, s)
        for j in range(h_q if len(pg) else 0):
            x = (rows(c, "k", s, j // g) @ q[s, j]) * scale
            e = np.exp(x - x.max())
            out[s, j] = (e / e.sum() * c["v_scale"][pg, j // g, r].astype(np.float64)).max()
    return out


def rotate(x, w, eps, angle, interleaved):
    """x [T, H, D] fp64, angle [T, R/2]: the norm (w not None) and the rotation.
    Returns (y, |a| + |b| of every element's pair)."""
    x = x.copy()
    if w is not None:
        x = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * w
    half = angle.shape[1]
    i = np.arange(half)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    y, size = x.copy(), np.abs(x)
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    size[..., ia] = size[..., ib] = np.abs(a) + np.abs(b)
    return y, size


def evict_moves(mass, order, keep, seen, sink, recent):
    """(kept rows, [(from, to)]) of one sequence and KV head with n = len(mass) rows."""
    n = len(mass)
    if n <= keep:
        return list(range(n)), []

    def rank(i):
        safe = order is not None and (order[i] < sink or (recent and order[i] >= seen - recent))
        m = -np.inf if np.isnan(mass[i]) else float(mass[i])
        return (0 if safe else 1, 0.0 if safe else -m, i)

    kept = sorted(sorted(range(n), key=rank)[:keep])
    holes = sorted(set(range(keep)) - set(kept))
    movers = [i for i in kept if i >= keep]
    return kept, list(zip(movers, holes))

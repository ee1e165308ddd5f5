"""Speculative decoding from the 4-bit cache in plain loops: what kvc_kv4_append_rotated, kvc_kv4_tree_attention and
kvc_kv4_keep are compared with.  Written from the definitions in kvc.h."""
from __future__ import annotations

import numpy as np


def table(n_positions, rot, base=10000.0):
    """Cosines, then sines, of position * base^(-2i/rot), computed in 64 bits."""
    angle = np.arange(n_positions, dtype=np.float64)[:, None] * base ** (-2.0 * np.arange(rot // 2) / rot)
    return np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)


def rotate(x, tab, positions, interleaved):
    """x [T][heads][D] float32 turned in fp32, every operation rounded on its own."""
    x = np.asarray(x, np.float32)
    y, rot = x.copy(), tab.shape[1]
    cs = tab[positions][:, None]
    with np.errstate(over="ignore", invalid="ignore"):
        for i in range(rot // 2):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
            cos, sin = cs[..., i], cs[..., rot // 2 + i]
            y[..., a] = x[..., a] * cos - x[..., b] * sin
            y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def path(parents, i):
    """Token i's path from the tree's first level, itself the last."""
    out = []
    while i >= 0:
        out.append(i)
        i = parents[i]
    return out[::-1]


def sees(parents, length, window):
    """[n][length]: the keys that each of the n drafted tokens sees, those of positions at most window - 1 back."""
    n = len(parents)
    base, ok = length - n, np.zeros((n, max(length, 0)), bool)
    for i in range(n):
        way = path(parents, i)
        pos = base + len(way) - 1
        for key in range(max(base, 0)):
            ok[i, key] = not window or key > pos - window
        for step, tok in enumerate(way):
            if base + tok >= 0 and (not window or base + step > pos - window):
                ok[i, base + tok] = True
    return ok


def attention(q, k, v, ok, softcap, scale):
    """q [n][R][D], k and v [len][D] float64, ok [n][len] -> out [n][R][D], lse [n][R]; -inf for a row without a key."""
    n, R, D = q.shape
    out, lse = np.zeros((n, R, D)), np.full((n, R), -np.inf)
    for i in range(n):
        if not ok[i].any():
            continue
        x = q[i] @ k[ok[i]].T * scale
        if softcap:
            x = softcap * np.tanh(x / softcap)
        m = x.max(-1, keepdims=True)
        e = np.exp(x - m)
        out[i] = e @ v[ok[i]] / e.sum(-1, keepdims=True)
        lse[i] = m[:, 0] + np.log(e.sum(-1))
    return out, lse


def spread(q, k, v, ok, softcap, scale):
    """sum_j p_j |v_j - out|, p normalised, of attention's rows: what one rounding of every p moves out by, for each
    unit of its relative size."""
    n, R, D = q.shape
    out = np.zeros((n, R, D))
    for i in range(n):
        if not ok[i].any():
            continue
        x = q[i] @ k[ok[i]].T * scale
        if softcap:
            x = softcap * np.tanh(x / softcap)
        p = np.exp(x - x.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        for r in range(R):
            out[i, r] = p[r] @ np.abs(v[ok[i]] - p[r] @ v[ok[i]])
    return out


def random_tree(n, rng, shape="bushy"):
    if shape == "chain":
        return list(range(-1, n - 1))
    if shape == "flat":
        return [-1] * n
    return [int(rng.integers(-1, i)) if rng.random() < 0.3 else int(rng.integers(max(-1, i // 3 - 1), max(0, i - i // 2)))
            for i in range(n)]


def keep(pool, slots, base, way):
    """In a kv4_ref.Pool: token base + way[i] moves to base + i; slots: the sequence's, by position."""
    to, of = slots[base:base + len(way)], slots[base + np.asarray(way, int)]
    for x in (pool.code, pool.s, pool.lo):
        x[:, to] = x[:, of]

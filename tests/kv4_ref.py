"""The resident 4-bit cache in 64 bits and plain loops: what the kernels of
kvc_kv4_* are compared with.  Written from the definition in kvc.h."""
from __future__ import annotations

import numpy as np

F32, F64 = np.float32, np.float64


def to16(x):
    """fp32 to fp16, round to nearest even."""
    with np.errstate(over="ignore"):
        return np.asarray(x, F32).astype(np.float16)


def quantise(x, G):
    """x [..., D] fp32 values -> codes uint8 [..., D], s and lo float16 [..., D/G]; every fp32 step rounded once."""
    x = np.asarray(x, F32)
    g = x.reshape(*x.shape[:-1], -1, G)
    bad = ~np.isfinite(g).all(-1)
    c = np.clip(np.where(np.isfinite(g), g, F32(0)), F32(-65504), F32(65504)).astype(F32)
    mn, mx = c.min(-1), c.max(-1)
    lo = to16(mn)
    s = to16((mx - mn) * (F32(1) / F32(15)))
    with np.errstate(divide="ignore"):
        inv = np.where(s > 0, F32(1) / s.astype(F32), F32(0)).astype(F32)
    r = np.rint((c - lo.astype(F32)[..., None]) * inv[..., None])
    code = np.clip(r, 0, 15).astype(np.uint8)
    code[bad] = 0
    s = np.where(bad, np.float16(0), s)
    lo = np.where(bad, np.float16("nan"), lo)
    return code.reshape(x.shape), s, lo


def pack_k(code):
    """codes [D] of one K row -> D/2 bytes, byte by byte from the layout."""
    D = code.shape[-1]
    out = np.zeros(D // 2, np.uint8)
    for c in range(D):
        t, h, i = c // 32, c % 32 // 8, c % 8
        out[4 * (h * (D // 32) + t) + i // 2] |= int(code[c]) << (4 * (i % 2))
    return out


def v_byte(D, off, c):
    """Byte within a V block, and the nibble's shift, of token `off`, channel c."""
    u, i, n = c // 64, c % 64 // 16, c % 16
    return ((off // 4 * 16 + n) * (D // 64) + u) * 8 + off % 4 * 2 + i // 2, 4 * (i % 2)


def values(code, s, lo, G):
    """lo + code * s in float64 (exact: at most 53 bits)."""
    rep = lambda p: np.repeat(p.astype(F64), G, -1)  # noqa: E731
    return code.astype(F64) * rep(s) + rep(lo)


class Pool:
    """Codes and parameters of every slot, as arrays; `bytes` gives the device layout."""

    def __init__(self, H, D, G, P, n_pages):
        self.H, self.D, self.G, self.P, self.n = H, D, G, P, n_pages
        N = n_pages * P
        self.code = np.zeros((2, N, H, D), np.uint8)
        self.s = np.zeros((2, N, H, D // G), np.float16)
        self.lo = np.zeros((2, N, H, D // G), np.float16)

    def write(self, k, v, slots):
        for kv, x in enumerate((k, v)):
            c, s, lo = quantise(x, self.G)
            for t, slot in enumerate(slots):
                if 0 <= slot < self.n * self.P:
                    self.code[kv, slot], self.s[kv, slot], self.lo[kv, slot] = c[t], s[t], lo[t]

    def value(self, kv, slots):
        return values(self.code[kv, slots], self.s[kv, slots], self.lo[kv, slots], self.G)

    def codes_bytes(self):
        H, D, P = self.H, self.D, self.P
        out = np.zeros((self.n, 2, H, P * D // 2), np.uint8)
        for slot in range(self.n * P):
            page, off = divmod(slot, P)
            for h in range(H):
                out[page, 0, h, off * (D // 2):(off + 1) * (D // 2)] = pack_k(self.code[0, slot, h])
                for c in range(D):
                    b, sh = v_byte(D, off, c)
                    out[page, 1, h, b] |= int(self.code[1, slot, h, c]) << sh
        return out

    def params(self):
        H, P, NG = self.H, self.P, self.D // self.G
        x = np.stack([self.s, self.lo], -1).reshape(2, self.n, P, H, NG, 2)  # [kv][page][off][H][g][2]
        return np.ascontiguousarray(x.transpose(1, 0, 3, 4, 2, 5))


def attention(q, k, v, pos, n_keys, causal, window, softcap, scale):
    """q [n][R][D], k and v [len][D] float64 -> out [n][R][D], lse [n][R], and per row the largest
    sum_c |q_c| max_j |k_jc| (what a logit's rounding errors scale with)."""
    n, R, D = q.shape
    out, lse = np.zeros((n, R, D)), np.full((n, R), -np.inf)
    for i in range(n):
        hi = min(n_keys, pos[i] + 1) if causal else n_keys
        lo = max(0, pos[i] - window + 1) if window else 0
        if hi <= lo:
            continue
        x = q[i] @ k[lo:hi].T * scale
        if softcap:
            x = softcap * np.tanh(x / softcap)
        m = x.max(-1, keepdims=True)
        e = np.exp(x - m)
        out[i] = e @ v[lo:hi] / e.sum(-1, keepdims=True)
        lse[i] = m[:, 0] + np.log(e.sum(-1))
    return out, lse

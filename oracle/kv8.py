"""Slow references of the 8-bit paged KV cache, written from its description.

numpy only. ``Sequence`` holds what a cache holds for one sequence, call by call, so that
values can be compared bit for bit; ``decode`` reads a pool byte by byte from the layout's
formulas; ``select`` works on whole numbers; ``attention`` is the definition in fp64 over any
subset of the tokens. The rotation and the bookkeeping are those of the 4-bit cache (kv4.py).
"""
from __future__ import annotations

import numpy as np

from oracle.kv4 import attention as dense_attention
from oracle.kv4 import bf16, rotate  # noqa: F401  (the tests' references)

F = np.float32


def e4m3(x):
    """Numbers of magnitude up to 448 -> the nearest 8-bit floats, ties to even (fp64)."""
    x = np.asarray(x, np.float64)
    _, k = np.frexp(np.abs(x))
    step = np.exp2(np.maximum(k - 1, -6).astype(np.float64) - 3)
    return np.rint(x / step) * step


def exponent(most, top, least, largest):
    """The least e with most <= top 2^e, within [least, largest]."""
    most = np.asarray(most, np.float64)
    e = np.full(most.shape, least)
    while True:
        low = (most > top * np.exp2(e.astype(np.float64))) & (e < largest)
        if not low.any():
            return e
        e = e + low


class Sequence:
    """One sequence of one layer: k, v fp32 [n][H][D] as held, scales' exponents [blocks][H][2]."""

    def __init__(self, H, D):
        self.k, self.v = np.zeros((0, H, D), F), np.zeros((0, H, D), F)
        self.e = np.zeros((0, H, 2), int)

    def copy(self):
        other = Sequence(*self.k.shape[1:])
        other.k, other.v, other.e = self.k.copy(), self.v.copy(), self.e.copy()
        return other

    def append(self, k, v):
        """The new tokens' rotated k (fp32) and v of one call."""
        n0, n1 = len(self.k), len(self.k) + len(k)
        if n1 == n0:
            return
        ok = np.isfinite(k).all(-1) & np.isfinite(v).all(-1)
        new = [np.where(ok[..., None], np.clip(np.nan_to_num(x), -32768, 32768), 0).astype(np.float64) for x in (k, v)]
        held = [np.concatenate([h, np.zeros_like(x, F)]) for h, x in ((self.k, k), (self.v, v))]
        e = np.full((-(-n1 // 16), k.shape[1], 2), -24)
        e[:len(self.e)] = self.e
        for i in (0, 1):
            for b in range(n0 // 16, len(e)):
                lo, hi = max(16 * b, n0), min(16 * b + 16, n1)
                x = new[i][lo - n0:hi - n0]
                now = exponent(np.abs(x).max((0, 2)), 448.0, -24, 7)
                if lo > 16 * b:
                    now = np.maximum(now, e[b, :, i])
                    s = np.exp2(now.astype(np.float64))[None, :, None]
                    held[i][16 * b:lo] = e4m3(held[i][16 * b:lo] / s) * s
                e[b, :, i] = now
                s = np.exp2(now.astype(np.float64))[None, :, None]
                held[i][lo:hi] = e4m3(x / s) * s
        held[0][n0:] = np.where(ok[..., None], held[0][n0:], F("nan"))
        self.k, self.v, self.e = held[0], held[1], e


def bounds(k):
    """k [n][H][D] as held -> upper, lower (whole numbers [H][D]) and step [H]."""
    has = ~np.isnan(k).all(0)
    hi = np.where(has, np.where(np.isnan(k), -np.inf, k).max(0), 0).astype(np.float64)
    lo = np.where(has, np.where(np.isnan(k), np.inf, k).min(0), 0).astype(np.float64)
    step = np.exp2(exponent(np.maximum(np.abs(hi), np.abs(lo)).max(-1), 127.0, -30, 100).astype(np.float64))
    return np.ceil(hi / step[:, None]), np.floor(lo / step[:, None]), step


def decode(pool, page, layer, head, token, n_layers, n_heads, page_tokens, D):
    """(k, v) of one token of a page, and the page's (upper, lower, step), from the layout."""
    cells, size = page_tokens // 16, 32 * D + 16
    share = cells * size + 2 * D + 16
    base = (layer * n_heads + head) * share
    cell, i = pool[page, base + token // 16 * size:][:size], token % 16
    tail = pool[page, base + cells * size:base + share]

    def value(b):
        sign, e, m = -1.0 if b & 128 else 1.0, (b >> 3) & 15, b & 7
        if b & 127 == 127:
            return F("nan")
        return F(sign * (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)))

    scales = cell[32 * D:32 * D + 8].view(F)
    k, v = np.zeros(D, F), np.zeros(D, F)
    for ch in range(D):
        k[ch] = value(int(cell[(i // 8) * 8 * D + (ch // 64) * 512 + (i % 8) * 64 + ch % 64])) * scales[0]
        v[ch] = value(int(cell[16 * D + (ch // 4) * 64 + (i % 8) // 2 * 16 + (ch % 4) * 4 + i % 2 + 2 * (i // 8)])) * scales[1]
    return (k, v), (tail[:D].view(np.int8).astype(float), tail[D:2 * D].view(np.int8).astype(float), float(tail[2 * D:2 * D + 4].view(F)[0]))


def select(q, K, P, n_list, first, last):
    """The pages of the last query of a sequence: q fp32 [H][D], K fp32 [n][Hk][D] as held, up to its own
    position -> int [Hk][n_list]."""
    n, Hk, D = K.shape
    count = (n - 1) // P + 1
    out = np.full((Hk, n_list), -1)
    for h in range(Hk):
        if count <= n_list:
            out[h, :count] = np.arange(count)
            continue
        x = q.reshape(Hk, -1, D)[h].astype(F)
        x = np.clip(np.where(np.isfinite(x), x, F(0)), F(-2.0 ** 100), F(2.0 ** 100))
        p, m = np.zeros(D, F), np.zeros(D, F)
        for row in x:
            p, m = p + np.maximum(row, 0), m + np.minimum(row, 0)
        unit = 2.0 ** float(exponent(max(p.max(), -m.min()), 127.0, -100, 200))
        a, c = np.rint(p.astype(np.float64) / unit), np.rint(m.astype(np.float64) / unit)
        score = []
        for z in range(count - last):
            up, low, step = bounds(K[z * P:(z + 1) * P, h:h + 1])
            score.append(float((a * up[0] + c * low[0]).sum() * step[0]))
        rest = sorted(range(first, count - last), key=lambda z: (-score[z], z))
        out[h] = sorted(list(range(first)) + list(range(count - last, count)) + rest[:n_list - first - last])
    return out


def attention(q, K, V, length, scale, pages=None, P=0):
    """As kv4.attention; with pages [n][Hk][m] each query's heads see the tokens of those pages alone."""
    if pages is None:
        return dense_attention(q, K, V, length, scale)
    n, H, D = q.shape
    Hk = K.shape[1]
    r = H // Hk
    out, A = np.zeros((n, H, D)), np.zeros((n, H, D))
    lse, B = np.full((n, H), -np.inf), np.zeros((n, H))
    for i in range(n):
        seen = np.arange(max(0, length - n + i + 1))
        for h in range(Hk):
            at = seen[np.isin(seen // P, pages[i, h])]
            o, l, a, b = dense_attention(q[i:i + 1, h * r:(h + 1) * r], K[at][:, h:h + 1], V[at][:, h:h + 1], len(at), scale)
            out[i, h * r:(h + 1) * r], lse[i, h * r:(h + 1) * r] = o[0], l[0]
            A[i, h * r:(h + 1) * r], B[i, h * r:(h + 1) * r] = a[0], b[0]
    return out, lse, A, B


def listed(entries, count):
    """The entries of one list that count, for a sequence of `count` pages, and whether others are reported: the first -1
    ends it; before that, those in range and above all in range before them."""
    taken, faults = [], False
    for e in entries:
        if e == -1:
            break
        if 0 <= e < count and (not taken or e > taken[-1]):
            taken.append(int(e))
        else:
            faults = True
    return taken, faults

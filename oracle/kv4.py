"""Slow references of the 4-bit paged KV cache, written from its description.

numpy only. ``quantise`` follows the format's fp32 arithmetic operation by
operation, so codes and parameters can be compared bit for bit; ``decode`` reads
a pool byte by byte from the layout's formulas; ``attention`` is the definition in
fp64; ``Pages`` does the bookkeeping one entry at a time.
"""
from __future__ import annotations

import numpy as np

F = np.float32


def bf16(x):
    """fp32 -> the nearest bf16 (ties to even), as fp32; NaN stays NaN."""
    x = np.ascontiguousarray(x, dtype=F)
    b = x.view(np.uint32)
    r = ((b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(F)
    return np.where(np.isnan(x), x, r)


def rotate(x, cos, sin):
    """x fp32 [T][H][D], cos and sin fp32 [T][D/2]: halves turned, every operation rounded to fp32."""
    h = x.shape[-1] // 2
    a, b = x[..., :h], x[..., h:]
    c, s = cos[:, None].astype(F), sin[:, None].astype(F)
    return np.concatenate([(a * c) - (b * s), (b * c) + (a * s)], -1).astype(F)


def quantise(k, v):
    """fp32 k, v [T][H][D] -> the values the cache holds for them, fp32 (K of a token and head with
    a non-finite k or v: NaN)."""
    bad = ~(np.isfinite(k).all(-1) & np.isfinite(v).all(-1))
    out = []
    for x in (k, v):
        x = np.where(np.isnan(x), F(0), np.clip(x, F(-32768), F(32768))).astype(F)
        g = x.reshape(*x.shape[:-1], -1, 64)
        lo, hi = g.min(-1, keepdims=True), g.max(-1, keepdims=True)
        s = bf16((hi - lo) * F(1 / 15)).astype(np.float16).astype(F)
        mid = (lo + s * F(8)).astype(np.float16).astype(F)
        with np.errstate(divide="ignore", invalid="ignore"):
            u = np.where(s > 0, np.rint((g - mid) / s), F(0))
        u = np.clip(u, F(-8), F(7))
        out.append(((u * s) + mid).astype(F).reshape(x.shape))
    out[0] = np.where(bad[..., None], F("nan"), out[0])
    return out


def decode(pool, page, layer, head, token, n_layers, n_heads, page_tokens, D):
    """(k, v) fp32 [D] of one token of a page, from the layout: pool uint8 [pages][page bytes]."""
    G = D // 64
    size = 16 * (D + 8 * G)
    cells = page_tokens // 16
    base = ((layer * n_heads + head) * cells + token // 16) * size
    cell, i = pool[page, base:base + size], token % 16
    f16 = cell.view(np.float16)
    k, v = np.zeros(D, F), np.zeros(D, F)
    for ch in range(D):
        g, x = divmod(ch, 64)
        kb = i * (D // 2) + (x // 16) * 8 * G + g * 8 + (x % 16) // 2
        vb = 8 * D + g * 512 + (x // 8) * 64 + ((i // 2) % 4) * 16 + (i // 8) * 8 + ((x // 4) % 2) * 4 + (i % 2) * 2 \
            + (x % 4) // 2
        kp = (16 * D + (i * G + g) * 4) // 2
        vp = (16 * D + 64 * G + ((i // 2) * G + g) * 8) // 2 + i % 2
        for out, byte, s, mid in ((k, kb, f16[kp], f16[kp + 1]), (v, vb, f16[vp], f16[vp + 2])):
            code = (int(cell[byte]) >> (4 * (ch % 2))) & 15
            out[ch] = F(F(code - 8) * F(s)) + F(mid)
    return k, v


def attention(q, K, V, length, scale):
    """q [n][H][D], K, V [length][Hk][D] (all as fp64): causal attention of the last n positions.
    Returns (out, lse, A, B): A = sum_t weight |v| per output, B = the largest sum_d |q k| scale of a row."""
    n, H, D = q.shape
    r = H // K.shape[1]
    out, A = np.zeros((n, H, D)), np.zeros((n, H, D))
    lse, B = np.full((n, H), -np.inf), np.zeros((n, H))
    for i in range(n):
        m = length - n + i + 1
        if m <= 0:
            continue
        for h in range(H):
            k, v = K[:m, h // r], V[:m, h // r]
            with np.errstate(invalid="ignore", over="ignore"):
                s = k @ q[i, h] * scale
                top = s.max()
                p = np.exp(s - top)
                lse[i, h] = top + np.log(p.sum())
                p = p / p.sum()
                out[i, h], A[i, h] = p @ v, p @ np.abs(v)
                B[i, h] = (np.abs(k) @ np.abs(q[i, h])).max() * abs(scale)
    return out, lse, A, B


class Pages:
    """The bookkeeping: lens, refs, tables (lists), info = [free, result, moved]."""

    def __init__(self, n_pages, page_tokens, max_seqs, max_pages):
        self.P, self.max_pages = page_tokens, max_pages
        self.refs, self.lens = [0] * n_pages, [0] * max_seqs
        self.tables = [[-1] * max_pages for _ in range(max_seqs)]
        self.result = self.moved = 0
        self.copies = []  # (source page, destination page, tokens) of the last fork, (source, destination) of a compact

    def free_pages(self):
        return [p for p, r in enumerate(self.refs) if r == 0]

    def _pages(self, n):
        return -(-n // self.P)

    def reserve(self, seqs, new):
        if len(set(seqs)) < len(seqs) or any(s < 0 or s >= len(self.lens) for s in seqs) or \
                any(n < 0 or self._pages(self.lens[s] + n) > self.max_pages for s, n in zip(seqs, new)):
            self.result = -1
            return
        need = [self._pages(self.lens[s] + n) - self._pages(self.lens[s]) for s, n in zip(seqs, new)]
        free = self.free_pages()
        self.result = max(0, sum(need) - len(free))
        if self.result:
            return
        for s, n, k in zip(seqs, new, need):
            for _ in range(k):
                p = free.pop(0)
                self.tables[s][self.tables[s].index(-1)] = p
                self.refs[p] = 1
            self.lens[s] += n

    def fork(self, src, dst):
        self.copies = []
        if any(s < 0 or s >= len(self.lens) for s in list(src) + list(dst)) or len(set(dst)) < len(dst) or \
                set(src) & set(dst) or any(self.lens[d] for d in dst):
            self.result = -1
            return
        free = self.free_pages()
        self.result = max(0, sum(self.lens[s] % self.P > 0 for s in src) - len(free))
        if self.result:
            return
        for s, d in zip(src, dst):
            full, rest = divmod(self.lens[s], self.P)
            for k in range(full):
                self.tables[d][k] = self.tables[s][k]
                self.refs[self.tables[s][k]] += 1
            if rest:
                p = free.pop(0)
                self.copies.append((self.tables[s][full], p, rest))
                self.tables[d][full] = p
                self.refs[p] = 1
            self.lens[d] = self.lens[s]

    def free(self, seqs):
        for s in seqs:
            for k in range(self._pages(self.lens[s])):
                self.refs[self.tables[s][k]] -= 1
                self.tables[s][k] = -1
            self.lens[s] = 0

    def compact(self):
        live = sum(r > 0 for r in self.refs)
        holes = [p for p in range(live) if self.refs[p] == 0]
        movers = [p for p in range(live, len(self.refs)) if self.refs[p] > 0]
        self.copies, self.moved = list(zip(movers, holes)), len(holes)
        for a, b in self.copies:
            self.refs[b], self.refs[a] = self.refs[a], 0
            for t in self.tables:
                for k, p in enumerate(t):
                    if p == a:
                        t[k] = b

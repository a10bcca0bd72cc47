"""The operators around the layer, written out plainly in float64 and loops.

Test infrastructure only (see the package docstring for who may import it).

* ``step``: a step's tables, one request and one page at a time;
* ``KvCache``: NVFP4 rows by slot (``nvfp4.quantize`` with a static global
  scale) and the byte layout of a pool's 16-token blocks;
* ``attention``: one query row at a time over cached values;
* ``block_norm``: norm, gate, residual, norm;
* ``rope``: pairs as complex numbers, angles of exact fractions of a turn;
* ``grid``, ``block_mean``, ``picks``: a block's mean key on its grid, and the
  blocks that one query picks.

Pinned by tests/test_oracle_block.py, the last two groups by tests/test_sparse_host.py.
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np

from . import nvfp4

# 2 pi to 60 decimal places
TWO_PI = Fraction(6283185307179586476925286766559005768394338798750211641949889, 10 ** 60)


def step(ctx, new, table, free, count, P, tokens):
    """A step's tables; returns a dict of new arrays (the inputs are not changed).

    ``table`` int ``[B, W]``, ``free[:count]`` a stack. Pinned by: no page
    handed out twice, every granted token's slot inside a page of its own
    request, refusals in request order (tests).
    """
    table = np.array(table)
    B, W = table.shape
    bad = False
    cu, kv, slots, pos = [0], [], [], []
    left, short = int(count), False
    for b in range(B):
        c, n = int(ctx[b]), int(new[b])
        bad |= c < 0 or n < 0
        c, n = max(c, 0), max(n, 0)
        have, want = -(-c // P), -(-(c + n) // P)
        ok = c + n <= W * P
        if ok and want > have:
            short |= want - have > left      # once one goes short, every later one that needs a page does
            ok = not short
        if ok:
            for j in range(have, want):
                left -= 1
                table[b, j] = free[left]
        bad |= not ok
        kv.append(c + n if ok else c)
        cu.append(cu[-1] + n)
        for i in range(n):
            pos.append(c + i)
            slots.append(table[b, (c + i) // P] * P + (c + i) % P if ok else -1)
    bad |= len(slots) > tokens
    pad = max(0, tokens - len(slots))
    return dict(table=table, kv_len=np.array(kv), cu_q=np.array(cu), bad=bool(bad), free_count=left,
                slots=np.array((slots + [-1] * pad)[:tokens], dtype=np.int64),
                positions=np.array((pos + [0] * pad)[:tokens], dtype=np.int64))


class KvCache:
    """Quantised rows by slot; values as the codes stand for, in float64."""

    def __init__(self, pages, P, heads, dim, k_gs, v_gs):
        self.P, self.heads, self.dim, self.gs = P, heads, dim, (k_gs, v_gs)
        n = pages * P
        self.codes = np.zeros((2, n, heads, dim), np.uint8)
        self.sf = np.zeros((2, n, heads, dim // 16), np.uint8)

    def append(self, k, v, slots):
        for which, x in ((0, k), (1, v)):
            x = np.where(np.isnan(x), np.float32(0), np.asarray(x, np.float32))
            rows = x.reshape(-1, self.dim)
            codes, sf, _ = nvfp4.quantize(rows, self.gs[which])
            codes, sf = codes.reshape(x.shape), sf.reshape(x.shape[:2] + (self.dim // 16,))
            for t, s in enumerate(slots):
                if s >= 0:
                    self.codes[which, s], self.sf[which, s] = codes[t], sf[t]

    def values(self, which, slots):
        s = np.asarray(slots)
        out = nvfp4.dequantize(self.codes[which, s].reshape(-1, self.dim), self.sf[which, s].reshape(-1, self.dim // 16),
                               self.gs[which])
        return out.reshape(len(s), self.heads, self.dim)

    def pool(self):
        """The pool's bytes: [pages, heads, P / 16, 18 dim]."""
        D, pages = self.dim, self.codes.shape[1] // self.P
        out = np.empty((pages, self.heads, self.P // 16, 18 * D), np.uint8)
        for pg in range(pages):
            for h in range(self.heads):
                for blk in range(self.P // 16):
                    s = slice(pg * self.P + blk * 16, pg * self.P + blk * 16 + 16)
                    out[pg, h, blk] = np.concatenate([
                        part.reshape(-1) for w in (0, 1)
                        for part in (nvfp4.pack(self.codes[w, s, h]), self.sf[w, s, h])])
        return out


def attention(q, keys, values, scale, position, window=0):
    """One query row: ``q`` [D], ``keys`` / ``values`` [n, D]; sees token j with
    ``j <= position`` (and ``j > position - window``). Returns (out, lse,
    sum p |v|, largest |scale| sum |q k|): the last two enter error bounds.
    """
    j = np.arange(len(keys))
    see = j <= position
    if window:
        see &= j > position - window
    if not see.any():
        return np.zeros(len(q)), -np.inf, np.zeros(len(q)), 0.0
    s = (keys[see] @ q) * scale
    m = s.max()
    p = np.exp(s - m)
    lse = m + np.log(p.sum())
    p /= p.sum()
    v = values[see]
    return p @ v, lse, p @ np.abs(v), abs(scale) * (np.abs(keys[see]) @ np.abs(q)).max()


def block_norm(x, residual, gate=None, w_post=None, w_pre=None, a=1.0, b=1.0, eps=1e-6, offset=0.0):
    """(r, out) in float64; ``out`` is None without ``w_pre``."""
    def rms(v, w):
        return v / np.sqrt((v * v).mean(-1, keepdims=True) + eps) * (w + offset)
    r = a * residual
    if x is not None:
        n = x if w_post is None else rms(x, w_post)
        r = r + b * (n if gate is None else gate * n)
    return r, None if w_pre is None else rms(r, w_pre)


def turns(inv_freq, position):
    """The fraction of a turn, in [0, 1), by which a pair of this frequency turns at a position: exact up to the
    60 places of pi."""
    return Fraction(float(inv_freq)) * int(position) / TWO_PI % 1


def rope(x, positions, inv_freq, axis, pairs, scale=1.0, inverse=False):
    """``x`` [T, heads, D] turned; ``positions`` [axes, T]. Returns (y, sum |a| + |b| of each element's pair, scaled)."""
    T, _, D = x.shape
    half = len(inv_freq)
    lo, hi = ((np.arange(half), half + np.arange(half)) if pairs == "half" else (2 * np.arange(half), 2 * np.arange(half) + 1))
    angle = np.array([[float(turns(f, positions[a][t])) for f, a in zip(inv_freq, axis)] for t in range(T)])
    z = np.exp((-2j if inverse else 2j) * np.pi * angle.reshape(T, half))[:, None]
    y, size = x.copy(), np.abs(x)
    w = (x[..., lo] + 1j * x[..., hi]) * z * scale
    y[..., lo], y[..., hi] = w.real, w.imag
    size[..., lo] = size[..., hi] = (np.abs(x[..., lo]) + np.abs(x[..., hi])) * abs(scale)
    return y, size


def grid(x, bits):
    """``x`` rounded, ties to even, to multiples of 2^(E - bits), E the exponent of its largest magnitude (at least
    -100). Returns (the multiples, the step)."""
    top = max(np.abs(x).max(), 2.0 ** -100)
    step = 2.0 ** (np.frexp(top)[1] - 1 - bits)
    return np.rint(x / step), step


def block_mean(rows):
    """Mean of a block's rows [tokens, D] (code * scale, not divided by gs), on its grid of 8 bits."""
    n, step = grid(np.asarray(rows, np.float64).sum(0) / len(rows), 6)
    return n * step


def picks(q, means, position, block_tokens, top, sink, local):
    """One query's blocks for one head: ``q`` [group, D], ``means`` [blocks, D] (None where the page is bad)."""
    if position < 0:
        return []
    seen = position // block_tokens + 1
    if seen <= top:
        return list(range(seen))
    u = grid(np.where(np.isfinite(q), q, 0.0), 5)[0].sum(0)
    ranked = range(sink, seen - local)
    score = {j: -np.inf if means[j] is None else float(u @ means[j]) for j in ranked}
    best = sorted(ranked, key=lambda j: (-score[j], j))[:top - sink - local]
    return sorted(list(range(sink)) + best + list(range(seen - local, seen)))

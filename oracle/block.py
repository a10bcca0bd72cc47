"""The operators around the layer, written out plainly in float64 and loops.

Test infrastructure only (see the package docstring for who may import it).

* ``step``: a step's tables, one request and one page at a time;
* ``KvCache``: NVFP4 rows by slot (``nvfp4.quantize`` with a static global
  scale) and the byte layout of a pool's 16-token blocks;
* ``attention``: one query row at a time over cached values;
* ``block_norm``: norm, gate, residual, norm.

Each is pinned by tests/test_oracle_block.py.
"""
from __future__ import annotations

import numpy as np

from . import nvfp4


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

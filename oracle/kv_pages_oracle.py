"""CPU oracle of the paged FP8 KV cache and the attention over it, written
from the definitions in include/nvfp4.h in float64 numpy."""
from __future__ import annotations

import numpy as np

from oracle.nvfp4_oracle import E4M3_VALUES

MAGNITUDES = np.asarray(E4M3_VALUES, dtype=np.float64)  # of the codes 0 .. 0x7E
_MIDPOINTS = (MAGNITUDES[1:] + MAGNITUDES[:-1]) / 2


def quantize_rows(x):
    """x [..., D] (float32 values) -> codes uint8 [..., D], scale bytes uint8 [...]."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(x).max(-1)
    e = np.full(a.shape, -126)
    for k in range(-126, 121):  # the least e with a <= 448 * 2^e
        e = np.where(a > 448.0 * 2.0 ** k, k + 1, e)
    y = np.abs(x) / 2.0 ** e[..., None].astype(np.float64)
    up = np.searchsorted(_MIDPOINTS, y, side="left")     # midpoints below y
    tie = np.searchsorted(_MIDPOINTS, y, side="right") != up
    codes = up + (tie & (up % 2 == 1))                    # a tie goes to the even code
    return (codes | (np.signbit(x) << 7)).astype(np.uint8), (e + 127).astype(np.uint8)


def values(codes, scales):
    """float64 values of codes [..., D] with scale bytes [...]."""
    mag = MAGNITUDES[np.minimum(codes & 0x7F, 0x7E)]
    v = np.where(codes & 0x80, -mag, mag)
    return v * 2.0 ** (scales.astype(np.float64) - 127)[..., None]


def key_index(o, d, dim):
    """Byte of token o, dimension d in a key block."""
    return o // 4 * (4 * dim) + d // 16 * 64 + o % 4 * 16 + d % 16


def value_index(o, d):
    return d * 16 + o


class Pages:
    """A cache on the host: k_codes, v_codes [n_pages, heads * page * dim],
    k_scales, v_scales [n_pages, heads * page], all uint8."""

    def __init__(self, n_pages, heads, dim, page, fill=0xA5):
        self.n_pages, self.heads, self.dim, self.page = n_pages, heads, dim, page
        self.k_codes = np.full((n_pages, heads * page * dim), fill, np.uint8)
        self.v_codes = self.k_codes.copy()
        self.k_scales = np.full((n_pages, heads * page), fill, np.uint8)
        self.v_scales = self.k_scales.copy()

    def _at(self, slot, head):
        page, i = divmod(int(slot), self.page)
        return page, (head * self.page + i // 16 * 16) * self.dim, i % 16, head * self.page + i

    def write(self, k, v, slots):
        """k, v [rows, heads * dim]; rows outside the cache are dropped."""
        d = np.arange(self.dim)
        kc, ks = quantize_rows(np.reshape(k, (len(slots), self.heads, self.dim)))
        vc, vs = quantize_rows(np.reshape(v, (len(slots), self.heads, self.dim)))
        for r, slot in enumerate(slots):
            if not 0 <= slot < self.n_pages * self.page:
                continue
            for h in range(self.heads):
                page, block, o, s = self._at(slot, h)
                self.k_codes[page, block + key_index(o, d, self.dim)] = kc[r, h]
                self.v_codes[page, block + value_index(o, d)] = vc[r, h]
                self.k_scales[page, s], self.v_scales[page, s] = ks[r, h], vs[r, h]

    def read(self, slots):
        """Keys and values [rows, heads, dim] float64 of slots inside the cache."""
        d = np.arange(self.dim)
        k = np.empty((len(slots), self.heads, self.dim))
        v = np.empty_like(k)
        for r, slot in enumerate(slots):
            for h in range(self.heads):
                page, block, o, s = self._at(slot, h)
                k[r, h] = values(self.k_codes[page, block + key_index(o, d, self.dim)], self.k_scales[page, s])
                v[r, h] = values(self.v_codes[page, block + value_index(o, d)], self.v_scales[page, s])
        return k, v


def attention(q, pages, q_heads, scale, table, lens, q_len, prefix_pages, prefix_len, max_len=None):
    """(o, wv): o [batch * q_len, q_heads, dim] float64 and sum_t w_t |v_t|
    (what the rounding of the softmax weights scales with); rows of negative
    length are NaN in o."""
    batch = len(lens)
    group = q_heads // pages.heads
    q = np.asarray(q, np.float64).reshape(batch, q_len, q_heads, pages.dim)
    o = np.zeros(q.shape)
    wv = np.zeros(q.shape)

    def tokens(ids, n):
        slots, ok = [], []
        for t in range(n):
            page = int(ids[t // pages.page])
            ok.append(0 <= page < pages.n_pages)
            slots.append((page if ok[-1] else 0) * pages.page + t % pages.page)
        k, v = pages.read(slots)
        return k, v, np.asarray(ok, bool)

    kp, vp, okp = tokens(prefix_pages, prefix_len)
    for b in range(batch):
        n = int(lens[b]) if max_len is None else min(int(lens[b]), max_len)
        if n < 0:
            o[b] = np.nan
            continue
        ks, vs, oks = tokens(table[b] if table is not None else [], n)
        k, v = np.concatenate([kp, ks]), np.concatenate([vp, vs])
        for j in range(q_len):
            seen = np.concatenate([okp, oks & (np.arange(n) < n - q_len + 1 + j)])
            if not seen.any():
                continue
            for h in range(q_heads):
                kk, vv = k[seen, h // group], v[seen, h // group]
                x = kk @ q[b, j, h] * scale
                p = np.exp(x - x.max())
                p /= p.sum()
                o[b, j, h] = p @ vv
                wv[b, j, h] = p @ np.abs(vv)
    return o.reshape(batch * q_len, q_heads, -1), wv.reshape(batch * q_len, q_heads, -1)

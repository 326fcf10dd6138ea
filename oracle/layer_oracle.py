"""CPU oracle of the 8-bit linear layers, the query/key norm with rotation and
the short convolution, written from the definitions in include/nvfp4.h in
float64 numpy.  (The gated delta rule's next tokens are held to
``nvfp4_oracle.gdn_recurrence``.)"""
from __future__ import annotations

import numpy as np

from oracle.kv_pages_oracle import MAGNITUDES

_MIDPOINTS = (MAGNITUDES[1:] + MAGNITUDES[:-1]) / 2
NAN_CODE = 0x7F


def _spread(scales, block_rows, rows, cols):
    """Scales [row blocks, column blocks] for every element."""
    return np.repeat(np.repeat(scales, block_rows, 0)[:rows], 128, 1)[:, :cols]


def fp8_quantize(x, block_rows=1, pow2=False):
    """x [R, C] (float32 values) -> codes uint8 [R, C], float32 scales [ceil(R / block_rows), ceil(C / 128)]."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    fine = np.isfinite(x)
    scales = np.zeros((-(-rows // block_rows), -(-cols // 128)), np.float32)
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            at = np.s_[i * block_rows: (i + 1) * block_rows, j * 128: (j + 1) * 128]
            a = np.abs(x[at][fine[at]]).max(initial=0.0)
            if pow2:
                e = -126
                while a > 448.0 * 2.0 ** e:
                    e += 1
                scales[i, j] = 2.0 ** e
            else:
                scales[i, j] = np.float32(a / 448.0)
    s = _spread(scales.astype(np.float64), block_rows, rows, cols)
    y = np.divide(np.where(fine, np.abs(x), 0.0), s, out=np.zeros_like(x), where=s > 0)
    up = np.searchsorted(_MIDPOINTS, y, side="left")     # midpoints below y
    tie = np.searchsorted(_MIDPOINTS, y, side="right") != up
    codes = np.where(fine, up + (tie & (up % 2 == 1)), NAN_CODE)  # a tie goes to the even code
    return (codes | (np.signbit(x) << 7)).astype(np.uint8), scales


def fp8_values(codes, scales, block_rows):
    """float64 values of the codes (NaN for the NaN code)."""
    mag = np.append(MAGNITUDES, np.nan)[codes & 0x7F]
    return np.where(codes & 0x80, -mag, mag) * _spread(scales.astype(np.float64), block_rows, *codes.shape)


def fp8_gemm(a_codes, a_scales, w_codes, w_scales):
    """(A W^T, |A| |W|^T) in float64."""
    a, w = fp8_values(a_codes, a_scales, 1), fp8_values(w_codes, w_scales, 128)
    return a @ w.T, np.abs(a) @ np.abs(w).T


def qk_norm_rope(x, head_dim, weight=None, eps=1e-6, weight_offset=0.0, positions=None, inv_freq=None, axis=None,
                 interleaved=False):
    """x [T, heads, head_dim] -> (result, |z_i| + |z_j| of each element's pair)."""
    z = np.array(x, dtype=np.float64)
    if weight is not None:
        z = z / np.sqrt((z * z).mean(-1, keepdims=True) + eps) * (np.asarray(weight, np.float64) + weight_offset)
    out, size = z.copy(), np.abs(z)
    if inv_freq is None:
        return out, size
    half = len(inv_freq)
    pos = np.atleast_2d(positions).astype(np.float64)
    for i in range(half):
        p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        row = 0 if axis is None else min(int(axis[i]), len(pos) - 1)
        turn = (pos[row] * np.float64(np.float32(inv_freq[i])))[:, None]
        u, v = z[..., p], z[..., q]
        out[..., p], out[..., q] = u * np.cos(turn) - v * np.sin(turn), v * np.cos(turn) + u * np.sin(turn)
        size[..., p] = size[..., q] = np.abs(u) + np.abs(v)
    return out, size


def causal_conv(x, weight, starts, bias=None, silu=True, state=None, slots=None, fresh=None):
    """x [T, C], state [n, W - 1, C] -> (y with zeros outside the sequences, size, new state, rows written).  size: sum |w in| + |bias|."""
    x, weight = np.asarray(x, np.float64), np.asarray(weight, np.float64)
    old_count = weight.shape[1] - 1
    y, size = np.zeros_like(x), np.zeros_like(x)
    written = np.zeros(len(x), bool)
    new = None if state is None else np.array(state, np.float64)
    for b in range(len(starts) - 1):
        i, j = (min(max(int(v), 0), len(x)) for v in starts[b: b + 2])
        if j <= i:
            continue
        slot = -1 if state is None else b if slots is None else int(slots[b])
        kept = slot >= 0 and slot < len(state)
        past = np.zeros((old_count, x.shape[1]))
        if kept and (fresh is None or not fresh[b]):
            past = np.asarray(state[slot], np.float64)
        line = np.concatenate([past, x[i:j]])
        for t in range(j - i):
            taps = weight.T * line[t: t + old_count + 1]
            u = taps.sum(0) + (0.0 if bias is None else np.asarray(bias, np.float64))
            size[i + t] = np.abs(taps).sum(0) + (0.0 if bias is None else np.abs(bias))
            y[i + t] = u / (1 + np.exp(-u)) if silu else u
        written[i:j] = True
        if kept:
            new[slot] = line[j - i:]
    return y, size, new, written

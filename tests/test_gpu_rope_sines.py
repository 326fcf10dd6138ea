"""Sines and cosines of the rotation, as a rotation of ones and zeros leaves them.

The angle a = position * frequency (exact in 64 bits: 20 and 24 bits) is turned into turns by a product with 1 / 2 pi, whose
own rounding and that of the product are 2^-53 of the angle each, and the difference from the nearest integer is exact: with
one 2^-53 for the reference's own, the angle is off by at most 3 * 2^-53 |a|, the 64-bit sine by 2^-50, and its rounding to float32
by half a step of the value, 2^-24.
"""
import numpy as np
import pytest
import torch

import bit_linear_layer_amd as nv
from tests.gpu_util import DEV, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,top", [(1, 10), (700, 700), (5000, 1 << 20)])
def test_sines_are_rounded_once(tokens, top, interleaved):
    say(f"rope sines {tokens} {top} {interleaved}")
    half = 64
    freq = (1e4 ** (-np.arange(half) / half)).astype(np.float32)
    pos = np.random.default_rng(tokens).integers(0, top, tokens)
    x = torch.zeros(tokens, 2, half, device=DEV)
    x[:, 0] = 1  # the first of each pair: (cos, sin)
    if interleaved:
        x = x.transpose(1, 2)
    q, _ = nv.qk_norm_rope(x.reshape(tokens, 128).contiguous(), x.reshape(tokens, 128).contiguous(), 128, torch.from_numpy(pos).to(DEV),
                           nv.Rope(torch.from_numpy(freq).to(DEV), interleaved=interleaved))
    q = q.double().cpu().numpy()
    cosine, sine = (q[:, 0::2], q[:, 1::2]) if interleaved else (q[:, :half], q[:, half:])
    turn = pos[:, None].astype(np.float64) * freq.astype(np.float64)
    for got, ref in ((cosine, np.cos(turn)), (sine, np.sin(turn))):
        assert np.all(np.abs(got - ref) <= 2.0 ** -24 * np.abs(ref) + 3 * 2.0 ** -53 * turn + 2.0 ** -50), np.max(np.abs(got - ref)) * 2 ** 24

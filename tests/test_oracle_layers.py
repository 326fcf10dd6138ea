"""Pins of the oracle of the 8-bit linear layers, the norm with rotation and the
short convolution: against torch's own roundings and transforms, closed forms
and worked examples (CPU)."""
import numpy as np
import pytest
import torch

from oracle import layer_oracle as L


def e4m3(codes):
    return torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy()


@pytest.mark.parametrize("block_rows", [1, 128])
def test_codes_are_torchs_for_power_of_two_scales(block_rows):
    """x / 2^e is exact in float32, so torch's cast gives the nearest code."""
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((200, 304)) * 10.0 ** rng.uniform(-4, 4, (200, 1))).astype(np.float32)
    x[3] = 0
    codes, scales = L.fp8_quantize(x, block_rows, pow2=True)
    s = L._spread(scales, block_rows, *x.shape)
    want = torch.from_numpy(x / s).to(torch.float8_e4m3fn)
    assert np.array_equal(codes, want.view(torch.uint8).numpy())
    top = np.abs(L.fp8_values(codes, scales, block_rows) / s).max()
    assert 224 < top <= 448


def test_scale_and_worked_codes():
    x = np.zeros((1, 144), np.float32)
    x[0, :6] = [448, -1.0625, 1.1875, 0.001, -0.0, 17]
    x[0, 128:131] = [7, np.nan, -np.inf]
    codes, scales = L.fp8_quantize(x)
    assert scales.tolist() == [[1.0, 7 / 448]]
    # 1.0625 lies between 1 and 1.125 (codes 0x38, 0x39): a tie, to the even one; 1.1875 between 0x39 and 0x3A likewise;
    # 17 between 16 (0x58) and 18 (0x59)
    assert codes[0, :6].tolist() == [0x7E, 0xB8, 0x3A, 0x01, 0x80, 0x58]
    assert codes[0, 128:131].tolist() == [0x7E, 0x7F, 0xFF]
    assert L.fp8_quantize(np.zeros((2, 16), np.float32))[1].max() == 0


def test_values_and_product():
    rng = np.random.default_rng(1)
    x, w = rng.standard_normal((5, 272)).astype(np.float32), rng.standard_normal((130, 272)).astype(np.float32)
    (ac, as_), (wc, ws) = L.fp8_quantize(x), L.fp8_quantize(w, 128)
    out, size = L.fp8_gemm(ac, as_, wc, ws)
    want = np.zeros((5, 130))
    for b in range(3):
        at = np.s_[:, b * 128: (b + 1) * 128]
        want += e4m3(ac)[at].astype(float) @ e4m3(wc)[at].T.astype(float) * as_[:, b: b + 1] * np.repeat(ws[:, b], 128)[:130]
    assert np.allclose(out, want, rtol=1e-12, atol=1e-12) and np.all(np.abs(out) <= size * (1 + 1e-12))
    assert np.abs(out - x.astype(float) @ w.T).max() < 0.05 * size.max()  # 2^-4 each way at most


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((7, 3, 64))
    pos = np.stack([np.arange(7), np.arange(7) * 1000, 1 << np.arange(7)])
    freq = (10000.0 ** (-np.arange(16) / 16)).astype(np.float32)
    axis = np.arange(16) % 4  # 3 counts as 2
    out, _ = L.qk_norm_rope(x, 64, positions=pos, inv_freq=freq, axis=axis, interleaved=interleaved)
    turn = pos[np.minimum(axis, 2)].T * freq.astype(float)
    z = x[..., 0:32:2] + 1j * x[..., 1:32:2] if interleaved else x[..., :16] + 1j * x[..., 16:32]
    z = z * np.exp(1j * turn)[:, None]
    got = out[..., 0:32:2] + 1j * out[..., 1:32:2] if interleaved else out[..., :16] + 1j * out[..., 16:32]
    assert np.allclose(got, z, atol=1e-12) and np.array_equal(out[..., 32:], x[..., 32:])


def test_norm():
    rng = np.random.default_rng(3)
    x, w = rng.standard_normal((4, 2, 128)), rng.standard_normal(128)
    out, _ = L.qk_norm_rope(x, 128, weight=w, weight_offset=1.0, eps=1e-5)
    t = torch.nn.functional.rms_norm(torch.from_numpy(x), (128,), torch.from_numpy(w + 1), 1e-5)
    assert np.allclose(out, t.numpy(), rtol=1e-12)


def test_convolution_is_torchs_and_splits():
    rng = np.random.default_rng(4)
    x, w, bias = rng.standard_normal((23, 16)), rng.standard_normal((16, 4)), rng.standard_normal(16)
    y, size, _, written = L.causal_conv(x, w, [0, 23], bias, silu=False)
    t = torch.nn.functional.conv1d(torch.from_numpy(x.T)[None], torch.from_numpy(w)[:, None], torch.from_numpy(bias), padding=3, groups=16)
    assert np.allclose(y, t[0, :, :23].T.numpy(), rtol=1e-12) and np.all(np.abs(y) <= size + 1e-12) and written.all()
    # one sequence in pieces of 1, 2, 0 and 20 rows, the state carried in slot 1 of 3
    whole = L.causal_conv(x, w, [0, 23], bias)[0]
    state, parts, at = rng.standard_normal((3, 3, 16)), [], 0
    untouched = state[[0, 2]].copy()
    for i, n in enumerate([1, 2, 0, 20]):
        y, _, state, _ = L.causal_conv(x[at: at + n], w, [0, n], bias, state=state, slots=[1], fresh=[i == 0])
        parts.append(y)
        at += n
    assert np.allclose(np.concatenate(parts), whole, rtol=1e-12)
    assert np.array_equal(state[1], x[-3:]) and np.array_equal(state[[0, 2]], untouched)

"""The oracle of the paged FP8 KV cache: scale exponents and codes against
brute force over every code, the layout as a bijection, the attention
against closed forms."""
import numpy as np
import pytest

from oracle import kv_pages_oracle as P


@pytest.mark.parametrize("a,e", [(448.0, 0), (np.nextafter(np.float32(448), np.float32(1e9)), 1), (224.0, -1), (1.0, -8),
                                 (1.75, -8), (1.7500001, -7), (0.0, -126), (2.0 ** -149, -126), (3.4e38, 120)])
def test_scale_is_the_least_power_of_two_that_holds_the_row(a, e):
    x = np.zeros(64, np.float32)
    x[5] = -np.float32(a)
    codes, byte = P.quantize_rows(x)
    assert int(byte) - 127 == e
    assert a <= 448 * 2.0 ** e and (e == -126 or a > 448 * 2.0 ** (e - 1))


def test_codes_are_nearest_with_ties_to_even():
    rng = np.random.default_rng(0)
    mids = (P.MAGNITUDES[1:] + P.MAGNITUDES[:-1]) / 2
    x = np.concatenate([mids, P.MAGNITUDES, rng.uniform(0, 448, 200), [448.0]]).astype(np.float32)
    x *= rng.choice([-1, 1], x.size)
    codes, byte = P.quantize_rows(x)
    assert int(byte) == 127
    for v, c in zip(x.astype(np.float64), codes):
        dist = np.abs(P.MAGNITUDES - abs(v))
        best = np.flatnonzero(dist == dist.min())
        want = best[0] if best.size == 1 else best[best % 2 == 0][0]
        assert c & 0x7F == want and (c >> 7) == (v < 0)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_block_layout_is_a_bijection(dim):
    o, d = np.divmod(np.arange(16 * dim), dim)
    for at in (P.key_index(o, d, dim), P.value_index(o, d)):
        assert np.array_equal(np.sort(at), np.arange(16 * dim))


def test_write_then_read_keeps_the_nearest_values():
    rng = np.random.default_rng(1)
    pages = P.Pages(3, 2, 64, 32)
    slots = rng.permutation(96)[:40]
    k, v = (rng.standard_normal((40, 128)).astype(np.float32) for _ in range(2))
    pages.write(k, v, np.concatenate([slots[:39], [96]]))  # the last one is outside
    kk, vv = pages.read(slots[:39])
    for got, x in ((kk, k), (vv, v)):
        x = x[:39].reshape(39, 2, 64).astype(np.float64)
        step = np.maximum(np.abs(x) / 16, np.abs(x).max(-1, keepdims=True) / 224 * 2.0 ** -10)
        assert np.all(np.abs(got - x) <= step)


def test_attention_of_equal_keys_is_the_mean_and_masks_hold():
    rng = np.random.default_rng(2)
    pages = P.Pages(4, 1, 64, 16)
    v = rng.standard_normal((40, 64)).astype(np.float32)
    pages.write(np.ones((40, 64), np.float32), v, np.arange(40))
    _, vq = pages.read(np.arange(40))
    q = rng.standard_normal((3, 64))
    o, _ = P.attention(q, pages, 1, 0.125, np.array([[1, 2]]), [20], 3, [0], 16)
    for j in range(3):  # the prefix (slots 0..15) and 18 + j own tokens (slots 16..)
        assert np.allclose(o[j, 0], vq[: 16 + 18 + j, 0].mean(0), rtol=1e-12, atol=1e-12)
    o, _ = P.attention(q[:1], pages, 1, 0.125, np.array([[7, 2]]), [17], 1, [], 0)  # page 7 does not exist
    assert np.allclose(o[0, 0], vq[32, 0])
    o, _ = P.attention(q, pages, 1, 0.125, np.array([[1, 2]] * 3), [0, -1, 2], 1, [], 0)
    assert np.all(o[0] == 0) and np.all(np.isnan(o[1])) and np.allclose(o[2, 0], vq[16:18, 0].mean(0), atol=0.2)


def test_attention_is_one_softmax_over_prefix_and_own_tokens():
    rng = np.random.default_rng(3)
    pages = P.Pages(4, 2, 64, 16)
    pages.write(rng.standard_normal((50, 128)), rng.standard_normal((50, 128)), np.arange(50))
    k, v = pages.read(np.arange(50))
    q = rng.standard_normal((1, 4 * 64))
    o, wv = P.attention(q, pages, 4, 0.125, np.array([[2, 3]]), [18], 1, [0, 1], 32)
    for h in range(4):
        x = k[:, h // 2] @ q.reshape(4, 64)[h] * 0.125
        w = np.exp(x) / np.exp(x).sum()
        assert np.allclose(o[0, h], w @ v[:, h // 2]) and np.allclose(wv[0, h], w @ np.abs(v[:, h // 2]))

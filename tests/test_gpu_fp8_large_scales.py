"""The 8-bit linear layers' products where the product of two scales is beyond
float32's range: the result counts as it is -- sums of 0 add 0, small sums add
finite numbers.  All codes are positive, so that nothing cancels; a block beyond the range rounds
two times more than others, which the (K / 128 + 136) 2^-23 of the other tests holds too."""
import numpy as np
import pytest
import torch

import bit_linear_layer_amd as nv
from oracle import layer_oracle as L
from tests.gpu_util import DEV, say

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
TOP = float(np.finfo(np.float32).max)


def on(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


@pytest.mark.parametrize("m,n,k", [(3, 700, 272), (20, 300, 400), (50, 515, 272), (100, 130, 1040), (200, 1500, 6400), (600, 12900, 336)])
@pytest.mark.parametrize("out_dtype,cut", [(BF16, False), (F32, False), (BF16, True)])
def test_products_of_scales_beyond_float32(m, n, k, out_dtype, cut):
    say(f"fp8 large scales {m}x{n}x{k} {out_dtype} {cut}")
    rng = np.random.default_rng(m + n)
    blocks = -(-k // 128)
    # few small codes (1 to 9 times 2^-9), some rows with none at all
    a, w = (np.where(rng.random((rows, k)) < 0.02, rng.integers(1, 10, (rows, k)), 0).astype(np.uint8) for rows in (m, n))
    a[m // 2], w[n // 2] = 0, 0
    sa = rng.choice([2.0 ** -30, 0.7, 3.0 * 2.0 ** 40, 1.1 * 2.0 ** 100, TOP / 448], (m, blocks)).astype(np.float32)
    sw = rng.choice([0.9, 2.0 ** 9, 1.3 * 2.0 ** 20, 1.7 * 2.0 ** 38], (-(-n // 128), blocks)).astype(np.float32)
    ref, size = L.fp8_gemm(a, sa, w, sw)
    with np.errstate(over="ignore"):
        assert np.isinf(sa[:, None] * sw[None]).any()
    out = nv.fp8_gemm(nv.FP8Tensor(on(a), on(sa), m, k, 1), nv.FP8Tensor(on(w), on(sw), n, k, 128), out_dtype, cut_sums=cut)
    got = out.double().cpu().numpy()
    tol = (k / 128 + 136) * 2.0 ** -23 * size + (2.0 ** -10 * size if cut else 0.0)
    if out_dtype == BF16:
        tol = tol + 2.0 ** -8 * (ref + tol)
    finite, beyond = ref < TOP * 0.99, ref > TOP * 1.01
    assert finite.any() and beyond.any() and (ref[finite] > TOP * 2.0 ** -20).any()
    bad = np.argwhere(~(np.abs(got - ref) <= tol + 2.0 ** -126) & finite)
    assert bad.size == 0, f"{len(bad)} outside, first {bad[:3].tolist()}: {[(got[i, j], ref[i, j]) for i, j in bad[:3]]}"
    assert np.all(np.isposinf(got[beyond]))
    assert np.all(got[m // 2] == 0) and np.all(got[:, n // 2] == 0)

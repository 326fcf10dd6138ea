"""SiLU of the short convolution with float32 outputs, over its whole range.

The taps leave u itself.  In units of 2^-24 of the result: the exponential is
off by at most 2 (one ulp of the hardware's), its correction rounds once, 1 + e
once, the quotient twice, the product with u once: at most 8; results below
2^-126 round to a multiple of 2^-149 besides."""
import numpy as np
import pytest
import torch

import bit_linear_layer_amd as nv
from tests.gpu_util import DEV, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("single", [False, True])
@pytest.mark.parametrize("width", [2, 4])
def test_float32_silu_is_float32(width, single):
    say(f"conv silu float32 W={width} single {single}")
    rng = np.random.default_rng(width)
    u = np.concatenate([np.linspace(-110, 110, 40000), rng.standard_normal(20000), -10.0 ** rng.uniform(-30, 2, 4000),
                        [0.0, -0.0, 1e30, -1e30, 88.0, -87.4, -103.9, 200.0, -200.0, 3e38, -3e38, 0.5, -0.5, 1.0, -1.0, 2.0]])
    u = u.astype(np.float32).reshape(-1, 8)
    w = torch.zeros(8, width, device=DEV)
    w[:, -1] = 1
    x = torch.from_numpy(u).to(DEV)
    y = nv.causal_conv(x, w, len(u) if single else 1).double().cpu().numpy()
    u = u.astype(np.float64)
    with np.errstate(over="ignore"):
        ref = u / (1 + np.exp(-u))
    off = np.abs(y - ref) - 2.0 ** -149
    bad = np.argwhere(~(off <= 8 * 2.0 ** -24 * np.abs(ref)))
    assert bad.size == 0, f"{len(bad)} outside, first {[(u[i, j], y[i, j], ref[i, j]) for i, j in bad[:4]]}"


def test_infinities_and_nan():
    say("conv silu infinities")
    x = torch.tensor([[np.inf, -np.inf, np.nan, 1.0, -1.0, 0.0, 5.0, -5.0]], device=DEV)
    w = torch.zeros(8, 2, device=DEV)
    w[:, -1] = 1
    y = nv.causal_conv(x, w).cpu()[0]
    assert y[0] == np.inf and bool(y[1:3].isnan().all()) and bool(y[3:].isfinite().all())

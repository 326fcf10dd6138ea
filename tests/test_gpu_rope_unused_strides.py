"""Strides that are not used change nothing: one token's rows, one head's heads."""
import pytest
import torch

import bit_linear_layer_amd as nv
from tests.gpu_util import DEV, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,heads", [(1, 5), (7, 1), (1, 1)])
@pytest.mark.parametrize("odd", [-3, 1, 1 << 62])
def test_unused_strides(tokens, heads, odd):
    say(f"rope unused strides {tokens} {heads} {odd}")
    x = torch.randn(tokens, heads * 128, device=DEV)
    w = torch.rand(128, device=DEV)
    want = torch.empty_like(x)
    nv.nvfp4_qk_norm_rope(x, None, want, None, 128, q_weight=w)
    out = torch.zeros_like(x)
    ld, head = (odd if tokens == 1 else heads * 128), (odd if heads == 1 else 128)
    rows = nv._HEAD_ROWS(x.data_ptr(), ld, head, out.data_ptr(), ld, head, w.data_ptr(), heads)
    assert nv.load().nvfp4_qk_norm_rope(rows, None, nv.DTYPE_F32, tokens, 128, 1e-6, 0.0, None, torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert torch.equal(out, want)

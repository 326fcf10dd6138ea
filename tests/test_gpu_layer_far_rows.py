"""Rows, states and outputs whose offsets pass 32 bits: the same bits as the
same call on dense tensors."""
import pytest
import torch

import bit_linear_layer_amd as nv
from tests.gpu_util import DEV, say

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def far(t, ld):
    """t's rows (all but the first dimension kept dense) ld elements apart, beyond 2^31 elements in all."""
    assert len(t) * ld > 2 ** 31
    out = torch.empty(len(t) * ld, dtype=t.dtype, device=DEV).as_strided(t.shape, (ld, *t.stride()[1:]))
    out.copy_(t)
    return out


def normal(seed, *shape, dtype=BF16):
    g = torch.Generator(DEV).manual_seed(seed)
    return torch.randn(*shape, device=DEV, generator=g).to(dtype)


@pytest.mark.parametrize("rows", [3, 40, 100, 600])
@pytest.mark.parametrize("out_dtype", [BF16, F32])
def test_far_weight_codes(rows, out_dtype):
    say(f"far weight codes {rows} {out_dtype}")
    x, w = normal(1, rows, 272), nv.fp8_quantize(normal(2, 600, 272), 128)
    wide = nv.FP8Tensor(far(w.codes, 2 ** 22 - 16), w.scales, w.rows, w.cols, 128)
    assert torch.equal(nv.fp8_linear(x, wide, out_dtype), nv.fp8_linear(x, w, out_dtype))


@pytest.mark.parametrize("n,k", [(1000, 6400), (20000, 528)])
def test_far_activations_and_outputs(n, k):
    """The first product is shared out in steps, the second goes to whole tiles."""
    say(f"far activations {n}x{k}")
    x, w = normal(3, 600, k), nv.fp8_quantize(normal(4, n, k), 128)
    want, q = nv.fp8_linear(x, w), nv.fp8_quantize(x)
    xf = far(x, 2 ** 22)
    codes = nv.FP8Tensor(far(torch.zeros_like(q.codes), 2 ** 22 - 16), torch.empty_like(q.scales), 600, k)
    nv.nvfp4_fp8_quantize(xf, codes)
    assert torch.equal(codes.codes, q.codes) and torch.equal(codes.scales, q.scales)
    out = far(torch.zeros_like(want), 2 ** 22)
    nv.nvfp4_fp8_gemm(codes, w, out, nv.fp8_gemm_workspace(600))
    assert torch.equal(out, want)
    out.zero_()
    nv.nvfp4_fp8_linear(xf, w, out, nv.fp8_linear_workspace(600, k))
    assert torch.equal(out, want)


def test_far_heads():
    say("far heads")
    q, k = normal(5, 270, 4 * 128), normal(6, 270, 128)
    rope = nv.Rope(1e4 ** (-torch.arange(32, device=DEV, dtype=F32) / 32))
    pos, w = torch.arange(270, device=DEV) * 11, normal(7, 128, dtype=F32)
    want = nv.qk_norm_rope(q, k, 128, pos, rope, w, w)
    got = far(torch.zeros_like(q), 2 ** 23), far(torch.zeros_like(k), 2 ** 23)
    nv.nvfp4_qk_norm_rope(far(q, 2 ** 23), far(k, 2 ** 23), *got, 128, pos, rope, w, w)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("each", [1, 3])
def test_far_convolution(each):
    say(f"far convolution {each}")
    x, w, state = normal(8, 270 * each, 64), normal(9, 64, 4, dtype=F32), normal(10, 270, 3, 64)
    kept, slots = far(state, 2 ** 23), torch.randperm(270, device=DEV).int()
    want = nv.causal_conv(x, w, 270, state=state, slots=slots)
    got = far(torch.zeros_like(x), 2 ** 23)
    nv.nvfp4_causal_conv(far(x, 2 ** 23), w, got, 270, state=kept, slots=slots)
    assert torch.equal(got, want) and torch.equal(kept, state)


def test_far_states():
    say("far states")
    q, k, v, beta, g = normal(11, 12, 128), normal(12, 12, 128), normal(13, 12, 256), normal(14, 12, 2).sigmoid(), -normal(15, 12, 2).abs()
    state, slots = normal(16, 270, 2, 128, 128, dtype=F32), torch.tensor([269, 0, 268, -1, 100, 270], dtype=torch.int32, device=DEV)
    pool = far(state, 2 ** 23)
    o = torch.zeros(12, 256, device=DEV)
    got = o.clone()
    nv.nvfp4_gdn_step(q, k, v, beta, g, o, 1, 2, state, slots, 2)
    nv.nvfp4_gdn_step(q, k, v, beta, g, got, 1, 2, pool, slots, 2)
    assert torch.equal(got, o) and torch.equal(pool, state) and bool((o[:2] != 0).all()) and bool((o[6:8] == 0).all())

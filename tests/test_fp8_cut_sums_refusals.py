"""Cut sums are for bf16 outputs only (CPU: refused before any HIP call, or nothing to do)."""
import bit_linear_layer_amd as nv
from tests.test_layer_refusals import fp8, gemm, linear

BF16, F32 = nv.DTYPE_BF16 | nv.FP8_CUT_SUMS, nv.DTYPE_F32 | nv.FP8_CUT_SUMS


def test_cut_sums_take_bf16_outputs():
    assert gemm(dt=F32) == -9 and linear(odt=F32) == -9
    assert gemm(dt=BF16 | 2) == -3 and gemm(dt=0x200) == -3 and linear(odt=BF16 | 2) == -3
    # the other checks follow as they do without
    assert gemm(dt=BF16, ld=129) == -4 and gemm(dt=BF16, out=None) == -1 and linear(odt=BF16, ws=None) == -8
    assert gemm(dt=BF16, a=fp8(rows=0)) == 0 and linear(odt=BF16, rows=0) == 0

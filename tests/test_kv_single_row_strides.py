"""The strides that the binding passes on for one row and for one page."""
import torch

import bit_linear_layer_amd as nv


def test_one_row():
    cpu = torch.device("cpu")
    t = torch.zeros(4, 130, dtype=torch.bfloat16)
    assert nv._row_stride(t[0:1, :128], 1, 128, cpu, "x") == 128
    assert nv._row_stride(t[:, :128], 4, 128, cpu, "x") == 130  # (refused by the C ABI)
    assert nv._row_stride(t[0:0, :128], 0, 128, cpu, "x") == 128
    assert nv._row_stride(t[0:1].expand(1, 130)[:, :64], 1, 64, cpu, "x") == 64

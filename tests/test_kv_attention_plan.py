"""Which batches have their shared prefix computed once for all sequences, seen
on the CPU through the workspace that the attention asks for.

Where each sequence reads the prefix for itself, the workspace holds the partial
results of one pass: a slot of `tile` rows for each tile and share, with two
floats and head_dim sums a row, and two ints a tile -- or nothing, if a tile is
one unit of work.  A pass over the prefix for all sequences adds its own.
"""
import pytest
import torch

import bit_linear_layer_amd as nv

BF16, F32 = torch.bfloat16, torch.float32


def up(a, b):
    return -(-a // b)


def one_pass_bytes(batch, heads, group, dim, q_len, max_len, prefix, dtype):
    """The workspace where each sequence reads the prefix for itself."""
    rows = q_len * group
    wide = dtype == BF16 and rows > 16
    wm = (1 if rows <= 32 else 2 if rows <= 64 else 4) if wide else 0
    tile = 32 * wm if wide else 16
    step = 32 if wide and dim == 256 else 64
    waves = 4 // wm if wide else 4
    per_cu = (1 if wm == 1 else 2) if wide else (1 if dtype == F32 or dim == 256 else 2)
    tiles = batch * heads * up(rows, tile)
    solo = tile == 16 and tiles >= 1024 and batch > 1
    waves = 1 if solo else waves
    steps = up(prefix, step) + up(max_len, step)
    units = tiles * max(1, up(steps, waves))
    shares = 4 * min(up(units, 4), 256 * per_cu) if solo else min(units, 256 * per_cu)
    if steps <= waves:
        return 16
    return 16 + 4 * ((tiles + shares) * tile * (2 + dim) + up(2 * tiles, 4) * 4)


def workspace(batch, heads, group, dim, q_len, max_len, prefix, dtype):
    """What the attention asks for (through the C ABI, without a device)."""
    import ctypes
    p = nv._KVPages(0, 0, 0, 0, 1 << 20, 0, 0, heads, dim, 16)
    b = nv._KVBatch(batch, q_len, None, max_len, None, 0, 0, None, prefix)
    return nv.load().nvfp4_kv_pages_attention_workspace_bytes(ctypes.byref(p), ctypes.byref(b), heads * group,
                                                              nv.DTYPE_BF16 if dtype == BF16 else nv.DTYPE_F32)


def prefix_is_shared(batch, heads, group, dim, q_len, max_len, prefix, dtype):
    need, alone = workspace(batch, heads, group, dim, q_len, max_len, prefix, dtype), \
        one_pass_bytes(batch, heads, group, dim, q_len, max_len, prefix, dtype)
    assert need > 0 and (need == alone or need >= one_pass_bytes(batch, heads, group, dim, q_len, max_len, 0, dtype))
    return need != alone


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("batch,heads,group,q_len", [
    (1, 1, 1, 1), (1, 8, 4, 512), (3, 2, 8, 2), (64, 8, 4, 1), (200, 8, 2, 1), (7, 3, 5, 4), (9, 1, 1, 64), (4, 2, 9, 7)])
def test_without_a_prefix_there_is_one_pass(batch, heads, group, q_len, dim, dtype):
    for max_len in (0, 1, 64, 65, 256, 257, 5000, 1 << 20):
        args = (batch, heads, group, dim, q_len, max_len, 0, dtype)
        assert workspace(*args) == one_pass_bytes(*args)


RULE = [
    # batch, heads, rows of a sequence and head, dim, prefix, dtype, shared
    (1, 8, 4, 128, 1 << 20, BF16, False),   # one sequence has nothing to share
    (16, 8, 4, 128, 1023, BF16, False), (16, 8, 4, 128, 1024, BF16, True),
    (16, 8, 16, 256, 1023, BF16, False), (16, 8, 16, 256, 1024, BF16, True),
    (16, 8, 1, 64, 1023, F32, False), (16, 8, 1, 64, 1024, F32, True),
    (2, 2, 4, 128, 16383, BF16, False), (2, 2, 4, 128, 16384, BF16, True),    # 2^16 in all
    (8, 2, 4, 256, 4095, BF16, False), (8, 2, 4, 256, 4096, BF16, True),
    (5, 2, 4, 128, 6553, F32, False), (5, 2, 4, 128, 6554, F32, True),
    (64, 8, 4, 128, 1535, BF16, False), (64, 8, 4, 128, 1536, BF16, True),    # 512 own tiles
    (127, 8, 4, 64, 1535, BF16, False), (127, 8, 4, 64, 1536, BF16, True),
    (63, 8, 4, 128, 1024, BF16, True), (128, 8, 4, 128, 1024, BF16, True),    # 504, 1024
    (64, 8, 4, 256, 1024, BF16, True), (64, 8, 4, 128, 1024, F32, True),
    (255, 8, 4, 128, 512, BF16, False), (256, 8, 4, 128, 511, BF16, False), (256, 8, 4, 128, 512, BF16, True),
    (256, 8, 4, 256, 512, F32, True),
    (16, 8, 17, 128, 12287, BF16, False), (16, 8, 17, 128, 12288, BF16, True),  # 17 to 48 rows: 3 * 2^19 in all
    (16, 8, 48, 256, 12287, BF16, False), (16, 8, 48, 256, 12288, BF16, True),
    (16, 8, 49, 128, 1 << 20, BF16, False),
]


@pytest.mark.parametrize("batch,heads,rows,dim,prefix,dtype,shared", RULE)
def test_the_rule(batch, heads, rows, dim, prefix, dtype, shared):
    for max_len in (64, 1000):
        assert prefix_is_shared(batch, heads, rows, dim, 1, max_len, prefix, dtype) == shared

"""One row (a decode step of one sequence) and one page may carry any stride:
it is never used, so no call is refused for it."""
import pytest
import torch

import bit_linear_layer_amd as nv
from tests.gpu_util import DEV, say

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pad", [1, 2, 3, 7])
def test_one_row_of_a_padded_buffer(pad, dtype):
    say(f"kv one row {pad} {dtype}")
    heads, dim, page = 2, 64, 16
    g = torch.Generator(device=DEV).manual_seed(pad)
    rand = lambda *shape: torch.randn(shape, generator=g, device=DEV).to(dtype)  # noqa: E731
    row = lambda width: rand(3, width + pad)[0:1, :width]  # noqa: E731
    a, b = (nv.empty_kv_pages(3, heads, dim, page) for _ in range(2))
    slots = torch.tensor([20], device=DEV)
    k, v, q = row(heads * dim), row(heads * dim), row(4 * heads * dim)
    assert q.stride(0) == 4 * heads * dim + pad
    nv.kv_pages_write(a, k, v, slots)
    nv.kv_pages_write(b, k.contiguous(), v.contiguous(), slots)
    outs = [torch.full((3, heads * dim + pad), 5.0, dtype=dtype, device=DEV) for _ in range(2)]
    nv.nvfp4_kv_pages_read(a, slots, *(t[0:1, : heads * dim] for t in outs))
    for got, want in zip(outs, nv.kv_pages_read(b, slots, dtype)):
        assert torch.equal(got[0:1, : heads * dim], want)
        assert torch.all(got[1:] == 5.0) and torch.all(got[0, heads * dim:] == 5.0)
    table = torch.tensor([[1]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([5], dtype=torch.int32, device=DEV)
    for t in (a, b):
        nv.kv_pages_write(t, *(torch.arange(4 * heads * dim, device=DEV).remainder(7).to(dtype).view(4, -1) for _ in range(2)),
                          torch.arange(16, 20, device=DEV))
    wide = torch.full((3, q.shape[1] + pad), 5.0, dtype=dtype, device=DEV)
    nv.kv_pages_attention(q, a, table, lens, out=wide[0:1, : q.shape[1]])
    assert torch.equal(wide[0:1, : q.shape[1]], nv.kv_pages_attention(q.contiguous(), b, table, lens))
    assert torch.all(wide[1:] == 5.0) and torch.all(wide[0, q.shape[1]:] == 5.0)


@pytest.mark.parametrize("pad", [1, 4, 8, 24])
def test_one_page_of_a_padded_buffer(pad):
    say(f"kv one page {pad}")
    heads, dim, page = 1, 64, 16
    tensors = [torch.full((4, width + pad), 0xFF, dtype=torch.uint8, device=DEV)
               for width in (page * dim, page * dim, page, page)]
    whole = [t[0:1] for t in tensors]  # rows as wide as the buffer's, of an odd stride
    cut = [t[0:1, :w] for t, w in zip(tensors, (page * dim, page * dim, page, page))]
    x = torch.randn((7, dim), device=DEV).to(BF16)
    slots = torch.arange(3, 10, device=DEV)
    dense = nv.empty_kv_pages(1, heads, dim, page)
    nv.kv_pages_write(dense, x, -x, slots)
    want = nv.kv_pages_read(dense, slots)
    for part in (whole, cut):
        pages = nv.KVPages(*part, heads, dim, page)
        nv.kv_pages_write(pages, x, -x, slots)
        for got, w in zip(nv.kv_pages_read(pages, slots), want):
            assert torch.equal(got, w)
    assert all(torch.all(t[1:] == 0xFF) for t in tensors)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_calls_with_nothing_in_them(dtype):
    """No rows, no sequences, a table without pages, nothing to attend to."""
    say(f"kv empty calls {dtype}")
    pages = nv.empty_kv_pages(3, 2, 64, 16)
    for t in (pages.k_codes, pages.v_codes, pages.k_scales, pages.v_scales):
        t.fill_(0xFF)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    empty, slots = torch.empty((0, 128), dtype=dtype, device=DEV), torch.empty(0, dtype=torch.int64, device=DEV)
    nv.kv_pages_write(pages, empty, empty, slots)
    assert [tuple(t.shape) for t in nv.kv_pages_read(pages, slots, dtype)] == [(0, 128)] * 2
    assert nv.kv_pages_attention(torch.empty((0, 256), dtype=dtype, device=DEV), pages, none.view(0, 1)[:, :0], none).shape == (0, 256)
    q = torch.ones((4, 256), dtype=dtype, device=DEV)
    assert torch.all(nv.kv_pages_attention(q, pages, q_len=2) == 0)
    lens = torch.zeros(4, dtype=torch.int32, device=DEV)
    assert torch.all(nv.kv_pages_attention(q, pages, torch.zeros((4, 0), dtype=torch.int32, device=DEV), lens) == 0)
    assert torch.all(nv.kv_pages_attention(q, pages, torch.zeros((4, 2), dtype=torch.int32, device=DEV), lens) == 0)

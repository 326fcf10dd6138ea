"""GPU parity of the 8-bit linear layers: the quantizer bit for bit against the
oracle, the product within the derived bound.

With A = sum |a w| over a row and column (K terms in blocks of 128):
  float32 output: products of two E4M3 values are exact in float32; a block's
    sum and the matrix unit's steps round at most 128 times, the scales' product
    once, its fma once per block, each by at most 2^-23 of the magnitudes so
    far: (K / 128 + 136) 2^-23 A.
  bf16 output: in the 8-bit instructions the 7 smaller of 8 products are cut
    by less than 2^-13 of the largest's power of two each: less than 2^-10 A
    more; then the output's rounding, half a step: 2^-8 |out|.
"""
import numpy as np
import pytest
import torch

import bit_linear_layer_amd as nv
from oracle import layer_oracle as L
from tests.gpu_util import DEV, say, x_f32

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def matrix(rng, rows, cols, dtype):
    """Loud columns, tiny and zero rows and pieces, exact ties."""
    x = rng.standard_normal((rows, cols)) * 10.0 ** rng.uniform(-3, 3, (rows, 1))
    x[:, rng.integers(0, cols, max(1, cols // 60))] *= 40
    if rows > 2:
        x[1] = 0
        mids = (L.MAGNITUDES[1:] + L.MAGNITUDES[:-1]) / 2
        x[2] = rng.choice(mids, cols) * rng.choice([-1.0, 1.0], cols)
        x[2, ::128] = 448
    if cols > 128:
        x[0, :128] = -0.0
    return torch.from_numpy(x.astype(np.float32)).to(dtype).to(DEV)


def host(q):
    torch.cuda.synchronize()
    return q.codes[:, : q.cols].cpu().numpy(), q.scales[:, : -(-q.cols // 128)].cpu().numpy()


def same(q, x, block_rows, pow2=False):
    codes, scales = host(q)
    want = L.fp8_quantize(x_f32(x), block_rows, pow2)
    assert np.array_equal(scales.view(np.uint32), want[1].view(np.uint32)), np.argwhere(scales != want[1])[:4]
    bad = np.argwhere(codes != want[0])
    assert bad.size == 0, f"{len(bad)} codes differ, first {bad[:4].tolist()}"


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 128), (3, 144), (5, 1040), (67, 272), (130, 2064), (700, 5120)])
def test_rows_bit_exact(rows, cols, dtype):
    say(f"fp8 quantize rows {rows}x{cols} {dtype}")
    x = matrix(np.random.default_rng(rows + cols), rows, cols, dtype)
    for pow2 in (False, True):
        same(nv.fp8_quantize(x, 1, nv.FP8_SCALE_POW2 if pow2 else nv.FP8_SCALE_F32), x, 1, pow2)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", [(1, 16), (127, 128), (129, 144), (300, 1040), (256, 512)])
def test_blocks_bit_exact(rows, cols, dtype):
    say(f"fp8 quantize blocks {rows}x{cols} {dtype}")
    x = matrix(np.random.default_rng(rows + cols), rows, cols, dtype)
    for pow2 in (False, True):
        same(nv.fp8_quantize(x, 128, nv.FP8_SCALE_POW2 if pow2 else nv.FP8_SCALE_F32), x, 128, pow2)


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("pow2", [False, True])
def test_extreme_values(block_rows, pow2):
    """Largest and smallest magnitudes, scales that vanish, infinities and NaN in a block's middle."""
    say(f"fp8 quantize extremes {block_rows} {pow2}")
    rng = np.random.default_rng(7)
    tops = [3.4e38, 448.0, 2.0 ** -80, 2.0 ** -81, 2.0 ** -117, 2.0 ** -126, 2.0 ** -140, 2.0 ** -149, 1e30, 7.0, 0.0]
    x = (rng.uniform(-1, 1, (len(tops) * 2, 272)) * np.repeat(tops, 2)[:, None]).astype(np.float32)
    x[:, 0] = x[:, 128] = np.repeat(tops, 2)
    x[::2, 5] = np.inf
    x[::2, 130:132] = [np.nan, -np.inf]
    x[3, :128] = np.nan
    x = torch.from_numpy(x).to(DEV)
    for part in x.split(1) if block_rows == 128 else [x]:
        part = part.contiguous()
        same(nv.fp8_quantize(part, block_rows, nv.FP8_SCALE_POW2 if pow2 else nv.FP8_SCALE_F32), part, block_rows, pow2)


def test_strides_and_what_is_left_alone():
    say("fp8 quantize strides")
    rng = np.random.default_rng(8)
    wide = matrix(rng, 70, 512, BF16)
    x = wide[:, 16: 16 + 272]
    for block in (1, 128):
        high = 70 if block == 1 else 1
        codes = torch.full((70, 320), 0xAB, dtype=torch.uint8, device=DEV)
        scales = torch.full((high, 5), -7.0, device=DEV)
        q = nv.FP8Tensor(codes, scales, 70, 272, block)
        nv.nvfp4_fp8_quantize(x, q)
        same(q, x, block)
        assert bool((codes[:, 272:] == 0xAB).all()) and bool((scales[:, 3:] == -7).all())
    assert nv.fp8_quantize(x[:0]).codes.shape == (0, 272)


def operands(rng, m, n, k, dtype=BF16):
    return nv.fp8_quantize(matrix(rng, m, k, dtype)), nv.fp8_quantize(matrix(rng, n, k, dtype) * 0.02, 128)


def close(out, a, w, extra=0.0):
    ref, size = L.fp8_gemm(*host(a), *host(w))
    tol = (a.cols / 128 + 136) * 2.0 ** -23 * size
    if out.dtype == BF16:
        tol = tol + 2.0 ** -10 * size
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    err = np.abs(out.float().cpu().numpy().astype(np.float64) - ref)
    bad = np.argwhere(~(err <= tol + 2.0 ** -126))
    assert bad.size == 0, f"{len(bad)} of {err.size} outside, first {bad[:3].tolist()}: {[(err[i, j], tol[i, j]) for i, j in bad[:3]]}"


SHAPES = [(1, 1, 16), (300, 300, 16), (129, 70, 128), (240, 256, 144), (1000, 40, 272), (130, 1, 16), (4, 384, 6400), (16, 200, 17408), (30, 640, 3600), (100, 130, 6400), (130, 130, 9984), (224, 128, 16384), (225, 192, 400), (1, 128, 128), (2, 130, 144), (3, 1000, 272), (5, 4096, 1040), (15, 64, 4096), (16, 129, 2064), (17, 257, 128),
          (33, 100, 640), (64, 512, 1024), (65, 384, 2064), (77, 1000, 400), (128, 128, 128), (129, 640, 256), (200, 1111, 912),
          (257, 513, 384), (300, 256, 3200), (511, 1280, 512)]


@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product(m, n, k, out_dtype):
    say(f"fp8 gemm {m}x{n}x{k} {out_dtype}")
    a, w = operands(np.random.default_rng(m * 7 + n), m, n, k)
    close(nv.fp8_gemm(a, w, out_dtype), a, w)


@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("m,n,k", [(1, 34816, 1024), (9, 5120, 5120), (40, 5120, 8192), (150, 2048, 17408), (1030, 1300, 1024), (2048, 2560, 512), (200, 17000, 400),
                                   (500, 5120, 1200), (700, 12900, 272)])
def test_product_of_large_operands(m, n, k, out_dtype):
    say(f"fp8 gemm large {m}x{n}x{k} {out_dtype}")
    a, w = operands(np.random.default_rng(m + n), m, n, k)
    close(nv.fp8_gemm(a, w, out_dtype), a, w)


@pytest.mark.parametrize("m", [2, 40, 300])
def test_products_of_any_codes(m):
    """Every code but NaN, evenly: products over the whole range of exponents, where the 8-bit instructions cut most."""
    say(f"fp8 gemm any codes {m}")
    rng = np.random.default_rng(m)

    def codes(rows, cols):
        c = rng.integers(0, 256, (rows, cols))
        return torch.from_numpy(np.where(c & 127 == 127, c ^ 1, c).astype(np.uint8)).to(DEV)
    a = nv.FP8Tensor(codes(m, 768), torch.rand(m, 6, device=DEV) + 0.1, m, 768, 1)
    w = nv.FP8Tensor(codes(300, 768), torch.rand(3, 6, device=DEV) + 0.1, 300, 768, 128)
    for out_dtype in (BF16, F32):
        close(nv.fp8_gemm(a, w, out_dtype), a, w)


@pytest.mark.parametrize("m", [1, 16, 50, 200, 600])
@pytest.mark.parametrize("n", [7, 256, 515])
def test_output_strides_and_neighbours(m, n):
    """Rows of the output at odd places, nothing written beside them."""
    say(f"fp8 gemm strides {m}x{n}")
    a, w = operands(np.random.default_rng(m + n), m, n, 272)
    ws = nv.fp8_gemm_workspace(m)
    for out_dtype in (BF16, F32):
        whole = nv.fp8_gemm(a, w, out_dtype)
        for lead, pad in ((0, 8), (1, 0), (3, 2)):
            buf = torch.full((m + 1, lead + n + pad), -7.0, dtype=out_dtype, device=DEV)
            nv.nvfp4_fp8_gemm(a, w, buf[:m, lead: lead + n], ws)
            assert torch.equal(buf[:m, lead: lead + n], whole)
            buf[:m, lead: lead + n] = -7
            assert bool((buf == -7).all())


@pytest.mark.parametrize("m", [3, 40, 300])
@pytest.mark.parametrize("out_dtype", [BF16, F32])
def test_nan_stays_in_its_row_or_column(m, out_dtype):
    say(f"fp8 gemm NaN {m} {out_dtype}")
    a, w = operands(np.random.default_rng(m), m, 300, 400)
    clean = nv.fp8_gemm(a, w, out_dtype)
    a.codes[1, 399] = 0x7F
    w.codes[299, 0] = 0xFF
    out = nv.fp8_gemm(a, w, out_dtype)
    assert bool(out[1].isnan().all()) and bool(out[:, 299].isnan().all())
    out[1], out[:, 299] = clean[1], clean[:, 299]
    assert torch.equal(out, clean)


@pytest.mark.parametrize("m", [1, 20, 100])
def test_bytes_behind_the_columns_do_not_matter(m):
    """cols ends inside a block of 128: NaN codes behind it, in both operands, are not read into the sums."""
    say(f"fp8 gemm padding {m}")
    a, w = operands(np.random.default_rng(m), m, 140, 336)
    want = nv.fp8_gemm(a, w)

    def padded(q):
        codes = torch.full((q.rows + 1, 400), 0x7F, dtype=torch.uint8, device=DEV)
        scales = torch.full((q.scales.shape[0] + 1, 9), float("nan"), device=DEV)
        codes[: q.rows, :336], scales[: q.scales.shape[0], :3] = q.codes[:, :336], q.scales
        return nv.FP8Tensor(codes[: q.rows], scales[: q.scales.shape[0]], q.rows, 336, q.block_rows)
    assert torch.equal(nv.fp8_gemm(padded(a), padded(w)), want)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("m,n,k", [(1, 512, 272), (4, 5120, 5120), (16, 130, 2064), (17, 300, 1024), (90, 640, 1040), (700, 1024, 512), (150, 1030, 4112), (180, 20000, 528), (1500, 5120, 272)])
def test_linear_is_quantize_and_product(m, n, k, dtype):
    say(f"fp8 linear {m}x{n}x{k} {dtype}")
    rng = np.random.default_rng(m + k)
    x, w = matrix(rng, m, k + 16, dtype)[:, 16:], nv.fp8_quantize(matrix(rng, n, k, F32), 128)
    ws = nv.fp8_linear_workspace(m, k)
    for out_dtype in (BF16, F32):
        ws.fill_(float("nan"))
        assert torch.equal(nv.fp8_linear(x, w, out_dtype, workspace=ws), nv.fp8_gemm(nv.fp8_quantize(x), w, out_dtype))


@pytest.mark.parametrize("m", [1, 12, 60, 400])
def test_linear_in_a_graph_and_on_a_stream(m):
    say(f"fp8 linear graph {m}")
    rng = np.random.default_rng(m)
    x, w = matrix(rng, m, 1040, BF16), nv.fp8_quantize(matrix(rng, 700, 1040, F32), 128)
    out, ws = torch.empty(m, 700, dtype=BF16, device=DEV), nv.fp8_linear_workspace(m, 1040)
    nv.fp8_linear(x, w, out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nv.fp8_linear(x, w, out=out, workspace=ws)
    for i in range(4):
        x.copy_(matrix(rng, m, 1040, BF16))
        want = nv.fp8_linear(x, w)  # eager, between the replays
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = torch.empty_like(out)
    nv.nvfp4_fp8_linear(x, w, got, ws, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    for _ in range(3):  # the same bits again
        assert torch.equal(nv.fp8_linear(x, w), want)


def test_no_rows():
    say("fp8 no rows")
    w = nv.fp8_quantize(torch.ones(130, 128, device=DEV), 128)
    assert nv.fp8_linear(torch.ones(0, 128, device=DEV), w).shape == (0, 130)
    assert nv.fp8_gemm(nv.empty_fp8(0, 128), w).shape == (0, 130)

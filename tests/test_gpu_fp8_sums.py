"""The sums of the 8-bit linear layers' products, exact by default and cut where
the caller allows it.

With A = sum |a w| over a row and column (K terms in blocks of 128), exact
products and float32 sums are within (K / 128 + 136) 2^-23 A, as for float32
outputs; a bf16 output adds half a step, 2^-8.  With cut sums the 7 smaller of 8
neighbouring products lose less than 2^-13 of the largest's power of two each:
less than 2^-10 A more.  On normally distributed data these losses are independent
and of either sign, a product's less than 2^-13 of a number near its own
root mean square, so that relative to the result their root mean square stays below 2^-13."""
import numpy as np
import pytest
import torch

import bit_linear_layer_amd as nv
from oracle import layer_oracle as L
from tests.gpu_util import DEV, say
from tests.test_gpu_fp8 import BF16, F32, host, matrix, operands
from tests.test_gpu_layer_far_rows import far

pytestmark = pytest.mark.gpu


def close(out, ref, size, k, cut=False):
    tol = (k / 128 + 136) * 2.0 ** -23 * size + (2.0 ** -10 * size if cut else 0.0)
    if out.dtype == BF16:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    err = np.abs(out.double().cpu().numpy() - ref)
    bad = np.argwhere(~(err <= tol + 2.0 ** -126))
    assert bad.size == 0, f"{len(bad)} of {err.size} outside, first {bad[:3].tolist()}: {[(err[i, j], tol[i, j]) for i, j in bad[:3]]}"


def against_oracle(out, a, w, cut=False):
    close(out, *L.fp8_gemm(*host(a), *host(w)), a.cols, cut)


def any_codes(rng, rows, cols):
    c = rng.integers(0, 256, (rows, cols))
    return np.where(c & 127 == 127, c ^ 1, c).astype(np.uint8)


@pytest.mark.parametrize("m,n", [(3, 700), (16, 4096), (30, 4096), (64, 2000), (128, 1111), (200, 1500), (450, 900), (600, 12900)])
@pytest.mark.parametrize("out_dtype", [BF16, F32])
def test_sums_that_cancel(m, n, out_dtype):
    """Every product once with either sign, in two blocks and in another order in the second: the result is 0."""
    say(f"fp8 cancelling sums {m}x{n} {out_dtype}")
    rng = np.random.default_rng(m)
    order = rng.permutation(128)
    a, w = any_codes(rng, m, 128), any_codes(rng, n, 128)
    a, w = np.concatenate([a, a[:, order]], 1), np.concatenate([w, w[:, order] ^ 0x80], 1)
    sa, sw = rng.uniform(0.1, 1, (m, 1)).astype(np.float32), rng.uniform(0.1, 1, (-(-n // 128), 1)).astype(np.float32)
    sa, sw = np.repeat(sa, 2, 1), np.repeat(sw, 2, 1)
    _, size = L.fp8_gemm(a, sa, w, sw)

    def on(*v):
        return [torch.from_numpy(np.ascontiguousarray(x)).to(DEV) for x in v]
    out = nv.fp8_gemm(nv.FP8Tensor(*on(a, sa), m, 256, 1), nv.FP8Tensor(*on(w, sw), n, 256, 128), out_dtype)
    close(out, np.zeros((m, n)), size, 256)
    if out_dtype is BF16:
        out = nv.fp8_gemm(nv.FP8Tensor(*on(a, sa), m, 256, 1), nv.FP8Tensor(*on(w, sw), n, 256, 128), cut_sums=True)
        close(out, np.zeros((m, n)), size, 256, cut=True)


@pytest.mark.parametrize("m,n,k,cut", [(2048, 5120, 5120, False), (2048, 5120, 5120, True), (200, 2048, 5120, False), (96, 1000, 2064, False)])
def test_root_mean_square_error(m, n, k, cut):
    """By rows and by columns: one product left out of 5120 would be an error of 1.4e-2."""
    say(f"fp8 rms {m}x{n}x{k} {cut}")
    g = torch.Generator(DEV).manual_seed(m + k)
    a = nv.fp8_quantize(torch.randn(m, k, device=DEV, generator=g))
    w = nv.fp8_quantize(torch.randn(n, k, device=DEV, generator=g) * 0.02, 128)
    out = nv.fp8_gemm(a, w, cut_sums=cut).double()
    va, vw = (torch.from_numpy(L.fp8_values(*host(q), q.block_rows)).to(DEV) for q in (a, w))
    ref = torch.mm(va, vw.t().contiguous())
    limit = 2.0 ** -8 + (2.0 ** -13 if cut else (k / 128 + 136) * 2.0 ** -23 * k ** 0.5)  # sum |a w| is below k^1/2 times the result's
    for dim in (0, 1):
        off = ((out - ref).square().mean(dim) / ref.square().mean(dim)).sqrt().max().item()
        assert off <= limit, (dim, off, limit)


CUT = [(130, 1, 16), (129, 70, 128), (225, 192, 400), (240, 256, 144), (257, 513, 384), (300, 300, 16), (511, 1280, 512), (1000, 40, 272),
       (1030, 1300, 1024), (700, 12900, 272), (448, 515, 912), (2048, 2560, 512), (3, 200, 400), (100, 300, 640), (500, 5120, 3600)]


@pytest.mark.parametrize("m,n,k", CUT)
def test_cut_sums(m, n, k):
    say(f"fp8 cut sums {m}x{n}x{k}")
    rng = np.random.default_rng(m + n)
    a, w = operands(rng, m, n, k)
    out = nv.fp8_gemm(a, w, cut_sums=True)
    against_oracle(out, a, w, cut=True)
    x = matrix(rng, m, k + 16, BF16)[:, 16:]
    ws = nv.fp8_linear_workspace(m, k).fill_(float("nan"))
    assert torch.equal(nv.fp8_linear(x, w, workspace=ws, cut_sums=True), nv.fp8_gemm(nv.fp8_quantize(x), w, cut_sums=True))
    buf = torch.full((m + 1, n + 5), -7.0, dtype=BF16, device=DEV)
    nv.nvfp4_fp8_gemm(a, w, buf[:m, 3: 3 + n], nv.fp8_gemm_workspace(m), cut_sums=True)
    assert torch.equal(buf[:m, 3: 3 + n], out)
    buf[:m, 3: 3 + n] = -7
    assert bool((buf == -7).all())


@pytest.mark.parametrize("cut", [False, True])
def test_nan_and_bytes_behind_the_columns_in_whole_tiles(cut):
    say(f"fp8 whole tiles NaN {cut}")
    a, w = operands(np.random.default_rng(1), 700, 12900, 336)
    clean = nv.fp8_gemm(a, w, cut_sums=cut)

    def padded(q):
        codes = torch.full((q.rows + 1, 400), 0x7F, dtype=torch.uint8, device=DEV)
        scales = torch.full((q.scales.shape[0] + 1, 9), float("nan"), device=DEV)
        codes[: q.rows, :336], scales[: q.scales.shape[0], :3] = q.codes[:, :336], q.scales
        return nv.FP8Tensor(codes[: q.rows], scales[: q.scales.shape[0]], q.rows, 336, q.block_rows)
    assert torch.equal(nv.fp8_gemm(padded(a), padded(w), cut_sums=cut), clean)
    a.codes[699, 335] = 0x7F
    w.codes[12899, 0] = 0xFF
    out = nv.fp8_gemm(a, w, cut_sums=cut)
    assert bool(out[699].isnan().all()) and bool(out[:, 12899].isnan().all())
    out[699], out[:, 12899] = clean[699], clean[:, 12899]
    assert torch.equal(out, clean)


@pytest.mark.parametrize("cut", [False, True])
def test_far_rows_in_whole_tiles(cut):
    say(f"fp8 whole tiles far rows {cut}")
    g = torch.Generator(DEV).manual_seed(3)
    a, w = nv.fp8_quantize(torch.randn(600, 272, device=DEV, generator=g)), nv.fp8_quantize(torch.randn(12900, 272, device=DEV, generator=g), 128)
    want = nv.fp8_gemm(a, w, cut_sums=cut)
    wide = [nv.FP8Tensor(far(q.codes, 2 ** 22 - 16), q.scales, q.rows, q.cols, q.block_rows) for q in (a, w)]
    out = far(torch.zeros_like(want), 2 ** 22)
    nv.nvfp4_fp8_gemm(*wide, out, nv.fp8_gemm_workspace(600), cut_sums=cut)
    assert torch.equal(out, want)


def test_cut_sums_in_a_graph():
    say("fp8 cut sums graph")
    rng = np.random.default_rng(5)
    x, w = matrix(rng, 600, 272, BF16), nv.fp8_quantize(matrix(rng, 12900, 272, F32), 128)
    out, ws = torch.empty(600, 12900, dtype=BF16, device=DEV), nv.fp8_linear_workspace(600, 272)
    for cut in (False, True):
        nv.fp8_linear(x, w, out=out, workspace=ws, cut_sums=cut)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            nv.fp8_linear(x, w, out=out, workspace=ws, cut_sums=cut)
        for i in range(3):
            x.copy_(matrix(rng, 600, 272, BF16))
            want = nv.fp8_linear(x, w, cut_sums=cut)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want), (cut, i)

"""Calls as long as prompts, where a thread or workgroup takes several pieces,
tokens or passes: the same bits as the same rows or channels in calls so small that
it takes one, which the other tests hold to the oracle."""
import numpy as np
import pytest
import torch

import bit_linear_layer_amd as nv
from oracle import layer_oracle as L
from tests.gpu_util import DEV, say, x_f32

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def normal(seed, *shape, dtype=F32):
    return torch.randn(*shape, device=DEV, generator=torch.Generator(DEV).manual_seed(seed)).to(dtype)


def loud(seed, rows, cols, dtype):
    """Rows of unequal size, some elements not finite, some rows zero."""
    x = normal(seed, rows, cols) * torch.exp(3 * normal(seed + 1, rows, 1))
    x[::97] = 0
    x[5::131, cols // 2] = float("nan")
    x[7::251, cols - 1] = float("-inf")
    return x.to(dtype)


# A call of 32768 pieces of 128 columns at most gives each group of 16 lanes one piece.
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", [(4100, 1040), (33000, 16), (40001, 128), (20000, 272), (3000, 17408), (16500, 17408)])
def test_quantizer_of_many_pieces(rows, cols, dtype):
    say(f"fp8 quantize long {rows}x{cols} {dtype}")
    wide = loud(rows, rows, cols + 16, dtype)
    x, pieces = wide[:, 16:], -(-cols // 128)
    assert rows * pieces > 32768
    codes = torch.full((rows, cols + 16), 0xAB, dtype=torch.uint8, device=DEV)
    scales = torch.full((rows, pieces + 1), -7.0, device=DEV)
    for flags in (nv.FP8_SCALE_F32, nv.FP8_SCALE_POW2):
        q = nv.FP8Tensor(codes, scales, rows, cols)
        nv.nvfp4_fp8_quantize(x, q, flags)
        step = max(1, 32768 // pieces)
        for r in range(0, rows, step):
            part = nv.fp8_quantize(x[r: r + step], 1, flags)
            assert torch.equal(codes[r: r + step, :cols], part.codes[:, :cols]), r
            assert torch.equal(scales[r: r + step, :pieces], part.scales), r
        assert bool((codes[:, cols:] == 0xAB).all()) and bool((scales[:, pieces:] == -7).all())
    if rows == 4100:
        want = L.fp8_quantize(x_f32(x), 1, True)
        assert np.array_equal(codes[:, :cols].cpu().numpy(), want[0])
        assert np.array_equal(scales[:, :pieces].cpu().numpy().view(np.uint32), want[1].view(np.uint32))


@pytest.mark.parametrize("rows,cols,outs", [(4100, 1040, 200), (9000, 640, 2000)])
def test_linear_of_many_pieces(rows, cols, outs):
    say(f"fp8 linear long {rows}x{outs}x{cols}")
    x, w = normal(1, rows, cols, dtype=BF16), nv.fp8_quantize(normal(2, outs, cols), 128)
    for cut in (False, True):
        assert torch.equal(nv.fp8_linear(x, w, cut_sums=cut), nv.fp8_gemm(nv.fp8_quantize(x), w, cut_sums=cut))


def lens_of(rng, total):
    """Sequences of all kinds, empty ones among them, that end at every place of a run of 32."""
    lens = []
    while sum(lens) < total:
        n = int(rng.choice([0, 1, 2, 3, 4, 5, 15, 16, 17, 31, 32, 33, 63, 65, int(rng.integers(6, 700))]))
        lens.append(min(n, total - sum(lens)))
    return lens


# Runs of 4 tokens up to 2^19 pieces of 8 channels, then of 8, from 2^21 of 16, from 2^25 of 32.
@pytest.mark.parametrize("dtype,width", [(BF16, 4), (BF16, 2), (F32, 3), (F32, 4)])
@pytest.mark.parametrize("tokens,channels,run", [(450, 10240, 8), (1701, 10240, 16), (26300, 10240, 32), (70000, 64, 8), (300001, 64, 16)])
def test_convolution_of_long_runs(tokens, channels, run, dtype, width):
    say(f"conv long {tokens}x{channels} {dtype} W={width}")
    places = tokens * channels // 8
    assert run == (32 if places >= 2 ** 25 else 16 if places >= 2 ** 21 else 8) and places >= 2 ** 19
    rng = np.random.default_rng(tokens + width)
    lead = 5
    lens = lens_of(rng, tokens - lead - 2)
    n = len(lens)
    starts = torch.from_numpy(np.concatenate([[0], np.cumsum(lens)]) + lead).int().to(DEV)
    x, w, b = normal(1, tokens, channels, dtype=dtype), normal(2, channels, width), normal(3, channels)
    state = normal(4, n + 2, width - 1, channels, dtype=dtype)
    slots = rng.permutation(n + 2)[:n]
    slots[rng.random(n) < 0.1] = -1
    slots, fresh = torch.from_numpy(slots).int().to(DEV), torch.from_numpy(rng.integers(0, 2, n)).to(torch.uint8).to(DEV)
    before, y = state.clone(), torch.full_like(x, -7)
    nv.nvfp4_causal_conv(x, w, y, n, starts, b, True, state, slots, fresh)
    some = 8 * (2 ** 19 // tokens // 2)  # channels of a call with runs of 4
    some = min(channels // 2, max(8, some - some % 8))
    assert tokens * some // 8 < 2 ** 19
    picks = [0, channels // 2 // 8 * 8, channels - some] if channels > 4 * some else range(0, channels, some)
    for c in picks:
        part = slice(c, min(c + some, channels))
        kept, out = before[:, :, part].contiguous(), torch.full_like(x[:, part], -7)
        nv.nvfp4_causal_conv(x[:, part], w[part].contiguous(), out, n, starts, b[part].contiguous(), True, kept, slots, fresh)
        assert torch.equal(y[:, part], out), c
        assert torch.equal(state[:, :, part], kept), c
    assert bool((y[:lead] == -7).all()) and bool((y[tokens - 2:] == -7).all())


def test_convolution_of_long_runs_against_the_oracle():
    say("conv long against the oracle")
    rng = np.random.default_rng(9)
    lens = lens_of(rng, 1700)
    starts = np.concatenate([[0], np.cumsum(lens)])
    x, w, b = normal(1, 1700, 10240), normal(2, 10240, 4), normal(3, 10240)
    state = normal(4, len(lens), 3, 10240)
    before, y = state.clone(), torch.empty_like(x)
    nv.nvfp4_causal_conv(x, w, y, len(lens), torch.from_numpy(starts).int().to(DEV), b, False, state)
    at = rng.choice(10240, 24, replace=False)
    mine = [v.double().cpu().numpy() for v in (x[:, at], w[at], b[at], before[..., at], y[:, at], state[..., at])]
    ref, size, new, written = L.causal_conv(mine[0], mine[1], starts, mine[2], False, mine[3])
    assert written.all() and np.array_equal(mine[5], new)
    assert np.all(np.abs(mine[4] - ref) <= 4 * 2.0 ** -24 * size)  # W fmas from the bias on


# A workgroup takes one pass over rows (tokens x heads) up to 1024 workgroups' worth, then 3 or 5, from 16384 on 8, and as many
# tokens as fill it.
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("t,hq,hk,d,r,axes,inter", [
    (1001, 32, 8, 128, 128, 3, False), (8195, 32, 8, 128, 128, 3, False), (8195, 32, 8, 128, 96, 1, True), (9001, 16, 4, 64, 64, 3, True),
    (33333, 16, 4, 64, 32, 1, False), (60001, 2, 1, 64, 16, 1, False), (3001, 6, 2, 256, 256, 2, False), (20003, 6, 1, 256, 64, 3, True),
    (1100, 64, 8, 256, 64, 1, False)])
def test_rotation_of_long_prompts(t, hq, hk, d, r, axes, inter, dtype):
    say(f"rope long {t} {hq}+{hk}x{d} rotary {r} axes {axes} {inter} {dtype}")
    slots = 256 // (d // 8)
    assert t * (hq + hk) // slots >= 1024
    x = normal(t, t, (hq + 2 * hk) * d, dtype=dtype)
    q, k = x[:, : hq * d], x[:, hq * d: (hq + hk) * d]
    rng = np.random.default_rng(t)
    rope = nv.Rope((1e4 ** (-torch.arange(r // 2, device=DEV) / (r // 2))).float(),
                   torch.from_numpy(rng.integers(0, axes, r // 2)).to(torch.uint8).to(DEV) if axes > 1 else None, inter)
    pos = torch.from_numpy(rng.integers(0, 1 << 20, (axes, t))).to(DEV)
    qw, kw = normal(1, d), normal(2, d)
    outs = [torch.full((t + 1, h * d), -7.0, dtype=dtype, device=DEV) for h in (hq, hk)]
    nv.nvfp4_qk_norm_rope(q, k, outs[0][:t], outs[1][:t], d, pos if axes > 1 else pos[0], rope, qw, kw, weight_offset=1.0)
    step = 1023 * slots // (hq + hk)
    for a in range(0, t, step):
        p = pos[:, a: a + step].contiguous()
        want = nv.qk_norm_rope(q[a: a + step], k[a: a + step], d, p if axes > 1 else p[0], rope, qw, kw, weight_offset=1.0)
        for out, part in zip(outs, want):
            assert torch.equal(out[a: min(a + step, t)], part), a
    assert all(bool((out[t] == -7).all()) for out in outs)


@pytest.mark.parametrize("in_place", [False, True])
def test_one_of_both_in_a_long_prompt(in_place):
    """Queries alone, without a norm, or keys in place."""
    say(f"rope long, one of both {in_place}")
    t, h, d = 5001, 8, 128
    x, pos = normal(3, t, h * d, dtype=BF16), torch.arange(t, device=DEV) * 3
    rope = nv.Rope((1e4 ** (-torch.arange(32, device=DEV) / 32)).float())
    want = torch.cat([nv.qk_norm_rope(x[a: a + 500], x[a: a + 500], d, pos[a: a + 500], rope)[0] for a in range(0, t, 500)])
    out = x.clone() if in_place else torch.empty_like(x)
    src = out if in_place else x
    if in_place:
        nv.nvfp4_qk_norm_rope(None, src, None, out, d, pos, rope)
    else:
        nv.nvfp4_qk_norm_rope(src, None, out, None, d, pos, rope)
    assert torch.equal(out, want)

"""GPU parity of the query/key norm with rotation.

Tolerance, u = 2^-24: the sum of squares rounds at most 8 + 5 times and the
norm's factor (halved by the root) a few times more, a sine or cosine is off by
at most 4 u absolutely (the angle's fraction rounds to 2^-25 of half a turn; two
ulps of the function), and the rotation rounds twice: together at most 32 u
(|z_i| + |z_j|) over the pair; bf16 adds half a step, 2^-8 of the result."""
import numpy as np
import pytest
import torch

import bit_linear_layer_amd as nv
from oracle import layer_oracle as L
from tests.gpu_util import DEV, say

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def close(out, x, head_dim, **kw):
    ref, size = L.qk_norm_rope(x.double().cpu().numpy().reshape(len(x), -1, head_dim), head_dim, **kw)
    got = out.double().cpu().numpy().reshape(ref.shape)
    tol = 32 * 2.0 ** -24 * size
    if out.dtype == BF16:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    bad = np.argwhere(~(np.abs(got - ref) <= tol + 2.0 ** -126))
    assert bad.size == 0, f"{len(bad)} outside, first {bad[:3].tolist()}"


def rope_of(dim, axes, interleaved, rng, theta=1e4):
    half = dim // 2
    freq = (theta ** (-np.arange(half) / half)).astype(np.float32)
    axis = rng.integers(0, axes, half).astype(np.uint8) if axes > 1 else None
    return nv.Rope(torch.from_numpy(freq).to(DEV), None if axis is None else torch.from_numpy(axis).to(DEV), interleaved), freq, axis


CASES = [  # tokens, q heads, k heads, head_dim, rotary_dim, axes, interleaved, norm, offset
    (1, 1, 1, 64, 64, 1, False, True, 0.0), (1, 24, 4, 256, 64, 3, False, True, 1.0), (5, 3, 1, 64, 16, 1, True, True, 0.0),
    (7, 8, 8, 128, 128, 3, True, False, 0.0), (64, 32, 8, 128, 128, 1, False, True, 0.0), (33, 40, 5, 128, 96, 2, False, True, 1.0),
    (19, 2, 2, 256, 256, 4, True, True, 0.0), (130, 12, 4, 64, 48, 3, False, False, 0.0), (300, 64, 8, 256, 32, 1, True, True, 1.0),
    (3, 300, 7, 64, 32, 1, False, True, 0.0),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("t,hq,hk,d,r,axes,inter,norm,offset", CASES)
def test_norm_and_rotation(t, hq, hk, d, r, axes, inter, norm, offset, dtype):
    say(f"rope {t} {hq}+{hk}x{d} rotary {r} axes {axes} {inter} {norm} {dtype}")
    rng = np.random.default_rng(t + d)
    x = torch.from_numpy(rng.standard_normal((t, (hq + 2 * hk) * d)) * 10.0 ** rng.uniform(-4, 4, (t, 1))).to(dtype).to(DEV)
    q, k = x[:, : hq * d], x[:, hq * d: (hq + hk) * d]  # columns of one projection
    pos = rng.integers(0, 1 << 20, (axes, t))
    pos[:, 0] = [0, (1 << 24) - 1, 123456789, 5][:axes]
    rope, freq, axis = rope_of(r, axes, inter, rng)
    w = [torch.from_numpy(rng.standard_normal(d)).float().to(DEV) if norm else None for _ in range(2)]
    p = torch.from_numpy(pos).to(DEV)
    got = nv.qk_norm_rope(q, k, d, p if axes > 1 else p[0], rope, *w, weight_offset=offset, eps=1e-5)
    for out, inp, weight in zip(got, (q, k), w):
        close(out, inp, d, weight=None if weight is None else weight.cpu().numpy(), weight_offset=offset, eps=1e-5, positions=pos,
              inv_freq=freq, axis=axis, interleaved=inter)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_far_and_negative_positions(dtype):
    """Up to 2^31 a turn's fraction is formed from 64 bits: off by at most 2^31 2^-52 of a turn, below 2^-24 of half a turn."""
    say(f"rope far {dtype}")
    rng = np.random.default_rng(1)
    pos = np.array([0, 1, -1, 1 << 20, (1 << 24) + 1, -(1 << 26) - 3, (1 << 31) - 1, -(1 << 31)])
    x = torch.from_numpy(rng.standard_normal((8, 2 * 128))).to(dtype).to(DEV)
    rope, freq, _ = rope_of(128, 1, False, rng, 1e7)
    q, k = nv.qk_norm_rope(x, x[:, :128], 128, torch.from_numpy(pos).to(DEV), rope)
    close(q, x, 128, positions=pos, inv_freq=freq)
    assert torch.equal(k, q[:, :128])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strided_heads_in_place_and_one_of_both(dtype):
    """Queries with a gate beside each head, as three-dimensional views; written in place; keys alone; no rotation; no norm."""
    say(f"rope views {dtype}")
    rng = np.random.default_rng(2)
    t, h, d = 11, 5, 128
    both = torch.from_numpy(rng.standard_normal((t, h, 2 * d))).to(dtype).to(DEV)
    before = both.clone()
    pos = torch.arange(t, device=DEV) * 37
    rope, freq, _ = rope_of(64, 1, False, rng)
    w = torch.from_numpy(rng.standard_normal(d)).float().to(DEV)
    q = both[..., :d]
    nv.nvfp4_qk_norm_rope(q, None, q, None, d, pos, rope, q_weight=w)
    kw = dict(weight=w.cpu().numpy(), positions=pos.cpu().numpy(), inv_freq=freq)
    close(q.reshape(t, -1), before[..., :d].reshape(t, -1), d, **kw)
    assert torch.equal(both[..., d:], before[..., d:])
    # keys alone, all tokens of a head together in memory, and as usual
    k = before[..., :d].transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.empty_like(k)
    assert out.stride() == k.stride() == (d, t * d, 1)
    nv.nvfp4_qk_norm_rope(None, k, None, out, d, pos, rope, k_weight=w)
    assert torch.equal(out, q)
    with pytest.raises(nv.NVFP4Error):  # heads that overlap
        nv.nvfp4_qk_norm_rope(None, k.as_strided(k.shape, (d, (t - 1) * d, 1)), None, out, d, pos, rope)
    k = before[..., :d].contiguous()
    out = torch.empty_like(k)
    nv.nvfp4_qk_norm_rope(None, k, None, out, d, pos, rope, k_weight=w)
    assert torch.equal(out, q)
    nv.nvfp4_qk_norm_rope(None, k, None, out, d, k_weight=w)
    close(out.view(t, -1), k.view(t, -1), d, weight=kw["weight"])
    nv.nvfp4_qk_norm_rope(k, None, out, None, d)
    assert torch.equal(out, k)
    one = torch.empty_like(k[:1])
    nv.nvfp4_qk_norm_rope(k[:1].expand(1, h, d), None, one, None, d, pos[:1], rope)
    close(one.view(1, -1), k[:1].reshape(1, -1), d, positions=pos[:1].cpu().numpy(), inv_freq=freq)
    empty = nv.qk_norm_rope(k.view(t, -1)[:0], k.view(t, -1)[:0], d, pos[:0], rope)
    assert empty[0].shape == (0, h * d)


def test_infinite_and_nan_rows_stay_alone():
    say("rope non-finite")
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.standard_normal((6, 4 * 64))).float().to(DEV)
    rope, freq, _ = rope_of(64, 1, False, rng)
    pos, w = torch.arange(6, device=DEV), torch.ones(64, device=DEV)
    want, _ = nv.qk_norm_rope(x, x, 64, pos, rope, w, w)
    y = x.clone()
    y[2, 70], y[4, 3] = float("nan"), float("inf")
    got, _ = nv.qk_norm_rope(y, y, 64, pos, rope, w, w)
    bad = torch.zeros(6, 4, dtype=torch.bool, device=DEV)
    bad[2, 1] = bad[4, 0] = True
    assert bool(got.view(6, 4, 64)[bad].isnan().any(-1).all())
    assert torch.equal(got.view(6, 4, 64)[~bad], want.view(6, 4, 64)[~bad])
    zero = torch.zeros_like(x)
    assert bool((nv.qk_norm_rope(zero, zero, 64, pos, rope, w, w)[0] == 0).all())


def test_axis_values_beyond_the_axes_and_bad_plans():
    say("rope axes")
    rng = np.random.default_rng(4)
    x = torch.from_numpy(rng.standard_normal((9, 2 * 64))).float().to(DEV)
    rope, freq, _ = rope_of(64, 1, False, rng)
    rope = nv.Rope(rope.inv_freq, torch.arange(32, device=DEV).to(torch.uint8) * 8)
    pos = torch.from_numpy(rng.integers(0, 5000, (2, 9))).to(DEV)
    got, _ = nv.qk_norm_rope(x, x, 64, pos, rope)
    close(got, x, 64, positions=pos.cpu().numpy(), inv_freq=freq, axis=rope.axis.cpu().numpy())

    shared = pos[:1].expand(2, 9)  # one row for all axes
    assert torch.equal(nv.qk_norm_rope(x, x, 64, shared, rope)[0], nv.qk_norm_rope(x, x, 64, shared.contiguous(), rope)[0])

    def refused(**kw):
        a = dict(positions=pos, rope=rope)
        a.update(kw)
        with pytest.raises(nv.NVFP4Error):
            nv.qk_norm_rope(x, x, 64, **a)
    refused(positions=pos.int())
    refused(positions=pos[:, :8])
    refused(positions=pos.cpu())
    refused(positions=None)
    refused(rope=nv.Rope(rope.inv_freq))
    for args in ((rope.inv_freq.double(), rope.axis), (rope.inv_freq, rope.axis[:31]), (rope.inv_freq, rope.axis.int()),
                 (rope.inv_freq, rope.axis.cpu()), (rope.inv_freq[::2], None), (rope.inv_freq.view(2, 16), None)):
        with pytest.raises(nv.NVFP4Error):
            nv.Rope(*args)
    refused(rope=nv.Rope(rope.inv_freq.cpu(), rope.axis.cpu()))
    refused(rope=nv.Rope(rope.inv_freq[:31], rope.axis[:31]))
    refused(q_weight=torch.ones(63, device=DEV))
    refused(q_weight=torch.ones(64, device=DEV).double())
    refused(q_weight=torch.ones(64, device=DEV), eps=0.0)
    with pytest.raises(nv.NVFP4Error):
        nv.qk_norm_rope(x, x.to(BF16), 64, pos, rope)


def test_in_a_graph():
    say("rope graph")
    rng = np.random.default_rng(5)
    x = torch.from_numpy(rng.standard_normal((40, 6 * 128))).to(BF16).to(DEV)
    pos = torch.zeros(3, 40, dtype=torch.int64, device=DEV)
    rope, _, _ = rope_of(128, 3, False, rng)
    w, out = torch.ones(128, device=DEV), torch.empty_like(x)
    nv.nvfp4_qk_norm_rope(x, None, out, None, 128, pos, rope, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nv.nvfp4_qk_norm_rope(x, None, out, None, 128, pos, rope, w)
    for i in range(4):
        x.copy_(torch.from_numpy(rng.standard_normal(x.shape)))
        pos.copy_(torch.from_numpy(rng.integers(0, 9999, pos.shape)))
        want, _ = nv.qk_norm_rope(x, x, 128, pos, rope, w, w)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i

"""GPU parity of the short causal convolution and its states.

Tolerance, u = 2^-24, S = sum |w in| + |bias|: W fmas from the bias on, 4 u S at
most; SiLU's slope is at most 1.1 and its own evaluation is off by at most
(|u| + 16) 2^-23 of its value (the exponent's product rounds to 2^-24 |u|); bf16
adds half a step, 2^-8 of the result.  The states are copies: equal bit for bit."""
import numpy as np
import pytest
import torch

import bit_linear_layer_amd as nv
from oracle import layer_oracle as L
from tests.gpu_util import DEV, say

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def bound(ref, size, silu, dtype):
    tol = 1.1 * 4 * 2.0 ** -24 * size + ((size + 16) * 2.0 ** -23 * np.abs(ref) if silu else 0.0)
    return tol + (2.0 ** -8 * (np.abs(ref) + tol) if dtype == BF16 else 0.0) + 2.0 ** -126


def inputs(rng, rows, channels, width, dtype, n_states=9, bias=True):
    x = torch.from_numpy(rng.standard_normal((rows, channels)) * 10.0 ** rng.uniform(-2, 1, (1, channels))).to(dtype).to(DEV)
    w = torch.from_numpy(rng.standard_normal((channels, width))).float().to(DEV)
    b = torch.from_numpy(rng.standard_normal(channels)).float().to(DEV) if bias else None
    state = torch.from_numpy(rng.standard_normal((n_states, width - 1, channels))).to(dtype).to(DEV)
    return x, w, b, state


def check(x, w, y, starts, b=None, silu=True, before=None, after=None, slots=None, fresh=None):
    n = [None if t is None else t.double().cpu().numpy() for t in (x, w, b, before)]
    ref, size, new, written = L.causal_conv(n[0], n[1], starts, n[2], silu, n[3], slots, fresh)
    got = y.double().cpu().numpy()
    bad = np.argwhere(~(np.abs(got - ref) <= bound(ref, size, silu, y.dtype)) & written[:, None])
    assert bad.size == 0, f"{len(bad)} outside, first {bad[:4].tolist()}"
    assert np.all(got[~written] == -7)
    if after is not None:
        assert np.array_equal(after.double().cpu().numpy(), new)


def lens_cases(rng):
    return {
        "one token": [1], "two": [2], "three": [3], "a run and a bit": [17], "prompt": [700],
        "mixed": [1, 0, 5, 2, 0, 0, 40, 3, 1, 16, 15, 33],
        "all empty but one": [0, 0, 4, 0],
        "short ones": list(rng.integers(0, 4, 50)),
        "ones": [1] * 37,
        "long and short": [129, 1, 2, 300, 0, 1],
    }


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("width", [2, 3, 4])
@pytest.mark.parametrize("channels", [8, 104, 640])
def test_batches(channels, width, dtype):
    rng = np.random.default_rng(channels + width)
    for i, (name, lens) in enumerate(lens_cases(rng).items()):
        say(f"conv {name} C={channels} W={width} {dtype}")
        n, total, silu, lead = len(lens), sum(lens), i % 2 == 0, i % 3
        x, w, b, state = inputs(rng, lead + total + 2, channels, width, dtype, n + 3, bias=i % 4 != 1)
        starts = np.concatenate([[0], np.cumsum(lens)]) + lead
        slots = rng.permutation(n + 3)[:n]
        if n > 2:
            slots[1], slots[2] = -1, n + 3  # no state
        fresh = rng.integers(0, 2, n) if i % 2 else None
        before = state.clone()
        y = torch.full_like(x, -7)
        nv.nvfp4_causal_conv(x, w, y, n, torch.from_numpy(starts).int().to(DEV), b, silu, state, torch.from_numpy(slots).int().to(DEV),
                             None if fresh is None else torch.from_numpy(fresh).to(torch.uint8).to(DEV))
        check(x, w, y, starts, b, silu, before, state, slots, fresh)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_uniform_batches_without_starts_slots_or_states(dtype):
    rng = np.random.default_rng(1)
    for batch, each in ((1, 1), (5, 1), (64, 1), (3, 2), (4, 33), (1, 515)):
        say(f"conv uniform {batch}x{each} {dtype}")
        x, w, b, state = inputs(rng, batch * each, 64, 4, dtype, batch)
        starts = np.arange(batch + 1) * each
        y = torch.full_like(x, -7)
        nv.nvfp4_causal_conv(x, w, y, batch)
        check(x, w, y, starts)
        before = state.clone()
        y = torch.full_like(x, -7)
        nv.nvfp4_causal_conv(x, w, y, batch, state=state, bias=b)  # sequence b has state b
        check(x, w, y, starts, b, True, before, state)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("width", [2, 3, 4])
def test_next_tokens_of_a_padded_batch(width, dtype):
    """One row a sequence without starts: places without a state, fresh ones, strides, a pool with more states than places."""
    say(f"conv next tokens W={width} {dtype}")
    rng = np.random.default_rng(20 + width)
    for n, silu in ((1, True), (7, False), (33, True)):
        wide, w, b, pool = inputs(rng, n, 72, width, dtype, n + 4)
        w, b = w[:40].contiguous(), b[:40].contiguous()
        x, state = wide[:, 16:56], pool[:, :, :40].contiguous()
        slots, fresh = rng.permutation(n + 4)[:n], rng.integers(0, 2, n)
        if n > 4:
            slots[[0, 2, 4]] = -1, n + 4, -2 ** 31
            fresh[0], fresh[2] = 0, 1
        before, out = state.clone(), torch.full((n, 64), -7.0, dtype=dtype, device=DEV)
        nv.nvfp4_causal_conv(x, w, out[:, 8:48], n, None, b, silu, state, torch.from_numpy(slots).int().to(DEV),
                             torch.from_numpy(fresh).to(torch.uint8).to(DEV))
        check(x, w, out[:, 8:48], np.arange(n + 1), b, silu, before, state, slots, fresh)
        assert bool((out[:, :8] == -7).all()) and bool((out[:, 48:] == -7).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_prompt_in_chunks_and_single_tokens(dtype):
    """The same rows as one call, as chunks and token by token: the same bits, and the same state at the end."""
    say(f"conv chunks {dtype}")
    rng = np.random.default_rng(2)
    x, w, b, state = inputs(rng, 150, 256, 4, dtype, 4)
    whole = nv.causal_conv(x, w, 1, bias=b)
    at, parts, slot = 0, [], torch.tensor([2], dtype=torch.int32, device=DEV)
    other = state[[0, 1, 3]].clone()
    for i, n in enumerate([1, 1, 64, 2, 1, 50, 31]):
        fresh = torch.tensor([i == 0], dtype=torch.uint8, device=DEV)
        parts.append(nv.causal_conv(x[at: at + n], w, 1, None, b, True, state, slot, fresh))
        at += n
    assert at == 150 and torch.equal(torch.cat(parts), whole)
    assert torch.equal(state[2], x[-3:]) and torch.equal(state[[0, 1, 3]], other)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strides(dtype):
    """x and y as columns of wider tensors, states of a pool with room between them."""
    say(f"conv strides {dtype}")
    rng = np.random.default_rng(3)
    wide, w, b, _ = inputs(rng, 90, 80, 4, dtype)
    w, b = w[:56].contiguous(), b[:56].contiguous()
    x = wide[:, 8:64]
    pool = torch.from_numpy(rng.standard_normal((6, 5, 56))).to(dtype).to(DEV)
    before, state = pool.clone(), pool[:, 1:4]
    out = torch.full((90, 72), -7.0, dtype=dtype, device=DEV)
    starts = np.array([0, 30, 31, 88])
    slots = [5, 0, 3]
    nv.nvfp4_causal_conv(x, w, out[:, 8:64], 3, torch.from_numpy(starts).int().to(DEV), b, True, state,
                         torch.tensor(slots, dtype=torch.int32, device=DEV))
    check(x, w, out[:, 8:64], starts, b, True, before[:, 1:4], state, slots)
    assert bool((out[:, :8] == -7).all()) and bool((out[:, 64:] == -7).all())
    assert torch.equal(pool[:, [0, 4]], before[:, [0, 4]])


def test_starts_beyond_the_rows():
    """Starts above the number of rows, or below zero, count as these: nothing outside is read or written."""
    say("conv clamped starts")
    rng = np.random.default_rng(4)
    x, w, b, state = inputs(rng, 20, 32, 4, F32, 4)
    starts = np.array([-5, 3, 9, 50, 60])
    before, y = state.clone(), torch.full_like(x, -7)
    nv.nvfp4_causal_conv(x, w, y, 4, torch.from_numpy(starts).int().to(DEV), b, True, state)
    check(x, w, y, starts, b, True, before, state)


def test_nan_stays_in_its_channel_and_reach():
    say("conv NaN")
    rng = np.random.default_rng(5)
    x, w, b, state = inputs(rng, 40, 32, 4, F32, 3)
    starts = torch.tensor([0, 25, 40], dtype=torch.int32, device=DEV)
    clean = nv.causal_conv(x, w, 2, starts, b)
    x[23, 7] = float("nan")
    y = nv.causal_conv(x, w, 2, starts, b)
    assert bool(y[23:25, 7].isnan().all())  # not into the next sequence
    y[23:25, 7] = clean[23:25, 7]
    assert torch.equal(y, clean)
    state.fill_(float("nan"))  # a state that is not looked at
    y = nv.causal_conv(x[:20], w, 1, None, b, True, state, torch.tensor([1], dtype=torch.int32, device=DEV),
                       torch.ones(1, dtype=torch.uint8, device=DEV))
    assert torch.equal(y, clean[:20]) and torch.equal(state[1], x[17:20])


@pytest.mark.parametrize("u", [-120.0, -90.0, -30.0, -1e-30, 0.0, 30.0, 120.0])
def test_silu_over_its_range(u):
    say(f"conv silu {u}")
    x = torch.full((3, 8), u, device=DEV)
    w = torch.tensor([[0.0, 0.0, 0.0, 1.0]], device=DEV).repeat(8, 1)
    y = nv.causal_conv(x, w).double().cpu().numpy()
    ref = u / (1 + np.exp(-np.float64(np.float32(u))))
    assert np.all(np.abs(y - ref) <= bound(np.array(ref), np.array(abs(u)), True, F32))


def test_in_a_graph():
    say("conv graph")
    rng = np.random.default_rng(6)
    x, w, b, state = inputs(rng, 33, 512, 4, BF16, 40)
    slots = torch.randperm(40, device=DEV)[:33].int()
    y, mine = torch.empty_like(x), state.clone()
    nv.nvfp4_causal_conv(x, w, y, 33, None, b, True, mine.clone(), slots)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nv.nvfp4_causal_conv(x, w, y, 33, None, b, True, mine, slots)
    for i in range(4):
        x.copy_(torch.from_numpy(rng.standard_normal(x.shape)))
        want = nv.causal_conv(x, w, 33, None, b, True, state, slots)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(mine, state), i


def test_refusals_of_the_binding():
    say("conv refusals")
    x, w, b, state = inputs(np.random.default_rng(7), 12, 64, 4, F32, 5)
    i32 = torch.arange(5, dtype=torch.int32, device=DEV)

    def refused(**kw):
        a = dict(x=x, weight=w, batch=3, state=state)
        a.update(kw)
        with pytest.raises(nv.NVFP4Error):
            nv.causal_conv(**a)
    refused(x=x[:, :60])
    refused(x=x.half())
    refused(weight=w.double())
    refused(weight=w[:60])
    refused(weight=torch.zeros(64, 5, device=DEV), state=None)
    refused(bias=b[:63])
    refused(state=state.to(BF16))
    refused(state=state[:, :2])
    refused(state=state[:0])
    refused(state=state[:2])  # three sequences, two states, no slots
    refused(state=None, slots=i32[:3])
    refused(slots=i32[:2])
    refused(slots=i32[:3].long())
    refused(starts=i32[:3])
    refused(fresh=i32[:3])
    refused(batch=5)  # 12 rows
    refused(slots=i32[:3].cpu())
    with pytest.raises(nv.NVFP4Error):
        nv.nvfp4_causal_conv(x, w, x, 3)
    nothing = nv.causal_conv(x[:0], w, 0)
    assert nothing.shape == (0, 64)

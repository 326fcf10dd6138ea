"""GPU parity of the gated delta rule's next tokens against the oracle's
sequential float64 definition.

Tolerance, u = 2^-24, per row i of a state (value dimension i) and token: keys
and queries (normalized or unit) are off by at most 16 u relative (a sum of 128
squares over 8 lanes: 16 + 3 roundings, halved by the root; root, quotient,
product), a product with a row by 19 u more, the decay by 2 u, the update by
a few: with B = |S_i| + |v_i| at its largest over the tokens, each token adds at
most 64 u B to the row and the output is off by at most 64 u (tokens + 1) B |q|,
|q| = 128^-1/2 or its norm; the output's rounding in bf16 adds 2^-8 of it."""
import numpy as np
import pytest
import torch

import bit_linear_layer_amd as nv
from oracle import nvfp4_oracle as O
from tests.gpu_util import DEV, say

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def inputs(rng, rows, hk, hv, dtype, decay=1.0):
    q, k, v = (rng.standard_normal((rows, h * 128)) for h in (hk, hk, hv))
    beta = 1 / (1 + np.exp(-2 * rng.standard_normal((rows, hv))))
    g = -rng.uniform(1, 16, hv) * np.log1p(np.exp(rng.standard_normal((rows, hv)) - 4)) * decay
    return [torch.from_numpy(x).to(dtype).to(DEV) for x in (q, k, v, beta, g)]


def check(ins, o, before, after, hk, hv, slots, q_len, fresh=None, normalize=True):
    n = [t.double().cpu().numpy() for t in ins]
    got, o_rows = after.double().cpu().numpy(), o.double().cpu().numpy()
    start = before.double().cpu().numpy()
    left = np.ones(len(start), bool)
    for b, slot in enumerate(slots):
        at = slice(b * q_len, (b + 1) * q_len)
        if not 0 <= slot < len(start):
            assert np.all(o_rows[at] == -7)
            continue
        left[slot] = False
        s0 = np.zeros_like(start[slot]) if fresh is not None and fresh[b] else start[slot]
        q, k, v = (x[at].reshape(q_len, -1, 128) for x in n[:3])
        size, s = np.linalg.norm(s0, axis=-1), s0
        top = size.copy()
        for t in range(q_len):
            one, s = O.gdn_recurrence(q[t: t + 1], k[t: t + 1], v[t: t + 1], n[3][at][t: t + 1], n[4][at][t: t + 1], s0=s, normalize=normalize)
            top = np.maximum(top, np.linalg.norm(s, axis=-1)) + np.abs(v[t])
            qn = 128 ** -0.5 if normalize else np.repeat(np.linalg.norm(q[t], axis=-1), hv // hk)[:, None]
            tol = 64 * 2.0 ** -24 * (t + 2) * top * qn
            if o.dtype == BF16:
                tol = tol + 2.0 ** -8 * (np.abs(one[0]) + tol)
            err = np.abs(o_rows[at][t].reshape(hv, 128) - one[0])
            assert np.all(err <= tol), (b, t, (err / tol).max())
        err = np.linalg.norm(got[slot] - s, axis=-1)
        assert np.all(err <= 64 * 2.0 ** -24 * (q_len + 1) * top), (b, (err / top).max())
    assert np.array_equal(got[left], start[left])


@pytest.mark.parametrize("dtype,o_dtype", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("batch,q_len,hk,hv", [(1, 1, 1, 1), (1, 1, 16, 48), (3, 1, 2, 6), (5, 4, 1, 3), (2, 9, 2, 2), (40, 1, 1, 4), (1, 70, 1, 2)])
def test_next_tokens(batch, q_len, hk, hv, dtype, o_dtype):
    say(f"gdn step {batch}x{q_len} {hk}/{hv} {dtype} {o_dtype}")
    rng = np.random.default_rng(batch + q_len + hv)
    ins = inputs(rng, batch * q_len, hk, hv, dtype)
    states = torch.from_numpy(rng.standard_normal((batch + 2, hv, 128, 128))).float().to(DEV)
    slots = rng.permutation(batch + 2)[:batch]
    if batch > 2:
        slots[1], slots[2] = -1, batch + 2
    fresh = rng.integers(0, 2, batch) if batch > 1 else None
    before = states.clone()
    o = torch.full((batch * q_len, hv * 128), -7.0, dtype=o_dtype, device=DEV)
    nv.nvfp4_gdn_step(*ins, o, hk, hv, states, torch.from_numpy(slots).int().to(DEV), q_len,
                      fresh=None if fresh is None else torch.from_numpy(fresh).to(torch.uint8).to(DEV))
    check(ins, o, before, states, hk, hv, slots, q_len, fresh)


def test_without_normalization_and_slots():
    say("gdn step raw")
    rng = np.random.default_rng(1)
    ins = inputs(rng, 12, 2, 4, F32)
    ins[1] = torch.nn.functional.normalize(ins[1].view(12, 2, 128), dim=-1).reshape(12, 256)
    states = torch.from_numpy(rng.standard_normal((7, 4, 128, 128))).float().to(DEV)
    before = states.clone()
    o = torch.full((12, 512), -7.0, device=DEV)
    nv.nvfp4_gdn_step(*ins, o, 2, 4, states, None, 2, normalize_qk=False)
    check(ins, o, before, states, 2, 4, range(6), 2, normalize=False)


def test_a_zero_key_and_full_decay():
    say("gdn step corners")
    rng = np.random.default_rng(2)
    ins = inputs(rng, 3, 1, 2, F32)
    ins[1][0] = 0
    ins[0][1] = 0
    ins[4][2] = -200.0  # exp(g) = 0: the state starts anew
    states = torch.from_numpy(rng.standard_normal((3, 2, 128, 128))).float().to(DEV)
    before = states.clone()
    o = torch.full((3, 256), -7.0, device=DEV)
    nv.nvfp4_gdn_step(*ins, o, 1, 2, states)
    check(ins, o, before, states, 1, 2, range(3), 1)
    assert bool((o[1] == 0).all())


def test_strides_and_what_is_left_alone():
    """Inputs as columns of one tensor, a pool with room between the states, o inside a wider one; a fresh state's NaN is not read."""
    say("gdn step strides")
    rng = np.random.default_rng(3)
    hk, hv, rows = 2, 4, 6
    wide = torch.from_numpy(rng.standard_normal((rows, 8 + 2 * 256 + 512 + 8))).to(BF16).to(DEV)
    q, k, v = wide[:, 8:264], wide[:, 264:520], wide[:, 520:1032]
    gates = torch.from_numpy(rng.uniform(0, 1, (rows, 10))).to(BF16).to(DEV)
    ins = [q, k, v, gates[:, 1:5], -gates[:, 5:9]]
    pool = torch.from_numpy(rng.standard_normal((8, hv + 1, 128, 128))).float().to(DEV)
    pool[3, :hv] = float("nan")
    before = pool.clone()
    out = torch.full((rows, 8 + 512 + 3), -7.0, dtype=BF16, device=DEV)
    slots, fresh = [7, 3, 0], [0, 1, 0]
    nv.nvfp4_gdn_step(*ins, out[:, 8:520], hk, hv, pool[:, :hv], torch.tensor(slots, dtype=torch.int32, device=DEV), 2,
                      fresh=torch.tensor(fresh, dtype=torch.uint8, device=DEV))
    check(ins, out[:, 8:520], before[:, :hv].nan_to_num(), pool[:, :hv], hk, hv, slots, 2, fresh)
    assert bool((out[:, :8] == -7).all()) and bool((out[:, 520:] == -7).all()) and torch.equal(pool[:, hv:], before[:, hv:])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_continues_the_recurrence(dtype):
    """A prompt by the recurrence, then its next tokens here, is the whole by the recurrence (both within float32 of it)."""
    say(f"gdn step after recurrence {dtype}")
    rng = np.random.default_rng(4)
    hk, hv, n, more = 2, 4, 130, 7
    ins = inputs(rng, n + more, hk, hv, dtype)
    whole, last = nv.gdn_recurrence(*ins, hk, hv, return_state=True)
    _, state = nv.gdn_recurrence(*[x[:n] for x in ins], hk, hv, return_state=True)
    pool = state[None].clone()
    parts = [nv.gdn_step(*[x[i: i + 1].contiguous() for x in ins], hk, hv, pool) for i in range(n, n + more)]
    # the recurrence is held to 2e-4 of |S| |q| a token; both sides are
    size = float(last.norm(dim=(1, 2)).max() + 12 * more)
    assert float((torch.cat(parts) - whole[n:]).abs().max()) <= 4e-4 * size * 128 ** -0.5
    assert float((pool[0] - last).norm(dim=(1, 2)).max()) <= 4e-4 * size


def test_in_a_graph():
    say("gdn step graph")
    rng = np.random.default_rng(5)
    ins = inputs(rng, 9, 2, 6, BF16)
    states = torch.from_numpy(rng.standard_normal((12, 6, 128, 128))).float().to(DEV)
    slots = torch.randperm(12, device=DEV)[:9].int()
    mine, o = states.clone(), torch.empty(9, 768, dtype=BF16, device=DEV)
    nv.nvfp4_gdn_step(*ins, o, 2, 6, mine.clone(), slots)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nv.nvfp4_gdn_step(*ins, o, 2, 6, mine, slots)
    for i in range(4):
        for t, new in zip(ins, inputs(rng, 9, 2, 6, BF16)):
            t.copy_(new)
        want = nv.gdn_step(*ins, 2, 6, states, slots, out_dtype=BF16)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(mine, states), i


def test_refusals_of_the_binding():
    say("gdn step refusals")
    ins = inputs(np.random.default_rng(6), 4, 1, 2, F32)
    states = torch.zeros(4, 2, 128, 128, device=DEV)

    def refused(*a, **kw):
        with pytest.raises(nv.NVFP4Error):
            nv.gdn_step(*a, **kw)
    refused(*ins, 1, 2, states.double())
    refused(*ins, 1, 2, states[:, :1])
    refused(*ins, 1, 2, states[:3])
    refused(*ins, 1, 2, states[:0])
    refused(*ins, 1, 2, states.transpose(2, 3))
    refused(*ins, 2, 2, states)
    refused(*ins, 1, 2, states, torch.arange(4, device=DEV))
    refused(*ins, 1, 2, states, torch.arange(3, device=DEV).int())
    refused(*ins, 1, 2, states, q_len=3)
    refused(*ins, 1, 2, states, fresh=torch.zeros(4, device=DEV))
    refused(*ins[:4], ins[4].to(BF16), 1, 2, states)
    refused(ins[0][:, :120], *ins[1:], 1, 2, states)
    assert nv.gdn_step(*[x[:0] for x in ins], 1, 2, states).shape == (0, 256)

"""The operators of a hybrid model's layers one after another, as a server runs
them: a prompt, then single tokens of two sequences; each stage is held to the
oracle on what the stage before it gave."""
import numpy as np
import pytest
import torch

import bit_linear_layer_amd as nv
from oracle import layer_oracle as L
from tests.gpu_util import DEV, say
from tests.test_gpu_causal_conv import check as check_conv
from tests.test_gpu_fp8 import close as close_product
from tests.test_gpu_rope import close as close_rope

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def weight(gen, n, k):
    return nv.fp8_quantize(torch.randn(n, k, generator=gen, device=DEV) * k ** -0.5, 128)


def linear(x, w, out_dtype=BF16):
    out = nv.fp8_linear(x, w, out_dtype)
    close_product(out, nv.fp8_quantize(x), w)
    return out


def test_an_attention_layer_around_the_paged_cache():
    say("chain attention")
    gen = torch.Generator(device=DEV).manual_seed(0)
    hidden, hq, hk, d, page, prompts, steps = 384, 6, 2, 64, 16, (45, 130), 4
    w_in, w_out = weight(gen, (hq + 2 * hk) * d, hidden), weight(gen, hidden, hq * d)
    qw, kw = (1 + 0.1 * torch.randn(d, generator=gen, device=DEV) for _ in range(2))
    half = 24  # 48 of 64 dimensions turn
    freq = (1e4 ** (-np.arange(half) / half)).astype(np.float32)
    axis = np.arange(half) % 3
    rope = nv.Rope(torch.from_numpy(freq).to(DEV), torch.from_numpy(axis.astype(np.uint8)).to(DEV))
    pages = nv.empty_kv_pages(20, hk, d, page)
    for t in (pages.k_codes, pages.v_codes, pages.k_scales, pages.v_scales):
        t.fill_(0xFF)
    table = torch.randperm(20, generator=gen, device=DEV)[:18].int().view(2, 9).contiguous()

    def slots(b, at):
        return table.long()[b, at // page] * page + at % page

    def layer(x, positions, write_to, attend):
        qkv = linear(x, w_in)
        q, k, v = qkv[:, : hq * d], qkv[:, hq * d: (hq + hk) * d], qkv[:, (hq + hk) * d:]
        qn, kn = nv.qk_norm_rope(q, k, d, positions, rope, qw, kw)
        for out, x_in, w in ((qn, q, qw), (kn, k, kw)):
            close_rope(out, x_in, d, weight=w.cpu().numpy(), positions=positions.cpu().numpy(), inv_freq=freq, axis=axis)
        nv.kv_pages_write(pages, kn, v, write_to)
        o = attend(qn)
        return qn, o, linear(o, w_out, F32)

    def held(o, q, at):
        """Attention of rows (sequence, tokens seen) over the cache as it is, in 64 bits: 2^-8 for the weights, 2^-8 for the output,
        float32 work below 2^-11 of the sum of magnitudes (scores below 2^7)."""
        for i, (b, n) in enumerate(at):
            k, v = (t.view(n, hk, d).double() for t in nv.kv_pages_read(pages, slots(b, torch.arange(n, device=DEV)), F32))
            qq = q[i].view(hk, hq // hk, d).double()
            for h in range(hk):
                p = torch.softmax(qq[h] @ k[:, h].t() * d ** -0.5, -1)
                want, size = p @ v[:, h].contiguous(), p @ v[:, h].abs().contiguous()
                err = (o[i].view(hk, hq // hk, d)[h].double() - want).abs()
                assert bool((err <= (2.0 ** -8 + 2.0 ** -11) * size + 2.0 ** -8 * want.abs()).all()), (i, h)

    lens = torch.zeros(2, dtype=torch.int32, device=DEV)
    for b, n in enumerate(prompts):
        at = torch.arange(n, device=DEV)
        lens[b] = n
        x = torch.randn(n, hidden, generator=gen, device=DEV).to(BF16)
        q, o, _ = layer(x, torch.stack([at, at // 7, at % 7]), slots(b, at),
                        lambda q: nv.kv_pages_attention(q, pages, table[b: b + 1], lens[b: b + 1], q_len=len(q)))
        held(o[-3:], q[-3:], [(b, n - 2), (b, n - 1), (b, n)])
    for _ in range(steps):
        at = lens.long().clone()
        lens += 1
        write_to = torch.stack([slots(b, at[b]) for b in range(2)])
        x = torch.randn(2, hidden, generator=gen, device=DEV).to(BF16)
        q, o, y = layer(x, at.expand(3, 2).contiguous(), write_to, lambda q: nv.kv_pages_attention(q, pages, table, lens))
        held(o, q, [(b, int(lens[b])) for b in range(2)])
        assert y.shape == (2, hidden) and bool(y.isfinite().all())


def test_a_gated_delta_layer():
    """Two prompts in one convolution call and a recurrence each, states into the pools, then single tokens of both."""
    say("chain gated delta")
    gen = torch.Generator(device=DEV).manual_seed(1)
    hidden, hk, hv, prompts, steps = 256, 2, 4, (70, 131), 5
    channels = (2 * hk + hv) * 128
    w_in = weight(gen, channels + 2 * hv, hidden)
    taps = 0.5 * torch.randn(channels, 4, generator=gen, device=DEV)
    tails = torch.randn(5, 3, channels, generator=gen, device=DEV).to(BF16)
    states = torch.randn(5, hv, 128, 128, generator=gen, device=DEV)
    slots = torch.tensor([4, 1], dtype=torch.int32, device=DEV)
    fresh = torch.ones(2, dtype=torch.uint8, device=DEV)
    rows = sum(prompts)
    x = torch.randn(rows, hidden, generator=gen, device=DEV).to(BF16)
    more = torch.randn(steps, 2, hidden, generator=gen, device=DEV).to(BF16)

    def parts(y, z):
        gates = z[:, channels:].float()
        return [t.contiguous() if t.dtype == F32 else t for t in (
            y[:, : hk * 128], y[:, hk * 128: 2 * hk * 128], y[:, 2 * hk * 128:], torch.sigmoid(gates[:, :hv]).to(BF16),
            -torch.nn.functional.softplus(gates[:, hv:] - 3).to(BF16))]

    z = linear(x, w_in)
    starts = np.array([0, prompts[0], rows])
    before, y = tails.clone(), torch.empty(rows, channels, dtype=BF16, device=DEV)
    nv.nvfp4_causal_conv(z[:, :channels], taps, y, 2, torch.from_numpy(starts).int().to(DEV), None, True, tails, slots, fresh)
    check_conv(z[:, :channels], taps, y, starts, None, True, before, tails, [4, 1], [1, 1])
    whole_z, whole_y = [], []
    for b in range(2):
        at = slice(starts[b], starts[b + 1])
        _, s = nv.gdn_recurrence(*[t[at] for t in parts(y, z)], hk, hv, return_state=True)
        states[slots[b]] = s
        whole_z.append(z[at])
    outs = []
    for t in range(steps):
        z1 = linear(more[t], w_in)
        before, old = tails.clone(), states.clone()
        y1 = nv.causal_conv(z1[:, :channels], taps, 2, state=tails, slots=slots)
        check_conv(z1[:, :channels], taps, y1, np.arange(3), None, True, before, tails, [4, 1])
        outs.append(nv.gdn_step(*parts(y1, z1), hk, hv, states, slots))
        assert torch.equal(states[[0, 2, 3]], old[[0, 2, 3]])
        whole_z = [torch.cat([whole_z[b], z1[b: b + 1]]) for b in range(2)]
    # the same rows as one prompt each: the convolution to the bit, the recurrence within its own bound on both sides
    for b in range(2):
        whole_y = nv.causal_conv(whole_z[b][:, :channels], taps)
        o, s = nv.gdn_recurrence(*parts(whole_y, whole_z[b]), hk, hv, return_state=True)
        got = torch.stack([out[b] for out in outs])
        v_size = whole_y[-steps:, 2 * hk * 128:].float().view(steps, hv, 128).norm(dim=-1).sum()
        size = float(s.norm(dim=(1, 2)).max() + v_size)
        assert float((got - o[-steps:]).abs().max()) <= 4e-4 * size * 128 ** -0.5
        assert float((states[slots[b]] - s).norm(dim=(1, 2)).max()) <= 4e-4 * size

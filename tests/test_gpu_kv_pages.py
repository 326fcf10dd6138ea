"""GPU parity of the paged FP8 KV cache (write and read back bit for bit
against the oracle, untouched bytes included) and of the attention over it.

Tolerance of the attention, per element.  With w_t the exact softmax weights
and A = sum_t w_t |v_t|:
  float32 work: scores s_t are sums of D products, so their error is at most
    (D + 8) 2^-24 S with S >= scale * sum_d |q_d k_td|, plus a few roundings of
    numbers up to S in the exponent; a score error of d changes a weight by a
    factor within 1 +- 2 d (numerator and denominator).  The sums over n
    tokens round at most n + 64 times each, in numerator and denominator.
    Together F = 2^-24 (4 (D + 16) S + 2 (n + 64) + 16) times A.
  bf16: each weight is rounded once (half a step: 2^-8 relative), at most
    2^-8 A in the sum; the output is rounded once, 2^-8 |o|.
  float32 in three bf16 terms leaves 2^-24 of each query element and weight,
    which F covers; the output's rounding is 2^-24 |o|.
"""
import numpy as np
import pytest
import torch

import bit_linear_layer_amd as nv
from oracle import kv_pages_oracle as P
from tests.gpu_util import DEV, say, x_f32

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def to_dev(pages, extra=0):
    """The host cache on the GPU; extra: bytes between pages beyond the dense stride (a multiple of 16)."""
    def up(a, fill):
        t = torch.full((a.shape[0], a.shape[1] + extra), fill, dtype=torch.uint8, device=DEV)
        t[:, : a.shape[1]] = torch.from_numpy(a).to(DEV)
        return t
    return nv.KVPages(*(up(a, 0x7F) for a in (pages.k_codes, pages.v_codes, pages.k_scales, pages.v_scales)),
                      pages.heads, pages.dim, pages.page)


def rows(rng, n, width, dtype, dim=None):
    """Rows with outliers, tiny and zero rows, exact ties and a full-range spread."""
    x = rng.standard_normal((n, width)) * 10.0 ** rng.uniform(-3, 2, (n, 1))
    x[:, rng.integers(0, width, max(1, width // 40))] *= 30
    if n > 2:
        x[1] = 0
        x[2] = rng.choice(P.MAGNITUDES, width) * rng.choice([-1.0, 1.0], width) * 2.0 ** -3
    if n > 3:
        mids = (P.MAGNITUDES[1:] + P.MAGNITUDES[:-1]) / 2
        x[3] = rng.choice(mids, width)
        x[3, 0] = 448
    return torch.from_numpy(x.astype(np.float32)).to(dtype).to(DEV)


def same_bytes(dev, host):
    torch.cuda.synchronize()
    for name in ("k_codes", "v_codes", "k_scales", "v_scales"):
        want = getattr(host, name)
        got = getattr(dev, name).cpu().numpy()
        bad = np.argwhere(got[:, : want.shape[1]] != want)
        assert bad.size == 0, f"{name}: {len(bad)} bytes differ, first {bad[:4].tolist()}"
        assert np.all(got[:, want.shape[1]:] == 0x7F), f"{name}: bytes between pages were written"


def slot_patterns(rng, n_slots):
    whole = np.arange(48)
    return {
        "one": np.array([n_slots - 1]),
        "whole blocks": whole + 16,
        "odd start": np.arange(5, 70),
        "15 rows": np.arange(16, 31),
        "17 rows": np.arange(15, 32),
        "two runs and a gap": np.concatenate([np.arange(3, 21), np.arange(64, 100)]),
        "backwards": whole[::-1].copy(),
        "scattered": rng.permutation(n_slots)[:53],
        "outside": np.concatenate([np.arange(16, 32), [-1, n_slots, 2 ** 40, -2 ** 62], np.arange(n_slots - 16, n_slots + 3)]),
    }


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim,heads,page", [(64, 3, 16), (128, 1, 128), (128, 2, 32), (256, 2, 64)])
def test_write_and_read_bit_exact(dim, heads, page, dtype):
    rng = np.random.default_rng(dim + heads)
    n_pages = 512 // page
    for name, slots in slot_patterns(rng, n_pages * page).items():
        say(f"kv pages write D={dim} H={heads} page={page} {dtype} {name}")
        host = P.Pages(n_pages, heads, dim, page)
        dev = to_dev(host, extra=16 if name == "odd start" else 0)
        k, v = (rows(rng, len(slots), heads * dim, dtype) for _ in range(2))
        if name == "two runs and a gap":  # strided rows
            k = torch.cat([k, k[:, :16]], 1)[:, : heads * dim]
        nv.kv_pages_write(dev, k, v, torch.from_numpy(slots).to(DEV))
        host.write(x_f32(k), x_f32(v), slots)
        same_bytes(dev, host)

        good = (slots >= 0) & (slots < n_pages * page)
        again = np.concatenate([slots, slots[:3]])  # a slot may be read twice
        kept = np.concatenate([good, good[:3]])
        for out_dtype in (BF16, F32):
            outs = [torch.full((len(again), heads * dim), -7.0, dtype=out_dtype, device=DEV) for _ in range(2)]
            nv.nvfp4_kv_pages_read(dev, torch.from_numpy(again).to(DEV), *outs)
            torch.cuda.synchronize()
            for out, want in zip(outs, host.read(again[kept])):
                got = x_f32(out)
                assert np.array_equal(got[kept], want.reshape(kept.sum(), -1).astype(np.float32)), (name, out_dtype)
                assert np.all(got[~kept] == -7.0)


def test_extreme_rows():
    """Largest and smallest magnitudes, the 448 border of the scale, signed zeros."""
    say("kv pages extreme rows")
    rng = np.random.default_rng(5)
    x = np.zeros((48, 64), np.float32)
    tops = [3.3e38, 448.0, np.nextafter(np.float32(448), np.float32(500)), 2.0 ** -126, 2.0 ** -149, 2.0 ** -118 * 1.75, 1.75, 1.7500001]
    for i in range(48):
        x[i] = rng.uniform(-1, 1, 64) * tops[i % 8]
        x[i, i % 64] = tops[i % 8] * (-1 if i % 2 else 1)
        x[i, (i + 1) % 64] = -0.0
    x = x.astype(np.float32)
    host = P.Pages(4, 1, 64, 16)
    dev = to_dev(host)
    t = torch.from_numpy(x).to(DEV)
    nv.kv_pages_write(dev, t, t, torch.arange(7, 55, device=DEV))
    host.write(x, x, np.arange(7, 55))
    same_bytes(dev, host)
    k, _ = nv.kv_pages_read(dev, torch.arange(7, 55, device=DEV), F32)
    want = host.read(np.arange(7, 55))[0].reshape(48, 64)
    normal = np.abs(want) >= 2.0 ** -126  # below, float32 results may be flushed
    with np.errstate(over="ignore"):  # the largest rows may round up past float32's range
        assert np.array_equal(k.cpu().numpy()[normal], want.astype(np.float32)[normal])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_elements_that_are_not_finite(dtype):
    """They read back as NaN; a NaN leaves the rest of its row as it would be
    without it, and other rows are untouched."""
    say(f"kv pages not finite {dtype}")
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn((40, 2 * 64), generator=g, device=DEV).to(dtype)
    y = x.clone()
    bad = torch.zeros(x.shape, dtype=torch.bool, device=DEV)
    for r, c, v in ((0, 3, float("nan")), (17, 64, float("nan")), (17, 100, float("inf")), (30, 9, float("-inf"))):
        y[r, c], bad[r, c] = v, True
    x[0, 3] = x[17, 64] = 0
    a, b = (nv.empty_kv_pages(4, 2, 64, 16) for _ in range(2))
    slots = torch.arange(3, 43, device=DEV)
    nv.kv_pages_write(a, x, x, slots)
    nv.kv_pages_write(b, y, y, slots)
    same = torch.ones(40, 2, dtype=torch.bool, device=DEV)
    same[17, 1] = same[30, 0] = False  # heads with an infinity have its scale
    same = same.repeat_interleave(64, 1)
    for want, got in zip(nv.kv_pages_read(a, slots, F32), nv.kv_pages_read(b, slots, F32)):
        assert torch.isnan(got[bad]).all() and torch.isfinite(got[~bad]).all()
        assert torch.equal(want[same & ~bad], got[same & ~bad])


# ------------------------------------------------------------- attention

class Setup:
    """A batch over a host cache whose unused bytes are all 0xFF (NaN codes,
    scale byte 255), with pages in random order."""

    def __init__(self, seed, dim, heads, group, page, lens, q_len=1, prefix=0, dtype=BF16, amp=1.0, spare_cols=0):
        rng = np.random.default_rng(seed)
        self.rng, self.q_len, self.prefix, self.dtype = rng, q_len, prefix, dtype
        self.lens = np.asarray(lens, np.int32)
        self.batch, self.q_heads, self.dim = len(lens), heads * group, dim
        cols = max(1, -(-max(int(self.lens.max()), 1) // page)) + spare_cols
        shared = -(-prefix // page)
        n_pages = self.batch * cols + shared + 1
        ids = rng.permutation(n_pages).astype(np.int32)
        self.table = ids[: self.batch * cols].reshape(self.batch, cols)
        self.prefix_pages = ids[self.batch * cols: self.batch * cols + shared]
        self.host = P.Pages(n_pages, heads, dim, page, fill=0xFF)
        slots = [self.prefix_pages[t // page] * page + t % page for t in range(prefix)]
        for b, n in enumerate(self.lens):
            slots += [self.table[b, t // page] * page + t % page for t in range(n)]
        n = len(slots)
        self.host.write((rng.standard_normal((n, heads * dim)) * 1.3).astype(np.float32),
                        (rng.standard_normal((n, heads * dim)) * 10.0 ** rng.uniform(-1, 1, (n, 1))).astype(np.float32), slots)
        self.dev = to_dev(self.host)
        q = rng.standard_normal((self.batch * q_len, self.q_heads * dim)) * amp
        self.q = torch.from_numpy(q.astype(np.float32)).to(dtype).to(DEV)

    def args(self):
        return dict(table=torch.from_numpy(self.table).to(DEV), lens=torch.from_numpy(self.lens).to(DEV), q_len=self.q_len,
                    prefix_pages=torch.from_numpy(self.prefix_pages).to(DEV), prefix_len=self.prefix)

    def run(self, **more):
        return nv.kv_pages_attention(self.q, self.dev, **{**self.args(), **more})

    def check(self, out, scale=None, max_len=None, lens=None):
        scale = self.dim ** -0.5 if scale is None else scale
        lens = self.lens if lens is None else lens
        q = x_f32(self.q)
        o, a = P.attention(q, self.host, self.q_heads, scale, self.table, lens, self.q_len, self.prefix_pages, self.prefix,
                           max_len)
        torch.cuda.synchronize()
        got = x_f32(out).astype(np.float64).reshape(o.shape)
        n = self.prefix + max(int(lens.max()), 0)
        qn = np.sqrt((q.reshape(o.shape) ** 2).sum(-1)).max()
        kn = self.key_norm()
        f = 2.0 ** -24 * (4 * (self.dim + 16) * scale * qn * kn + 2 * (n + 64) + 16)
        half = 2.0 ** -8 if self.dtype == BF16 else 0.0
        out_half = 2.0 ** -8 if self.dtype == BF16 else 2.0 ** -24
        tol = (half + f) * a * (1 + out_half) + out_half * np.abs(o) + 1e-30
        live = ~np.isnan(o)
        err = np.abs(got - o)
        bad = np.argwhere(live & ~(err <= tol))
        assert bad.size == 0, (len(bad), bad[0], got[tuple(bad[0])], o[tuple(bad[0])], tol[tuple(bad[0])])
        return live, got

    def key_norm(self):
        """The largest norm of a written key row."""
        worst = 0.0
        page = self.host.page
        lists = [(self.prefix_pages, self.prefix)] + [(self.table[b], max(int(n), 0)) for b, n in enumerate(self.lens)]
        for ids, n in lists:
            slots = [int(ids[t // page]) * page + t % page for t in range(n)]
            slots = [s for s in slots if 0 <= s < self.host.n_pages * page]
            if slots:
                worst = max(worst, np.sqrt((self.host.read(slots)[0] ** 2).sum(-1)).max())
        return worst


CASES = [
    # dim, kv heads, group, page, lens, q_len, prefix
    (128, 1, 1, 16, [1], 1, 0),
    (128, 2, 4, 16, [0], 1, 0),
    (64, 2, 1, 16, [1, 15, 16, 17, 63, 64, 65], 1, 0),
    (128, 2, 4, 64, [255, 256, 257, 0, 300, 3], 1, 0),
    (256, 1, 6, 64, [700], 1, 0),
    (256, 2, 3, 32, [129, 64], 1, 100),          # one pass over prefix and own tokens
    (128, 2, 4, 16, [1, 0, 33, 128, 5], 1, 257),
    (128, 1, 8, 128, [40] * 9, 1, 513),
    (64, 3, 5, 32, [70, 9, 200], 4, 0),          # drafted tokens, 20 rows a head
    (64, 1, 2, 16, [3, 7, 0], 7, 300),           # more queries than own tokens
    (64, 1, 2, 16, [3, 7], 7, 0),                # ... and rows that see nothing
    (256, 1, 2, 64, [90, 75], 33, 40),           # a chunk
    (128, 1, 1, 16, [50, 200], 50, 333),
    (64, 1, 16, 16, [20] * 40, 1, 1000),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", CASES, ids=[str(c).replace(" ", "") for c in CASES])
def test_attention(case, dtype):
    dim, heads, group, page, lens, q_len, prefix = case
    say(f"kv attention {case} {dtype}")
    s = Setup(7, dim, heads, group, page, lens, q_len, prefix, dtype, amp=2.0)
    s.check(s.run())


@pytest.mark.parametrize("prefix", [0, 300])
def test_attention_of_long_unequal_sequences(prefix):
    """More shares than tiles: every tile is cut several times."""
    say(f"kv attention unequal {prefix}")
    s = Setup(8, 64, 1, 2, 64, [4000, 1, 900, 0, 2500, 64], 1, prefix)
    s.check(s.run())


def test_attention_places_without_sequence_and_length_bounds():
    say("kv attention padded batch")
    for prefix in (0, 260):
        s = Setup(9, 128, 2, 2, 16, [30, 40, 50, 60, 70], 1, prefix, spare_cols=2)
        lens = s.lens.copy()
        lens[1] = -1
        lens[3] = -2 ** 31
        lens[4] = 10 ** 6  # counts as max_len
        out = torch.full_like(s.q, 3.0)
        before = out.clone()
        s.run(lens=torch.from_numpy(lens).to(DEV), out=out, max_len=70)
        live, got = s.check(out, max_len=70, lens=lens)
        assert not live[1].any() and not live[3].any() and live[[0, 2, 4]].all()
        assert torch.equal(out[[1, 3]], before[[1, 3]])


def test_attention_skips_pages_that_do_not_exist():
    say("kv attention bad pages")
    s = Setup(10, 64, 1, 4, 16, [100, 64, 40], 2, 290)
    s.table[0, 2] = s.host.n_pages
    s.table[1] = -5          # nothing of its own left
    s.table[2, 0] = 2 ** 30
    s.prefix_pages[3] = -1
    s.check(s.run())
    s = Setup(11, 64, 1, 4, 16, [100, 64], 1, 0)
    s.table[1] = 2 ** 31 - 1  # a row that sees nothing
    out = s.run()
    s.check(out)
    assert torch.all(out[1] == 0)


def test_attention_scale_and_large_scores():
    say("kv attention scales")
    for scale, amp in ((1.0, 8.0), (1e-6, 1.0), (0.3, 30.0)):
        s = Setup(12, 128, 1, 2, 16, [90, 200], 1, 0, F32, amp=amp)
        s.check(s.run(scale=scale), scale=scale)


def test_attention_strided_rows_and_reused_workspace():
    """Column slices of a fused projection as q and out; a workspace full of NaN."""
    say("kv attention strides")
    s = Setup(13, 64, 2, 3, 16, [300, 20, 700], 1, 280)
    w = s.q.shape[1]
    wide = torch.full((3, w + 72), float("nan"), dtype=BF16, device=DEV)
    wide[:, 64: 64 + w] = s.q
    out = torch.full((3, w + 8), 5.0, dtype=BF16, device=DEV)
    s.q = wide[:, 64: 64 + w]
    ws = nv.kv_pages_attention_workspace(s.q, s.dev, 3, 1, s.table.shape[1] * 16, 280)
    ws.fill_(float("nan"))
    s.run(out=out[:, :w], workspace=ws)
    s.q = s.q.contiguous()
    s.check(out[:, :w].contiguous())
    assert torch.all(out[:, w:] == 5.0)


def test_attention_repeats_its_bits():
    say("kv attention determinism")
    s = Setup(14, 128, 2, 4, 16, [500, 3, 260, 77], 1, 300)
    first = s.run()
    for _ in range(5):
        assert torch.equal(s.run(), first)


def test_attention_on_a_side_stream_and_in_a_graph():
    """Captured once, replayed on new queries, lengths and cache contents,
    with eager work in between; each replay equals the eager call."""
    say("kv attention graph")
    s = Setup(15, 64, 2, 2, 16, [400, 90, 33], 1, 270)
    args = s.args()
    cap = s.table.shape[1] * 16
    ws = nv.kv_pages_attention_workspace(s.q, s.dev, 3, 1, cap, 270)
    out = torch.zeros_like(s.q)
    new = torch.zeros((3, 2 * 64), dtype=BF16, device=DEV)
    slots = torch.from_numpy(np.array([s.table[b, 1] * 16 + b for b in range(3)], np.int64)).to(DEV)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        nv.kv_pages_write(s.dev, new, new, slots)
        nv.kv_pages_attention(s.q, s.dev, out=out, workspace=ws, max_len=cap, **args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nv.kv_pages_write(s.dev, new, new, slots)
        nv.kv_pages_attention(s.q, s.dev, out=out, workspace=ws, max_len=cap, **args)
    for i in range(4):
        say(f"kv attention graph replay {i}")
        s.q.copy_(torch.randn_like(s.q, dtype=F32))
        new.copy_(torch.randn_like(new, dtype=F32))
        args["lens"].copy_(torch.tensor([400 - 100 * i, 90, 17 * i], dtype=torch.int32))
        out.fill_(9.0)
        graph.replay()
        got = out.clone()
        torch.cuda.synchronize()
        k, _ = nv.kv_pages_read(s.dev, slots, F32)
        assert (k - new.float()).abs().max() <= new.float().abs().max() / 16
        # bits, since a length past the written tokens attends to the NaN codes there
        assert torch.equal(nv.kv_pages_attention(s.q, s.dev, **args).view(torch.int16), got.view(torch.int16))


def test_two_streams_with_a_workspace_each():
    say("kv attention two streams")
    a, b = Setup(16, 128, 1, 4, 16, [900, 40], 1, 270), Setup(17, 128, 1, 4, 16, [10, 800], 1, 500)
    want = [a.run(), b.run()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for s, st in zip((a, b), streams):
        with torch.cuda.stream(st):
            got.append(s.run())
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_cache_beyond_32_bit_offsets():
    """Pages that lie more than 4 GiB into the codes."""
    say("kv pages 4 GiB")
    heads, dim, page = 8, 128, 64
    n_pages = (1 << 32) // (heads * dim * page) + 40
    dev = nv.empty_kv_pages(n_pages, heads, dim, page)
    rng = np.random.default_rng(18)
    ids = np.array([n_pages - 1, 3, n_pages - 20], np.int32)
    slots = np.concatenate([i * page + np.arange(page) for i in ids.astype(np.int64)])
    k, v = (rows(rng, len(slots), heads * dim, BF16) for _ in range(2))
    nv.kv_pages_write(dev, k, v, torch.from_numpy(slots).to(DEV))
    kq, vq = nv.kv_pages_read(dev, torch.from_numpy(slots).to(DEV), F32)
    host = P.Pages(3, heads, dim, page)
    host.write(x_f32(k), x_f32(v), np.arange(192))
    want = host.read(np.arange(192))
    for got, w in zip((kq, vq), want):
        assert np.array_equal(got.cpu().numpy().reshape(w.shape), w.astype(np.float32))
    q = torch.randn((1, heads * dim), device=DEV).to(BF16)
    small = to_dev(host)
    args = dict(lens=torch.tensor([180], dtype=torch.int32, device=DEV))
    far = nv.kv_pages_attention(q, dev, table=torch.from_numpy(ids[None]).to(DEV), **args)
    near = nv.kv_pages_attention(q, small, table=torch.tensor([[0, 1, 2]], dtype=torch.int32, device=DEV), **args)
    assert torch.equal(far, near)


def test_a_decode_loop_over_a_shared_prefix():
    """As a server runs it: the prompt is written once, then each step writes
    a token of every sequence and attends; compared with dense attention over
    everything read back."""
    say("kv pages decode loop")
    heads, group, dim, page, batch, prefix, steps = 2, 3, 64, 16, 5, 275, 20
    g = torch.Generator(device=DEV).manual_seed(0)
    dev = nv.empty_kv_pages(40, heads, dim, page)
    for t in (dev.k_codes, dev.v_codes, dev.k_scales, dev.v_scales):
        t.fill_(0xFF)

    def rand(n, w):
        return torch.randn((n, w), generator=g, device=DEV).to(BF16)

    order = torch.randperm(40, generator=g, device=DEV).int()
    prefix_pages, table = order[:18], order[18: 18 + 2 * batch].view(batch, 2).contiguous()
    at = torch.arange(prefix, device=DEV)
    prefix_slots = prefix_pages.long()[at // page] * page + at % page
    nv.kv_pages_write(dev, rand(prefix, heads * dim), rand(prefix, heads * dim), prefix_slots)
    lens = torch.zeros(batch, dtype=torch.int32, device=DEV)
    ws = nv.kv_pages_attention_workspace(rand(batch, heads * group * dim), dev, batch, 1, 2 * page, prefix)
    for step in range(steps):
        slots = table.long()[:, step // page] * page + step % page
        nv.kv_pages_write(dev, rand(batch, heads * dim), rand(batch, heads * dim), slots)
        lens += 1
        q = rand(batch, heads * group * dim)
        out = nv.kv_pages_attention(q, dev, table, lens, prefix_pages=prefix_pages, prefix_len=prefix, workspace=ws)
        at = torch.arange(step + 1, device=DEV)
        for b in range(batch):
            k, v = nv.kv_pages_read(dev, torch.cat([prefix_slots, table.long()[b, at // page] * page + at % page]), F32)
            k, v = (t.view(-1, heads, dim).double().cpu() for t in (k, v))
            qq = q[b].view(heads, group, dim).double().cpu()
            p = torch.softmax(torch.einsum("hgd,thd->hgt", qq, k) * dim ** -0.5, -1)
            want = torch.einsum("hgt,thd->hgd", p, v)
            scale = torch.einsum("hgt,thd->hgd", p, v.abs())
            err = (out[b].view(heads, group, dim).double().cpu() - want).abs()
            # 2^-8 for the weights, 2^-8 for the output, and float32 work below 2^-12 (see the top of the file)
            assert torch.all(err <= (2.0 ** -8 + 2.0 ** -12) * scale + 2.0 ** -8 * want.abs())

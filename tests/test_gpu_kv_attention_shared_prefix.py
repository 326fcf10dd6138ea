"""The prefix of all sequences computed once: each kernel of the joint launch,
the launches of their own for 17 to 48 query rows, and the join, with every
irregularity that the other paths are tested with.  Every case asserts that its
prefix is in fact computed once (see test_kv_attention_plan.py).

The reference is 64-bit attention over the tokens read back from the cache (the
read is tested bit for bit); the tolerance is the one derived at the top of
test_gpu_kv_pages.py.
"""
import numpy as np
import pytest
import torch

import bit_linear_layer_amd as nv
from oracle import kv_pages_oracle as P
from tests.gpu_util import DEV, say
from tests.test_gpu_kv_pages import BF16, F32
from tests.test_kv_attention_plan import prefix_is_shared

pytestmark = pytest.mark.gpu


class Batch:
    """Sequences over a cache whose unused bytes are all 0xFF (NaN codes, scale byte 255)."""

    def __init__(self, seed, dim, heads, group, page, lens, q_len, prefix, dtype, bad=False, keys=None):
        self.dim, self.heads, self.group, self.page, self.q_len, self.prefix, self.dtype = dim, heads, group, page, q_len, prefix, dtype
        self.lens = [int(n) for n in lens]
        self.batch, self.q_heads = len(lens), heads * group
        rng = np.random.default_rng(seed)
        g = self.g = torch.Generator(device=DEV).manual_seed(seed)
        cols, shared = max(1, -(-max(self.lens) // page)), -(-prefix // page)
        self.n_pages = self.batch * cols + shared + 1
        ids = rng.permutation(self.n_pages).astype(np.int32)
        self.table, self.prefix_pages = ids[: self.batch * cols].reshape(self.batch, cols), ids[self.batch * cols: -1]
        self.pages = nv.empty_kv_pages(self.n_pages, heads, dim, page)
        for t in (self.pages.k_codes, self.pages.v_codes, self.pages.k_scales, self.pages.v_scales):
            t.fill_(0xFF)
        for ids, n, t0 in [(self.prefix_pages, prefix, 0)] + [(self.table[b], n, prefix) for b, n in enumerate(self.lens)]:
            if n > 0:
                k = torch.randn((n, heads * dim), generator=g, device=DEV) * 1.3 if keys is None else keys(t0, n)
                v = torch.randn((n, heads * dim), generator=g, device=DEV) * 10.0 ** (2 * torch.rand((n, 1), generator=g, device=DEV) - 1)
                nv.kv_pages_write(self.pages, k, v, self.slots(ids, n)[0])
        if bad:
            for _ in range(1 + self.table.size // 12):
                at = rng.integers(self.batch), rng.integers(cols)
                self.table[at] = rng.choice([-1, self.n_pages, 2 ** 31 - 1, -2 ** 31])
            self.prefix_pages[rng.integers(shared)] = -7
        self.q = (torch.randn((self.batch * q_len, self.q_heads * dim), generator=g, device=DEV) * 2).to(dtype)
        assert prefix_is_shared(self.batch, heads, group, dim, q_len, cols * page, prefix, dtype)

    def slots(self, ids, n):
        """Cache slots of n tokens, and which of them exist."""
        at = np.arange(max(n, 0))
        page = ids[at // self.page].astype(np.int64) if n > 0 else np.zeros(0, np.int64)
        ok = (page >= 0) & (page < self.n_pages)
        return torch.from_numpy(page * self.page + at % self.page).to(DEV), torch.from_numpy(ok).to(DEV)

    def args(self):
        return dict(table=torch.from_numpy(self.table).to(DEV), lens=torch.tensor(self.lens, dtype=torch.int32, device=DEV),
                    q_len=self.q_len, prefix_pages=torch.from_numpy(self.prefix_pages).to(DEV), prefix_len=self.prefix)

    def run(self, **more):
        return nv.kv_pages_attention(self.q, self.pages, **{**self.args(), **more})

    def check(self, out, before=None):
        """out against the definition; rows of missing sequences against what they held."""
        heads, group, dim, q_len = self.heads, self.group, self.dim, self.q_len
        out = out.view(self.batch, q_len, heads, group, dim)
        half, last = (2.0 ** -8, 2.0 ** -8) if self.dtype == BF16 else (0.0, 2.0 ** -24)
        first = self.slots(self.prefix_pages, self.prefix)
        for b, n in enumerate(self.lens):
            if n < 0:
                assert before is None or torch.all(out[b] == before), b
                continue
            own = self.slots(self.table[b], n)
            slots, ok = (torch.cat(t) for t in zip(first, own))
            # token t of its own is seen by query j where t < n - q_len + 1 + j
            last_own = torch.cat([torch.full((self.prefix,), -2 ** 40, device=DEV), torch.arange(n, device=DEV)])[ok]
            sees = last_own[None, :] < n - q_len + 1 + torch.arange(q_len, device=DEV)[:, None]
            k, v = (t.view(-1, heads, dim).transpose(0, 1).double().contiguous() for t in nv.kv_pages_read(self.pages, slots[ok], F32))
            q = self.q.view(self.batch, q_len, heads, group, dim)[b].permute(1, 0, 2, 3).reshape(heads, q_len * group, dim).double().contiguous()
            x = torch.matmul(q, k.transpose(1, 2).contiguous()) * dim ** -0.5
            x = x.masked_fill(~sees.repeat_interleave(group, 0), float("-inf"))
            p = torch.softmax(x, -1)
            size = dim ** -0.5 * float(q.norm(dim=-1).max() * k.norm(dim=-1).max())
            f = 2.0 ** -24 * (4 * (dim + 16) * size + 2 * (k.shape[1] + 64) + 16)
            back = lambda t: t.view(heads, q_len, group, dim).permute(1, 0, 2, 3)  # noqa: E731
            want, scale = back(torch.matmul(p, v)), back(torch.matmul(p, v.abs()))
            over = (out[b].double() - want).abs() - ((half + f) * scale * (1 + last) + last * want.abs() + 1e-30)
            assert float(over.max()) <= 0, (b, n, float(over.max()))


def ragged(n, most, q_len=1):
    some = [x for x in (-1, 0, 1, 2, 15, 16, 17, 33, 63, 64, 65, 127, 128, 129, most) if x <= most]
    return np.random.default_rng(n).choice(some, n)


# dim, kv heads, group, page, sequences, longest, q_len, prefix, dtype
JOINT = [(dim, *c, dtype) for dim in (64, 128, 256) for dtype, cases in (
    (BF16, [(8, 4, 16, 8, 129, 1, 1100),      # tiles of 16 rows for the prefix
            (8, 4, 32, 12, 129, 1, 1030),     # ... 64
            (4, 4, 64, 24, 300, 1, 1024),     # ... 128
            (4, 2, 16, 24, 70, 6, 1090),      # drafted tokens, more of them than some have tokens
            (32, 1, 16, 32, 70, 1, 1100),     # the same with a wave to each own tile
            (16, 1, 16, 64, 70, 1, 1100),
            (8, 1, 32, 130, 129, 1, 1030),
            (8, 2, 16, 128, 40, 3, 1100)]),
    (F32, [(8, 4, 16, 24, 129, 1, 1100),
           (8, 2, 16, 24, 70, 7, 1030),
           (16, 1, 16, 64, 70, 1, 1100)])) for c in cases]
BESIDE = [  # 17 to 48 query rows: two launches and the join
    (64, 16, 1, 16, 64, 70, 18, 1600, BF16), (64, 16, 1, 16, 64, 70, 40, 1700, BF16),
    (128, 16, 1, 16, 64, 70, 20, 1600, BF16), (128, 16, 4, 64, 48, 129, 12, 2100, BF16), (128, 8, 3, 32, 64, 129, 11, 3100, BF16),
    (256, 16, 1, 16, 64, 70, 20, 1600, BF16), (256, 16, 2, 64, 48, 129, 24, 2100, BF16), (256, 16, 6, 32, 40, 70, 6, 2500, BF16),
]
name = lambda c: "-".join(str(x) for x in c[:8]) + "-" + str(c[8])[6:]  # noqa: E731


@pytest.mark.parametrize("bad", [False, True], ids=["", "bad-pages"])
@pytest.mark.parametrize("case", JOINT + BESIDE, ids=name)
def test_ragged_batches(case, bad):
    dim, heads, group, page, batch, longest, q_len, prefix, dtype = case
    say(f"kv attention shared prefix {case} {bad}")
    s = Batch(61, dim, heads, group, page, ragged(batch, longest), q_len, prefix, dtype, bad)
    out = torch.full_like(s.q, 3.0)
    s.run(out=out)
    s.check(out, 3.0)


# one case of each kind of kernel, for what follows
KINDS = [
    (64, 8, 4, 16, [70, 3, 40, 0, 129, 64, 17, 1], 1, 1100, BF16),      # 16-row tiles
    (128, 8, 4, 16, [70, 3, 40, 0, 129, 64, 17, 1] * 2, 1, 1030, BF16),  # 64
    (64, 4, 4, 16, [70, 3, 40, 0, 129, 64, 17, 1] * 3, 1, 1100, BF16),   # 128
    (128, 4, 4, 32, [70, 3, 40, 2, 129, 64, 17, 1] * 3, 2, 1030, BF16),
    (256, 4, 4, 16, [70, 3, 40, 0, 129, 64, 17, 1] * 3, 1, 1025, BF16),
    (256, 8, 2, 16, [70, 3, 40, 0, 129, 64, 17, 1] * 3, 1, 1025, BF16),
    (128, 16, 1, 16, [70, 3, 40, 0, 129, 64, 17, 1] * 8, 1, 1025, BF16),  # a wave to each own tile
    (128, 16, 1, 16, [70, 3, 40, 2, 12, 64, 17, 1] * 8, 18, 1600, BF16),  # two launches
    (64, 8, 4, 16, [70, 3, 40, 0, 129, 64, 17, 1] * 3, 1, 1100, F32),
    (128, 16, 1, 16, [70, 3, 40, 0, 129, 64, 17, 1] * 8, 1, 1025, F32),
]
kind = lambda c: f"{c[0]}-{c[1]}-{c[2]}-{len(c[4])}-{c[5]}-{str(c[7])[6:]}"  # noqa: E731


@pytest.mark.parametrize("case", KINDS, ids=kind)
def test_a_query_that_is_not_a_number(case):
    say(f"kv attention shared nan {kind(case)}")
    s = Batch(62, *case)
    want = s.run()
    rows, heads = s.batch * s.q_len, s.q_heads
    spoilt = [(0, heads - 1), (rows // 2, 0), (rows - 1, heads // 2)]
    for r, h in spoilt:
        s.q.view(rows, heads, s.dim)[r, h, 5] = float("nan")
    got = s.run().view(rows, heads, s.dim)
    nan = torch.zeros((rows, heads, 1), dtype=torch.bool, device=DEV)
    for r, h in spoilt:
        nan[r, h] = True
    assert int((torch.isnan(got) != nan).sum()) == 0
    assert int((torch.where(nan, 0, got) != torch.where(nan, 0, want.view(got.shape))).sum()) == 0


@pytest.mark.parametrize("growth", [0.01, 0.3, 20.0, -0.3])
@pytest.mark.parametrize("case", KINDS, ids=kind)
def test_scores_that_grow(case, growth):
    """Every token's score exceeds the last one's, through the prefix and into the own tokens."""
    say(f"kv attention shared growth {kind(case)} {growth}")
    dim, heads = case[0], case[1]
    u = torch.from_numpy(np.random.default_rng(63).choice([-1.0, 1.0], dim)).to(DEV)

    def keys(t0, n):  # scale * q . k = growth * t for q = u
        t = torch.arange(t0, t0 + n, device=DEV, dtype=torch.float64)
        return (growth * t[:, None] * dim ** -0.5 * u).repeat(1, heads).float()
    s = Batch(63, *case, keys=keys)
    s.q = u.repeat(s.q.shape[0], s.q_heads).to(s.dtype)
    s.check(s.run())


@pytest.mark.parametrize("case", KINDS, ids=kind)
def test_only_a_prefix(case):
    """No tokens of the sequences' own: neither table nor lengths are given."""
    say(f"kv attention shared prefix only {kind(case)}")
    s = Batch(64, *case)
    assert prefix_is_shared(s.batch, s.heads, s.group, s.dim, s.q_len, 0, s.prefix, s.dtype)
    s.lens = [0] * s.batch
    s.check(nv.kv_pages_attention(s.q, s.pages, q_len=s.q_len, prefix_pages=s.args()["prefix_pages"], prefix_len=s.prefix))


@pytest.mark.parametrize("case", KINDS, ids=kind)
def test_strided_rows_a_spoilt_workspace_and_equal_bits(case):
    """Column slices as q and out, a workspace full of NaN, and the same bits each time."""
    say(f"kv attention shared strides {kind(case)}")
    s = Batch(65, *case)
    want = s.run()
    s.check(want)
    rows, w = s.q.shape
    wide = torch.full((rows, w + 72), float("nan"), dtype=s.dtype, device=DEV)
    wide[:, 64: 64 + w] = s.q
    out = torch.full((rows, w + 8), 5.0, dtype=s.dtype, device=DEV)
    ws = nv.kv_pages_attention_workspace(s.q, s.pages, s.batch, s.q_len, s.table.shape[1] * s.page, s.prefix)
    s.q = wide[:, 64: 64 + w]
    for _ in range(3):
        ws.fill_(float("nan"))
        out.fill_(5.0)
        s.run(out=out[:, :w], workspace=ws)
        assert torch.equal(out[:, :w], want)
        assert torch.all(out[:, w:] == 5.0)


def put_nan_code(s, ids, token, head, d):
    """A NaN code as dimension d of a token's value."""
    at = (head * s.page + token % s.page // 16 * 16) * s.dim + P.value_index(token % 16, d)
    s.pages.v_codes[int(ids[token // s.page]), at] = 0x7F


DRAFTS = [KINDS[3], KINDS[7], (64, 16, 2, 16, [70, 3, 40, 2, 129, 64, 17, 1], 6, 1100, BF16), (256, 8, 2, 16, [70, 3, 40, 2, 12] * 5, 8, 1030, BF16),
          (128, 8, 2, 16, [70, 3, 40, 2, 12] * 5, 7, 1030, F32)]


@pytest.mark.parametrize("case", DRAFTS, ids=kind)
def test_values_that_are_not_numbers(case):
    """In the last drafted tokens, for the rows that see them, and in the prefix, for all."""
    say(f"kv attention shared nan values {kind(case)}")
    s = Batch(69, *case)
    want = s.run().view(s.batch, s.q_len, s.heads, s.group, s.dim)
    nan = torch.zeros(want.shape, dtype=torch.bool, device=DEV)
    for b, n in enumerate(s.lens):
        for back in (1, 2):
            if n >= back:
                h, d = (b + back) % s.heads, (7 * b + 5 * back) % s.dim
                put_nan_code(s, s.table[b], n - back, h, d)
                nan[b, max(0, s.q_len - back):, h, :, d] = True  # queries j with n - back < n - q_len + 1 + j
    put_nan_code(s, s.prefix_pages, s.prefix - 1, 0, 9)
    nan[:, :, 0, :, 9] = True
    got = s.run().view(want.shape)
    assert int((torch.isnan(got) != nan).sum()) == 0
    assert int((torch.where(nan, 0, got) != torch.where(nan, 0, want)).sum()) == 0


@pytest.mark.parametrize("case", KINDS, ids=kind)
def test_a_prefix_token_of_no_weight(case):
    """Its weight is 0 in float32 beside the later tokens'; a NaN in its value
    is one in every row all the same."""
    say(f"kv attention shared no weight {kind(case)}")
    dim, heads = case[0], case[1]
    u = torch.from_numpy(np.random.default_rng(70).choice([-1.0, 1.0], dim)).to(DEV)

    def keys(t0, n):  # scale * q . k = 4 t for q = u
        t = torch.arange(t0, t0 + n, device=DEV, dtype=torch.float64)
        return (4.0 * t[:, None] * dim ** -0.5 * u).repeat(1, heads).float()
    s = Batch(70, *case, keys=keys)
    s.q = u.repeat(s.q.shape[0], s.q_heads).to(s.dtype)
    want = s.run().view(-1, s.heads, s.group, dim)
    put_nan_code(s, s.prefix_pages, 5, heads - 1, 3)
    got = s.run().view(want.shape)
    nan = torch.zeros(want.shape, dtype=torch.bool, device=DEV)
    nan[:, heads - 1, :, 3] = True
    assert int((torch.isnan(got) != nan).sum()) == 0
    assert int((torch.where(nan, 0, got) != torch.where(nan, 0, want)).sum()) == 0


def test_two_streams_with_a_workspace_each():
    say("kv attention shared two streams")
    batches = [Batch(66 + i, *c) for i, c in enumerate(KINDS)]
    want = [s.run() for s in batches]
    args = [s.args() for s in batches]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for i, s in enumerate(batches):
        with torch.cuda.stream(streams[i % 2]):
            got.append(s.run(**args[i]))
    torch.cuda.synchronize()
    for i, (g, w) in enumerate(zip(got, want)):
        assert torch.equal(g, w), i


LARGE = [  # more units than the chip holds: the joint launch divides itself by the lengths
    (64, 8, 4, 64, 64, 3000, 1, 1600, BF16), (128, 8, 4, 64, 96, 2000, 1, 1600, BF16), (128, 8, 1, 64, 48, 5000, 1, 3000, BF16),
    (256, 4, 6, 64, 64, 1000, 1, 1100, BF16), (128, 8, 4, 64, 260, 300, 1, 520, BF16), (64, 8, 2, 16, 96, 700, 4, 4100, BF16),
    (128, 8, 4, 64, 96, 1000, 1, 1100, F32),
]


@pytest.mark.parametrize("case", LARGE, ids=name)
def test_large_batches(case):
    dim, heads, group, page, batch, longest, q_len, prefix, dtype = case
    say(f"kv attention shared large {case}")
    lens = np.random.default_rng(67).integers(0, longest + 1, batch)
    lens[:3] = longest, -1, 0
    s = Batch(67, dim, heads, group, page, lens, q_len, prefix, dtype)
    out = torch.full_like(s.q, 3.0)
    s.run(out=out)
    s.check(out, 3.0)


@pytest.mark.parametrize("case", [KINDS[3], KINDS[7], KINDS[8]], ids=kind)
def test_in_a_graph(case):
    """Captured once; lengths and queries change between replays."""
    say(f"kv attention shared graph {kind(case)}")
    s = Batch(68, *case)
    args, out = s.args(), torch.zeros_like(s.q)
    most = args["lens"].clone()
    ws = nv.kv_pages_attention_workspace(s.q, s.pages, s.batch, s.q_len, s.table.shape[1] * s.page, s.prefix)
    s.run(out=out, workspace=ws, **args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nv.kv_pages_attention(s.q, s.pages, out=out, workspace=ws, **args)
    for i in range(4):
        s.q.copy_(torch.randn(s.q.shape, generator=s.g, device=DEV))
        args["lens"].copy_(torch.minimum(most, torch.tensor([129, 20, -1, 40][i], device=DEV).int()))
        out.fill_(9.0)
        graph.replay()
        got = out.clone()
        torch.cuda.synchronize()
        want = torch.full_like(out, 9.0)
        nv.kv_pages_attention(s.q, s.pages, out=want, **args)
        assert torch.equal(want, got), i

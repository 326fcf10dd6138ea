"""The attention over the paged FP8 cache in each of its tile shapes: 16 to 128
query rows, waves or workgroups to a tile, with the prefix in the same launch
or without; tiles cut into many shares; and in each of them rows that see
nothing, places without a sequence, pages that do not exist and unused bytes
that are NaN codes.  The tolerance is derived in test_gpu_kv_pages.py.
"""
import numpy as np
import pytest
import torch

import bit_linear_layer_amd as nv
from tests.gpu_util import DEV, say
from tests.test_gpu_kv_pages import BF16, F32, Setup, to_dev

pytestmark = pytest.mark.gpu


def ragged(rng, n, most):
    """n lengths around the steps' borders, empty and missing sequences among them."""
    some = [-1, 0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, most]
    return rng.choice([x for x in some if x <= most], n).astype(np.int32)


def spoil(s, rng):
    """Some pages of the tables and of the prefix do not exist."""
    for _ in range(1 + s.table.size // 12):
        s.table[rng.integers(s.table.shape[0]), rng.integers(s.table.shape[1])] = rng.choice([-1, s.host.n_pages, 2 ** 31 - 1, -2 ** 31])
    if len(s.prefix_pages) > 2:
        s.prefix_pages[rng.integers(len(s.prefix_pages))] = -7


def run(seed, dim, heads, group, page, lens, q_len, prefix, dtype, bad):
    s = Setup(seed, dim, heads, group, page, lens, q_len, prefix, dtype, amp=2.0)
    if bad:
        spoil(s, s.rng)
    out = torch.full_like(s.q, 3.0)
    s.run(out=out)
    live, got = s.check(out)
    assert np.all(got[~live] == 3.0)  # places without a sequence are left as they were


MANY = [
    # dim, kv heads, group, page, batch, longest, q_len, prefix, dtype: at least 1024 tiles of 16 rows
    (64, 8, 2, 16, 140, 200, 1, 300, BF16),   # with a prefix of their own pass
    (128, 8, 1, 32, 130, 130, 1, 256, BF16),
    (128, 8, 1, 16, 40, 70, 8, 257, BF16),    # fewer tiles: a workgroup to each
    (256, 16, 1, 16, 64, 70, 1, 256, BF16),
    (256, 16, 2, 64, 65, 70, 1, 260, BF16),
    (128, 8, 1, 16, 130, 130, 1, 0, BF16),    # own tokens only
    (64, 4, 3, 64, 257, 64, 1, 0, BF16),      # ... a step each
    (256, 16, 1, 16, 64, 130, 2, 20, BF16),   # ... with a short prefix
    (64, 8, 4, 16, 64, 70, 5, 40, F32),       # two tiles to a head
    (64, 8, 1, 16, 128, 65, 1, 256, F32),
    (256, 16, 1, 64, 64, 65, 1, 256, F32),
]


@pytest.mark.parametrize("case", MANY, ids=[str(c[:8]).replace(" ", "") + str(c[8])[6:] for c in MANY])
def test_many_short_sequences(case):
    dim, heads, group, page, batch, longest, q_len, prefix, dtype = case
    say(f"kv attention many {case}")
    rng = np.random.default_rng(31)
    run(31, dim, heads, group, page, ragged(rng, batch, longest), q_len, prefix, dtype, bad=True)


ROWS = [
    # dim, kv heads, group, page, lens, q_len, prefix
    (64, 2, 1, 16, [200, 70, 5], 20, 0),        # 20 rows: 32-row tiles
    (128, 1, 4, 32, [333, 0, 31], 7, 30),
    (256, 1, 1, 16, [130, 70], 31, 0),
    (64, 1, 2, 16, [300, 12], 25, 65),          # 50 rows: 64-row tiles
    (128, 2, 1, 64, [500, -1, 64], 63, 0),
    (256, 1, 1, 16, [400, 30], 50, 0),
    (64, 1, 2, 32, [500, 0, 3], 70, 0),         # 140 rows: two tiles of 128
    (128, 2, 4, 16, [300, 40, 129], 33, 70),
    (256, 1, 2, 64, [400, 65], 66, 33),
    (128, 1, 8, 128, [5000], 20, 0),            # a tile in many shares
    (256, 1, 2, 64, [3000], 40, 0),
    (64, 1, 2, 64, [4100], 20, 100),
    (64, 1, 1, 16, [9, 40], 12, 2000),          # the prefix of 24 rows, with the own tokens
    (128, 1, 5, 16, [9, 40, 0, 77, 3], 2, 1500),  # ... 50
    (256, 2, 1, 16, [9, 40, 0, 77, 3, 33, 1, 18, 90, 5, 2, 60], 8, 700),
    (64, 1, 4, 16, [150, 40, 70], 12, 600),
]


@pytest.mark.parametrize("bad", [False, True], ids=["", "bad-pages"])
@pytest.mark.parametrize("case", ROWS, ids=[str(c).replace(" ", "") for c in ROWS])
def test_many_rows(case, bad):
    dim, heads, group, page, lens, q_len, prefix = case
    say(f"kv attention rows {case} {bad}")
    run(33, dim, heads, group, page, lens, q_len, prefix, BF16, bad)


def test_a_whole_prompt():
    """Row tiles whose first sees 16 tokens and whose last sees 1000."""
    say("kv attention whole prompt")
    run(34, 64, 5, 8, 32, [1000], 1000, 0, BF16, False)


def dense(s_q, dev, slots, q_len, heads, group, dim):
    """Attention of q_len queries in 64 bits over the tokens read back, the
    scale of its rounding errors, and F of the top of test_gpu_kv_pages.py."""
    k, v = nv.kv_pages_read(dev, slots, F32)
    k, v = (t.view(-1, heads, dim).transpose(0, 1).double().contiguous() for t in (k, v))
    q = s_q.view(q_len, heads, group, dim).permute(1, 0, 2, 3).reshape(heads, q_len * group, dim).double().contiguous()
    x = torch.matmul(q, k.transpose(1, 2).contiguous()) * dim ** -0.5
    n = k.shape[1]
    sees = n - q_len + torch.arange(q_len, device=DEV).repeat_interleave(group)
    x = x.masked_fill(torch.arange(n, device=DEV)[None, :] > sees[:, None], float("-inf"))
    p = torch.softmax(x, -1)
    size = dim ** -0.5 * float(q.norm(dim=-1).max() * k.norm(dim=-1).max())
    f = 2.0 ** -24 * (4 * (dim + 16) * size + 2 * (n + 64) + 16)
    back = lambda t: t.view(heads, q_len, group, dim).permute(1, 0, 2, 3).reshape(q_len, -1)
    return back(torch.matmul(p, v)), back(torch.matmul(p, v.abs())), f


LARGE = [
    # dim, kv heads, group, page, batch, longest, prefix, dtype
    (128, 8, 4, 64, 512, 300, 0, BF16),    # a wave to a tile, several tiles to a wave
    (64, 8, 2, 16, 512, 300, 0, F32),
    (128, 8, 4, 64, 96, 4096, 0, BF16),    # a workgroup to a tile, several units
    (256, 4, 6, 64, 96, 4096, 0, BF16),
    (64, 8, 1, 128, 96, 4096, 0, F32),
    (128, 8, 4, 64, 300, 300, 2100, BF16), # with a shared prefix: the launch divides itself
    (256, 4, 6, 64, 64, 1000, 3000, BF16),
    (64, 8, 4, 64, 64, 3000, 700, BF16),
    (128, 8, 1, 64, 24, 5000, 3000, BF16),
]


@pytest.mark.parametrize("case", LARGE, ids=[str(c[:7]).replace(" ", "") + str(c[7])[6:] for c in LARGE])
def test_large_batches(case):
    """More units than the chip holds, against 64-bit attention over the
    tokens read back."""
    dim, heads, group, page, batch, longest, prefix, dtype = case
    say(f"kv attention large {case}")
    g = torch.Generator(device=DEV).manual_seed(5)
    cols, shared = -(-longest // page), -(-prefix // page)
    n_pages = batch * cols + shared
    dev = nv.empty_kv_pages(n_pages, heads, dim, page)
    for i in range(0, n_pages * page, 1 << 15):
        n = min(1 << 15, n_pages * page - i)
        k, v = (torch.randn((n, heads * dim), generator=g, device=DEV).to(BF16) for _ in range(2))
        nv.kv_pages_write(dev, k, v, torch.arange(i, i + n, device=DEV))
    ids = torch.randperm(n_pages, generator=g, device=DEV).int()
    table, prefix_pages = ids[: batch * cols].view(batch, cols).contiguous(), ids[batch * cols:].contiguous()
    lens = torch.randint(0, longest + 1, (batch,), generator=g, device=DEV).int()
    lens[:3] = torch.tensor([longest, -1, 0], dtype=torch.int32)
    q = torch.randn((batch, heads * group * dim), generator=g, device=DEV).to(dtype)
    out = nv.kv_pages_attention(q, dev, table, lens, prefix_pages=prefix_pages, prefix_len=prefix)
    at = torch.arange(prefix, device=DEV)
    before = prefix_pages.long()[at // page] * page + at % page
    half, last = (2.0 ** -8, 2.0 ** -8) if dtype == BF16 else (0.0, 2.0 ** -24)
    for b, n in enumerate(lens.tolist()):
        if n < 0:
            continue
        at = torch.arange(n, device=DEV)
        slots = torch.cat([before, table.long()[b, at // page] * page + at % page])
        if slots.numel() == 0:
            assert torch.all(out[b] == 0)
            continue
        want, scale, f = dense(q[b], dev, slots, 1, heads, group, dim)
        err = (out[b].double() - want[0]).abs()
        tol = (half + f) * scale[0] * (1 + last) + last * want[0].abs()
        assert torch.all(err <= tol), (b, n, float((err - tol).max()))


@pytest.mark.parametrize("q_len,prefix,dtype", [(1, 0, BF16), (1, 300, BF16), (40, 300, BF16), (80, 0, BF16), (1, 300, F32)])
def test_a_query_that_is_not_a_number(q_len, prefix, dtype):
    """NaN in one query row and head: NaN there, also where pieces are joined,
    and every other row as without it."""
    say(f"kv attention nan {q_len} {prefix} {dtype}")
    s = Setup(35, 64, 2, 2, 16, [700, 300], q_len, prefix, dtype)
    want = s.run()
    s.q.view(2 * q_len, 4, 64)[q_len, 3, 5] = float("nan")
    got = s.run()
    a, b = got.view(2 * q_len, 4, 64), want.view(2 * q_len, 4, 64).clone()
    assert torch.isnan(a[q_len, 3]).all()
    b[q_len, 3] = a[q_len, 3]
    assert torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))


@pytest.mark.parametrize("growth", [0.01, 0.3, 20.0, -0.3])
@pytest.mark.parametrize("dim,group,q_len,prefix,dtype", [
    (128, 1, 1, 0, BF16), (64, 2, 1, 0, F32), (64, 2, 10, 0, BF16), (128, 1, 40, 0, BF16), (128, 2, 40, 0, BF16),
    (256, 2, 40, 0, BF16), (64, 1, 1, 300, BF16)])
def test_scores_that_grow(dim, group, q_len, prefix, dtype, growth):
    """Every token's score exceeds the last one's, by little or by much (or
    falls): the running maximum lags behind, is caught up, or stays."""
    say(f"kv attention growth {dim} {group} {q_len} {prefix} {dtype} {growth}")
    s = Setup(36, dim, 1, group, 16, [600, 330], q_len, prefix, dtype)
    u = s.rng.choice([-1.0, 1.0], dim)
    # scale * q . k = growth * t for q = u, k = growth * t * u / sqrt(dim)
    lists = [(s.prefix_pages, prefix, 0)] + [(s.table[b], int(n), prefix) for b, n in enumerate(s.lens)]
    for ids, n, t0 in lists:
        t = np.arange(n)
        if n:
            k = (growth * (t0 + t) * dim ** -0.5)[:, None] * u[None, :]
            v = s.rng.standard_normal((n, dim))
            s.host.write(k.astype(np.float32), v.astype(np.float32), [int(ids[i // 16]) * 16 + i % 16 for i in t])
    s.dev = to_dev(s.host)
    s.q = torch.from_numpy(np.tile(u.astype(np.float32), (s.q.shape[0], group))).to(dtype).to(DEV)
    s.check(s.run())


@pytest.mark.parametrize("q_len,prefix,dtype", [(1, 300, BF16), (1, 100, BF16), (50, 300, BF16), (80, 257, BF16), (3, 300, F32)])
def test_only_a_prefix(q_len, prefix, dtype):
    """No tokens of the sequences' own: neither table nor lengths are given."""
    say(f"kv attention prefix only {q_len} {prefix} {dtype}")
    s = Setup(37, 64, 2, 1, 16, [0, 0, 0], q_len, prefix, dtype)
    out = nv.kv_pages_attention(s.q, s.dev, q_len=q_len, prefix_pages=s.args()["prefix_pages"], prefix_len=prefix)
    # every query sees the whole prefix and nothing else
    s.check(out)


def test_the_largest_pages():
    say("kv attention pages of 4096")
    for q_len, prefix in ((1, 300), (40, 0)):
        run(38, 128, 1, 2, 4096, [4200, 300], q_len, prefix, BF16, False)


SHARED = [
    # dim, kv heads, group, page, lens or (batch, longest), q_len, prefix, dtype: the prefix for all at once
    (64, 8, 2, 16, (140, 200), 1, 1030, BF16),   # 128-row tiles beside a wave to each own tile
    (128, 8, 1, 32, (130, 130), 1, 1024, BF16),
    (256, 16, 2, 64, (65, 70), 1, 1024, BF16),
    (256, 16, 1, 16, (64, 70), 1, 1024, BF16),   # 64-row tiles
    (64, 16, 1, 16, (64, 70), 1, 1025, BF16),
    (128, 16, 1, 64, (64, 70), 1, 1025, BF16),
    (64, 16, 1, 16, (64, 70), 1, 1025, F32),     # 16-row tiles
    (256, 16, 1, 64, (64, 65), 1, 1024, F32),
    (128, 8, 1, 16, (40, 70), 8, 1100, BF16),    # a workgroup to each own tile
    (64, 1, 5, 16, [9, 40, 0, 77, 3], 2, 1100, BF16),
    (256, 1, 5, 16, [9, 40, -1, 77, 3], 2, 1100, BF16),
    (256, 2, 1, 16, [9, 40, 0, 77, 3, 33, 1, 18, 90, 5, 2, 60], 8, 1100, BF16),
    (64, 1, 16, 16, [20] * 40, 1, 1040, BF16),
    (128, 2, 4, 16, [1, 0, 33, 128, 5], 1, 1025, BF16),
    (256, 2, 2, 32, [30, 0, 50], 2, 1200, BF16),
    (128, 2, 4, 16, [1, 0, 33, 128, 5], 1, 1030, F32),
    (64, 16, 1, 64, (64, 40), 17, 1600, BF16),   # 17 own rows: two launches
]


@pytest.mark.parametrize("bad", [False, True], ids=["", "bad-pages"])
@pytest.mark.parametrize("case", SHARED, ids=[str(c[:7]).replace(" ", "") + str(c[7])[6:] for c in SHARED])
def test_a_shared_prefix(case, bad):
    dim, heads, group, page, lens, q_len, prefix, dtype = case
    say(f"kv attention shared {case} {bad}")
    if isinstance(lens, tuple):
        lens = ragged(np.random.default_rng(39), *lens)
    run(39, dim, heads, group, page, lens, q_len, prefix, dtype, bad)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_shared_prefix_in_a_graph(dtype):
    """Lengths change between replays, and with them the division of the launch."""
    say(f"kv attention shared graph {dtype}")
    s = Setup(40, 64, 8, 2, 16, [200] * 72, 1, 1100, dtype)
    args, out = s.args(), torch.zeros_like(s.q)
    ws = nv.kv_pages_attention_workspace(s.q, s.dev, 72, 1, s.table.shape[1] * 16, 1100)
    s.run(out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nv.kv_pages_attention(s.q, s.dev, out=out, workspace=ws, **args)
    for i in range(4):
        s.q.copy_(torch.randn_like(s.q, dtype=F32))
        args["lens"].copy_(torch.randint(-1, (200, 1, 60, 200)[i] + 1, (72,), dtype=torch.int32))
        out.fill_(9.0)
        graph.replay()
        got = out.clone()
        torch.cuda.synchronize()
        want = torch.full_like(out, 9.0)
        nv.kv_pages_attention(s.q, s.dev, out=want, **args)
        assert torch.equal(want, got)

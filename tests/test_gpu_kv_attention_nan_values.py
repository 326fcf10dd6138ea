"""Values that are not finite in tokens that only some of the query rows see
(drafted tokens, chunks of a prompt): the cache holds them as NaN codes, and
they belong to the rows that see their token and to no other.

The rows are compared with a run on the same cache whose codes at these places
are ordinary numbers: rows that do not see the token keep every bit, and rows
that do get a NaN in the element's dimension and keep the bits of the others.
"""
import numpy as np
import pytest
import torch

import bit_linear_layer_amd as nv
from oracle import kv_pages_oracle as P
from tests.gpu_util import DEV, say
from tests.test_gpu_kv_pages import BF16, F32, Setup, to_dev

pytestmark = pytest.mark.gpu


def poison(s, places):
    """NaN codes in s.host's values at places (sequence, own token, head, dimension)."""
    page = s.host.page
    for n, (b, t, h, d) in enumerate(places):
        slot = int(s.table[b, t // page]) * page + t % page
        p, block, o, _ = s.host._at(slot, h)
        s.host.v_codes[p, block + P.value_index(o, d)] = (0x7F, 0xFF)[n % 2]
    s.dev = to_dev(s.host)


def check(s, places):
    """Both runs, and what the places change."""
    want = torch.full_like(s.q, 3.0)
    s.run(out=want)
    s.check(want)
    poison(s, places)
    got = torch.full_like(s.q, 3.0)
    s.run(out=got)
    torch.cuda.synchronize()
    group = s.q_heads // s.host.heads
    nan = torch.zeros((s.batch, s.q_len, s.q_heads, s.dim), dtype=torch.bool, device=DEV)
    for b, t, h, d in places:
        first = max(0, t - int(s.lens[b]) + s.q_len)  # the first query that sees token t
        nan[b, first:, h * group: (h + 1) * group, d] = True
    got, want = (x.view(nan.shape) for x in (got, want))
    leaked = (torch.isnan(got) & ~nan).nonzero().tolist()
    assert not leaked, f"{len(leaked)} elements of rows that do not see the token, first {leaked[0]}"
    lost = (~torch.isnan(got) & nan).nonzero().tolist()
    assert not lost, f"{len(lost)} NaN lost, first {lost[0]}"
    changed = int((torch.where(nan, 0, got) != torch.where(nan, 0, want)).sum())
    assert changed == 0


def tail(rng, s, count):
    """Places in the last q_len tokens of every sequence (and in the last token of all)."""
    out = []
    for b, n in enumerate(s.lens.tolist()):
        for k in range(count if n > 0 else 0):
            t = n - 1 if k == 0 else int(rng.integers(max(0, n - s.q_len), n))
            out.append((b, t, int(rng.integers(s.host.heads)), int(rng.integers(s.dim))))
    return out


CASES = [
    # dim, kv heads, group, page, lens, q_len, prefix, dtype
    (64, 2, 2, 16, [70, 130, 5], 5, 0, BF16),            # tiles of 16 rows
    (128, 2, 1, 32, [64, 65, 190, 3], 3, 40, BF16),
    (128, 1, 4, 64, [700, 1030], 4, 0, BF16),            # ... cut into pieces
    (256, 1, 2, 16, [31, 300], 8, 20, BF16),
    (64, 1, 3, 16, [3, 0, 2, 7], 7, 0, BF16),            # rows that see nothing
    (64, 2, 2, 16, [70, 130, 5], 9, 0, F32),
    (128, 1, 2, 16, [40, 333], 30, 20, F32),
    (256, 1, 1, 64, [40, 90], 20, 0, F32),
    (64, 8, 2, 16, [20, 66, 3, 0, 130, 64, 33, 1] * 17, 2, 0, BF16),  # a wave to a tile
    (256, 16, 2, 16, [20, 66, 3, 0] * 16, 3, 0, BF16),
    (64, 8, 1, 16, [20, 66, 3, 0, 130, 64, 33, 1] * 17, 4, 0, F32),
    (64, 2, 1, 16, [200, 70, 5], 20, 20, BF16),          # 32 rows
    (128, 1, 4, 32, [333, 0, 31], 7, 30, BF16),
    (256, 1, 1, 16, [130, 70], 31, 0, BF16),
    (64, 1, 2, 16, [300, 12], 25, 65, BF16),             # 64 rows
    (128, 2, 1, 64, [500, -1, 64], 63, 0, BF16),
    (256, 1, 1, 16, [400, 30], 50, 0, BF16),
    (64, 1, 2, 32, [500, 0, 3], 70, 0, BF16),            # 128 rows
    (128, 2, 4, 16, [300, 40, 129], 33, 70, BF16),
    (128, 1, 1, 16, [700, 128], 128, 0, BF16),
    (256, 1, 2, 64, [400, 65], 66, 33, BF16),
    (64, 1, 5, 16, [9, 40, 0, 77, 3], 2, 1100, BF16),    # after a long prefix
    (128, 2, 1, 16, [9, 40, 0, 77, 3, 33, 1, 18, 90, 5, 2, 60], 8, 1100, BF16),
    (256, 1, 2, 16, [9, 40, -1, 77, 3], 2, 1100, BF16),
    (64, 16, 1, 64, [40, 3, 17, 0] * 16, 17, 1600, BF16),
    (128, 2, 4, 16, [1, 0, 33, 128, 5], 3, 1030, F32),
]


@pytest.mark.parametrize("case", CASES, ids=[str(c[:4]).replace(" ", "") + f"x{len(c[4])}-{c[5]}-{c[6]}-{str(c[7])[6:]}" for c in CASES])
def test_a_value_belongs_to_the_rows_that_see_it(case):
    dim, heads, group, page, lens, q_len, prefix, dtype = case
    say(f"kv attention nan values {case[:4]} {len(lens)} {q_len} {prefix} {dtype}")
    s = Setup(51, dim, heads, group, page, lens, q_len, prefix, dtype)
    check(s, tail(s.rng, s, 3))


def test_every_token_and_dimension_of_a_step():
    """A NaN in each of the last tokens in turn, in another dimension each."""
    for dim, group, q_len, page in ((64, 1, 12, 16), (128, 2, 14, 16), (64, 2, 30, 64), (128, 2, 60, 16), (256, 2, 60, 16)):
        say(f"kv attention nan values diagonal {dim} {group} {q_len}")
        s = Setup(52, dim, 1, group, page, [q_len + 5], q_len, 0)
        check(s, [(0, t, 0, (37 * t + 11) % dim) for t in range(q_len + 5)])


def test_beside_pages_that_do_not_exist():
    say("kv attention nan values, bad pages")
    for dim, group, q_len in ((64, 2, 8), (64, 2, 14), (128, 2, 30), (128, 2, 70), (256, 2, 70)):
        s = Setup(53, dim, 2, group, 16, [150, 90], q_len, 33)
        s.table[0, 2] = -1
        s.table[1, (90 - q_len) // 16 - 1] = s.host.n_pages
        # (0, 16): beside the missing page, in a step that all rows see
        check(s, [(0, 149, 1, 5), (0, 148, 0, dim - 1), (1, 89, 0, 0), (1, 90 - q_len, 1, 7), (0, 16, 0, 3)])


def test_drafted_tokens_as_they_are_written():
    """Through the public calls: an infinity and a NaN in the last drafted
    tokens' values, which some of the drafts see."""
    say("kv attention nan values, written")
    heads, dim, page, batch, q_len = 2, 128, 16, 3, 6
    g = torch.Generator(device=DEV).manual_seed(2)
    pages = nv.empty_kv_pages(batch * 4, heads, dim, page)
    table = torch.randperm(batch * 4, generator=g, device=DEV).int().view(batch, 4)
    lens = torch.tensor([50, 6, 33], dtype=torch.int32, device=DEV)
    q = torch.randn((batch * q_len, 4 * dim), generator=g, device=DEV).to(BF16)
    outs = []
    at = torch.arange(64, device=DEV)
    slots = (table.long()[:, at // page] * page + at % page)[at[None] < lens[:, None]]
    k, v = (torch.randn((len(slots), heads * dim), generator=g, device=DEV).to(BF16) for _ in range(2))
    for bad in (False, True):
        if bad:
            v[49, 3], v[55, dim + 5], v[54, 9] = float("inf"), float("nan"), float("-inf")
        nv.kv_pages_write(pages, k, v, slots)
        outs.append(nv.kv_pages_attention(q, pages, table, lens, q_len=q_len).view(batch, q_len, heads, 2, dim))
    want, got = outs
    for a, b in ((got[0, :5], want[0, :5]), (got[1, :4], want[1, :4]), (got[2], want[2])):
        assert int((a != b).sum()) == 0
    nan = torch.isnan(got)
    expected = torch.zeros_like(nan)
    expected[0, 5:, 0, :, 3] = expected[1, 5:, 1, :, 5] = expected[1, 4:, 0, :, 9] = True
    assert int((nan != expected).sum()) == 0


@pytest.mark.parametrize("dim,group,lens,q_len,prefix,dtype", [
    (64, 1, [4000], 1, 0, BF16), (128, 2, [3000, 700], 1, 0, F32), (64, 2, [300, 200, 150], 1, 1100, BF16),
    (128, 1, [900], 40, 0, BF16), (128, 2, [1000], 80, 0, BF16), (256, 1, [900], 80, 0, BF16)])
def test_a_token_of_no_weight(dim, group, lens, q_len, prefix, dtype):
    """Scores grow so much that the first tokens' weights are 0 in float32, as
    are those of whole pieces of the sequence.  A NaN in one of their values
    stays a NaN wherever the sequence is cut (0 * NaN)."""
    say(f"kv attention nan values, no weight {dim} {group} {lens} {q_len} {prefix} {dtype}")
    s = Setup(54, dim, 1, group, 16, lens, q_len, prefix, dtype)
    u = s.rng.choice([-1.0, 1.0], dim)
    for ids, n, t0 in [(s.prefix_pages, prefix, 0)] + [(s.table[b], n, prefix) for b, n in enumerate(lens)]:
        if n:  # scale * q . k = 4 t for token t
            k = (4.0 * (t0 + np.arange(n)) * dim ** -0.5)[:, None] * u[None, :]
            slots = [int(ids[t // 16]) * 16 + t % 16 for t in range(n)]
            s.host.write(k.astype(np.float32), s.rng.standard_normal((n, dim)).astype(np.float32), slots)
    s.q = torch.from_numpy(np.tile(u.astype(np.float32), (s.q.shape[0], group))).to(dtype).to(DEV)
    s.dev = to_dev(s.host)
    if prefix:
        want = s.run()
        page, block, o, _ = s.host._at(int(s.prefix_pages[0]) * 16 + 5, 0)
        s.host.v_codes[page, block + P.value_index(o, 3)] = 0x7F
        s.dev = to_dev(s.host)
        got = s.run().view(-1, dim)
        assert torch.isnan(got[:, 3]).all()
        keep = torch.arange(dim, device=DEV) != 3
        assert int((got[:, keep] != want.view(-1, dim)[:, keep]).sum()) == 0
    else:
        check(s, [(b, 7 * b + 2, 0, 5 * b + 1) for b in range(len(lens))] + [(0, lens[0] // 3, 0, 0), (0, lens[0] - 1, 0, dim - 1)])

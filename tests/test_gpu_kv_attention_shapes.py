"""The attention over the paged FP8 cache in each of its tile shapes: 16 to 128
query rows, waves or workgroups to a tile, with the prefix in the same launch
or without; tiles cut into many shares; and in each of them rows that see
nothing, places without a sequence, pages that do not exist and unused bytes
that are NaN codes.  The tolerance is derived in test_gpu_kv_pages.py.
"""
import numpy as np
import pytest
import torch

from tests.gpu_util import say
from tests.test_gpu_kv_pages import BF16, F32, Setup

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
    (64, 8, 2, 16, 140, 200, 1, 300, BF16),   # with the prefix's 128-row tiles in one launch
    (128, 8, 1, 32, 130, 130, 1, 256, BF16),
    (128, 8, 1, 16, 40, 70, 8, 257, BF16),    # fewer tiles: a workgroup to each
    (256, 16, 1, 16, 64, 70, 1, 256, BF16),   # ... 64-row tiles
    (256, 16, 2, 64, 65, 70, 1, 260, BF16),   # ... 128-row tiles of 256 dimensions
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
    (128, 1, 5, 16, [9, 40, 0, 77, 3], 2, 1500),  # ... of 50
    (256, 2, 1, 16, [9, 40, 0, 77, 3, 33, 1, 18, 90, 5, 2, 60], 8, 700),  # ... of 96
    (64, 1, 4, 16, [150, 40, 70], 12, 600),     # 48 own rows: two launches
]


@pytest.mark.parametrize("bad", [False, True], ids=["", "bad-pages"])
@pytest.mark.parametrize("case", ROWS, ids=[str(c).replace(" ", "") for c in ROWS])
def test_many_rows(case, bad):
    dim, heads, group, page, lens, q_len, prefix = case
    say(f"kv attention rows {case} {bad}")
    run(33, dim, heads, group, page, lens, q_len, prefix, BF16, bad)

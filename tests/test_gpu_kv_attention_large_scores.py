"""Scores so large that neighbouring float32 numbers among them are many powers
of two of weight apart.  The softmax is then the mean over the tokens of the
largest score, as long as the others are further away than a score's rounding.

Queries and keys are multiples of one vector of signs, with factors that are
small integers times powers of two: every product and sum is exact, so equal
factors give equal scores in any order of summation.  The values' mean is exact
up to the kernels' roundings: 2^-8 for each weight and 2^-8 for the output in
bf16, 2^-24 (n + 2) for the sums of n equal weights in float32.
"""
import numpy as np
import pytest
import torch

import bit_linear_layer_amd as nv
from tests.gpu_util import DEV, say
from tests.test_gpu_kv_attention_shared_prefix import KINDS, Batch, kind
from tests.test_gpu_kv_pages import BF16, F32

pytestmark = pytest.mark.gpu

ALONE = [
    # dim, kv heads, group, page, lens, q_len, dtype
    (64, 2, 2, 16, [700, 90, 5], 1, BF16), (128, 2, 4, 16, [700, 90, 5], 3, BF16), (256, 1, 2, 16, [700, 90, 5], 1, BF16),
    (64, 16, 2, 16, [70, 9, 5] * 30, 1, BF16),
    (128, 1, 1, 16, [700, 90], 20, BF16), (128, 1, 1, 16, [700, 90], 40, BF16), (128, 1, 2, 16, [700, 90], 60, BF16),
    (64, 1, 2, 16, [700, 90], 60, BF16), (256, 1, 1, 16, [700, 90], 20, BF16), (256, 1, 1, 16, [700, 90], 40, BF16),
    (256, 1, 2, 16, [700, 90], 60, BF16),
    (64, 2, 2, 16, [700, 90, 5], 1, F32), (128, 1, 2, 16, [700, 90, 5], 20, F32), (256, 1, 2, 16, [700, 90, 5], 1, F32),
]
# The exponent of the queries' factor: scores from about 2^18 to 2^106; the largest of them positive or negative.
SIZES = [(p, s) for p in (2, 8, 11, 12, 13, 14, 15, 17, 20, 40, 90) for s in (1, -1)]


def mean_of_the_best(factors, values, seen, sign):
    """Mean of the values of the tokens with the largest score; factors [n] > 0."""
    f = torch.where(seen, sign * factors, -torch.inf)
    best = f == f.max()
    return values[best].mean(0), values[best].abs().mean(0), int(best.sum())


def check(out, want, scale, n, dtype):
    half, last = (2.0 ** -8, 2.0 ** -8) if dtype == BF16 else (0.0, 2.0 ** -24)
    tol = (half + 2.0 ** -24 * (n + 2)) * scale * (1 + last) + last * want.abs()
    over = (out.double() - want).abs() - tol
    assert float(over.max()) <= 0, float(over.max())


def factor(rng, n):
    """256 times small integers, each largest one (15) several times."""
    return torch.from_numpy(256.0 * rng.integers(1, 16, n)).to(DEV)


@pytest.mark.parametrize("power,sign", SIZES)
@pytest.mark.parametrize("case", ALONE, ids=lambda c: f"{c[0]}-{c[1]}-{c[2]}-{len(c[4])}-{c[5]}-{str(c[6])[6:]}")
def test_large_scores(case, power, sign):
    dim, heads, group, page, lens, q_len, dtype = case
    say(f"kv attention large scores {case[:4]} {len(lens)} {q_len} {dtype} {power} {sign}")
    rng = np.random.default_rng(71)
    u = torch.from_numpy(rng.choice([-1.0, 1.0], dim)).to(DEV)
    cols = -(-max(lens) // page)
    pages = nv.empty_kv_pages(len(lens) * cols, heads, dim, page)
    for t in (pages.k_codes, pages.v_codes, pages.k_scales, pages.v_scales):
        t.fill_(0xFF)
    table = torch.from_numpy(rng.permutation(len(lens) * cols).astype(np.int32)).to(DEV).view(len(lens), cols)
    factors, values = [], []
    for b, n in enumerate(lens):
        at = torch.arange(n, device=DEV)
        slots = table.long()[b, at // page] * page + at % page
        factors.append(factor(rng, n))
        v = torch.from_numpy(rng.standard_normal((n, heads * dim)).astype(np.float32)).to(DEV)
        nv.kv_pages_write(pages, (factors[-1][:, None] * u).repeat(1, heads).float(), v, slots)
        values.append(nv.kv_pages_read(pages, slots, F32)[1].double().view(n, heads, dim))
    q = (sign * 2.0 ** power * u).repeat(len(lens) * q_len, heads * group).to(dtype)
    out = nv.kv_pages_attention(q, pages, table, torch.tensor(lens, dtype=torch.int32, device=DEV), q_len=q_len)
    out = out.view(len(lens), q_len, heads, group, dim)
    for b, n in enumerate(lens):
        for j in range(q_len):
            seen = torch.arange(n, device=DEV) < n - q_len + 1 + j
            if not seen.any():
                assert torch.all(out[b, j] == 0)
                continue
            want, scale, k = mean_of_the_best(factors[b], values[b], seen, sign)
            check(out[b, j], want[:, None], scale[:, None], k, dtype)


@pytest.mark.parametrize("power,sign", SIZES)
@pytest.mark.parametrize("case", KINDS, ids=kind)
def test_large_scores_with_a_shared_prefix(case, power, sign):
    say(f"kv attention large scores, shared {kind(case)} {power} {sign}")
    dim, heads = case[0], case[1]
    rng = np.random.default_rng(72)
    u = torch.from_numpy(rng.choice([-1.0, 1.0], dim)).to(DEV)
    factors = []

    def keys(t0, n):
        factors.append(factor(rng, n))
        return (factors[-1][:, None] * u).repeat(1, heads).float()
    s = Batch(72, *case, keys=keys)
    s.q = (sign * 2.0 ** power * u).repeat(s.q.shape[0], s.q_heads).to(s.dtype)
    out = s.run().view(s.batch, s.q_len, heads, s.group, dim)
    first = s.slots(s.prefix_pages, s.prefix)[0]
    f, rest = factors[0], iter(factors[1:])
    for b, n in enumerate(s.lens):
        own = next(rest) if n > 0 else f[:0]
        slots = torch.cat([first, s.slots(s.table[b], n)[0]])
        values = nv.kv_pages_read(s.pages, slots, F32)[1].double().view(-1, heads, dim)
        for j in {0, s.q_len - 1}:
            seen = torch.cat([torch.ones_like(f, dtype=torch.bool), torch.arange(n, device=DEV) < n - s.q_len + 1 + j])
            want, scale, k = mean_of_the_best(torch.cat([f, own]), values, seen, sign)
            check(out[b, j], want[:, None], scale[:, None], k, s.dtype)


@pytest.mark.parametrize("q_len,dtype", [(1, BF16), (5, F32), (20, BF16), (40, BF16), (80, BF16)])
def test_a_tiny_scale(q_len, dtype):
    """scale as small as a float: every token that a row sees has the same
    weight, and a row that sees none gets zeros beside rows that do."""
    say(f"kv attention tiny scale {q_len} {dtype}")
    dim, n = 64, q_len - 3 if q_len > 3 else 50
    g = torch.Generator(device=DEV).manual_seed(73)
    pages = nv.empty_kv_pages(8, 1, dim, 16)
    slots = torch.arange(n, device=DEV)
    k, v = (torch.randn((n, dim), generator=g, device=DEV) for _ in range(2))
    nv.kv_pages_write(pages, k, v, slots)
    values = nv.kv_pages_read(pages, slots, F32)[1].double()
    q = torch.randn((q_len, dim), generator=g, device=DEV).to(dtype)
    table = torch.arange(8, device=DEV).int()[None]
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    for scale in (1e-12, 1e-20, 1e-30, 1e-38, 1e-45):
        out = nv.kv_pages_attention(q, pages, table, lens, q_len=q_len, scale=scale)
        for j in range(q_len):
            seen = n - q_len + 1 + j
            if seen <= 0:
                assert torch.all(out[j] == 0)
            else:
                check(out[j], values[:seen].mean(0), values[:seen].abs().mean(0), seen, dtype)

"""The norm with rotation does not look at a stride that it does not use: the row
strides of one token, the head strides of one head (CPU: the calls are refused for the
weight, which is checked after the strides)."""
import pytest

from tests.test_layer_refusals import FAKE, rope, rows_of

ODD = [-1, -128, 0, 3, 130, 1 << 31, 1 << 62, -(1 << 63), (1 << 63) - 1]


@pytest.mark.parametrize("odd", ODD)
def test_strides_that_are_not_used(odd):
    reached = dict(w=FAKE + 2)
    for kw in (dict(ld=odd), dict(ldo=odd), dict(ld=odd, ldo=odd)):
        assert rope(tokens=1, q=rows_of(**kw, **reached)) == -5
        assert rope(tokens=0, q=rows_of(**kw)) == 0  # no rows: nothing else is looked at
    for kw in (dict(head=odd), dict(heado=odd), dict(head=odd, heado=odd)):
        assert rope(q=rows_of(heads=1, **kw, **reached)) == -5
    assert rope(tokens=1, q=rows_of(heads=1, ld=odd, ldo=odd, head=odd, heado=odd, **reached)) == -5


@pytest.mark.parametrize("odd", [v for v in ODD if v != 130 and v != 0])
def test_strides_that_are_used_are_refused(odd):
    for kw in (dict(ld=odd), dict(ldo=odd), dict(head=odd), dict(heado=odd)):
        assert rope(q=rows_of(**kw)) in (-4, -11)
    for kw in (dict(head=odd), dict(heado=odd)):
        assert rope(tokens=1, q=rows_of(**kw)) in (-4, -11)
    for kw in (dict(ld=odd), dict(ldo=odd)):
        assert rope(q=rows_of(heads=1, **kw)) in (-4, -11)

"""What the gated projections' gradient reserves (no GPU): the products in float32
only where float16 computes them again, sums of dhidden only where it comes in
parts."""

import pytest
from test_gated_linear_abi import INVALID, at, grad

import collective_communication_reduction_way_amd as rr

size = rr.gated_linear_workspace_size
SHAPES = [(1, 1, 1, 1), (2, 200, 64, 100), (3, 333, 770, 2050), (8, 8192, 4096, 16384), (64, 7, 5, 100)]


def up(n, k):
    return (n + k - 1) // k * k


def columns(p, ffn):
    return 2 * sum(up((r + 1) * ffn // p - r * ffn // p, 64) for r in range(p))


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_given_products_are_not_reserved(shape):
    p, tokens, dim, ffn = shape
    for dtype in ("float32", "bfloat16"):
        assert size(*shape, dtype, grad=True, kept=True) == size(*shape, dtype, grad=True)
    more = size(*shape, "float16", grad=True) - size(*shape, "float16", grad=True, kept=True)
    assert more == up(tokens * columns(p, ffn) * 4, 256)
    for dtype in ("float32", "bfloat16", "float16"):
        assert size(*shape, dtype, kept=True) == size(*shape, dtype)


def test_one_product_reserves_no_sums():
    # 256 tiles of 256 x 256, one for every compute unit; the weights are one piece where they are copied
    tokens, dim, ffn = 8192, 2048, 4096
    need = tokens * 2 * ffn * 2 + tokens * dim * 2 + 2 * ffn * dim * 2
    assert size(1, tokens, dim, ffn, "bfloat16", grad=True) == need


def test_the_call_checks_its_own_form():
    shape = (2, 200, 64, 100)
    whole, given = (size(*shape, "float16", grad=True, kept=k) for k in (False, True))
    assert given < whole
    f16 = dict(dt=3, pre=3)
    for kw, need in ((f16, given), (dict(f16, a=None, u=None), whole)):
        st, msg = grad(wsb=need - 1, **kw)
        assert st == INVALID and f"the {need} needed" in msg
        st, msg = grad(wsb=need, dx=at(0), **kw)  # (as far as the check after it)
        assert st == INVALID and "overlap" in msg

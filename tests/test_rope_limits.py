"""CPU-only checks of dsa_rope at the ends of what it takes: refused before any CUDA work."""

import pytest

from test_prompt_abi import P, P2, _rope, lib                # noqa: F401  (a fixture)

TOKENS, HEADS, STRIDE = (1 << 26) - 1, 1 << 16, 1 << 36      # the largest


@pytest.mark.parametrize("kw", [
    dict(heads=HEADS + 1, xt=1 << 24, ot=1 << 24), dict(xt=STRIDE + 8), dict(xh=STRIDE + 8), dict(ot=STRIDE + 8),
    dict(oh=STRIDE + 8, ot=64),
])
def test_just_past_the_limits(lib, kw):                      # noqa: F811
    assert _rope(lib, **kw) == 1


@pytest.mark.parametrize("x,out", [(P, P), (P, P2), (P2, P)])
def test_overlap_of_the_largest(lib, x, out):                # noqa: F811
    """x spans 2^63 + 2^53 bytes, more than a signed size holds, and out lies inside of it, or begins below it and runs into it."""
    a = dict(t=TOKENS, heads=HEADS, x=x, xt=STRIDE, xh=STRIDE, out=out, ot=STRIDE, oh=1 << 19)
    assert _rope(lib, **a) == 1

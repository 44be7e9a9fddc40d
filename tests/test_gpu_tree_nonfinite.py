"""A new row that holds a NaN or an infinity, wherever in its 576 values:
every row that sees it gets NaN throughout, all others their own results."""

import pytest
import torch

import sparse_attention_gb300 as dsa
from tree_case import Step, check_attention

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from sparse_attention_gb300 import build as B
    B.build()
    dsa.load_library()


def _check(st, hurt, places, bad, fill=0.0):
    """New row hurt[b] of sequence b (None: no such row) gets `bad` at `places`."""
    q, kv = st.inputs(fill=fill)
    sees = set()
    for b, j in enumerate(hurt):
        if j is None:
            continue
        kv[int(st.row(b, st.c[b] + j)), places] = bad
        sees |= {int(st.off[b]) + i for i in range(j, st.m[b]) if int(st.masks[b][i]) >> j & 1}
    out, lse = st.attention(q, kv)
    assert st.status() == 0
    assert sees and len(sees) < st.T
    for r in sorted(sees):
        assert torch.isnan(out[r]).all(), f"row {r}: {int((~torch.isnan(out[r])).any(1).sum())} heads with numbers"
        assert torch.isnan(lse[r]).all()
    check_attention(st, q, kv, out, lse, set(range(st.T)) - sees)


@pytest.mark.parametrize("bad", [INF, -INF, NAN])
@pytest.mark.parametrize("place", [0, 5, 300, 511, 512, 575])
@pytest.mark.parametrize("page", [0, 16])
def test_one_value(bad, place, page):
    """A head whose query has the other sign there scores -inf, not +inf."""
    st = Step([200, 131, 60], [9, 2, 5], page, seed=3)
    _check(st, [4, 1, None], [place], bad, fill=bad)


@pytest.mark.parametrize("bad", [INF, -INF])
@pytest.mark.parametrize("c,m,hurt", [
    ([0], [64], [40]),                        # nothing committed: the tile of the new rows alone
    ([120], [64], [7]), ([120], [64], [8]),   # the last row of a tile, and the first of the next
    ([60], [10], [5]), ([60], [10], [3]),     # either side of the middle of a tile
    ([1280, 50], [3, 2], [1, None]),          # new rows behind the last whole tile
    ([30000, 40], [3, 1], [1, None]),         # one sequence in many pieces
    ([700] * 30, [7] * 30, [3] * 30),         # many items
])
def test_places_in_a_tile(c, m, hurt, bad):
    st = Step(c, m, 64, seed=7)
    _check(st, hurt, [9], bad)


@pytest.mark.parametrize("places", [[3, 4], [3, 560], list(range(576))])
def test_several_values(places):
    st = Step([90, 33], [12, 6], 32, seed=5)
    _check(st, [2, 0], places, -INF, fill=NAN)


def test_a_row_that_sees_it_and_nothing_else():
    st = Step([0, 10], [3, 1], 16, seed=8, masks=[[1, 2, 4], [1]])
    _check(st, [1, None], [20], INF)


def test_minus_infinity_of_finite_rows_is_no_weight():
    """A product beyond fp32 is no infinity of the row: the position has no weight, as in 64 bits (exp of less
    than -1e37), and the row's results are those without it, bit for bit."""
    got = []
    for masks in ([1, 3, 5], [1, 1, 5]):
        st = Step([40], [3], 16, seed=9, masks=[masks])
        q, kv = st.inputs(fill=0.0)
        q[:, :, 0] = 4 * (q[:, :, 0].abs() + 1)
        kv[int(st.row(0, 41)), 0] = -3e38
        got.append(st.attention(q, kv))
        assert st.status() == 0
    check_attention(st, q, kv, *got[1])
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])

"""NaN and infinities in caches behind shared prefixes: every (row, head) that sees one shows it, as the formula does,
and no other changes."""

import numpy as np
import pytest
import torch

import sparse_attention_gb300 as dsa
from test_gpu_prefix import Shared
from tree_case import D_V, check_attention

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from sparse_attention_gb300 import build as B
    B.build()
    dsa.load_library()


def _same(a, b, rows):
    return torch.equal(a.cpu()[rows], b.cpu()[rows])


def _check_committed(st, q, kv, clean, b, pos, col, value, rows):
    """Committed position `pos` holds `value` in column `col` < 512, and packed rows `rows` see it.  Its score is the
    value times the query's: NaN, +inf and 0 times an infinity make the row and head NaN throughout; -inf is a weight of
    0, and 0 times the value is NaN in that column alone, the others are what they are without the position."""
    hurt = kv.clone()
    hurt[int(st.row(b, pos)), col] = value
    out, lse = st.prefix(q, hurt)
    assert st.status() == 0
    rest = [r for r in range(st.T) if r not in rows]
    assert _same(out, clean[0], rest) and _same(lse, clean[1], rest)
    out, lse = out.cpu()[rows], lse.cpu()[rows]
    least = q[rows][..., col].float() * value == -INF            # [rows, heads]
    assert out[~least].isnan().all() and lse[~least].isnan().all()
    assert out[least][:, col].isnan().all() and lse[least].isfinite().all()
    other = torch.arange(D_V) != col
    kept = out[least][:, other]
    assert kept.isfinite().all()
    # without the position: its row of K and V away from the sum, in 64 bits
    for n, r in enumerate(rows):
        if not least[n].any():
            continue
        s = int(np.searchsorted(st.off, r, "right")) - 1
        seen = [p for p in st.seen(s, r - int(st.off[s])) if p != (pos if s == b or st.of[s] == st.of[b] else -1)]
        k = kv[torch.from_numpy(st.row(s, np.asarray(seen)))].double()
        z = q[r][least[n]].double() @ k.T / 16
        p = torch.softmax(z, -1)
        ref, big = p @ k[:, :D_V], p @ k[:, :D_V].abs()
        # weights and results rounded to bf16; scores off by at most 576 fp32 steps of some 576 * 0.8^2 / 16 = 23
        tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 * 1.01 + 2 * 576 * 2.0 ** -24 * 40 + len(seen) * 2.0 ** -24) * big
        assert ((out[n][least[n]].double() - ref).abs() <= tol)[:, other].all(), r
        assert ((lse[n][least[n]].double() - torch.logsumexp(z, -1)).abs() <= 576 * 2.0 ** -24 * 40 + (len(seen) + 64) * 2.0 ** -24).all()


@pytest.mark.parametrize("page", [0, 16, 64])
@pytest.mark.parametrize("share", [0, 128, 1000])
@pytest.mark.parametrize("m", [[1, 1, 1, 1], [3, 1, 2, 5]])
def test_own_committed_rows(share, m, page):
    """Of one of two sequences whose rows may lie in one tile."""
    c = [share + x for x in (3, 700, 260, 129)] + [20000]        # (work enough that rows of two sequences are put together)
    st = Shared(c, m + [16], [0, 4, 5], [share, 0], page, seed=share + m[0])
    q, kv = st.inputs()
    clean = st.prefix(q, kv)
    for b in range(4):
        rows = list(range(int(st.off[b]), int(st.off[b + 1])))
        for value, pos, col in ((INF, c[b] - 1, 200), (-INF, c[b] - 1, 3), (NAN, c[b] - 1, 511), (-INF, share + c[b] % 3, 300)):
            _check_committed(st, q, kv, clean, b, pos, col, value, rows)


@pytest.mark.parametrize("page", [0, 32])
def test_shared_rows(page):
    """Of all sequences of a group, in whole tiles that are read once and in the shared rows behind them."""
    st = Shared([330, 401, 512, 200], [2, 1, 3, 2], [0, 3, 4], [320, 0], 0 if page == 0 else page, seed=8)
    q, kv = st.inputs()
    clean = st.prefix(q, kv)
    rows = list(range(int(st.off[3])))
    for value, pos, col in ((INF, 5, 7), (-INF, 255, 64), (NAN, 100, 0), (-INF, 300, 9)):
        hurt = kv.clone()
        for b in range(3):                                       # (one row with pages, each sequence's own copy without)
            hurt[int(st.row(b, pos)), col] = value
        out, lse = st.prefix(q, hurt)
        rest = list(range(int(st.off[3]), st.T))
        assert _same(out, clean[0], rest) and _same(lse, clean[1], rest)
        least = q[rows][..., col].float() * value == -INF
        out, lse = out.cpu()[rows], lse.cpu()[rows]
        assert out[~least].isnan().all() and lse[~least].isnan().all()
        assert out[least][:, col].isnan().all() and lse[least].isfinite().all()
        assert out[least][:, torch.arange(D_V) != col].isfinite().all()


@pytest.mark.parametrize("value", [INF, -INF, NAN])
@pytest.mark.parametrize("c,m,first,share,page", [
    ([131, 828, 388, 257, 20000], [3, 1, 2, 5, 16], [0, 4, 5], [128, 0], 16),      # tiles of two sequences
    ([30, 40, 128], [1, 1, 2], [0, 3], [30], 0),                                    # nothing shared is a whole tile
    ([40000, 40010], [1, 3], [0, 2], [39936], 64),                                  # cut into many pieces
    ([300] * 40, [1, 2] * 20, [0, 40], [256], 32),                                  # planned by a launch of its own
])
def test_new_rows(c, m, first, share, page, value):
    """Every row that sees a new row with such a value is NaN throughout; all others keep their bits."""
    st = Shared(c, m, first, share, page, seed=len(c))
    q, kv = st.inputs()
    clean = st.prefix(q, kv)
    some = set(int(x) for x in np.random.default_rng(1).integers(0, st.T, 12))
    check_attention(st, q, kv, *clean, rows=some)
    for b in sorted({0, 1, len(c) - 1}):
        for j, col in ((0, 5), (m[b] - 1, 575), (m[b] // 2, 511)):
            hurt = kv.clone()
            hurt[int(st.row(b, c[b] + j)), col] = value
            out, lse = st.prefix(q, hurt)
            assert st.status() == 0
            sees = [int(st.off[b]) + i for i in range(j, m[b]) if int(st.masks[b][i]) >> j & 1]
            rest = [r for r in range(st.T) if r not in sees]
            assert _same(out, clean[0], rest) and _same(lse, clean[1], rest)
            assert out.cpu()[sees].isnan().all() and lse.cpu()[sees].isnan().all(), (b, j, col)

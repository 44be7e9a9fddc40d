"""Drafted-step calls whose host bounds are far above the lengths (a graph
captured for the longest request), large pages, and tables in other forms."""

import numpy as np
import pytest
import torch

import sparse_attention_gb300 as dsa
from test_gpu_tree import Tables, _topk_ref
from tree_case import D_QK, D_V, H, SCALE, Step, check_attention

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from sparse_attention_gb300 import build as B
    B.build()
    dsa.load_library()


def _widen(st, max_q, max_ctx, more_rows=0):
    """The same step under larger bounds."""
    st.b = dsa.Batch(st.b.q_off, st.b.ctx_len, max_q, max_ctx, max(st.stride, max_ctx) if st.page else st.stride,
                     total_q=st.T + more_rows)
    if st.page:
        table = torch.full((st.B, -(-max_ctx // st.page)), -1, dtype=I32, device="cuda")
        table[:, :st.table.shape[1]] = torch.from_numpy(st.table).cuda()
        st.pages = dsa.make_pages(table, st.page, st.pool)
    st.ws = dsa.tree_workspace(st.b)


@pytest.mark.parametrize("page", [16, 64, 128, 1024])
@pytest.mark.parametrize("c,m", [([5], [1]), ([300, 0, 77], [4, 0, 9]), ([2500, 1023, 1024], [3, 1, 2])])
@pytest.mark.parametrize("max_ctx", [131072, 1 << 20])
def test_attention_under_wide_bounds(page, c, m, max_ctx):
    st = Step(c, m, page, seed=page)
    q, kv = st.inputs()
    _widen(st, 64, max_ctx)
    out, lse = st.attention(q, kv)
    assert st.status() == 0
    check_attention(st, q, kv, out, lse)


@pytest.mark.parametrize("c,m,k", [([5], [1], 4), ([300, 0, 77], [4, 0, 9], 64), ([9000, 40], [2, 3], 500),
                                   ([2100] * 20, [6] * 20, 2048)])
@pytest.mark.parametrize("bound", [4000, 20000, 40000, 131072, 500000])
@pytest.mark.parametrize("max_q", [9, 64])
def test_topk_under_wide_bounds(c, m, k, bound, max_q):
    if max(c) + max(m) > bound:
        bound = 9100
    st = Step(c, m, 0, seed=k, stride=bound)
    st.b = dsa.Batch(st.b.q_off, st.b.ctx_len, max_q, bound, bound, total_q=st.T)
    ld = (bound + 3) // 4 * 4
    sc = torch.randn((st.T, ld), generator=torch.Generator().manual_seed(k))
    idx = torch.full((st.T, k), -7, dtype=I32, device="cuda")
    dsa.tree_topk(st.b, sc.cuda(), st.mask, k, idx, ws=st.ws)
    assert st.status() == 0
    assert np.array_equal(idx.cpu().numpy(), _topk_ref(st, sc.numpy(), k))


@pytest.mark.parametrize("B,n", [(5, 64), (80, 30), (300, 9)])
@pytest.mark.parametrize("page", [0, 16])
def test_tables_of_trees_without_masks(B, n, page):
    rng = np.random.default_rng(B)
    t = Tables(rng.integers(0, 300, B), rng.integers(0, n + 1, B), page, True, pad=5, seed=B)
    assert t.run(mask=False) == 0
    t.check(mask=False)
    assert (t.mask == -9).all()


@pytest.mark.parametrize("B", [64, 256, 257, 1500])
@pytest.mark.parametrize("tree", [False, True])
def test_tables_in_place(B, tree):
    """More rows than one CTA writes: two launches in place."""
    rng = np.random.default_rng(B)
    t = Tables(rng.integers(0, 300, B), rng.integers(0, 33, B), 16, tree, pad=7, seed=B, max_q=64)
    assert t.run(inplace=True) == 0
    t.check(inplace=True)


@pytest.mark.parametrize("page", [256, 1024])
def test_tables_of_large_pages(page):
    t = Tables([0, page - 1, page, 3 * page + 5, 17], [1, 1, 1, 2 * page, page - 17], page, False, pad=1)
    assert t.run(mask=False) == 0
    t.check(mask=False)


def test_rows_of_a_wide_total():
    """total_q above the step's rows: what lies behind them is neither read nor written."""
    st = Step([700, 90], [5, 12], 64, seed=3)
    q, kv = st.inputs()
    _widen(st, 64, 4096, more_rows=40)
    more = torch.full((40, H, D_QK), float("nan")).to(torch.bfloat16)
    out = torch.full((st.T + 40, H, D_V), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((st.T + 40, H), 7.0, device="cuda")
    mask = torch.cat([st.mask, torch.full((40,), -1, dtype=torch.int64, device="cuda")])
    dsa.tree_mla_fwd(st.b, torch.cat([q, more]).cuda(), kv.cuda(), mask, SCALE, out, lse, pages=st.pages, ws=st.ws)
    assert st.status() == 0
    assert (out[st.T:] == 7).all() and (lse[st.T:] == 7).all()
    check_attention(st, q, kv, out[:st.T], lse[:st.T])

"""Drafted-step calls stay within the workspace that each asks for."""

import numpy as np
import pytest
import torch

import sparse_attention_gb300 as dsa
from tree_case import D_QK, H, SCALE, Step, check_attention, mask_of

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from sparse_attention_gb300 import build as B
    B.build()
    dsa.load_library()


class Guarded:
    """A workspace of n bytes, the status word cleared, in front of bytes that nothing may write."""

    def __init__(self, n):
        self.all = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        self.ws = self.all[:n]
        dsa.reset_device_status(self.ws)

    def check(self, status=0):
        assert dsa.read_device_status(self.ws) == status
        assert (self.all[self.ws.numel():] == 0xA5).all()


@pytest.mark.parametrize("B", [1, 7, 300])
def test_tables_and_commit_in_place(B):
    """In place a commit takes two launches, and tables of 300 sequences do: they pass something through the
    workspace."""
    rng = np.random.default_rng(B)
    st = Step(rng.integers(0, 60, B), np.maximum(rng.integers(0, 9, B), 1), 16, seed=B)
    g = Guarded(264 + 8 * B)
    c, m = (torch.tensor(np.asarray(x), dtype=I32).cuda() for x in (st.c, st.m))
    q_off, slots, pos = (torch.zeros(n, dtype=I32, device="cuda") for n in (B + 1, st.T, st.T))
    mask = torch.zeros(st.T, dtype=torch.int64, device="cuda")
    parent = torch.tensor([p for x in st.parents for p in x], dtype=I32).cuda()
    b = dsa.make_batch(q_off, c, int(max(st.m)), st.max_ctx, st.stride, total_q=st.T)
    held = torch.tensor([-(-x // 16) for x in st.L], dtype=I32).cuda()
    span = torch.zeros(2, dtype=I32, device="cuda")
    free = torch.zeros(st.pool, dtype=I32, device="cuda")
    dsa.step_tables(b, m, c, slots, pos, mask=mask, parent=parent, pages=st.pages, n_pages_old=held, n_pages=held,
                    free_pages=free, free_range=span, free_range_out=span, ws=g.ws)
    g.check()
    assert torch.equal(mask, st.mask) and c.tolist() == st.L
    want = np.concatenate([st.row(x, np.arange(st.c[x], st.L[x])) for x in range(B)])
    assert slots.tolist() == want.tolist()
    kv = torch.randn((st.rows, D_QK), device="cuda").to(torch.bfloat16)
    dsa.tree_commit(b, mask, m - 1, c, kv, pages=st.pages, ws=g.ws)
    g.check()
    assert c.tolist() == [x + bin(mask_of(p)[-1]).count("1") for x, p in zip(st.c, st.parents)]


@pytest.mark.parametrize("c,m", [([0], [1]), ([1500], [8]), ([30000], [3]), ([900] * 40, [5] * 40)])
def test_attention(c, m):
    st = Step(c, m, 64, seed=3)
    q, kv = st.inputs()
    g = Guarded(st.ws.numel())
    st.ws = g.ws
    out, lse = st.attention(q, kv)
    g.check()
    check_attention(st, q, kv, out, lse)


def test_a_tree_on_the_sparse_path():
    """Tables, indexer, selection, sparse attention and commit with the workspace of the path's calls."""
    st = Step([90, 33], [6, 9], 0, seed=5)
    q, kv = st.inputs()
    k = 128
    n = dsa.workspace_size(st.b, k)
    assert n < st.ws.numel()
    g = Guarded(n)
    c, m = (torch.tensor(x, dtype=I32).cuda() for x in (st.c, st.m))
    slots, pos = (torch.zeros(st.T, dtype=I32, device="cuda") for _ in range(2))
    mask = torch.zeros(st.T, dtype=torch.int64, device="cuda")
    parent = torch.tensor([p for x in st.parents for p in x], dtype=I32).cuda()
    dsa.step_tables(st.b, m, c, slots, pos, mask=mask, parent=parent, ws=g.ws)
    sc = torch.zeros((st.T, (st.max_ctx + 3) // 4 * 4), device="cuda")
    qi, ki = (torch.randn(s, device="cuda").to(torch.bfloat16) for s in ((st.T, 32, 128), (st.rows, 128)))
    w = torch.randn((st.T, 32), device="cuda")
    idx = torch.empty((st.T, k), dtype=I32, device="cuda")
    out = torch.empty((st.T, H, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((st.T, H), device="cuda")
    dsa.indexer_scores(st.b, qi, w, ki, sc, ws=g.ws)
    dsa.tree_topk(st.b, sc, mask, k, idx, ws=g.ws)
    dsa.sparse_mla_fwd(st.b, q.cuda(), kv.cuda(), idx, k, SCALE, out, lse, ws=g.ws)
    new = torch.zeros(2, dtype=I32, device="cuda")
    dsa.tree_commit(st.b, mask, m - 1, new, kv.cuda(), ws=g.ws)
    g.check()
    assert torch.equal(mask, st.mask)
    check_attention(st, q, kv, out, lse)
    assert new.tolist() == [x + bin(mask_of(p)[-1]).count("1") for x, p in zip(st.c, st.parents)]

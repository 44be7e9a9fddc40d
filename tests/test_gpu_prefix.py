"""Latent attention of sequences behind shared prefixes, against 64-bit
references and the calls that share nothing."""

import numpy as np
import pytest
import torch

import sparse_attention_gb300 as dsa
from tree_case import D_QK, D_V, H, SCALE, Step, check_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from sparse_attention_gb300 import build as B
    B.build()
    dsa.load_library()


class Shared(Step):
    """A Step whose group g (sequences first[g] .. first[g + 1] - 1) shares its
    first share[g] positions: whole pages by the tables, the rest by copies."""

    def __init__(self, c, m, first, share, page=0, seed=0, **kw):
        super().__init__(c, m, page, seed, **kw)
        self.first, self.share = list(first), list(share)
        self.of = [max(g for g in range(len(share)) if first[g] <= b) for b in range(self.B)]
        self.lead = [next((b for b in range(first[g], first[g + 1]) if m[b]), first[g]) for g in range(len(share))]
        if page:
            for b, g in enumerate(self.of):
                n = share[g] // page if min(c[b], c[self.lead[g]]) >= share[g] else 0
                self.table[b, :n] = self.table[self.lead[g], :n]
            self.pages = dsa.make_pages(torch.from_numpy(self.table).to(self.dev), page, self.pool)
        self.groups = self.make_groups(first, share)
        self.ws = dsa.prefix_workspace(self.b, self.groups, device=self.dev)

    def make_groups(self, first, share):
        f = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32).to(self.dev)  # noqa: E731
        return dsa.make_groups(f(first), f(share))

    def inputs(self, seed=1, fill=float("nan")):
        q, kv = super().inputs(seed, fill)
        for b, g in enumerate(self.of):
            if b != self.lead[g] and min(self.c[b], self.c[self.lead[g]]) >= self.share[g]:
                pos = np.arange(self.share[g])
                kv[torch.from_numpy(self.row(b, pos))] = kv[torch.from_numpy(self.row(self.lead[g], pos))]
        return q, kv

    def prefix(self, q, kv, lse=True, mask=True, groups=None, pages=None):
        out = torch.full((self.T, H, D_V), 7.0, dtype=torch.bfloat16, device=self.dev)
        ls = torch.full((self.T, H), 7.0, dtype=torch.float32, device=self.dev) if lse else None
        dsa.prefix_mla_fwd(self.b, groups or self.groups, q.to(self.dev), kv.to(self.dev), self.mask if mask else None,
                           SCALE, out, ls, pages=pages or self.pages, ws=self.ws)
        return out, ls


@pytest.mark.parametrize("page", [0, 16, 32, 128])
@pytest.mark.parametrize("c,m,first,share", [
    ([200], [1], [0, 1], [128]),
    ([300, 290], [1, 1], [0, 2], [288]),
    ([260, 400, 256, 300, 257], [1, 1, 1, 1, 1], [0, 5], [256]),
    ([130, 140, 700, 650, 9], [3, 1, 7, 2, 4], [0, 2, 4, 5], [130, 640, 0]),
    ([127, 127], [2, 2], [0, 2], [127]),                       # no whole tile is shared
    ([128, 128, 128], [64, 1, 63], [0, 3], [128]),             # nothing of their own but the new rows
    ([0, 520, 0, 600, 530], [0, 2, 0, 1, 3], [0, 5], [512]),   # sequences without new rows, and without a cache
    ([5, 6, 7], [1, 2, 3], [0, 1, 1, 3], [0, 9, 4]),           # an empty group
    ([384] * 9, [1, 2, 1, 2, 1, 2, 1, 2, 1], [0, 9], [384]),
])
@pytest.mark.parametrize("idle", [0, 40])                     # (more than 32 sequences are planned by a launch of their own)
def test_groups(c, m, first, share, page, idle):
    seed = len(c) + page
    if idle:
        c, m, first, share = c + [3] * idle, m + [0] * idle, first + [len(c) + idle], share + [0]
    st = Shared(c, m, first, share, page, seed=seed)
    q, kv = st.inputs()
    out, lse = st.prefix(q, kv)
    assert st.status() == 0
    check_attention(st, q, kv, out, lse)
    again, _ = st.prefix(q, kv, lse=False)
    assert torch.equal(out, again)


@pytest.mark.parametrize("b,n,share,own,page", [(1, 1, 20000, 3, 64), (2, 1, 60000, 100, 0), (33, 3, 4096, 200, 16), (64, 1, 9000, 300, 64)])
def test_cut_items(b, n, share, own, page):
    """Long prefixes are cut over many pairs, sequences' own parts over few."""
    rng = np.random.default_rng(b)
    st = Shared([share + int(x) for x in rng.integers(0, own, b)], [n] * b, [0, b], [share], page, seed=b)
    q, kv = st.inputs()
    out, lse = st.prefix(q, kv)
    assert st.status() == 0
    check_attention(st, q, kv, out, lse, rows=set(int(x) for x in rng.integers(0, b * n, 24)))


def test_chain_without_a_mask():
    st = Shared([200, 210, 190], [9, 64, 1], [0, 3], [190], 16, masks=[[(2 << i) - 1 for i in range(n)] for n in (9, 64, 1)])
    q, kv = st.inputs()
    a, la = st.prefix(q, kv)
    b, lb = st.prefix(q, kv, mask=False)
    assert torch.equal(a, b) and torch.equal(la, lb)
    check_attention(st, q, kv, a, la)


def test_rows_that_see_nothing():
    st = Shared([0, 0, 128], [3, 2, 2], [0, 2, 3], [0, 128], masks=[[0, 2, 0], [1, 1], [0, 3]])
    q, kv = st.inputs()
    out, lse = st.prefix(q, kv)
    assert st.status() == 0 and (out[0] == 0).all() and (lse[0] == -float("inf")).all()
    check_attention(st, q, kv, out, lse)


def test_against_the_calls_that_share_nothing():
    """Both are the same attention: each within its tolerance of the formula, so within two of each other."""
    st = Shared([900, 950, 1000, 700], [4, 1, 6, 2], [0, 3, 4], [896, 512], 64, seed=3)
    q, kv = st.inputs()
    out, lse = st.prefix(q, kv)
    ws = dsa.tree_workspace(st.b)
    ref, ref_lse = torch.empty_like(out), torch.empty_like(lse)
    dsa.tree_mla_fwd(st.b, q.cuda(), kv.cuda(), st.mask, SCALE, ref, ref_lse, pages=st.pages, ws=ws)
    check_attention(st, q, kv, ref, ref_lse)
    check_attention(st, q, kv, out, lse)


def test_rows_stay_apart():
    """Infinities in one sequence's own rows, committed or new, reach no other sequence."""
    st = Shared([300, 310, 400], [2, 1, 3], [0, 3], [256], 16, seed=5, masks=[[1, 3], [1], [1, 2, 5]])
    q, kv = st.inputs()
    clean, lclean = st.prefix(q, kv)
    kv[int(st.row(0, 290)), 5] = float("inf")        # committed, of sequence 0 alone
    kv[int(st.row(2, 401)), 7] = float("nan")        # new row 1 of sequence 2: row 1 sees it, 0 and 2 do not
    out, lse = st.prefix(q, kv)
    hurt = torch.tensor([True, True, False, False, True, False])
    assert torch.equal(out.cpu()[~hurt], clean.cpu()[~hurt]) and torch.equal(lse.cpu()[~hurt], lclean.cpu()[~hurt])
    assert out[4].isnan().all() and lse[4].isnan().all()
    assert not out[0].isfinite().all() and not out[1].isfinite().all()
    kv[int(st.row(0, 100)), 3] = float("nan")        # shared: everyone's
    out, lse = st.prefix(q, kv)
    assert out.isnan().all() and lse.isnan().all()


@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("share", [0, 128, 1000])
@pytest.mark.parametrize("m", [[1, 1, 1, 1], [3, 1, 2, 5]])
def test_a_tile_of_two_sequences(share, m, page):
    """Rows of neighbours in a group may lie in one tile: what either's own rows hold stays with it."""
    c = [share + x for x in (3, 700, 260, 129)] + [20000]        # (work enough that rows of two sequences are put together)
    st = Shared(c, m + [16], [0, 4, 5], [share, 0], page, seed=share + m[0])
    q, kv = st.inputs()
    clean, lclean = st.prefix(q, kv)
    assert st.status() == 0
    at = np.cumsum([0] + m)
    check_attention(st, q, kv, clean, lclean, rows=set(range(at[4] + 1)))
    for b in range(4):
        for value in (float("inf"), -float("inf"), float("nan")):
            hurt = kv.clone()
            hurt[int(st.row(b, c[b] - 1)), 200] = value          # the last committed one, its own
            out, lse = st.prefix(q, hurt)
            mine = torch.zeros(st.T, dtype=torch.bool)
            mine[at[b]:at[b + 1]] = True
            assert torch.equal(out.cpu()[~mine], clean.cpu()[~mine]) and torch.equal(lse.cpu()[~mine], lclean.cpu()[~mine])
            assert not out.cpu()[mine].isfinite().any(-1).all()


@pytest.mark.parametrize("b,n,share,own,page", [(12, 1, 128, 9000, 64), (3, 1, 0, 30000, 0), (9, 3, 256, 4000, 32), (15, 1, 300, 7000, 16)])
def test_cut_own_parts(b, n, share, own, page):
    """Long own parts: the pairs' cuts fall into either sequence of an item."""
    rng = np.random.default_rng(b)
    st = Shared([share + int(x) for x in rng.integers(own // 2, own, b)], [n] * b, [0, b], [share], page, seed=b)
    q, kv = st.inputs()
    out, lse = st.prefix(q, kv)
    assert st.status() == 0
    check_attention(st, q, kv, out, lse)
    again, _ = st.prefix(q, kv)
    assert torch.equal(out, again)


@pytest.mark.parametrize("first,share", [
    ([0, 2, 2], [128, 128]), ([1, 3, 4], [128, 128]), ([0, 3, 2], [128, 128]), ([0, 5, 4], [128, 128]), ([0, -1, 4], [128, 128]),
    ([0, 2, 4], [128, -1]), ([0, 2, 4], [128, 129]), ([0, 2, 4], [400, 128]), ([0, 2, 1 << 30], [128, 128]),
])
@pytest.mark.parametrize("idle", [0, 40])
def test_wrong_groups_share_nothing(first, share, idle):
    """Latched, and every sequence gets its attention all the same."""
    st = Shared([200, 210, 128, 140] + [2] * idle, [1, 2, 1, 3] + [0] * idle, [0, 2, 4 + idle], [128, 128], 32, seed=6)
    if idle:
        first = [x + (idle if 4 <= x <= 5 else 0) for x in first]
    q, kv = st.inputs()
    out, lse = st.prefix(q, kv, groups=st.make_groups(first, share))
    assert st.status() == 6
    check_attention(st, q, kv, out, lse)


@pytest.mark.parametrize("page", [0, 16, 32, 128])
def test_shared_length_beyond_a_sequence(page):
    """A member with fewer committed rows than the group shares: its group is computed one by one, and latched."""
    st = Shared([0, 500, 0, 600, 520], [0, 2, 0, 1, 3], [0, 5], [512], page, seed=5 + page)
    q, kv = st.inputs()
    out, lse = st.prefix(q, kv)
    assert st.status() == 6
    check_attention(st, q, kv, out, lse)


def test_wrong_lengths():
    """A sequence outside the bounds is left as it was; its group's others are computed."""
    st = Shared([200, 210, 300], [1, 2, 1], [0, 3], [128], 32, seed=7)
    q, kv = st.inputs()
    good, _ = st.prefix(q, kv)
    st.b.ctx_len[1] = st.max_ctx + 1
    out, lse = st.prefix(q, kv)
    assert st.status() == 6 and (out[1:3] == 7).all() and (lse[1:3] == 7).all()
    keep = torch.tensor([0, 3])
    o, l = out[keep.cuda()], lse[keep.cuda()]
    st.b.ctx_len[1] = 212
    full, lf = good.clone(), lse.clone()
    full[keep.cuda()], lf[keep.cuda()] = o, l
    check_attention(st, q, kv, full, lf, rows={0, 3})


def test_bad_pages():
    st = Shared([400, 410, 300], [1, 2, 1], [0, 2, 3], [384, 0], 16, seed=8)
    q, kv = st.inputs()
    good, lgood = st.prefix(q, kv)
    for b, col, rows in ((1, 25, [1, 2]), (0, 3, [0, 1, 2])):
        table = st.table.copy()
        table[b, col] = st.pool
        out, lse = st.prefix(q, kv, pages=dsa.make_pages(torch.from_numpy(table).cuda(), 16, st.pool))
        assert st.status() == 7
        dsa.reset_device_status(st.ws)
        hurt = torch.zeros(st.T, dtype=torch.bool)
        hurt[rows] = True
        assert (out.cpu()[hurt] == 7).all() and (lse.cpu()[hurt] == 7).all()
        assert torch.equal(out.cpu()[~hurt], good.cpu()[~hurt]) and torch.equal(lse.cpu()[~hurt], lgood.cpu()[~hurt])


def test_many_sequences():
    B = 65535
    c, m = np.zeros(B, np.int64), np.zeros(B, np.int64)
    c[:40], m[:40] = 150, 1
    c[40000:40010], m[40000:40010] = 129, 2
    m[B - 1] = 3
    first = [0, 50, 39000, 50000, B]
    st = Shared(list(c), list(m), first, [140, 0, 128, 0], 16, seed=9)
    q, kv = st.inputs()
    out, lse = st.prefix(q, kv)
    assert st.status() == 0
    check_attention(st, q, kv, out, lse)


@pytest.mark.parametrize("seed", range(12))
def test_random_batches(seed):
    rng = np.random.default_rng(100 + seed)
    c, m, first, share = [], [], [0], []
    for _ in range(int(rng.integers(1, 6))):
        share.append(int(rng.choice([0, 5, 127, 128, 256, 300, 700, 1500])))
        for _ in range(int(rng.integers(1, 13))):
            c.append(share[-1] + int(rng.choice([0, 1, 3, 60, 127, 128, 129, 400])))
            m.append(int(rng.choice([0, 1, 1, 1, 1, 2, 3, 5, 16, 64])))
        first.append(len(c))
    m[0] = max(m[0], 1)
    st = Shared(c, m, first, share, int(rng.choice([0, 16, 32, 64, 256])), seed=seed)
    q, kv = st.inputs()
    out, lse = st.prefix(q, kv)
    assert st.status() == 0
    check_attention(st, q, kv, out, lse, rows=set(int(x) for x in rng.integers(0, st.T, 40)))


def test_every_sequence_a_group():
    B = 300
    rng = np.random.default_rng(4)
    c, m = [int(x) for x in rng.integers(0, 400, B)], [int(x) for x in rng.integers(0, 3, B)]
    st = Shared(c, m, list(range(B + 1)), c, 16, seed=11)
    q, kv = st.inputs()
    out, lse = st.prefix(q, kv)
    assert st.status() == 0
    check_attention(st, q, kv, out, lse)


def test_captured_and_replayed():
    """One graph, lengths and groups that change on the device between replays."""
    st = Shared([700, 710, 800, 300], [2, 3, 1, 2], [0, 3, 4], [640, 128], 64, seed=12)
    q, kv = st.inputs()
    qd, kvd = q.cuda(), kv.cuda()
    out = torch.full((st.T, H, D_V), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((st.T, H), 7.0, device="cuda")
    call = lambda: dsa.prefix_mla_fwd(st.b, st.groups, qd, kvd, st.mask, SCALE, out, lse, pages=st.pages, ws=st.ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
        call()
    for cut, off in ((0, [0, 3, 4]), (37, [0, 3, 4]), (37, [0, 2, 4])):
        st.c = [x - cut for x in (700, 710, 800, 300)]
        st.L = [x + y for x, y in zip(st.c, st.m)]
        st.b.ctx_len.copy_(torch.tensor(st.L, dtype=torch.int32))
        st.groups.off.copy_(torch.tensor(off, dtype=torch.int32))
        if off[1] == 2:
            st.groups.shared.copy_(torch.tensor([640, 0], dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        assert st.status() == 0
        check_attention(st, q, kv, out, lse)


def test_two_streams():
    sts = [Shared([3000] * 8, [1] * 8, [0, 8], [2944], 64, seed=13), Shared([900, 950], [5, 6], [0, 2], [896], 16, seed=14)]
    ins = [tuple(t.cuda() for t in s.inputs()) for s in sts]
    refs = [s.prefix(*i) for s, i in zip(sts, ins)]
    torch.cuda.synchronize()
    ss = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [torch.zeros_like(r[0]) for r in refs]
    for _ in range(5):
        for s, i, o, x in zip(sts, ins, outs, ss):
            dsa.prefix_mla_fwd(s.b, s.groups, *i, s.mask, SCALE, o, None, pages=s.pages, ws=s.ws, stream=x)
    torch.cuda.synchronize()
    assert all(torch.equal(o, r[0]) for o, r in zip(outs, refs))


def test_a_step_behind_a_prefix():
    """Step tables, latent rows, shared-prefix attention and commit, as a server runs them."""
    page, share, B = 16, 256, 3
    st = Shared([256, 300, 260], [3, 4, 2], [0, 3], [share], page, seed=15)
    q, kv = st.inputs(fill=0.0)
    kvd = kv.cuda()
    i32 = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()  # noqa: E731
    held = [-(-x // page) for x in st.c]
    new = [int(st.table[b, k]) for b in range(B) for k in range(held[b], -(-st.L[b] // page))]
    free = i32(new + [0] * (st.pool - len(new)))
    table = st.table.copy()
    for b in range(B):
        table[b, held[b]:] = -1
    pages = dsa.make_pages(torch.from_numpy(table).cuda(), page, st.pool)
    parents = i32([p for par in st.parents for p in par])
    off, ctx = torch.zeros(B + 1, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    batch = dsa.Batch(off, ctx, max(st.m), st.max_ctx, st.max_ctx, total_q=st.T)
    slots, pos = (torch.zeros(st.T, dtype=torch.int32, device="cuda") for _ in (0, 1))
    mask = torch.zeros(st.T, dtype=torch.int64, device="cuda")
    tws, ws = dsa.tree_workspace(batch), dsa.prefix_workspace(batch, st.groups)
    dsa.step_tables(batch, i32(st.m), i32(st.c), slots, pos, mask=mask, parent=parents, pages=pages, n_pages_old=i32(held),
                    n_pages=torch.zeros(B, dtype=torch.int32, device="cuda"), free_pages=free, free_range=i32([0, len(new)]),
                    free_range_out=torch.zeros(2, dtype=torch.int32, device="cuda"), ws=tws)
    cos, sin = (torch.empty((512, 64), device="cuda") for _ in (0, 1))
    dsa.rope_table(cos, sin, 10000.0)
    x = torch.randn((st.T, D_QK), device="cuda", dtype=torch.bfloat16)
    dsa.latent_append(x, torch.ones(512, device="cuda"), 1e-5, cos, sin, pos, slots, kvd, ws=tws)
    qd = q.cuda()
    dsa.rope(qd[..., 512:], cos, sin, pos, ws=tws)
    out, lse = torch.empty((st.T, H, D_V), dtype=torch.bfloat16, device="cuda"), torch.empty((st.T, H), device="cuda")
    dsa.prefix_mla_fwd(batch, st.groups, qd, kvd, mask, SCALE, out, lse, pages=pages, ws=ws)
    assert dsa.read_device_status(tws) == 0 and dsa.read_device_status(ws) == 0
    assert torch.equal(pages.block_table.cpu(), torch.from_numpy(st.table))
    check_attention(st, qd.cpu(), kvd.cpu(), out, lse)
    dsa.tree_commit(batch, mask, i32([0, 2, 1]), ctx, kvd, pages=pages, ws=tws)
    want = [c + bin(st.masks[b][j] & ((2 << j) - 1)).count("1") for b, (c, j) in enumerate(zip(st.c, (0, 2, 1)))]
    assert ctx.tolist() == want


def test_refusals():
    st = Shared([200, 210], [1, 2], [0, 2], [128], seed=16)
    q, kv = (t.cuda() for t in st.inputs())
    out = torch.empty((st.T, H, D_V), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(TypeError):
        dsa.make_groups(st.groups.off.long(), st.groups.shared)
    with pytest.raises(ValueError):
        dsa.make_groups(st.groups.off[:1], st.groups.shared)
    with pytest.raises(dsa.DsaError):
        dsa.prefix_workspace(st.b, st.make_groups([0, 1, 2, 2], [0, 0, 0]))
    for kw, err in ((dict(q=q.float()), TypeError), (dict(kv=kv[:100]), ValueError), (dict(mask=st.mask[:1]), ValueError),
                    (dict(out=out.cpu()), ValueError), (dict(ws=st.ws[:256]), dsa.DsaError), (dict(ws=None), dsa.DsaError),
                    (dict(scale=0.0), dsa.DsaError)):
        a = dict(dict(q=q, kv=kv, mask=st.mask, out=out, ws=st.ws, scale=SCALE), **kw)
        with pytest.raises(err):
            dsa.prefix_mla_fwd(st.b, st.groups, a["q"], a["kv"], a["mask"], a["scale"], a["out"], ws=a["ws"])

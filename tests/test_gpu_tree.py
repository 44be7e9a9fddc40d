"""A step of drafted tokens over a cache, through the public entry points:
tables, latent append, tree attention, tree top-k, commit, and all of them
together, against 64-bit references."""

import numpy as np
import pytest
import torch

import sparse_attention_gb300 as dsa
from tree_case import D_IDX, D_QK, D_V, F32, H, HALF, SCALE, Step, check_attention, mask_of, parents_np, signed

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from sparse_attention_gb300 import build as B
    B.build()
    dsa.load_library()


def _dev(x, dtype=I32):
    return torch.as_tensor(np.asarray(x), dtype=dtype).cuda()


# ------------------------------------------------------------------ tables --

class Tables:
    def __init__(self, c, n, page, tree, pad=0, extra=5, held_more=0, width=None, max_ctx=None, seed=0, max_q=None):
        rng = np.random.default_rng(seed)
        self.c, self.n, self.page, self.B = list(c), list(n), page, len(c)
        self.T = sum(x for x in n if x > 0) + pad
        self.max_ctx = max_ctx or max(max(x + y for x, y in zip(c, n)), 1)
        self.parents = [parents_np(x, rng) for x in self.n] if tree else None
        o = lambda k, d=I32: torch.full((k,), -9, dtype=d, device="cuda")  # noqa: E731
        self.q_off, self.ctx = o(self.B + 1), o(self.B)
        self.batch = dsa.Batch(self.q_off, self.ctx, max(self.n) if max_q is None else max_q, self.max_ctx,
                               self.max_ctx + 2, total_q=self.T)
        self.slots, self.pos, self.mask = o(self.T), o(self.T), o(self.T, torch.int64)
        self.pages = None
        if page:
            self.held = [-(-x // page) + held_more for x in self.c]
            self.need = [max(h, -(-(x + y) // page)) for h, x, y in zip(self.held, self.c, self.n)]
            self.pool = sum(self.need) + max(extra, 0)
            order = rng.permutation(self.pool).astype(np.int32)
            self.table = np.full((self.B, width or max(max(self.need), 1)), -5, np.int32)
            at = 0
            for b, h in enumerate(self.held):
                self.table[b, :h] = order[at:at + h]
                at += h
            self.order, self.head = order, at
            self.tail = self.pool if extra >= 0 else self.pool + extra
            self.pages = dsa.make_pages(_dev(self.table), page, self.pool)
            self.held_old, self.held_new = _dev(self.held), o(self.B)
            self.free, self.range, self.range_out = _dev(order), _dev([self.head, self.tail]), o(2)
        self.ws = dsa.tree_workspace(self.batch)

    def run(self, mask=True, parents=None, c=None, n=None, inplace=False):
        par = parents if parents is not None else \
            [p for x in self.parents for p in x] + [-1] * (self.T - sum(self.n)) if self.parents is not None else None
        kw = {}
        ctx_old = _dev(self.c)
        if self.page:
            kw = dict(pages=self.pages, n_pages_old=self.held_old, n_pages=self.held_new, free_pages=self.free,
                      free_range=self.range, free_range_out=self.range_out)
        if inplace:
            self.ctx.copy_(ctx_old)
            ctx_old = self.ctx
            if self.page:
                kw.update(n_pages=self.held_old, free_range_out=self.range)
        dsa.step_tables(self.batch, _dev(self.n), ctx_old, self.slots, self.pos, mask=self.mask if mask else None,
                        parent=_dev(par) if par is not None else None, ws=self.ws, **kw)
        return dsa.read_device_status(self.ws)

    def check(self, mask=True, inplace=False):
        off = np.concatenate([[0], np.cumsum(self.n)])
        assert np.array_equal(self.q_off.cpu(), off)
        assert np.array_equal(self.ctx.cpu(), np.add(self.c, self.n))
        table = None
        if self.page:
            table, at = self.table.copy(), self.head
            for b in range(self.B):
                for p in range(self.held[b], self.need[b]):
                    table[b, p] = self.order[at]
                    at += 1
            assert np.array_equal(self.pages.block_table.cpu(), table)
            assert np.array_equal((self.held_old if inplace else self.held_new).cpu(), self.need)
            assert (self.range if inplace else self.range_out).tolist() == [at, self.tail]
        slots, pos, bits = [], [], []
        for b in range(self.B):
            m = mask_of(self.parents[b]) if self.parents is not None else [(2 << i) - 1 for i in range(self.n[b])]
            for i in range(self.n[b]):
                s = self.c[b] + i
                slots.append(table[b, s // self.page] * self.page + s % self.page if self.page
                             else b * (self.max_ctx + 2) + s)
                pos.append(self.c[b] + bin(m[i]).count("1") - 1 if self.parents is not None else s)
                bits.append(m[i])
        pad = self.T - int(off[-1])
        assert self.slots.tolist() == slots + [-1] * pad
        assert self.pos.tolist() == pos + [-1] * pad
        if mask:
            assert self.mask.tolist() == signed(bits) + [0] * pad


@pytest.mark.parametrize("page", [0, 16, 128])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("B,n", [(1, 1), (3, 64), (37, 13), (300, 40), (1025, 3)])
def test_tables(page, tree, B, n):
    rng = np.random.default_rng(B + n + page)
    m = rng.integers(0, n + 1, B)
    m[-1] = n
    t = Tables(rng.integers(0, 700, B), m, page, tree, pad=int(rng.integers(0, 70)), seed=n)
    assert t.run() == 0
    t.check()


def test_tables_of_long_prompts_and_in_place():
    t = Tables([0, 0, 100, 16], [5000, 0, 12001, 1], 16, False, pad=9)
    assert t.run(mask=False) == 0
    t.check(mask=False)
    u = Tables([0, 31, 100, 16], [33, 0, 64, 1], 32, True, pad=2)
    assert u.run(inplace=True) == 0
    u.check(inplace=True)
    # pages held beyond the length are used before new ones
    v = Tables([5, 40], [40, 1], 16, False, held_more=2)
    assert v.run() == 0
    v.check()


def _refused(t, code, **kw):
    table = t.pages.block_table.clone() if t.page else None
    assert t.run(**kw) == code
    assert t.q_off.tolist() == [0] * (t.B + 1)
    assert t.ctx.tolist() == list(t.c)
    assert t.slots.tolist() == [-1] * t.T and t.pos.tolist() == [-1] * t.T
    if t.page:
        assert torch.equal(t.pages.block_table, table)
        assert t.held_new.tolist() == t.held and t.range_out.tolist() == [t.head, t.tail]


def test_tables_refuse_the_whole_step():
    _refused(Tables([10, 20], [100, 60], 16, False, extra=-1, max_ctx=112), 9, mask=False)      # one page short
    _refused(Tables([10, 20], [100, 60], 16, False, width=6, max_ctx=96), 6, mask=False)        # past max_ctx
    _refused(Tables([10, 20], [4, 6], 16, False, max_q=5), 6)
    _refused(Tables([10, 20], [65, 6], 16, False), 6)                                           # > 64 with a mask
    _refused(Tables([10, 20, 3], [4, -1, 2], 0, False), 6)
    _refused(Tables([10, 20, 3], [4, 5, 2], 0, False, pad=-1), 6)                               # more than total_q
    t = Tables([10, 20], [4, 6], 16, False)
    t.held_old[1] = 1000
    t.held[1] = 1000
    _refused(t, 6)
    t = Tables([10, 20], [4, 6], 16, False)
    t.range[1] = t.head - 1
    t.tail = t.head - 1
    _refused(t, 6)


def test_tables_bad_parents_and_pages():
    t = Tables([3], [6], 0, True)
    t.parents = None
    assert t.run(parents=[-1, 0, 2, -2, 3, 77]) == 7
    assert t.mask.tolist() == [1, 3, 4, 8, 24, 32] and t.pos.tolist() == [3, 4, 3, 3, 4, 3]
    t = Tables([20, 3], [2, 2], 16, False)
    t.pages.block_table[0, 1] = t.pool
    assert t.run() == 7
    assert t.slots[:2].tolist() == [-1, -1] and (t.slots[2:] >= 0).all()


@pytest.mark.parametrize("B", [3, 300])
@pytest.mark.parametrize("page", [0, 16])
def test_tables_of_a_step_without_tokens(B, page):
    q_off, ctx = torch.full((B + 1,), 9, dtype=I32, device="cuda"), torch.zeros(B, dtype=I32, device="cuda")
    old, zero = torch.arange(B, dtype=I32, device="cuda") % 7, torch.zeros(B, dtype=I32, device="cuda")
    b = dsa.make_batch(q_off, ctx, 4, 16, 16, total_q=0)
    none = torch.empty(0, dtype=I32, device="cuda")
    kw = {}
    if page:
        held, span = torch.ones(B, dtype=I32, device="cuda"), _dev([0, B])
        kw = dict(pages=dsa.make_pages(torch.arange(B, dtype=I32, device="cuda").view(B, 1), page, B), n_pages_old=held,
                  n_pages=held.clone(), free_pages=torch.arange(B, dtype=I32, device="cuda"), free_range=span,
                  free_range_out=span.clone())
    ws = dsa.tree_workspace(b)
    dsa.step_tables(b, zero, old, none, none, ws=ws, **kw)
    assert dsa.read_device_status(ws) == 0
    assert not q_off.any() and torch.equal(ctx, old)


# ------------------------------------------------------------------ append --

@pytest.mark.parametrize("T,wide", [(1, 0), (7, 8), (129, 2048), (4001, 24)])
def test_latent_append(T, wide):
    g = torch.Generator().manual_seed(T)
    rows, eps = T + 9, 1e-5
    x = torch.randn((T, wide + D_QK), generator=g).to(torch.bfloat16)
    if T > 6:
        x[3], x[4, wide:wide + 512] = 0, 1e-3
    gamma = 1 + 0.1 * torch.randn(D_V, generator=g)
    pos = torch.randint(0, 500, (T,), generator=g)
    ang = torch.rand((500, 64), generator=g) * 6.28
    cos, sin = ang.cos(), ang.sin()
    slots = torch.randperm(rows, generator=g)[:T].to(I32)
    if T > 6:
        slots[2] = -1
    kv = torch.full((rows, D_QK), 3.0, dtype=torch.bfloat16)
    dev = kv.cuda()
    ws = dsa.tree_workspace()
    dsa.latent_append(x.cuda()[:, wide:], gamma.cuda(), eps, cos.cuda(), sin.cuda(), pos.to(I32).cuda(), slots.cuda(),
                      dev, ws=ws)
    assert dsa.read_device_status(ws) == 0
    z = x[:, wide:].double()
    lat = z[:, :D_V] / torch.sqrt((z[:, :D_V] ** 2).mean(1, keepdim=True) + eps) * gamma.double()
    pe, c, s = z[:, D_V:], cos[pos].double(), sin[pos].double()
    rot = torch.cat([pe[:, :32] * c[:, :32] - pe[:, 32:] * s[:, :32], pe[:, 32:] * c[:, 32:] + pe[:, :32] * s[:, 32:]], 1)
    # one rounding to bf16; before it the fp32 norm (512-term sum, root, two
    # products) and, for a rotation, two products and a sum of their sizes
    size = torch.cat([lat.abs(), torch.cat([pe[:, :32].abs() + pe[:, 32:].abs()] * 2, 1)], 1)
    ref = torch.cat([lat, rot], 1)
    live = slots >= 0
    want = kv.double()
    want[slots[live].long()] = ref[live]
    tol = torch.zeros_like(want)
    tol[slots[live].long()] = (HALF * ref.abs() + 520 * F32 * size)[live]
    assert ((dev.cpu().double() - want).abs() <= tol).all()


def test_latent_append_skips_bad_rows():
    T = 6
    x = torch.randn((T, D_QK)).to(torch.bfloat16).cuda()
    one, tab = torch.ones(D_V, device="cuda"), torch.ones((10, 64), device="cuda")
    kv = torch.zeros((8, D_QK), dtype=torch.bfloat16, device="cuda")
    ws = dsa.tree_workspace()
    dsa.latent_append(x, one, 1e-5, tab, tab, _dev([0, 10, -1, 3, 4, 5]), _dev([0, 1, 2, 8, -2, 5]), kv, ws=ws)
    assert dsa.read_device_status(ws) == 7
    assert (kv.abs().sum(1) > 0).tolist() == [True, False, False, False, False, True, False, False]


# --------------------------------------------------------------- attention --

@pytest.mark.parametrize("page", [0, 16, 32, 64, 256])
@pytest.mark.parametrize("c,m", [
    ([0], [1]), ([1], [1]), ([127], [1]), ([128], [2]), ([700], [3]), ([0], [64]), ([1000], [64]), ([4097], [5]),
    ([63, 64, 65, 0, 129, 511], [1, 2, 64, 7, 33, 1]),
])
def test_attention(page, c, m):
    st = Step(c, m, page, seed=sum(c) + page)
    q, kv = st.inputs()
    out, lse = st.attention(q, kv)
    assert st.status() == 0
    check_attention(st, q, kv, out, lse)


def test_attention_of_many_ragged_sequences():
    rng = np.random.default_rng(5)
    c, m = rng.integers(0, 900, 70), rng.integers(0, 12, 70)
    st = Step(c, m, 32, seed=6, stride=None)
    q, kv = st.inputs()
    out, lse = st.attention(q, kv)
    assert st.status() == 0
    rows = set(rng.choice(st.T, 60, replace=False).tolist())
    check_attention(st, q, kv, out, lse, rows)


@pytest.mark.parametrize("page", [0, 64])
def test_attention_over_long_contexts(page):
    st = Step([40001, 9000], [1, 6], page, seed=9)
    q, kv = st.inputs()
    q = (q.float() * 2).to(torch.bfloat16)          # sharper: a few positions carry a row
    out, lse = st.attention(q, kv)
    assert st.status() == 0
    check_attention(st, q, kv, out, lse)


@pytest.mark.parametrize("page", [0, 16])
def test_attention_masks(page):
    """Rows that see nothing, masks that are no tree, bits above the row's own."""
    m = [5, 4, 64]
    masks = [[0, 0, 0, 0, 0], [1, 0, 5, 0xF0F0F0F0F0F0F0F0 | 2], [(1 << 64) - 1] * 64]
    st = Step([0, 70, 0], m, page, seed=2, masks=masks)
    q, kv = st.inputs()
    out, lse = st.attention(q, kv)
    assert st.status() == 0
    check_attention(st, q, kv, out, lse)
    assert (out[:5] == 0).all() and torch.isinf(lse[:5]).all()


def test_attention_pieces_that_a_row_does_not_see():
    """Contexts that end on a tile: the last tile holds new rows alone, which some rows do not see."""
    masks = [[0, 2, 1, 0, 31], [0] * 3, [1], [0, 0, 7]]
    st = Step([1280, 128, 0, 0], [5, 3, 1, 3], 64, seed=13, masks=masks)
    q, kv = st.inputs()
    out, lse = st.attention(q, kv)
    assert st.status() == 0
    check_attention(st, q, kv, out, lse)


@pytest.mark.parametrize("way", ["rising", "falling", "flat", "spikes"])
def test_attention_moving_maximum(way):
    """Scores whose running maximum moves at every tile, never, or by hundreds at once."""
    st = Step([3500, 650], [2, 3], 16, seed=14)
    q, kv = st.inputs()
    q[:] = torch.randn((1, H, D_QK), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    along = q[0, 0].double() / (q[0, 0].double() ** 2).sum()
    for b in range(2):
        n = st.L[b]
        want = {"rising": torch.linspace(-300, 300, n), "falling": torch.linspace(300, -300, n),
                "flat": torch.zeros(n), "spikes": torch.where(torch.arange(n) % 500 == 499, 400.0, -100.0)}[way]
        rows = torch.from_numpy(st.row(b, np.arange(n)))
        kv[rows] = (kv[rows].double() * 0.05 + want.double()[:, None] / SCALE * along).to(torch.bfloat16)
    out, lse = st.attention(q, kv)
    assert st.status() == 0
    check_attention(st, q, kv, out, lse)


@pytest.mark.parametrize("what", ["page", "nan"])
def test_attention_of_a_long_sequence_cut_into_many_pieces(what):
    """A bad page leaves the rows unwritten, a NaN in a new row reaches its seers, whichever piece holds it."""
    st = Step([30000, 40], [3, 1], 64, seed=15, masks=[[1, 2, 7], [1]])
    q, kv = st.inputs()
    if what == "page":
        st.pages.block_table[0, 200] = -1
    else:
        kv[int(st.row(0, 30001)), 7] = float("nan")
    out, lse = st.attention(q, kv)
    assert st.status() == (7 if what == "page" else 0)
    if what == "page":
        assert (out[:3] == 7).all() and (lse[:3] == 7).all()
        check_attention(st, q, kv, out, lse, {3})
    else:
        assert torch.isnan(out[1:3]).all() and torch.isnan(lse[1:3]).all()
        check_attention(st, q, kv, out, lse, {0, 3})


def test_thousands_of_sequences():
    """Every call on 65,535 sequences, most of them empty."""
    rng = np.random.default_rng(8)
    B = 65535
    c, m = np.zeros(B, np.int64), np.zeros(B, np.int64)
    some = np.sort(rng.choice(B, 300, replace=False))
    some[-1] = B - 1
    c[some], m[some] = rng.integers(0, 60, 300), rng.integers(1, 4, 300)
    st = Step(c, m, 16, seed=16)
    q, kv = st.inputs()
    out, lse = st.attention(q, kv)
    assert st.status() == 0
    rows = set(rng.choice(st.T, 40, replace=False).tolist()) | {0, st.T - 1}
    check_attention(st, q, kv, out, lse, rows)
    t = Tables(c, m, 16, True, pad=3)
    assert t.run() == 0
    t.check()
    flat = Step(c, m, 0, seed=17)
    sc = torch.randn((flat.T, 64), generator=torch.Generator().manual_seed(2))
    idx = torch.full((flat.T, 20), -7, dtype=I32, device="cuda")
    dsa.tree_topk(flat.b, sc.cuda(), flat.mask, 20, idx, ws=flat.ws)
    assert flat.status() == 0
    assert np.array_equal(idx.cpu().numpy(), _topk_ref(flat, sc.numpy(), 20))
    kv1 = kv.clone().cuda()
    new = torch.zeros(B, dtype=I32, device="cuda")
    dsa.tree_commit(st.b, st.mask, _dev(m - 1), new, kv1, pages=st.pages, ws=st.ws)
    assert st.status() == 0
    want = [int(c[b]) + (bin(int(st.masks[b][-1])).count("1") if m[b] else 0) for b in range(B)]
    assert new.tolist() == want


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_attention_ignores_what_a_row_does_not_see(bad):
    """A new row with NaN or infinities reaches the rows that see it, and no others."""
    st = Step([200, 131], [9, 2], 32, seed=3)
    q, kv = st.inputs(fill=bad)
    hurt = 4
    kv[int(st.row(0, 200 + hurt)), 5] = bad
    kv[int(st.row(1, 132))] = bad
    out, lse = st.attention(q, kv)
    assert st.status() == 0
    sees = {i for i in range(9) if int(st.masks[0][i]) >> hurt & 1} | {10}
    assert hurt in sees and len(sees) < 10
    check_attention(st, q, kv, out, lse, set(range(11)) - sees)
    if bad != bad:
        for r in sees:
            assert torch.isnan(out[r]).all() and torch.isnan(lse[r]).all()


def test_attention_leaves_other_rows_alone():
    """Rows behind the last sequence, sequences of a bad batch or page, and no lse."""
    st = Step([90, 50, 10], [3, 2, 4], 16, seed=4)
    q, kv = st.inputs()
    st.pages.block_table[1, 2] = st.pool                 # a page that sequence 1 reads
    out, lse = st.attention(q, kv)
    assert st.status() == 7
    assert (out[3:5] == 7).all() and (lse[3:5] == 7).all()
    check_attention(st, q, kv, out, lse, {0, 1, 2, 5, 6, 7, 8})
    dsa.reset_device_status(st.ws)
    st.pages.block_table[1, 2] = int(st.table[1, 2])
    st.b.ctx_len[2] = 3                                   # fewer cached rows than new ones
    out, lse = st.attention(q, kv)
    assert st.status() == 6
    assert (out[5:] == 7).all()
    dsa.reset_device_status(st.ws)
    st.b.ctx_len[2] = 14
    st.b.q_off[3] = 7                                     # fewer rows than total_q: the last two stay
    st.b.ctx_len[2] = 12
    out, _ = st.attention(q, kv, lse=False)
    assert st.status() == 0
    assert (out[7:] == 7).all() and not (out[:7] == 7).all(-1).any()


# ------------------------------------------------------------------- top-k --

def _topk_ref(st, scores, k):
    idx = np.full((st.T, k), -1, np.int32)
    for b in range(st.B):
        for i in range(st.m[b]):
            r = int(st.off[b]) + i
            pos = st.seen(b, i)
            v = scores[r, pos]
            best = np.lexsort((pos, -(v + 0.0)))[:k]
            idx[r, :len(best)] = np.sort(pos[best])
    return idx


@pytest.mark.parametrize("c,m,k", [
    ([0], [1], 1), ([0], [64], 64), ([5, 0], [3, 9], 4), ([2046], [4], 2048), ([2047, 2300, 100], [64, 17, 1], 2048),
    ([9001] * 3, [5, 64, 33], 500), ([70001], [6], 2048), ([40000, 33000], [64, 64], 700),
])
@pytest.mark.parametrize("kind", ["normal", "ties", "inf"])
def test_tree_topk(c, m, k, kind):
    st = Step(c, m, 0, seed=k)
    ld = (st.max_ctx + 3) // 4 * 4
    rng = np.random.default_rng(k)
    sc = rng.standard_normal((st.T, ld)).astype(np.float32)
    if kind == "ties":
        sc = np.round(sc)                                 # many equal scores, both zeros
    elif kind == "inf":
        sc[rng.random(sc.shape) < 0.3] = -np.inf
        sc[rng.random(sc.shape) < 0.01] = np.inf
    for b in range(st.B):                                 # nothing may come from what a row does not see
        for i in range(st.m[b]):
            r = int(st.off[b]) + i
            hide = np.ones(ld, bool)
            hide[st.seen(b, i)] = False
            sc[r, hide] = np.nan
    idx = torch.full((st.T, k), -7, dtype=I32, device="cuda")
    dsa.tree_topk(st.b, torch.from_numpy(sc).cuda(), st.mask, k, idx, ws=st.ws)
    assert st.status() == 0
    assert np.array_equal(idx.cpu().numpy(), _topk_ref(st, sc, k))


_RANGES = {
    "offset": lambda x: 1e4 + x, "far": lambda x: 1e7 + x, "outlier": lambda x: np.where(x == x[0, 3], 1e30, x),
    "span": lambda x: np.clip(x, -3, 3) * 1.1e38, "tiny": lambda x: x * 1e-42,
    "lowest": lambda x: -3.4e38 * (1 - 1e-3 * np.abs(x) / 8),
}


@pytest.mark.parametrize("c,m,k", [
    ([700] * 5, [64] * 5, 333), ([11000] * 5, [64] * 5, 2047), ([26000] * 3, [60] * 3, 1001), ([900], [5], 30),
    ([20000], [5], 2048), ([255, 256, 257, 64], [64, 1, 63, 64], 250), ([50000], [3], 2046),
    ([30000, 3000, 29000, 8191], [9, 9, 5, 1], 2047), ([25000] * 7, [10] * 7, 100),
])
@pytest.mark.parametrize("kind", list(_RANGES))
def test_tree_topk_ranges(c, m, k, kind):
    """Scores whose range an even division does not fit, at row lengths and counts of every kernel; exact."""
    st = Step(c, m, 0, seed=k)
    ld = (st.max_ctx + 3) // 4 * 4
    x = np.random.default_rng(k).standard_normal((st.T, ld))
    sc = _RANGES[kind](x).astype(np.float32)
    assert np.isfinite(sc).all()
    idx = torch.full((st.T, k), -7, dtype=I32, device="cuda")
    dsa.tree_topk(st.b, torch.from_numpy(sc).cuda(), st.mask, k, idx, ws=st.ws)
    assert st.status() == 0
    assert np.array_equal(idx.cpu().numpy(), _topk_ref(st, sc, k))


@pytest.mark.parametrize("c,m,k", [([100000, 5000, 70000], [64, 64, 64], 1000), ([400000], [2], 2048),
                                   ([50000, 100], [64, 64], 7), ([99000] * 5, [62, 64, 1, 64, 64], 2048)])
@pytest.mark.parametrize("ties", [False, True])
def test_tree_topk_long(c, m, k, ties):
    """Rows longer than a CTA holds: clusters of every size, and the kernel that keeps candidates only."""
    st = Step(c, m, 0, seed=k)
    ld = (st.max_ctx + 3) // 4 * 4
    g = torch.Generator().manual_seed(k)
    sc = torch.randn((st.T, ld), generator=g)
    sc = sc.mul_(30).round_().div_(30) if ties else sc
    idx = torch.full((st.T, k), -7, dtype=I32, device="cuda")
    dsa.tree_topk(st.b, sc.cuda(), st.mask, k, idx, ws=st.ws)
    assert st.status() == 0
    rows = [0, 1, st.T // 2, st.T - 1]
    for r in rows:
        b = int(np.searchsorted(st.off, r, side="right")) - 1
        pos = st.seen(b, r - int(st.off[b]))
        v = sc[r].numpy()[pos]
        best = np.sort(pos[np.lexsort((pos, -(v + 0.0)))[:k]])
        assert np.array_equal(idx[r].cpu().numpy(), np.pad(best, (0, k - len(best)), constant_values=-1))
    # the others against a sort on the device
    own = torch.tensor([b for b in range(st.B) for _ in range(st.m[b])])
    for r in range(st.T):
        b = int(own[r])
        pos = torch.from_numpy(np.asarray(st.seen(b, r - int(st.off[b])))).cuda()
        v = sc[r].cuda()[pos] + 0.0
        best = pos[v.sort(descending=True, stable=True).indices[:k]].sort().values
        assert torch.equal(idx[r, :len(best)].long(), best.long()) and (idx[r, len(best):] == -1).all()


@pytest.mark.parametrize("B,longest", [(3, 2500), (40, 2500), (3, 30000)])
def test_tree_topk_right_behind_the_tables(B, longest):
    """Lengths and masks that the launch just before writes, changing from call to call."""
    rng = np.random.default_rng(B)
    m, T, k = 8, 8 * B, 100
    q_off, ctx = torch.zeros(B + 1, dtype=I32, device="cuda"), torch.zeros(B, dtype=I32, device="cuda")
    b = dsa.make_batch(q_off, ctx, m, longest + m, longest + m, total_q=T)
    ws = dsa.tree_workspace(b)
    slots, pos = (torch.zeros(T, dtype=I32, device="cuda") for _ in range(2))
    mask = torch.zeros(T, dtype=torch.int64, device="cuda")
    sc = torch.randn((T, (longest + m + 3) // 4 * 4), device="cuda")
    steps = []
    for _ in range(6):
        n = rng.integers(0, m + 1, B)
        par = np.full(T, -1, np.int32)
        at = 0
        for x in n:
            for i in range(x):
                par[at + i] = rng.integers(-1, i) if i else -1
            at += x
        steps.append((_dev(n.tolist()), _dev(rng.integers(0, longest + 1, B).tolist()), _dev(par.tolist())))

    def run(s, idx):
        dsa.step_tables(b, s[0], s[1], slots, pos, mask, parent=s[2], ws=ws)
        dsa.tree_topk(b, sc, mask, k, idx, ws=ws)
    want = []
    for s in steps:
        idx = torch.full((T, k), -7, dtype=I32, device="cuda")
        torch.cuda.synchronize()
        dsa.step_tables(b, s[0], s[1], slots, pos, mask, parent=s[2], ws=ws)
        torch.cuda.synchronize()
        dsa.tree_topk(b, sc, mask, k, idx, ws=ws)
        torch.cuda.synchronize()
        want.append(idx)
    order = rng.integers(0, len(steps), 300)
    got = torch.full((len(order), T, k), -7, dtype=I32, device="cuda")
    torch.cuda.synchronize()
    for x, s in enumerate(order):
        run(steps[s], got[x])
    assert dsa.read_device_status(ws) == 0
    for x, s in enumerate(order):
        assert torch.equal(got[x], want[s]), x


def test_tree_topk_from_two_threads():
    """Calls of two host threads, each with a stream and a workspace: long rows beside short ones."""
    import threading
    steps = [Step([20000], [2], 0, seed=1), Step([24000], [2], 0, seed=2)]
    wanted, jobs, wrong = [], [], []
    for st in steps:
        sc = torch.randn((st.T, (st.max_ctx + 3) // 4 * 4), generator=torch.Generator().manual_seed(st.max_ctx)).cuda()
        idx = torch.empty((st.T, 500), dtype=I32, device="cuda")
        dsa.tree_topk(st.b, sc, st.mask, 500, idx, ws=st.ws)
        wanted.append(idx.clone())
        jobs.append((st, sc, idx))
    torch.cuda.synchronize()

    def work(n):
        st, sc, idx = jobs[n]
        try:
            stream = torch.cuda.Stream()
            for _ in range(2000):
                dsa.tree_topk(st.b, sc, st.mask, 500, idx, ws=st.ws, stream=stream)
            stream.synchronize()
        except Exception as e:
            wrong.append(e)
    threads = [threading.Thread(target=work, args=(n,)) for n in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    for (st, _, idx), w in zip(jobs, wanted):
        assert st.status() == 0 and torch.equal(idx, w)


def test_tree_topk_of_a_chain_is_topk():
    st = Step([3000, 12], [7, 20], 0, masks=[[(2 << i) - 1 for i in range(n)] for n in (7, 20)])
    ld = (st.max_ctx + 3) // 4 * 4
    sc = torch.randn((st.T, ld), device="cuda")
    a, b = (torch.empty((st.T, 300), dtype=I32, device="cuda") for _ in range(2))
    dsa.tree_topk(st.b, sc, st.mask, 300, a, ws=st.ws)
    dsa.topk(st.b, sc, 300, b, ws=dsa.workspace(st.b, 300))
    assert torch.equal(a, b)


# ------------------------------------------------------------------ commit --

@pytest.mark.parametrize("page", [0, 16, 64])
@pytest.mark.parametrize("layers,inplace", [(1, False), (3, True)])
def test_commit(page, layers, inplace):
    rng = np.random.default_rng(page + layers)
    m = [1, 9, 64, 64, 17, 0, 30, 5]
    c = [0, 15, 40, 100, 1, 7, 63, 16]
    st = Step(c, m, page, seed=11)
    node = [0, 8, 63, 40, -1, -1, 29, 3]
    masks = [list(x) for x in st.masks]
    masks[3][40] = (1 << 41) - 1                           # a chain: nothing moves
    masks[2][63] = int(rng.integers(0, 1 << 62)) << 2 | 3 << 62
    masks[6][29] = 0                                       # a node that sees nothing
    st.mask = torch.tensor(signed([x for r in masks for x in r]), dtype=torch.int64).cuda()
    kv = torch.randn((layers, st.rows, D_QK)).to(torch.bfloat16)
    ki = torch.randn((layers, st.rows, D_IDX)).to(torch.bfloat16)
    want_kv, want_ki, want = kv.clone(), ki.clone(), []
    for b in range(st.B):
        path = [j for j in range(node[b] + 1) if int(masks[b][node[b]]) >> j & 1] if node[b] >= 0 else []
        for i, j in enumerate(path):
            to, of = int(st.row(b, c[b] + i)), int(st.row(b, c[b] + j))
            want_kv[:, to], want_ki[:, to] = kv[:, of], ki[:, of]
        want.append(c[b] + len(path))
    dkv, dki = kv.cuda(), ki.cuda()
    new = st.b.ctx_len if inplace else torch.full((st.B,), -3, dtype=I32, device="cuda")
    dsa.tree_commit(st.b, st.mask, _dev(node), new, dkv, dki, pages=st.pages, ws=st.ws)
    assert st.status() == 0
    assert new.tolist() == want
    assert torch.equal(dkv.cpu(), want_kv) and torch.equal(dki.cpu(), want_ki)


@pytest.mark.parametrize("inplace", [False, True])
def test_commit_refuses_a_sequence(inplace):
    st = Step([20, 30, 40], [4, 5, 6], 16, seed=1, masks=[[1, 2, 5, 9], [1, 2, 4, 8, 17], [1, 2, 4, 8, 16, 41]])
    kv = torch.randn((1, st.rows, D_QK)).to(torch.bfloat16).cuda()
    was = kv.clone()
    new = st.b.ctx_len if inplace else torch.zeros(3, dtype=I32, device="cuda")
    st.pages.block_table[1, 2] = -1                        # position 34 of sequence 1, on its path
    dsa.tree_commit(st.b, st.mask, _dev([4, 4, 5]), new, kv, pages=st.pages, ws=st.ws)
    assert st.status() == 7
    assert new.tolist() == [20, 30, 43]
    moved = [int(st.row(2, 41)), int(st.row(2, 42))]
    assert torch.equal(kv[0, moved[0]], was[0, int(st.row(2, 43))])
    assert torch.equal(kv[0, moved[1]], was[0, int(st.row(2, 45))])
    kv[0, moved] = was[0, moved]
    assert torch.equal(kv, was)
    # index keys alone, and lengths alone
    new2 = torch.zeros(3, dtype=I32, device="cuda")
    st2 = Step([20], [3], 0, seed=1, masks=[[1, 2, 5]])
    ki = torch.randn((st2.rows, D_IDX)).to(torch.bfloat16).cuda()
    was = ki.clone()
    dsa.tree_commit(st2.b, st2.mask, _dev([2]), new2, k_idx=ki, ws=st2.ws)
    assert torch.equal(ki[21], was[22]) and int(new2[0]) == 22
    dsa.tree_commit(st2.b, st2.mask, _dev([1]), new2, ws=st2.ws)
    assert int(new2[0]) == 21 and st2.status() == 0


def test_commit_refuses_other_shapes():
    st = Step([20], [3], 0, seed=1, masks=[[1, 2, 5]])
    new = torch.zeros(1, dtype=I32, device="cuda")
    kv, ki = (torch.zeros((2, st.rows, w), dtype=torch.bfloat16, device="cuda") for w in (D_QK, D_IDX))
    for bad in (dict(kv=kv[None]), dict(kv=kv.view(-1)), dict(kv=ki), dict(k_idx=kv), dict(kv=kv, k_idx=ki[0]),
                dict(kv=kv, k_idx=ki.view(1, -1, D_IDX)), dict(kv=kv[:, :, :D_IDX])):
        with pytest.raises(ValueError):
            dsa.tree_commit(st.b, st.mask, _dev([2]), new, ws=st.ws, **bad)
    with pytest.raises(dsa.DsaError):                      # fewer cache rows than the batch spans
        dsa.tree_commit(st.b, st.mask, _dev([2]), new, kv=kv[0, :-1], ws=st.ws)
    assert st.status() == 0 and not kv.any() and int(new[0]) == 0


@pytest.mark.parametrize("inplace", [False, True])
def test_calls_of_a_step_without_tokens(inplace):
    """No new token in any sequence: every call returns, and the lengths stay."""
    ctx = _dev([5, 0, 30])
    b = dsa.make_batch(torch.zeros(4, dtype=I32, device="cuda"), ctx, 4, 40, 40, total_q=0)
    ws = dsa.tree_workspace(b)
    kv = torch.randn((120, D_QK), device="cuda").to(torch.bfloat16)
    was = kv.clone()

    def none(*shape, dtype=torch.bfloat16):
        return torch.empty((0,) + shape, dtype=dtype, device="cuda")
    mask = none(dtype=torch.int64)
    dsa.latent_append(none(D_QK), torch.ones(D_V, device="cuda"), 1e-5, torch.ones((40, 64), device="cuda"),
                      torch.ones((40, 64), device="cuda"), none(dtype=I32), none(dtype=I32), kv, ws)
    dsa.tree_mla_fwd(b, none(64, D_QK), kv, mask, 0.06, none(64, D_V), none(64, dtype=torch.float32), ws=ws)
    dsa.tree_topk(b, none(40, dtype=torch.float32), mask, 8, none(8, dtype=I32), ws=ws)
    new = ctx if inplace else torch.zeros(3, dtype=I32, device="cuda")
    dsa.tree_commit(b, mask, _dev([-1, -1, -1]), new, kv=kv, ws=ws)
    assert dsa.read_device_status(ws) == 0
    assert new.tolist() == [5, 0, 30] and torch.equal(kv, was)


# ------------------------------------------------- the step, as it is used --

class Server:
    """Two decoding steps of a paged server: tables -> append -> attention -> commit."""

    def __init__(self, seed, B=5, page=16, pool=200):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.B, self.page, self.pool, self.T = B, page, pool, 8 * B
        self.kv = torch.zeros((pool * page, D_QK), dtype=torch.bfloat16, device="cuda")
        ang = torch.rand((2000, 64), generator=g) * 6.28
        self.cos, self.sin = ang.cos().cuda(), ang.sin().cuda()
        self.gamma = (1 + 0.1 * torch.randn(D_V, generator=g)).cuda()
        self.q_off, self.ctx = torch.zeros(B + 1, dtype=I32, device="cuda"), torch.zeros(B, dtype=I32, device="cuda")
        self.held = torch.zeros(B, dtype=I32, device="cuda")
        self.range = _dev([0, pool])
        self.free = _dev(rng.permutation(pool))
        self.pages = dsa.make_pages(torch.full((B, 40), -1, dtype=I32, device="cuda"), page, pool)
        self.batch = dsa.Batch(self.q_off, self.ctx, 8, 600, 600, total_q=self.T)
        self.ws = dsa.tree_workspace(self.batch)
        e = lambda d: torch.zeros(self.T, dtype=d, device="cuda")  # noqa: E731
        self.slots, self.pos, self.mask, self.parent = e(I32), e(I32), e(torch.int64), e(I32)
        self.n, self.accepted = torch.zeros(B, dtype=I32, device="cuda"), torch.zeros(B, dtype=I32, device="cuda")
        self.x = torch.zeros((self.T, D_QK), dtype=torch.bfloat16, device="cuda")
        self.q = torch.zeros((self.T, H, D_QK), dtype=torch.bfloat16, device="cuda")
        self.out = torch.zeros((self.T, H, D_V), dtype=torch.bfloat16, device="cuda")
        self.lse = torch.zeros((self.T, H), dtype=torch.float32, device="cuda")
        self.rng, self.hist = rng, [[] for _ in range(B)]

    def load(self, seed):
        """A step's host data: lengths, trees, inputs and what will be accepted."""
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.m = rng.integers(1, 9, self.B)
        self.par = [parents_np(int(n), rng) for n in self.m]
        flat = [p for x in self.par for p in x]
        self.n.copy_(_dev(self.m))
        self.parent.copy_(_dev(flat + [-1] * (self.T - len(flat))))
        self.acc = np.array([int(rng.integers(-1, n)) for n in self.m])
        self.accepted.copy_(_dev(self.acc))
        self.xh = torch.randn((self.T, D_QK), generator=g).to(torch.bfloat16)
        self.qh = torch.randn((self.T, H, D_QK), generator=g).to(torch.bfloat16)
        self.x.copy_(self.xh)
        self.q.copy_(self.qh)

    def step(self):
        dsa.step_tables(self.batch, self.n, self.ctx, self.slots, self.pos, mask=self.mask, parent=self.parent,
                        pages=self.pages, n_pages_old=self.held, n_pages=self.held, free_pages=self.free,
                        free_range=self.range, free_range_out=self.range, ws=self.ws)
        dsa.latent_append(self.x, self.gamma, 1e-5, self.cos, self.sin, self.pos, self.slots, self.kv, ws=self.ws)
        dsa.tree_mla_fwd(self.batch, self.q, self.kv, self.mask, SCALE, self.out, self.lse, pages=self.pages,
                         ws=self.ws)
        dsa.tree_commit(self.batch, self.mask, self.accepted, self.ctx, self.kv, pages=self.pages, ws=self.ws)

    def check(self):
        """Against a cache kept as lists of rows per sequence, in 64 bits from the same bf16 rows."""
        assert dsa.read_device_status(self.ws) == 0
        r = 0
        cos, sin, gamma = self.cos.cpu().double(), self.sin.cpu().double(), self.gamma.cpu().double()
        for b in range(self.B):
            masks = mask_of(self.par[b])
            rows = []
            for i in range(self.m[b]):
                z = self.xh[r + i].double()
                p = len(self.hist[b]) + bin(masks[i]).count("1") - 1
                lat = z[:D_V] / torch.sqrt((z[:D_V] ** 2).mean() + 1e-5) * gamma
                pe, c, s = z[D_V:], cos[p], sin[p]
                rot = torch.cat([pe[:32] * c[:32] - pe[32:] * s[:32], pe[32:] * c[32:] + pe[:32] * s[32:]])
                rows.append(torch.cat([lat, rot]))
            for i in range(self.m[b]):
                k = torch.stack(self.hist[b] + [rows[j] for j in range(i + 1) if masks[i] >> j & 1])
                z = self.qh[r + i].double() @ k.T * SCALE
                l = torch.logsumexp(z, -1)
                w = torch.exp(z - l[:, None])
                o, a = w @ k[:, :D_V], w @ k[:, :D_V].abs()
                # the cache rows are rounded too: a logit moves by at most HALF sum|qk| <= HALF |q||k|
                # (Cauchy-Schwarz), every weight by e^2d after normalising, every value by HALF
                d = HALF * SCALE * (self.qh[r + i].double().norm(dim=-1)[:, None] * k.norm(dim=-1)).amax(-1) + 1e-5
                tol = HALF * o.abs() + (2 * HALF + torch.expm1(2 * d)[:, None]) * 1.01 * a
                got = self.out[r + i].cpu().double()
                assert ((got - o).abs() <= tol).all(), (b, i)
                assert ((self.lse[r + i].cpu().double() - l).abs() <= d + 1e-5).all(), (b, i)
            if self.acc[b] >= 0:
                self.hist[b] += [rows[j] for j in range(self.acc[b] + 1) if masks[self.acc[b]] >> j & 1]
            r += int(self.m[b])
        assert self.ctx.tolist() == [len(h) for h in self.hist]


def test_steps_together():
    s = Server(1)
    for k in range(6):
        s.load(100 + k)
        s.step()
        s.check()


def test_steps_captured_and_replayed():
    """One graph serves every step: lengths, pages and trees change on the device."""
    s = Server(2)
    s.load(7)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.step()
    torch.cuda.current_stream().wait_stream(side)
    s.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.step()
    for k in range(4):
        s.load(300 + k)
        graph.replay()
        s.check()


def test_two_streams_at_once():
    servers = [Server(11, B=3), Server(12, B=7)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for k in range(3):
        for s in servers:
            s.load(500 + 10 * k + s.B)
        torch.cuda.synchronize()
        for s, st in zip(servers, streams):
            with torch.cuda.stream(st):
                s.step()
        torch.cuda.synchronize()
        for s in servers:
            s.check()


def test_a_stream_of_the_caller():
    st = Step([300, 41], [4, 7], 16, seed=22)
    q, kv = st.inputs()
    q, kv = q.cuda(), kv.cuda()
    out = torch.full((st.T, H, D_V), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((st.T, H), 7.0, dtype=torch.float32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    dsa.tree_mla_fwd(st.b, q, kv, st.mask, SCALE, out, lse, pages=st.pages, ws=st.ws, stream=side)
    side.synchronize()
    assert dsa.read_device_status(st.ws, stream=side) == 0
    check_attention(st, q.cpu(), kv.cpu(), out, lse)


def test_same_bits_every_time():
    st = Step([5000, 100, 2047, 0], [3, 64, 1, 9], 64, seed=21)
    q, kv = st.inputs()
    q, kv = q.cuda(), kv.cuda()
    first = st.attention(q, kv)
    for _ in range(3):
        again = st.attention(q, kv)
        assert torch.equal(first[0].view(torch.int16), again[0].view(torch.int16))
        assert torch.equal(first[1].view(I32), again[1].view(I32))


def test_dsa_of_a_tree():
    """indexer scores -> tree top-k -> sparse attention equals the dense tree
    attention while every visible position is selected, and the 64-bit
    attention over the selection when not."""
    st = Step([300, 90], [9, 20], 0, seed=31)
    q, kv = st.inputs()
    g = torch.Generator().manual_seed(5)
    qi = (torch.randn((st.T, 32, 128), generator=g) / 11).to(torch.bfloat16).cuda()
    ki = (torch.randn((st.rows, 128), generator=g) / 11).to(torch.bfloat16).cuda()
    w = (torch.randn((st.T, 32), generator=g) / 6).cuda()
    ld = (st.max_ctx + 3) // 4 * 4
    sc = torch.zeros((st.T, ld), device="cuda")
    for k in (512, 64):
        ws = dsa.workspace(st.b, k)
        idx = torch.empty((st.T, k), dtype=I32, device="cuda")
        out = torch.empty((st.T, H, D_V), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((st.T, H), device="cuda")
        dsa.indexer_scores(st.b, qi, w, ki, sc, ws=ws)
        dsa.tree_topk(st.b, sc, st.mask, k, idx, ws=ws)
        dsa.sparse_mla_fwd(st.b, q.cuda(), kv.cuda(), idx, k, SCALE, out, lse, ws=ws)
        assert dsa.read_device_status(ws) == 0
        assert np.array_equal(idx.cpu().numpy(), _topk_ref(st, sc.cpu().numpy(), k))
        if k == 512:
            check_attention(st, q, kv, out, lse)
        else:
            sel = idx.cpu().numpy()
            chosen = Step(st.c, st.m, 0, seed=31, stride=st.stride)
            where = [(b, i) for b in range(st.B) for i in range(st.m[b])]
            chosen.seen = lambda b, i: sel[where.index((b, i))][sel[where.index((b, i))] >= 0].astype(np.int64)
            check_attention(chosen, q, kv, out, lse)

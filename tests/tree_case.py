"""Seeded steps of drafted tokens over a cache, and their 64-bit references
(numpy / torch on the CPU, written from the definitions)."""

from __future__ import annotations

import numpy as np
import torch

import sparse_attention_gb300 as dsa

H, D_QK, D_V, D_IDX = 64, 576, 512, 128
SCALE = 1.0 / 16.0
HALF = 2.0 ** -8            # half a step of bf16, relative
F32 = 2.0 ** -24


def parents_np(n, rng, reach=8):
    return [-1] + [int(i - 1 - rng.integers(min(i, reach))) for i in range(1, n)] if n else []


def mask_of(parents):
    bits = []
    for i, p in enumerate(parents):
        bits.append((1 << i) | (bits[p] if p >= 0 else 0))
    return bits


def signed(bits):
    return [int(x) - (1 << 64) if int(x) >> 63 else int(x) for x in bits]


class Step:
    """c[b] committed and m[b] new rows; page 0 = contiguous caches."""

    def __init__(self, c, m, page=0, seed=0, masks=None, stride=None, spare=3, dev="cuda"):
        self.rng = rng = np.random.default_rng(seed)
        self.c, self.m, self.page, self.dev = list(c), list(m), page, dev
        self.B = len(self.c)
        self.off = np.concatenate([[0], np.cumsum(self.m)]).astype(np.int64)
        self.T = int(self.off[-1])
        self.L = [x + y for x, y in zip(self.c, self.m)]
        self.parents = [parents_np(n, rng) for n in self.m]
        self.masks = masks if masks is not None else [mask_of(p) for p in self.parents]
        self.max_ctx = max(max(self.L), 1)
        self.stride = stride or self.max_ctx
        if page:
            held = [-(-x // page) for x in self.L]
            self.pool = sum(held) + spare
            order = rng.permutation(self.pool)
            self.table = np.full((self.B, max(max(held), 1)), -1, np.int32)
            at = 0
            for b, h in enumerate(held):
                self.table[b, :h] = order[at:at + h]
                at += h
            self.rows = self.pool * page
        else:
            self.table, self.pool, self.rows = None, 0, self.B * self.stride
        self.mask = torch.tensor(signed([x for r in self.masks for x in r]), dtype=torch.int64).to(dev)
        self.b = dsa.make_batch(self.off.astype(np.int32), np.array(self.L, np.int32), max(max(self.m), 0),
                                self.max_ctx, self.stride, total_q=self.T, device=dev)
        self.pages = dsa.make_pages(torch.from_numpy(self.table).to(dev), page, self.pool) if page else None
        self.ws = dsa.tree_workspace(self.b, device=dev)

    def row(self, b, s):
        s = np.asarray(s)
        if not self.page:
            return b * self.stride + s
        return self.table[b][s // self.page].astype(np.int64) * self.page + s % self.page

    def seen(self, b, i):
        """Positions that new row i of sequence b sees."""
        bits = int(self.masks[b][i]) & ((2 << i) - 1)
        return np.array(list(range(self.c[b])) + [self.c[b] + j for j in range(self.m[b]) if bits >> j & 1], np.int64)

    def inputs(self, seed=1, fill=float("nan")):
        """q and a cache whose rows outside every sequence hold `fill`."""
        g = torch.Generator().manual_seed(seed)
        q = torch.randn((self.T, H, D_QK), generator=g).to(torch.bfloat16)
        kv = torch.randn((self.rows, D_QK), generator=g).to(torch.bfloat16)
        used = np.zeros(self.rows, bool)
        for b in range(self.B):
            if self.L[b]:
                used[self.row(b, np.arange(self.L[b]))] = True
        kv[~torch.from_numpy(used)] = fill
        return q, kv

    def attention(self, q, kv, sm_scale=SCALE, lse=True):
        out = torch.full((self.T, H, D_V), 7.0, dtype=torch.bfloat16, device=self.dev)
        ls = torch.full((self.T, H), 7.0, dtype=torch.float32, device=self.dev) if lse else None
        dsa.tree_mla_fwd(self.b, q.to(self.dev), kv.to(self.dev), self.mask, sm_scale, out, ls, pages=self.pages,
                         ws=self.ws)
        return out, ls

    def status(self):
        return dsa.read_device_status(self.ws)


def attention_ref(st: Step, q, kv, sm_scale=SCALE, rows=None):
    """(out, lse, tol_out, tol_lse) of packed rows, in 64 bits.

    Tolerance.  The result is rounded to bf16 (HALF |out|), and so is every
    softmax weight before it meets its value row (HALF sum p|v|).  Scores are
    fp32 sums of 576 exact products: off by at most 576 F32 sum|q k|, and a
    logit off by d moves every weight by at most a factor e^d, so out by
    2 d sum p|v| and lse by d; sums of n weights add n F32, the exponential
    and the merge of partial results a few F32 more (16 is ample)."""
    out, lse, to, tl = [], [], [], []
    for b in range(st.B):
        for i in range(st.m[b]):
            r = int(st.off[b]) + i
            if rows is not None and r not in rows:
                continue
            pos = st.seen(b, i)
            if len(pos) == 0:
                out.append(torch.zeros((H, D_V), dtype=torch.float64))
                lse.append(torch.full((H,), -np.inf, dtype=torch.float64))
                to.append(torch.zeros((H, D_V), dtype=torch.float64))
                tl.append(torch.zeros((H,), dtype=torch.float64))
                continue
            k = kv[torch.from_numpy(st.row(b, pos))].double()
            x = q[r].double()
            z = x @ k.T * sm_scale
            l = torch.logsumexp(z, -1)
            p = torch.exp(z - l[:, None])
            o = p @ k[:, :D_V]
            a = p @ k[:, :D_V].abs()
            d = 576 * F32 * sm_scale * (x.abs() @ k.abs().T).amax(-1)
            n = (len(pos) + 16) * F32
            out.append(o)
            lse.append(l)
            to.append(HALF * o.abs() + (HALF + 2 * (d[:, None] + n)) * a)
            tl.append(d + n + 4 * F32 * l.abs())
    return tuple(torch.stack(x) for x in (out, lse, to, tl))


def check_attention(st: Step, q, kv, out, lse, rows=None, sm_scale=SCALE):
    o, l, to, tl = attention_ref(st, q, kv, sm_scale, rows)
    pick = slice(None) if rows is None else sorted(rows)
    got = out.cpu()[pick].double()
    err = (got - o).abs() - to
    assert not torch.isnan(got).any(), "NaN in the output"
    assert err.max() <= 0, f"output off by {err.max():.3g} over its tolerance"
    if lse is not None:
        g = lse.cpu()[pick].double()
        empty = torch.isinf(l)
        assert torch.equal(torch.isinf(g), empty) and (g[empty] < 0).all()
        assert ((g - l).abs()[~empty] <= tl[~empty]).all(), f"lse off by {(g - l).abs()[~empty].max():.3g}"

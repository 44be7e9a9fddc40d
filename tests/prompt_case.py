"""Seeded prompts over latent caches and their expanded rows, and 64-bit
references (numpy / torch on the CPU, written from the definitions)."""

from __future__ import annotations

import numpy as np
import torch

import sparse_attention_gb300 as dsa

H, D_QK, D_LAT, D_NOPE, D_ROPE, D_HEAD, D_EXP = 64, 576, 512, 192, 64, 256, 448
SCALE = 1.0 / 16.0
HALF = 2.0 ** -8            # half a step of bf16, relative
F32 = 2.0 ** -24
ROOM = 128


def up(x, to=ROOM):
    return -(-x // to) * to


class Prompts:
    """c[b] kept and m[b] new rows; page 0 = contiguous caches."""

    def __init__(self, c, m, page=0, seed=0, gap=0, dev="cuda", max_q=None, max_ctx=None, pad=0):
        self.c, self.m, self.page, self.dev = list(c), list(m), page, dev
        self.B, self.gen = len(self.c), torch.Generator().manual_seed(seed)
        self.L = [x + y for x, y in zip(c, m)]
        self.off = np.concatenate([[0], np.cumsum(self.m)]).astype(np.int64)
        self.T = int(self.off[-1])
        self.max_ctx = max(max(self.L), 1) if max_ctx is None else max_ctx
        self.max_q = max(self.m) if max_q is None else max_q
        self.stride = self.max_ctx + 3
        room = [up(x) + gap for x in self.L]
        self.at = np.concatenate([[0], np.cumsum(room)]).astype(np.int64)
        self.rows_x = int(self.at[-1]) + pad
        self.i32 = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32).to(dev)
        self.batch = dsa.make_batch(self.i32(self.off), self.i32(self.L), self.max_q, self.max_ctx, self.stride,
                                    total_q=self.T + pad, device=dev)
        self.x_off = self.i32(self.at)
        if page:
            need = [-(-x // page) for x in self.L]
            self.pool = sum(need) + 2
            order = torch.randperm(self.pool, generator=self.gen).to(torch.int32)
            self.table = torch.full((self.B, max(max(need), -(-self.max_ctx // page), 1)), -1, dtype=torch.int32)
            at = 0
            for b, n in enumerate(need):
                self.table[b, :n] = order[at:at + n]
                at += n
            self.pages = dsa.make_pages(self.table.to(dev), page, self.pool)
            self.cache_rows = self.pool * page
        else:
            self.table, self.pages, self.cache_rows = None, None, self.B * self.stride
        self.ws = dsa.prompt_workspace(self.batch, device=dev)

    def normal(self, *shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=self.gen).to(dtype)

    def slots(self, b, lo, hi):
        """Cache rows of positions lo .. hi - 1 of sequence b."""
        p = torch.arange(lo, hi)
        if self.table is None:
            return b * self.stride + p
        return self.table[b].long()[p // self.page] * self.page + p % self.page

    def buffers(self, fill=float("nan")):
        """Expanded buffers that hold `fill` throughout."""
        kv = torch.full((self.rows_x, H, D_EXP), fill, dtype=torch.bfloat16, device=self.dev)
        k_pe = torch.full((self.rows_x, D_ROPE), fill, dtype=torch.bfloat16, device=self.dev)
        return dsa.make_expanded(self.x_off, kv, k_pe)

    def filled(self):
        """Random expanded rows, zeros behind each sequence, NaN in the rest."""
        x = self.buffers()                       # NaN
        for b in range(self.B):
            lo, n = int(self.at[b]), self.L[b]
            x.kv[lo:lo + n] = self.normal(n, H, D_EXP).to(self.dev)
            x.k_pe[lo:lo + n] = self.normal(n, D_ROPE).to(self.dev)
            x.kv[lo + n:lo + up(n, 16)] = 0
        return x


def expand_ref(rows, w):
    """rows [n, 576], w [64 * 448, 512] -> [n, 64, 448] and the products' sizes, in 64 bits."""
    c, w = rows[:, :D_LAT].double(), w.double()
    return (c @ w.t()).view(-1, H, D_EXP), (c.abs() @ w.abs().t()).view(-1, H, D_EXP)


def attention_ref(P, q, x, b, heads=range(H), rows=None):
    """out [n, heads, 256], lse and the largest |v| a row weighs, in 64 bits, for the new rows `rows` (all) of sequence b."""
    lo, n, c = int(P.at[b]), P.m[b], P.c[b]
    rows = torch.arange(n) if rows is None else torch.as_tensor(rows)
    q = q[int(P.off[b]):int(P.off[b]) + n].cpu()[rows].double()
    kv, pe = x.kv[lo:lo + P.L[b]].cpu(), x.k_pe[lo:lo + P.L[b]].cpu().double()
    seen = torch.arange(P.L[b])[None, :] <= (c + rows)[:, None]
    out, lse, big = [], [], []
    for h in heads:
        k = torch.cat([kv[:, h, :D_NOPE].double(), pe], 1)
        v = kv[:, h, D_NOPE:].double()
        s = torch.where(seen, q[:, h] @ k.t() * SCALE, float("-inf"))
        z = torch.logsumexp(s, -1)
        p = torch.exp(s - z[:, None])
        out.append(p @ v)
        big.append(p @ v.abs())
        lse.append(z)
    return torch.stack(out, 1), torch.stack(lse, 1), torch.stack(big, 1)


def check_attention(P, q, x, out, lse, heads=range(H), rows=None):
    """Scores are fp32 sums of 256 exact products in some order, each partial
    sum rounded: off by up to 256 F32 times the sum of the products' sizes,
    some 256 * 0.8^2 / 16 = 10 after scaling for N(0, 1) values (20 allowed); an
    error e of the scores moves weights by 2 e relative, and lse by e.  Weights
    are rounded to bf16 (HALF) and the result again; ex2 has 2 ulp, and the sums over
    positions again add some steps.  A maximum that lags by up to 2^8 costs nothing
    relative."""
    heads = list(heads)
    for b in range(P.B):
        if P.m[b] == 0:
            continue
        pick = None if rows is None else [r for r in rows if r < P.m[b]]
        if pick == []:
            continue
        ref, z, big = attention_ref(P, q, x, b, heads, pick)
        at = int(P.off[b]) + (torch.arange(P.m[b]) if pick is None else torch.as_tensor(pick))
        got = out.cpu()[at][:, heads].double()
        e = 256 * F32 * 20
        err = (got - ref).abs()
        tol = HALF * ref.abs() + (HALF * (1 + HALF) + 2 * e + 64 * F32) * big
        assert (err <= tol).all(), (b, (err / tol).max())
        if lse is not None:
            el = (lse.cpu()[at][:, heads].double() - z).abs()
            assert (el <= e + 16 * F32 * (1 + z.abs())).all(), (b, el.max())

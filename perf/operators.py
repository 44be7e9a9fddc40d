"""One step of drafted tokens over a cache: the operators' cases, their plain
forms and the framework's calls.

Sequence b holds c_b committed cache rows and gets n_b new ones; new row i of
sequence b is packed row q_off[b] + i and sits at cache position c_b + i.  Row
r sees every committed position and the new rows j of its own sequence whose
bit is set in mask[r].

  tables  lengths (and parent links) -> q_off, ctx_len, block table, slot map,
          rotary positions, visibility masks
  append  compressed KV projections -> RMSNorm | RoPE -> cache rows at slots
  attn    64-head latent attention of every new row over what it sees
  topk    the k best-scored positions of what every new row sees
  commit  the accepted path's rows moved behind the committed ones
"""

import math
import random

import torch

own = False

H, D_QK, D_V, D_IDX = 64, 576, 512, 128
SCALE = 1.0 / 16.0
EPS = 1e-5


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # a speculative step of a busy server: 64 requests, up to 16 drafted tokens each, pages of 64 rows
        dict(name="tables-tree-b64-n16", op="tables", b=64, n=16, ctx=8192, page=64, tree=True),
        # a prefill wave: 256 prompts of ragged lengths, 65,536 tokens at most, pages of 16 rows
        dict(name="tables-prompts-b256", op="tables", b=256, n=256, ctx=0, page=16, tree=False),
        # latent rows of a decode batch (64 tokens) and of a prefill chunk (8,192 tokens)
        dict(name="append-decode-t64", op="append", t=64, page=64, wide=0),
        dict(name="append-chunk-t8192", op="append", t=8192, page=64, wide=2048),
        # one request with a small tree over a short context: the smallest call, where latency counts
        dict(name="attn-one-b1-n8-ctx1500", op="attn", b=1, n=8, ctx=1500, page=64, ragged=False),
        # plain decode: one token for each of 64 sequences of 32,768 cached rows, contiguous caches
        dict(name="attn-decode-b64-ctx32768", op="attn", b=64, n=1, ctx=32767, page=0, ragged=False),
        # a served batch of odd trees and ragged contexts in pages of 16 rows
        dict(name="attn-ragged-b24-n13-ctx7001", op="attn", b=24, n=13, ctx=7001, page=16, ragged=True),
        # full trees: 16 requests of 64 drafted tokens over 8,192 rows (the tensor-bound end)
        dict(name="attn-full-b16-n64-ctx8192", op="attn", b=16, n=64, ctx=8192, page=64, ragged=False),
        # selection for 8 trees of 8 nodes over 32,768 positions, and for 64 ragged trees of 32 over 9,001
        dict(name="topk-b8-n8-ctx32768", op="topk", b=8, n=8, ctx=32760, k=2048, ragged=False),
        dict(name="topk-b64-n32-ctx9001", op="topk", b=64, n=32, ctx=9001, k=2048, ragged=True),
        # acceptance: one layer of 4 small trees, and 8 layers of 64 full trees in pages of 16 rows
        dict(name="commit-b4-n8", op="commit", b=4, n=8, ctx=200, page=0, layers=1),
        dict(name="commit-b64-n64-l8", op="commit", b=64, n=64, ctx=170, page=16, layers=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["tables", "append", "attn", "attn", "topk", "commit"])
    if op == "tables":
        tree = rng.random() < 0.5
        b = _log(rng, 1, 512)
        n = _log(rng, 1, 64) if tree else _log(rng, 1, max(1, 65536 // b // 2))
        return dict(op=op, b=b, n=n, ctx=_log(rng, 1, 20000) if b <= 128 else 0, page=rng.choice([16, 32, 64, 128]),
                    tree=tree)
    if op == "append":
        return dict(op=op, t=_log(rng, 1, 8192), page=rng.choice([16, 64, 256]), wide=rng.choice([0, 2048]))
    if op == "attn":
        b, n = _log(rng, 1, 64), _log(rng, 1, 64)
        most = max(1, min(100000, 8_000_000 // (b * n), 2_000_000 // b))
        return dict(op=op, b=b, n=n, ctx=_log(rng, 1, most), page=rng.choice([0, 16, 32, 64, 128]),
                    ragged=rng.random() < 0.5)
    if op == "topk":
        b, n = _log(rng, 1, 64), _log(rng, 1, 32)
        return dict(op=op, b=b, n=n, ctx=_log(rng, 1, max(1, min(100000, 6_000_000 // (b * n)))),
                    k=rng.choice([64, 500, 2048]), ragged=rng.random() < 0.5)
    return dict(op=op, b=_log(rng, 1, 64), n=_log(rng, 1, 64), ctx=_log(rng, 1, 190), page=rng.choice([0, 16, 64]),
                layers=rng.randint(1, 8))


def _lengths(case):
    """Committed and new rows of each sequence: fixed by the case, so that work() knows them."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    b, n, ctx = case["b"], case["n"], case["ctx"]
    if case["op"] == "tables":
        c = [rng.randint(0, ctx) for _ in range(b)]
        m = [rng.randint(0, n) if rng.random() < 0.9 else n for _ in range(b)]
    elif case.get("ragged"):
        c = [rng.randint(ctx // 3, ctx) for _ in range(b)]
        m = [rng.randint(1, n) for _ in range(b)]
    else:
        c, m = [ctx] * b, [n] * b
    return c, m


def _accepted(n, rng):
    """An accepted path of new rows: row 0, then rows that no move of the path overwrites, so that a
    second pass over the same caches moves the same values."""
    m = min(1 + n // 5, 8)
    rest = sorted(rng.sample(range(m, n), m - 1)) if m > 1 and n - m >= m - 1 else []
    return [0] + rest


def work(case):
    op = case["op"]
    if op == "append":
        t = case["t"]
        return {"bytes": t * (2 * 2 * D_QK + 2 * 4 * 64 + 8) + 4 * D_V, "flops": t * (4 * D_V + 6 * 64)}
    c, m = _lengths(case)
    rows = sum(m)
    if op == "tables":
        p = case["page"]
        new = sum(max(-(-(x + y) // p) - -(-x // p), 0) for x, y in zip(c, m))
        t = case["b"] * case["n"]
        return {"bytes": 4 * (6 * case["b"] + 1 + 2 * new + 2 * t) + (12 * t if case["tree"] else 0), "flops": 0}
    if op == "attn":
        seen = sum(y * x for x, y in zip(c, m))
        return {"bytes": 2 * D_QK * sum(x + y for x, y in zip(c, m)) + rows * (H * (2 * D_QK + 2 * D_V + 4) + 8),
                "flops": 2 * (D_QK + D_V) * H * seen}
    if op == "topk":
        return {"bytes": 4 * sum(y * (x + 1) for x, y in zip(c, m)) + 4 * rows * case["k"] + 8 * rows, "flops": 0}
    rng = random.Random(case["n"])
    moved = sum(len(_accepted(y, rng)) - 1 for y in m)
    return {"bytes": case["layers"] * moved * 2 * 2 * (D_QK + D_IDX) + 24 * case["b"], "flops": 0}


# ------------------------------------------------------------------ inputs --

def _dev(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype).cuda()


def _offsets(m):
    off = [0]
    for x in m:
        off.append(off[-1] + x)
    return off


def _parents(m, g):
    """Parent links of each sequence's tree: row 0 is the root, a later row hangs below one of the 8 rows before it."""
    out = []
    for n in m:
        out.append([-1] + [i - 1 - g.randrange(min(i, 8)) for i in range(1, n)] if n else [])
    return out


def _masks(parents):
    out = []
    for par in parents:
        bits = []
        for i, p in enumerate(par):
            bits.append((1 << i) | (bits[p] if p >= 0 else 0))
        out.append(bits)
    return out


def _signed(bits):
    return [x - (1 << 64) if x >> 63 else x for x in bits]


def _layout(c, m, page, gen):
    """Caches' layout: contiguous (page 0: stride and no table) or pages in random order. The last row is no sequence's."""
    longest = max(x + y for x, y in zip(c, m))
    if not page:
        return dict(stride=longest, table=None, pool=0, rows=len(c) * longest + 1)
    held = [-(-(x + y) // page) for x, y in zip(c, m)]
    pool = sum(held) + 1
    order = torch.randperm(pool - 1, generator=gen, device="cuda").to(torch.int32)
    width = max(max(held), 1)
    at = torch.arange(width, device="cuda")[None, :] + _dev(_offsets(held)[:-1], torch.int64)[:, None]
    table = torch.where(torch.arange(width, device="cuda")[None, :] < _dev(held)[:, None],
                        order[at.clamp(max=pool - 2)], -1).to(torch.int32).contiguous()
    return dict(stride=longest, table=table, pool=pool, rows=pool * page)


def _normal(shape, gen, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32 if dtype == torch.float32 else dtype)


def prepare(case, seed):
    g = random.Random(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = dict(case)
    if op == "append":
        t, page = case["t"], case["page"]
        pool = -(-(t + 100) // page) + 1
        s["rows"] = pool * page
        wide = _normal((t, case["wide"] + D_QK), gen)
        s["x"] = wide[:, case["wide"]:]
        s["gamma"] = 1 + 0.1 * _normal((D_V,), gen, torch.float32)
        s["positions"] = torch.randint(0, 32768, (t,), generator=gen, device="cuda", dtype=torch.int32)
        ang = torch.arange(32768, device="cuda", dtype=torch.float64)[:, None] / \
            10000.0 ** (torch.arange(32, device="cuda", dtype=torch.float64) / 32)[None, :]
        s["cos"], s["sin"] = (f(ang).float().repeat(1, 2).contiguous() for f in (torch.cos, torch.sin))
        s["slots"] = torch.randperm(s["rows"], generator=gen, device="cuda")[:t].to(torch.int32)
        s["kv"] = _normal((s["rows"], D_QK), gen)
        if own:
            import sparse_attention_gb300 as dsa
            s["ws"] = dsa.tree_workspace()
        return s

    c, m = _lengths(case)
    total = case["b"] * case["n"] if op == "tables" else sum(m)
    s["total"], s["off"] = total, _dev(_offsets(m))
    s["c"], s["m"] = _dev(c), _dev(m)
    s["ctx_len"] = _dev([x + y for x, y in zip(c, m)])
    longest = max(x + y for x, y in zip(c, m))
    s["longest"] = longest
    parents = _parents(m, g) if op != "tables" or case["tree"] else None

    if op == "tables":
        page = case["page"]
        held = [-(-x // page) for x in c]
        need = [-(-(x + y) // page) for x, y in zip(c, m)]
        pool = sum(need) + 40
        order = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
        width = max(max(need), 1)
        at = torch.arange(width, device="cuda")[None, :] + _dev(_offsets(held)[:-1], torch.int64)[:, None]
        s["table"] = torch.where(torch.arange(width, device="cuda")[None, :] < _dev(held)[:, None],
                                 order[at.clamp(max=pool - 1)], -1).to(torch.int32).contiguous()
        s["pool"], s["held"] = pool, _dev(held)
        # the free list: pages before `head` are in use, `tail` ends it
        s["free"] = order
        s["range"] = _dev([sum(held), pool])
        s["parent"] = _dev([p for par in parents for p in par] + [-1] * (total - sum(m))) if parents else None
        s["out"] = dict(q_off=torch.empty(case["b"] + 1, dtype=torch.int32, device="cuda"),
                        ctx_len=torch.empty(case["b"], dtype=torch.int32, device="cuda"),
                        n_pages=torch.empty(case["b"], dtype=torch.int32, device="cuda"),
                        range=torch.empty(2, dtype=torch.int32, device="cuda"),
                        slots=torch.empty(total, dtype=torch.int32, device="cuda"),
                        positions=torch.empty(total, dtype=torch.int32, device="cuda"))
        if case["tree"]:
            s["out"]["mask"] = torch.empty(total, dtype=torch.int64, device="cuda")
        if own:
            import sparse_attention_gb300 as dsa
            o = s["out"]
            s["batch"] = dsa.make_batch(o["q_off"], o["ctx_len"], case["n"], longest, longest, total_q=total)
            s["pages"] = dsa.make_pages(s["table"], page, pool)
            s["ws"] = dsa.tree_workspace(s["batch"])
        return s

    s["mask"] = _dev([x for bits in _masks(parents) for x in _signed(bits)], torch.int64)
    if op == "topk":
        ld = -(-longest // 4) * 4
        s["scores"] = _normal((total, ld), gen, torch.float32)
        s["idx"] = torch.empty((total, case["k"]), dtype=torch.int32, device="cuda")
        lay = dict(stride=longest, table=None, pool=0)
    else:
        lay = _layout(c, m, case["page"], gen)
    s.update(lay)
    if op == "attn":
        s["q"] = _normal((total, H, D_QK), gen)
        s["kv"] = _normal((lay["rows"], D_QK), gen)
        s["res"] = torch.empty((total, H, D_V), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty((total, H), dtype=torch.float32, device="cuda")
    if op == "commit":
        paths = [_accepted(n, g) for n in m]
        bits = [[(1 << i) for i in range(n)] for n in m]
        for par, path in zip(bits, paths):
            par[path[-1]] = sum(1 << j for j in path)
        s["mask"] = _dev([x for row in bits for x in _signed(row)], torch.int64)
        s["accepted"] = _dev([path[-1] for path in paths])
        s["kv"] = _normal((case["layers"], lay["rows"], D_QK), gen)
        s["k_idx"] = _normal((case["layers"], lay["rows"], D_IDX), gen)
        s["ctx_new"] = torch.empty(case["b"], dtype=torch.int32, device="cuda")
    if own:
        import sparse_attention_gb300 as dsa
        s["batch"] = dsa.make_batch(s["off"], s["ctx_len"], case["n"], longest, lay["stride"], total_q=total)
        s["pages"] = dsa.make_pages(lay["table"], case["page"], lay["pool"]) if lay["table"] is not None else None
        s["ws"] = dsa.tree_workspace(s["batch"])
    return s


# ------------------------------------------------------------- plain forms --

def _rows_of(off, total, b):
    """Sequence and place in it of every packed row."""
    r = torch.arange(total, device="cuda")
    seq = (torch.searchsorted(off.long(), r, right=True) - 1).clamp(max=b - 1)
    return r, seq, r - off.long()[seq]


def _slot(s, seq, pos):
    """Cache row of position `pos` of sequence `seq`."""
    if s["table"] is None:
        return seq * s["stride"] + pos
    return s["table"][seq, pos // s["page"]].long() * s["page"] + pos % s["page"]


def _plain_tables(s):
    b, n, total, page, o = s["b"], s["n"], s["total"], s["page"], s["out"]
    c, m, held = s["c"].long(), s["m"].long(), s["held"].long()
    off = torch.cat([m.new_zeros(1), m.cumsum(0)])
    need = (c + m + page - 1) // page
    new = (need - held).clamp(min=0)
    first = s["range"][0].long() + new.cumsum(0) - new
    col = torch.arange(s["table"].shape[1], device="cuda")[None, :] - held[:, None]
    fresh = (col >= 0) & (col < new[:, None])
    picked = s["free"][(first[:, None] + col).clamp(0, s["pool"] - 1)]
    s["table"].copy_(torch.where(fresh, picked, s["table"]))
    r, seq, i = _rows_of(off, total, b)
    live = r < off[b]
    pos = torch.where(live, c[seq] + i, 0)
    slots = torch.where(live, _slot(s, seq, pos), -1)
    out = dict(table=s["table"])
    if s["parent"] is not None:
        at = (off[:-1, None] + torch.arange(n, device="cuda")).clamp(max=total - 1)
        par = s["parent"].long()[at]
        used = torch.arange(n, device="cuda")[None, :] < m[:, None]
        link = (par[:, :, None] == torch.arange(n, device="cuda")) & used[:, :, None]
        reach = torch.linalg.matrix_power(torch.eye(n, device="cuda", dtype=torch.float64) + link.double(), 64) > 0
        bits = (reach.long() << torch.arange(n, device="cuda")).sum(-1)
        deep = reach.sum(-1) - 1
        inner = i.clamp(max=n - 1)
        out["mask"] = torch.where(live, bits[seq, inner], 0)
        pos = torch.where(live, c[seq] + deep[seq, inner], -1)
    out.update(q_off=off.int(), ctx_len=(c + m).int(), n_pages=torch.maximum(need, held).int(),
               range=torch.stack([s["range"][0] + new.sum(), s["range"][1]]).int(), slots=slots.int(),
               positions=torch.where(live, pos, -1).int())
    return out


def _plain_append(s):
    x = s["x"].float()
    lat, pe = x[:, :D_V], x[:, D_V:]
    lat = lat * torch.rsqrt((lat * lat).mean(1, keepdim=True) + EPS) * s["gamma"]
    cos, sin = s["cos"][s["positions"].long()], s["sin"][s["positions"].long()]
    pe = pe * cos + torch.cat([-pe[:, 32:], pe[:, :32]], 1) * sin
    s["kv"][s["slots"].long()] = torch.cat([lat, pe], 1).bfloat16()
    return s["kv"]


def _sees(s, length):
    """[rows, length]: which positions each packed row sees; and each row's sequence and place."""
    _, seq, i = _rows_of(s["off"], s["total"], s["b"])
    p = torch.arange(length, device="cuda")[None, :] - s["c"].long()[seq][:, None]
    bit = (s["mask"][:, None] >> p.clamp(0, 63)) & 1
    new = s["m"].long()[seq][:, None]
    return (p < 0) | ((p < new) & (p < 64) & (bit == 1)), seq, i


def _plain_attn(s):
    b, n, length = s["b"], s["n"], s["longest"]
    sees, seq, i = _sees(s, length)
    pos = torch.arange(length, device="cuda")[None, :].expand(b, -1)
    there = pos < s["ctx_len"][:, None]
    at = _slot(s, torch.arange(b, device="cuda")[:, None], torch.where(there, pos, 0))
    keys = s["kv"][at].float()
    q = torch.zeros((b, n, H, D_QK), device="cuda")
    q[seq, i] = s["q"].float()
    mask = torch.zeros((b, n, length), dtype=torch.bool, device="cuda")
    mask[seq, i] = sees
    logit = torch.matmul(q.view(b, n * H, D_QK), keys.transpose(1, 2)).view(b, n, H, length)
    logit = (logit * SCALE).masked_fill_(~mask[:, :, None, :], float("-inf"))
    top = logit.amax(-1, keepdim=True).clamp(min=-3e38)
    p = logit.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(b, n * H, length), keys[:, :, :D_V]).view(b, n, H, D_V) / total
    lse = (top + total.log()).squeeze(-1)
    return {"out": out[seq, i].bfloat16(), "lse": lse[seq, i]}


def _plain_topk(s):
    length = s["scores"].shape[1]
    sees, _, _ = _sees(s, length)
    order = s["scores"].masked_fill(~sees, float("-inf")).sort(dim=1, descending=True, stable=True).indices
    k = s["k"]
    best = order[:, :k]
    best = torch.where(sees.gather(1, best), best, length).sort(dim=1).values
    idx = torch.full((s["total"], k), -1, dtype=torch.int64, device="cuda")
    idx[:, :best.shape[1]] = torch.where(best < length, best, -1)
    return idx.int()


def _plain_commit(s):
    b, n, spare = s["b"], s["n"], s["rows"] - 1
    j = torch.arange(n, device="cuda")
    on = ((s["mask"][(s["off"][:-1] + s["accepted"]).long()][:, None] >> j) & 1) == 1
    count = on.sum(1)
    source = torch.sort((~on).long(), dim=1, stable=True).indices
    moves = j[None, :] < count[:, None]
    seq = torch.arange(b, device="cuda")[:, None]
    base = s["c"].long()[:, None]
    to = torch.where(moves, _slot(s, seq, torch.where(moves, base + j, 0)), spare).view(-1)
    of = torch.where(moves, _slot(s, seq, torch.where(moves, base + source, 0)), spare).view(-1)
    s["kv"][:, to] = s["kv"][:, of]
    s["k_idx"][:, to] = s["k_idx"][:, of]
    return {"ctx_len": (s["c"] + count).int(), "kv": s["kv"], "k_idx": s["k_idx"]}


def run(s):
    if not own:
        return {"tables": _plain_tables, "append": _plain_append, "attn": _plain_attn, "topk": _plain_topk,
                "commit": _plain_commit}[s["op"]](s)
    import sparse_attention_gb300 as dsa
    op = s["op"]
    if op == "tables":
        o = s["out"]
        dsa.step_tables(s["batch"], s["m"], s["c"], o["slots"], o["positions"], mask=o.get("mask"), parent=s["parent"],
                        pages=s["pages"], n_pages_old=s["held"], n_pages=o["n_pages"], free_pages=s["free"],
                        free_range=s["range"], free_range_out=o["range"], ws=s["ws"])
        return dict(o, table=s["table"])
    if op == "append":
        dsa.latent_append(s["x"], s["gamma"], EPS, s["cos"], s["sin"], s["positions"], s["slots"], s["kv"], ws=s["ws"])
        return s["kv"]
    if op == "attn":
        dsa.tree_mla_fwd(s["batch"], s["q"], s["kv"], s["mask"], SCALE, s["res"], s["lse"], pages=s["pages"],
                         ws=s["ws"])
        return {"out": s["res"], "lse": s["lse"]}
    if op == "topk":
        dsa.tree_topk(s["batch"], s["scores"], s["mask"], s["k"], s["idx"], ws=s["ws"])
        return s["idx"]
    dsa.tree_commit(s["batch"], s["mask"], s["accepted"], s["ctx_new"], s["kv"], k_idx=s["k_idx"], pages=s["pages"],
                    ws=s["ws"])
    return {"ctx_len": s["ctx_new"], "kv": s["kv"], "k_idx": s["k_idx"]}


# ----------------------------------------------------------------- 64 bits --

def exact(case, seed):
    op = case["op"]
    if op not in ("append", "attn"):
        return None          # whole numbers, or values that are only moved
    s = prepare(case, seed)
    if op == "append":
        kv, x = s["kv"].double(), s["x"].double()
        norm = (x[:, :D_V].pow(2).sum(1) / D_V + EPS).sqrt()
        row = torch.empty_like(x)
        row[:, :D_V] = x[:, :D_V] / norm[:, None] * s["gamma"].double()
        place = s["positions"].long()
        for i in range(32):
            a, b = x[:, D_V + i], x[:, D_V + 32 + i]
            row[:, D_V + i] = a * s["cos"][place, i].double() - b * s["sin"][place, i].double()
            row[:, D_V + 32 + i] = b * s["cos"][place, 32 + i].double() + a * s["sin"][place, 32 + i].double()
        kv[s["slots"].long()] = row
        return kv
    c, m = _lengths(case)
    parents = _parents(m, random.Random(seed))
    out = torch.empty((s["total"], H, D_V), dtype=torch.float64, device="cuda")
    lse = torch.empty((s["total"], H), dtype=torch.float64, device="cuda")
    first = 0
    for b in range(case["b"]):
        length = c[b] + m[b]
        where = torch.arange(length, device="cuda")
        if case["page"]:
            where = s["table"][b].long()[where // case["page"]] * case["page"] + where % case["page"]
        else:
            where = where + b * s["stride"]
        rows = s["kv"][where].double()
        seen = torch.zeros((m[b], length), dtype=torch.bool)
        seen[:, :c[b]] = True
        for i in range(m[b]):
            j = i
            while j >= 0:
                seen[i, c[b] + j] = True
                j = parents[b][j]
        seen = seen.cuda()[:, None, :]
        q = s["q"][first:first + m[b]].double()
        logit = torch.einsum("nhd,ld->nhl", q, rows) * SCALE
        logit = torch.where(seen, logit, float("-inf"))
        lse[first:first + m[b]] = torch.logsumexp(logit, -1)
        p = torch.exp(logit - lse[first:first + m[b], :, None])
        out[first:first + m[b]] = torch.einsum("nhl,ld->nhd", p, rows[:, :D_V])
        first += m[b]
    return {"out": out, "lse": lse}

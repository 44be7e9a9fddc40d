"""Prompts and shared prefixes over the latent cache: the operators' cases,
their plain forms and the framework's calls.

Sequence b holds ctx_len[b] cache rows of [512 latent | 64 rotary key], of
which the last n_b are new; its new row i is packed row q_off[b] + i at position
ctx_len[b] - n_b + i.

  table   rotary cos / sin rows of positions, plain or scaled for long contexts
  rope    part of every head rotated at the tokens' positions, in both layouts
  expand  latent rows -> each head's 192 key and 256 value columns (kv_b_proj)
  prompt  causal attention of new rows over expanded rows: 64 heads, 256 | 256
  prefix  latent attention of a batch whose groups of sequences share their
          first rows, and new rows under tree masks
"""

import math
import random

import torch

own = False

H, D_QK, D_V, D_LAT, D_NOPE, D_ROPE = 64, 576, 512, 512, 192, 64
D_HEAD, D_VAL, D_EXP = 256, 256, 448
SCALE = 1.0 / 16.0
ROOM = 128               # expanded rows of a sequence begin at a multiple of this


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # the tables that a server makes once: 32,768 positions, and 202,752 scaled from 16,384
        dict(name="table-32768", op="table", rows=32768, first=0, base=10000.0, factor=1.0, original=0),
        dict(name="table-yarn-202752", op="table", rows=202752, first=0, base=8000000.0, factor=12.375, original=16384),
        # the rotary part of 64 heads' queries of a decode batch, in place
        dict(name="rope-decode-t64", op="rope", t=64, heads=64, width=256, at=192, rot=64, table=32768, pairs="half",
             inverse=False, place=True),
        # a prefill chunk's index queries, the first 64 of 128 columns, neighbours as pairs, into a buffer of their own
        dict(name="rope-chunk-t8192", op="rope", t=8192, heads=32, width=128, at=0, rot=64, table=32768,
             pairs="neighbour", inverse=False, place=False),
        # eight short prompts in pages of 16 rows, and a chunk of 8,192 tokens behind 1,003 kept ones
        dict(name="expand-b8-n300", op="expand", b=8, n=300, kept=0, page=16, ragged=True),
        dict(name="expand-chunk-n8192", op="expand", b=1, n=8192, kept=1003, page=64, ragged=False),
        # one short question: the smallest call, where latency counts
        dict(name="prompt-one-n100", op="prompt", b=1, n=100, kept=0, ragged=False),
        # a wave of prompts below 2,048 tokens, where the sparse layers keep every position
        dict(name="prompt-wave-b12-n2047", op="prompt", b=12, n=2047, kept=0, ragged=True),
        # a whole prompt of 16,384 tokens (the tensor-bound end)
        dict(name="prompt-whole-n16384", op="prompt", b=1, n=16384, kept=0, ragged=False),
        # a few requests behind a system prompt: 4 x 1 row behind 2,000 shared rows
        dict(name="prefix-b4-s2000", op="prefix", b=4, g=1, n=1, shared=2000, own=40, page=64, ragged=False),
        # decode of 64 requests behind one prefix of 32,768 rows, and some 500 rows of their own
        dict(name="prefix-b64-s32768", op="prefix", b=64, g=1, n=1, shared=32768, own=500, page=64, ragged=True),
        # five documents with questions of their own and drafted trees, ragged, in pages of 16 rows
        dict(name="prefix-b40-g5-n6-s12001", op="prefix", b=40, g=5, n=6, shared=12001, own=900, page=16, ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["table", "rope", "expand", "prompt", "prompt", "prefix", "prefix"])
    if op == "table":
        scaled = rng.random() < 0.6
        return dict(op=op, rows=_log(rng, 1, 202752), first=rng.choice([0, 0, 1000, 1000003]),
                    base=rng.choice([10000.0, 1000000.0, 8000000.0]), factor=round(rng.uniform(1.5, 40.0), 2) if scaled else 1.0,
                    original=rng.choice([0, 4096, 32768]) if scaled else 0)
    if op == "rope":
        width = rng.choice([64, 128, 192, 256])
        rot = rng.choice([r for r in (32, 64, 128, 256) if r <= width])
        place = rng.random() < 0.5
        return dict(op=op, t=_log(rng, 1, 8192), heads=rng.choice([1, 5, 16, 32, 64]), width=width,
                    at=rng.choice([0, (width - rot) // 8 * 8]), rot=rot, table=_log(rng, 100, 32768),
                    pairs=rng.choice(["half", "neighbour"]), inverse=rng.random() < 0.3, place=place)
    if op == "expand":
        b = _log(rng, 1, 64)
        n = _log(rng, 1, max(1, 9000 // b))
        return dict(op=op, b=b, n=n, kept=rng.choice([0, 0, _log(rng, 1, 9000 // b)]), page=rng.choice([0, 16, 32, 64, 128]),
                    ragged=rng.random() < 0.5)
    if op == "prompt":
        b = _log(rng, 1, 32)
        n = _log(rng, 1, max(1, 16384 // b))
        most = min(65536 // b, 100_000_000 // (b * n) - n)
        return dict(op=op, b=b, n=n, kept=_log(rng, 1, most) if most > 1 and rng.random() < 0.5 else 0,
                    ragged=rng.random() < 0.5)
    b, n = _log(rng, 1, 64), rng.choice([1, 1, _log(rng, 1, 16)])
    shared = _log(rng, 1, max(1, min(60000, 6_000_000 // (b * n))))
    return dict(op=op, b=b, g=rng.randint(1, max(1, min(b, 8))), n=n, shared=shared, own=_log(rng, 1, 1200),
                page=rng.choice([0, 16, 32, 64, 128]), ragged=rng.random() < 0.6)


def _lengths(case):
    """Fixed by the case, so that work() knows them.  expand, prompt: kept and new rows of each sequence; prefix: also
    its group's shared rows (part of its kept ones), and the first sequence of each group."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    b, n = case["b"], case["n"]
    ragged = case["ragged"]
    m = [rng.randint(max(1, n // 3), n) if ragged else n for _ in range(b)]
    if case["op"] != "prefix":
        k = case["kept"]
        return [rng.randint(0, k) if ragged else k for _ in range(b)], m
    g, s = case["g"], case["shared"]
    first = [0] + sorted(rng.sample(range(1, b), g - 1)) + [b]
    share = [rng.randint(s // 2, s) if ragged else s for _ in range(g)]
    mine = [rng.randint(0, case["own"]) if ragged else case["own"] for _ in range(b)]
    of = [max(j for j in range(g) if first[j] <= x) for x in range(b)]
    return [share[of[x]] + mine[x] for x in range(b)], m, share, first, of


def work(case):
    op = case["op"]
    if op == "table":
        return {"bytes": case["rows"] * 2 * 4 * D_ROPE, "flops": 0}
    if op == "rope":
        t, r = case["t"], case["rot"]
        return {"bytes": t * (case["heads"] * 2 * 2 * r + 4 + 2 * 4 * r // 2), "flops": t * case["heads"] * 3 * r}
    if op == "expand":
        rows = sum(_lengths(case)[1])
        return {"bytes": rows * (2 * D_QK + 2 * H * D_EXP + 2 * D_ROPE) + 2 * H * D_EXP * D_LAT,
                "flops": 2 * rows * H * D_EXP * D_LAT}
    if op == "prompt":
        c, m = _lengths(case)
        pairs = sum(y * x + y * (y + 1) // 2 for x, y in zip(c, m))
        return {"bytes": sum(x + y for x, y in zip(c, m)) * 2 * (H * D_EXP + D_ROPE) +
                sum(m) * H * (2 * D_HEAD + 2 * D_VAL + 4), "flops": 2 * (D_HEAD + D_VAL) * H * pairs}
    c, m, share, first, of = _lengths(case)
    rows = sum(share) + sum(x + y - share[j] for x, y, j in zip(c, m, of))
    return {"bytes": 2 * D_QK * rows + sum(m) * (H * (2 * D_QK + 2 * D_V + 4) + 8),
            "flops": 2 * (D_QK + D_V) * H * sum(x * y for x, y in zip(c, m))}


# ------------------------------------------------------------------ inputs --

def _dev(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype).cuda()


def _offsets(m):
    off = [0]
    for x in m:
        off.append(off[-1] + x)
    return off


def _normal(shape, gen, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)


def _parents(m, g):
    """Parent links of each sequence's tree: row 0 is the root, a later row hangs below one of the 4 rows before it."""
    return [[-1] + [i - 1 - g.randrange(min(i, 4)) for i in range(1, n)] for n in m]


def _masks(parents):
    out = []
    for par in parents:
        bits = []
        for i, p in enumerate(par):
            bits.append((1 << i) | (bits[p] if p >= 0 else 0))
        out += bits
    return out


def _pages(lengths, page, gen, share=None, of=None, first=None):
    """Block table of pages in random order (None without pages), the pool's pages, and every sequence's cache rows.
    Whole pages of a group's shared rows are the same pages in each of its sequences' table rows."""
    longest = max(lengths)
    if not page:
        return None, 0, len(lengths) * longest
    need = [-(-x // page) for x in lengths]
    whole = [0] * len(lengths) if share is None else [share[j] // page for j in of]
    order, at = [], 0
    table = torch.full((len(lengths), max(need)), -1, dtype=torch.int64)
    for b, n in enumerate(need):
        lead = b if share is None else first[of[b]]
        from_lead = whole[b] if lead != b else 0
        table[b, :from_lead] = table[lead, :from_lead]
        table[b, from_lead:n] = torch.arange(at, at + n - from_lead)
        at += n - from_lead
    order = torch.randperm(at, generator=gen, device="cuda").cpu()
    table = torch.where(table >= 0, order[table.clamp(min=0)], -1)
    return table.to(torch.int32).cuda(), at + 1, (at + 1) * page


def prepare(case, seed):
    g = random.Random(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = dict(case)
    if own:
        import sparse_attention_gb300 as dsa
    if op == "table":
        # another seed is another base, as of another model
        s["base"] = case["base"] * (1 + g.random())
        s["cos"] = torch.empty((case["rows"], D_ROPE), device="cuda")
        s["sin"] = torch.empty((case["rows"], D_ROPE), device="cuda")
        if own:
            s["scaling"] = dsa.RopeScaling(case["factor"], case["original"], 32.0, 1.0, _mscale(case)) \
                if case["factor"] != 1.0 else None
        return s
    if op == "rope":
        t, r = case["t"], case["rot"]
        s["x"] = _normal((t, case["heads"], case["width"]), gen)
        s["out"] = s["x"][..., case["at"]:case["at"] + r] if case["place"] else \
            torch.zeros((t, case["heads"], r), dtype=torch.bfloat16, device="cuda")
        s["positions"] = torch.randint(0, case["table"], (t,), generator=gen, device="cuda", dtype=torch.int32)
        ang = torch.arange(case["table"], device="cuda", dtype=torch.float64)[:, None] / \
            10000.0 ** (torch.arange(r // 2, device="cuda", dtype=torch.float64) / (r // 2))[None, :]
        s["cos"], s["sin"] = (f(ang).float().repeat(1, 2).contiguous() for f in (torch.cos, torch.sin))
        if own:
            s["ws"] = dsa.tree_workspace()
        return s

    lay = _lengths(case)
    c, m = lay[:2]
    length = [x + y for x, y in zip(c, m)]
    s["lay"], s["longest"], s["total"] = lay, max(length), sum(m)
    s["off"], s["ctx_len"] = _dev(_offsets(m)), _dev(length)
    if op in ("expand", "prompt"):
        room = [-(-x // ROOM) * ROOM for x in length]
        s["at"] = _offsets(room)
        s["exp_off"] = _dev(s["at"])
        s["kvx"] = _normal((s["at"][-1], H, D_EXP), gen)
        s["k_pe"] = _normal((s["at"][-1], D_ROPE), gen)
        for b, x in enumerate(length):            # as the expansion leaves a sequence's room
            s["kvx"][s["at"][b] + x:s["at"][b + 1]] = 0
            s["k_pe"][s["at"][b] + x:s["at"][b + 1]] = 0
    if op == "prompt":
        s["q"] = _normal((s["total"], H, D_HEAD), gen)
        s["res"] = torch.empty((s["total"], H, D_VAL), dtype=torch.bfloat16, device="cuda")
    if op in ("expand", "prefix"):
        share, first, of = lay[2:] if op == "prefix" else (None, None, None)
        s["table"], s["pool"], rows = _pages(length, case["page"], gen, share, of, first)
        s["kv"] = _normal((rows, D_QK), gen)
    if op == "expand":
        s["first"] = _dev(c)
        s["w"] = (_normal((H * D_EXP, D_LAT), gen, torch.float32) / math.sqrt(D_LAT)).bfloat16()
    if op == "prefix":
        # the rows that members share but do not find on a shared page
        for b, j in enumerate(of):
            lo = share[j] // case["page"] * case["page"] if case["page"] else 0
            if first[j] != b and lo < share[j]:
                pos = torch.arange(lo, share[j], device="cuda")
                s["kv"][_slot(s, b, pos)] = s["kv"][_slot(s, first[j], pos)]
        s["group_off"], s["shared"] = _dev(first), _dev(share)
        bits = [x - (1 << 64) if x >> 63 else x for x in _masks(_parents(m, g))]
        s["mask"] = _dev(bits, torch.int64)
        s["q"] = _normal((s["total"], H, D_QK), gen)
        s["res"] = torch.empty((s["total"], H, D_V), dtype=torch.bfloat16, device="cuda")
    if op in ("prompt", "prefix"):
        s["lse"] = torch.empty((s["total"], H), dtype=torch.float32, device="cuda")
    if own:
        s["batch"] = dsa.make_batch(s["off"], s["ctx_len"], max(m), s["longest"], s["longest"], total_q=s["total"])
        s["paged"] = dsa.make_pages(s["table"], case["page"], s["pool"]) if s.get("table") is not None else None
        if op == "prefix":
            s["groups"] = dsa.make_groups(s["group_off"], s["shared"])
            s["ws"] = dsa.prefix_workspace(s["batch"], s["groups"])
        else:
            s["expanded"] = dsa.make_expanded(s["exp_off"], s["kvx"], s["k_pe"])
            s["ws"] = dsa.prompt_workspace(s["batch"])
    return s


# ------------------------------------------------------------- plain forms --

def _mscale(case):
    return 0.1 * math.log(case["factor"]) + 1.0 if case["original"] else 1.0


def _slot(s, b, pos):
    """Cache rows of positions `pos` of sequence b."""
    if s["table"] is None:
        return b * s["longest"] + pos
    return s["table"][b].long()[pos // s["page"]] * s["page"] + pos % s["page"]


def _plain_table(s):
    # angles of far positions need more than 32 bits
    half = D_ROPE // 2
    i = torch.arange(half, device="cuda", dtype=torch.float64)
    freq = s["base"] ** (-i / half)
    if s["original"]:
        turns = [D_ROPE * math.log(s["original"] / (x * 2 * math.pi)) / (2 * math.log(s["base"])) for x in (32.0, 1.0)]
        lo, hi = max(math.floor(turns[0]), 0), min(math.ceil(turns[1]), D_ROPE - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        freq = freq / s["factor"] * ramp + freq * (1 - ramp)
    else:
        freq = freq / s["factor"]
    pos = torch.arange(s["rows"], device="cuda", dtype=torch.float64) + s["first"]
    ang = (pos[:, None] * freq).repeat(1, 2)
    s["cos"].copy_(ang.cos() * _mscale(s))
    s["sin"].copy_(ang.sin() * _mscale(s))
    return {"cos": s["cos"], "sin": s["sin"]}


def _plain_rope(s):
    r = s["rot"]
    x = s["x"][..., s["at"]:s["at"] + r].float()
    p = s["positions"].long()
    c, w = s["cos"][p, None, :r // 2], s["sin"][p, None, :r // 2]
    if s["inverse"]:
        w = -w
    if s["pairs"] == "half":
        a, b = x[..., :r // 2], x[..., r // 2:]
        y = torch.cat([a * c - b * w, b * c + a * w], -1)
    else:
        a, b = x[..., 0::2], x[..., 1::2]
        y = torch.stack([a * c - b * w, b * c + a * w], -1).flatten(-2)
    s["out"].copy_(y.bfloat16())
    return s["x"] if s["place"] else s["out"]


def _plain_expand(s):
    w = s["w"].float()
    for b, (c, m) in enumerate(zip(*s["lay"])):
        rows = s["kv"][_slot(s, b, torch.arange(c, c + m, device="cuda"))]
        to = s["at"][b] + c
        s["kvx"][to:to + m] = (rows[:, :D_LAT].float() @ w.t()).bfloat16().view(m, H, D_EXP)
        s["k_pe"][to:to + m] = rows[:, D_LAT:]
    return {"kvx": s["kvx"], "k_pe": s["k_pe"]}


def _plain_prompt(s):
    first = 0
    for b, (c, m) in enumerate(zip(*s["lay"])):
        at, length = s["at"][b], c + m
        pe = s["k_pe"][at:at + length].float()
        for h in range(0, H, 8):
            kv = s["kvx"][at:at + length, h:h + 8].float().transpose(0, 1)
            k = torch.cat([kv[..., :D_NOPE], pe.expand(8, -1, -1)], -1).transpose(1, 2)
            v = kv[..., D_NOPE:].contiguous()
            for i in range(0, m, 2048):
                n = min(2048, m - i)
                end = c + i + n
                row = slice(first + i, first + i + n)
                logit = torch.matmul(s["q"][row, h:h + 8].float().transpose(0, 1), k[..., :end]) * SCALE
                late = torch.arange(end, device="cuda") > torch.arange(c + i, end, device="cuda")[:, None]
                logit.masked_fill_(late, float("-inf"))
                top = logit.amax(-1, keepdim=True)
                p = logit.sub_(top).exp_()
                total = p.sum(-1, keepdim=True)
                s["res"][row, h:h + 8] = (torch.matmul(p, v[:, :end]) / total).transpose(0, 1).bfloat16()
                s["lse"][row, h:h + 8] = (top + total.log()).squeeze(-1).t()
        first += m
    return {"out": s["res"], "lse": s["lse"]}


def _plain_prefix(s):
    first = 0
    for b, (c, m) in enumerate(zip(*s["lay"][:2])):
        keys = s["kv"][_slot(s, b, torch.arange(c + m, device="cuda"))].float()
        row = slice(first, first + m)
        j = torch.arange(m, device="cuda")
        seen = torch.ones((m, c + m), dtype=torch.bool, device="cuda")
        seen[:, c:] = ((s["mask"][row, None] >> j) & 1) == 1
        logit = torch.matmul(s["q"][row].float().view(m * H, D_QK), keys.t()).view(m, H, -1) * SCALE
        logit.masked_fill_(~seen[:, None], float("-inf"))
        top = logit.amax(-1, keepdim=True)
        p = logit.sub_(top).exp_()
        total = p.sum(-1, keepdim=True)
        s["res"][row] = (torch.matmul(p.view(m * H, -1), keys[:, :D_V]).view(m, H, D_V) / total).bfloat16()
        s["lse"][row] = (top + total.log()).squeeze(-1)
        first += m
    return {"out": s["res"], "lse": s["lse"]}


def run(s):
    if not own:
        return {"table": _plain_table, "rope": _plain_rope, "expand": _plain_expand, "prompt": _plain_prompt,
                "prefix": _plain_prefix}[s["op"]](s)
    import sparse_attention_gb300 as dsa
    op = s["op"]
    if op == "table":
        dsa.rope_table(s["cos"], s["sin"], s["base"], first=s["first"], scaling=s["scaling"])
        return {"cos": s["cos"], "sin": s["sin"]}
    if op == "rope":
        dsa.rope(s["x"][..., s["at"]:s["at"] + s["rot"]], s["cos"], s["sin"], s["positions"], s["out"],
                 interleaved=s["pairs"] == "neighbour", inverse=s["inverse"], ws=s["ws"])
        return s["x"] if s["place"] else s["out"]
    if op == "expand":
        dsa.mla_expand(s["batch"], s["kv"], s["w"], s["expanded"], first=s["first"], pages=s["paged"], ws=s["ws"])
        return {"kvx": s["kvx"], "k_pe": s["k_pe"]}
    if op == "prompt":
        dsa.prompt_mla_fwd(s["batch"], s["q"], s["expanded"], SCALE, s["res"], s["lse"], ws=s["ws"])
    else:
        dsa.prefix_mla_fwd(s["batch"], s["groups"], s["q"], s["kv"], s["mask"], SCALE, s["res"], s["lse"],
                           pages=s["paged"], ws=s["ws"])
    return {"out": s["res"], "lse": s["lse"]}


# ----------------------------------------------------------------- 64 bits --

def _exact_table(s):
    cos = torch.empty((s["rows"], D_ROPE), dtype=torch.float64, device="cuda")
    sin = torch.empty_like(cos)
    scale = 0.1 * math.log(s["factor"]) + 1.0 if s["original"] else 1.0
    pos = torch.arange(s["first"], s["first"] + s["rows"], device="cuda", dtype=torch.float64)
    for i in range(32):
        inv = s["base"] ** (-2 * i / D_ROPE)
        if s["original"]:
            # a pair that turns less than once in the original context is interpolated, one of 32 turns and more is not
            edge = [D_ROPE / 2 * math.log(s["original"] / (2 * math.pi * n), s["base"]) for n in (32, 1)]
            lo, hi = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), D_ROPE - 1)
            part = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            inv *= part / s["factor"] + 1 - part
        else:
            inv /= s["factor"]
        for col in (i, i + 32):
            cos[:, col], sin[:, col] = torch.cos(pos * inv) * scale, torch.sin(pos * inv) * scale
    return {"cos": cos, "sin": sin}


def _exact_rope(s):
    x, place = s["x"].double(), s["positions"].long()
    r = s["rot"]
    out = x.clone() if s["place"] else torch.empty((s["t"], s["heads"], r), dtype=torch.float64, device="cuda")
    to = s["at"] if s["place"] else 0
    for i in range(r // 2):
        p, q = (i, i + r // 2) if s["pairs"] == "half" else (2 * i, 2 * i + 1)
        turn = torch.complex(s["cos"][place, i].double(), s["sin"][place, i].double() * (-1 if s["inverse"] else 1))
        z = torch.complex(x[..., s["at"] + p], x[..., s["at"] + q]) * turn[:, None]
        out[..., to + p], out[..., to + q] = z.real, z.imag
    return out


def _exact_expand(s):
    kvx, k_pe, w = s["kvx"].double(), s["k_pe"].double(), s["w"].double().view(H, D_EXP, D_LAT)
    for b, (c, m) in enumerate(zip(*s["lay"])):
        where = torch.arange(c, c + m, device="cuda")
        if s["page"]:
            where = s["table"][b].long()[where // s["page"]] * s["page"] + where % s["page"]
        else:
            where = where + b * s["longest"]
        at = s["at"][b] + c
        kvx[at:at + m] = torch.einsum("td,hed->the", s["kv"][where, :D_LAT].double(), w)
        k_pe[at:at + m] = s["kv"][where, D_LAT:].double()
    return {"kvx": kvx, "k_pe": k_pe}


def _exact_prompt(s):
    out = torch.empty((s["total"], H, D_VAL), dtype=torch.float64, device="cuda")
    lse = torch.empty((s["total"], H), dtype=torch.float64, device="cuda")
    row = 0
    for b, (c, m) in enumerate(zip(*s["lay"])):
        rows = slice(s["at"][b], s["at"][b] + c + m)
        for h in range(H):
            k = torch.cat([s["kvx"][rows, h, :D_NOPE], s["k_pe"][rows]], 1).double()
            v = s["kvx"][rows, h, D_NOPE:].double()
            for i in range(0, m, 4096):
                n = min(4096, m - i)
                logit = s["q"][row + i:row + i + n, h].double() @ k[:c + i + n].t() * SCALE
                seen = torch.ones_like(logit, dtype=torch.bool).tril(c + i)
                logit = torch.where(seen, logit, float("-inf"))
                top = torch.logsumexp(logit, -1)
                lse[row + i:row + i + n, h] = top
                out[row + i:row + i + n, h] = torch.exp(logit - top[:, None]) @ v[:c + i + n]
        row += m
    return {"out": out, "lse": lse}


def _exact_prefix(s, seed):
    c, m = s["lay"][:2]
    parents = _parents(m, random.Random(seed))
    out = torch.empty((s["total"], H, D_V), dtype=torch.float64, device="cuda")
    lse = torch.empty((s["total"], H), dtype=torch.float64, device="cuda")
    first = 0
    for b in range(s["b"]):
        length = c[b] + m[b]
        where = torch.arange(length, device="cuda")
        if s["page"]:
            where = s["table"][b].long()[where // s["page"]] * s["page"] + where % s["page"]
        else:
            where = where + b * s["longest"]
        rows = s["kv"][where].double()
        seen = torch.zeros((m[b], length), dtype=torch.bool)
        seen[:, :c[b]] = True
        for i in range(m[b]):
            j = i
            while j >= 0:
                seen[i, c[b] + j] = True
                j = parents[b][j]
        q = s["q"][first:first + m[b]].double()
        logit = torch.einsum("nhd,ld->nhl", q, rows) * SCALE
        logit = torch.where(seen.cuda()[:, None, :], logit, float("-inf"))
        lse[first:first + m[b]] = torch.logsumexp(logit, -1)
        p = torch.exp(logit - lse[first:first + m[b], :, None])
        out[first:first + m[b]] = torch.einsum("nhl,ld->nhd", p, rows[:, :D_V])
        first += m[b]
    return {"out": out, "lse": lse}


def exact(case, seed):
    if work(case)["flops"] > 1e13:
        return None          # over 20 seconds in 64 bits
    s = prepare(case, seed)
    if case["op"] == "prefix":
        return _exact_prefix(s, seed)
    return {"table": _exact_table, "rope": _exact_rope, "expand": _exact_expand, "prompt": _exact_prompt}[case["op"]](s)

"""The expanded form of the latent attention through the public entry points:
expansion of cache rows, causal attention over expanded rows, and prompts
processed by both, against 64-bit references."""

import numpy as np
import pytest
import torch

import sparse_attention_gb300 as dsa
from prompt_case import (D_EXP, D_HEAD, D_LAT, D_QK, D_ROPE, F32, H, HALF, SCALE, Prompts, attention_ref, check_attention,
                         expand_ref, up)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from sparse_attention_gb300 import build as B
    B.build()
    dsa.load_library()


@pytest.fixture(scope="module")
def weight():
    g = torch.Generator().manual_seed(5)
    return (torch.randn((H * D_EXP, D_LAT), generator=g) / D_LAT ** 0.5).bfloat16()


# --------------------------------------------------------------- expansion --

def _check_expansion(P, x, kv, w, first, before=None):
    """Every buffer row: expanded, zeroed behind a sequence, or as it was."""
    got, pe = x.kv.cpu(), x.k_pe.cpu()
    want_nan = torch.ones(P.rows_x, dtype=torch.bool)
    for b in range(P.B):
        lo, f, n = int(P.at[b]), first[b], P.L[b]
        if f < n:
            rows = kv[P.slots(b, f, n)]
            ref, size = expand_ref(rows, w)
            err = (got[lo + f:lo + n].double() - ref).abs()
            # an fp32 sum of 512 exact products, and the rounding to bf16
            assert (err <= HALF * ref.abs() + 512 * F32 * (1 + HALF) * size).all(), b
            assert torch.equal(pe[lo + f:lo + n], rows[:, D_LAT:])
            want_nan[lo + f:lo + up(n, 16)] = False
            assert (got[lo + n:lo + up(n, 16)] == 0).all() and (pe[lo + n:lo + up(n, 16)] == 0).all()
    if before is None:
        assert got[want_nan].isnan().all() and pe[want_nan].isnan().all()
    else:
        assert torch.equal(got[want_nan], before[0][want_nan]) and torch.equal(pe[want_nan], before[1][want_nan])


@pytest.mark.parametrize("page", [0, 16, 64, 256])
@pytest.mark.parametrize("c,m", [
    ([0], [1]), ([0], [300]), ([5, 0, 200], [60, 0, 1]), ([0] * 40, [1] * 40),
    ([127, 128, 129, 0, 16, 15], [1, 1, 130, 128, 17, 1]), ([1000], [513]),
])
def test_expansion(weight, page, c, m):
    P = Prompts(c, m, page, seed=len(c), gap=128, pad=128)
    kv = P.normal(P.cache_rows, D_QK)
    x = P.buffers()
    dsa.mla_expand(P.batch, kv.cuda(), weight.cuda(), x, pages=P.pages, ws=P.ws)
    _check_expansion(P, x, kv, weight, [0] * P.B)
    y = P.buffers()
    dsa.mla_expand(P.batch, kv.cuda(), weight.cuda(), y, first=P.i32(c), pages=P.pages, ws=P.ws)
    _check_expansion(P, y, kv, weight, c)
    assert dsa.read_device_status(P.ws) == 0


def test_expansion_by_chunks(weight):
    """Chunks that keep what was expanded give the bits of one call."""
    P = Prompts([0, 0, 0], [700, 129, 5], 32, seed=9)
    kv = P.normal(P.cache_rows, D_QK).cuda()
    w = weight.cuda()
    one, many = P.buffers(), P.buffers()
    dsa.mla_expand(P.batch, kv, w, one, pages=P.pages, ws=P.ws)
    old = np.zeros(3, np.int64)
    for step in (3, 128, 250, 251, 700):
        new = np.minimum(P.L, step)
        b = dsa.make_batch(P.i32(np.zeros(4)), P.i32(new), 0, P.max_ctx, P.stride, total_q=0)
        dsa.mla_expand(b, kv, w, many, first=P.i32(old), pages=P.pages, ws=P.ws)
        old = new
    for a, b in ((one.kv, many.kv), (one.k_pe, many.k_pe)):
        assert torch.equal(a.nan_to_num(-7), b.nan_to_num(-7))
    assert dsa.read_device_status(P.ws) == 0


def test_expansion_keeps_values_finite(weight):
    """Rows with a NaN or an infinity anywhere: finite kv, NaN keys; leftovers behind a sequence reach nothing."""
    P = Prompts([0, 0], [200, 70], 64, seed=3)
    kv = P.normal(P.cache_rows, D_QK)
    clean = kv.clone()
    for b in range(2):
        n = P.L[b]
        end = up(n, 64)
        lost = P.slots(b, 0, n)[-1] + 1 + torch.arange(end - n)
        kv[lost] = float("nan")
    bad = {3: (0, 11, float("nan")), 130: (0, 511, float("inf")), 199: (0, 575, float("-inf")), 0: (1, 512, float("nan"))}
    for pos, (b, col, v) in bad.items():
        kv[P.slots(b, pos, pos + 1), col] = v
    w = weight.cuda()
    x, ref = P.buffers(), P.buffers()
    dsa.mla_expand(P.batch, kv.cuda(), w, x, pages=P.pages, ws=P.ws)
    dsa.mla_expand(P.batch, clean.cuda(), w, ref, pages=P.pages, ws=P.ws)
    hit = torch.zeros(P.rows_x, dtype=torch.bool)
    for pos, (b, _, _) in bad.items():
        hit[int(P.at[b]) + pos] = True
    hit = hit.cuda()
    same = lambda a, b: torch.equal(a[~hit].nan_to_num(-7), b[~hit].nan_to_num(-7))  # noqa: E731
    assert x.k_pe[hit].isnan().all() and same(x.k_pe, ref.k_pe) and same(x.kv, ref.kv)
    for b in range(2):
        assert x.kv[int(P.at[b]):int(P.at[b]) + up(P.L[b], 16)].isfinite().all()
    # overflow: kept at the largest value
    kv = torch.full((P.cache_rows, D_QK), 3e38, dtype=torch.bfloat16, device="cuda")
    dsa.mla_expand(P.batch, kv, w.abs() * 100, x, pages=P.pages, ws=P.ws)
    big = torch.finfo(torch.bfloat16).max
    assert (x.kv[:200] == big).all() and x.k_pe[:200].isfinite().all()
    dsa.mla_expand(P.batch, kv, w.abs() * -100, x, pages=P.pages, ws=P.ws)
    assert (x.kv[:200] == -big).all()


def test_expansion_skips_what_is_wrong(weight):
    P = Prompts([0, 0, 0], [40, 200, 10], 16, seed=4, gap=128, pad=128)
    kv = P.normal(P.cache_rows, D_QK)
    w = weight.cuda()
    table = P.table.clone()
    table[1, 3], table[1, 12] = P.pool, -1              # positions 48 .. 63 and 192 .. 199 of sequence 1
    x = P.buffers()
    dsa.mla_expand(P.batch, kv.cuda(), w, x, pages=dsa.make_pages(table.cuda(), 16, P.pool), ws=P.ws)
    assert dsa.read_device_status(P.ws) == 7
    dsa.reset_device_status(P.ws)
    lo = int(P.at[1])
    gone = torch.zeros(P.rows_x, dtype=torch.bool)
    gone[lo + 48:lo + 64] = True
    gone[lo + 192:lo + 200] = True
    assert x.kv[gone.cuda()].isnan().all() and x.k_pe[gone.cuda()].isnan().all()
    good = P.buffers()
    dsa.mla_expand(P.batch, kv.cuda(), w, good, pages=P.pages, ws=P.ws)
    assert torch.equal(x.kv[~gone.cuda()].nan_to_num(-7), good.kv[~gone.cuda()].nan_to_num(-7))
    assert torch.equal(x.k_pe[~gone.cuda()].nan_to_num(-7), good.k_pe[~gone.cuda()].nan_to_num(-7))
    assert dsa.read_device_status(P.ws) == 0
    for first, off in (([0, 201, 0], None), ([0, -1, 0], None), (None, [0, 64, 512, 768]), (None, [0, 256, 384, 10 ** 9]),
                       (None, [0, 512, 512, 768])):
        y = dsa.make_expanded(P.i32(off) if off else P.x_off, torch.full_like(x.kv, 5.0), torch.full_like(x.k_pe, 5.0))
        dsa.mla_expand(P.batch, kv.cuda(), w, y, first=P.i32(first) if first else None, pages=P.pages, ws=P.ws)
        assert dsa.read_device_status(P.ws) == 6
        dsa.reset_device_status(P.ws)
        o = off or [int(v) for v in P.at]
        if first or off == [0, 512, 512, 768]:          # sequence 1 alone
            assert torch.equal(y.kv[o[0]:o[0] + 40], good.kv[:40])
            lo = int(P.at[2])
            assert torch.equal(y.kv[o[2]:o[2] + 10], good.kv[lo:lo + 10])
            if first:
                assert (y.kv[o[1]:o[2]] == 5.0).all() and (y.k_pe[o[1]:o[2]] == 5.0).all()


# --------------------------------------------------------------- attention --

@pytest.mark.parametrize("c,m", [
    ([0], [1]), ([0], [2]), ([127], [1]), ([128], [1]), ([0], [128]), ([0], [129]), ([0], [256]), ([0], [257]),
    ([300], [5]), ([1], [255]), ([0, 0, 7, 513], [3, 0, 130, 260]), ([100] * 9, [1] * 9), ([2000], [300]),
    ([0, 31, 28, 0, 3], [32, 1, 4, 0, 29]), ([1020], [1]), ([500, 3, 0], [2, 1, 2]), ([5, 6, 7, 8], [5, 6, 7, 8]),
])
@pytest.mark.parametrize("max_ctx", [None, 20000])       # the bound on lengths, with that on new rows, chooses the kernel
def test_attention(c, m, max_ctx):
    P = Prompts(c, m, seed=sum(c) + sum(m), gap=128, pad=7, max_ctx=max_ctx)
    x = P.filled()
    q = P.normal(P.T + 7, H, D_HEAD).cuda()
    out = torch.full((P.T + 7, H, D_HEAD), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((P.T + 7, H), 9.0, device="cuda")
    dsa.prompt_mla_fwd(P.batch, q, x, SCALE, out, lse, ws=P.ws)
    assert dsa.read_device_status(P.ws) == 0
    check_attention(P, q, x, out, lse)
    assert (out[P.T:] == 9.0).all() and (lse[P.T:] == 9.0).all()
    again = torch.zeros_like(out)
    dsa.prompt_mla_fwd(P.batch, q, x, SCALE, again, None, ws=P.ws)
    assert torch.equal(out[:P.T], again[:P.T])


def test_long_attention():
    """More items than CTA pairs, and a long context: sampled rows and heads."""
    P = Prompts([0, 9000, 0], [3001, 700, 1024], seed=1)
    x = P.filled()
    q = P.normal(P.T, H, D_HEAD).cuda()
    out = torch.empty((P.T, H, D_HEAD), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((P.T, H), device="cuda")
    dsa.prompt_mla_fwd(P.batch, q, x, SCALE, out, lse, ws=P.ws)
    assert dsa.read_device_status(P.ws) == 0
    check_attention(P, q, x, out, lse, heads=[0, 1, 37, 63],
                    rows=[0, 1, 127, 128, 255, 256, 511, 699, 1023, 2000, 2815, 2816, 3000])


def test_moving_maxima():
    """Scores that grow along the context move the running maximum tile by tile; falling ones never."""
    P = Prompts([0, 0], [900, 900], seed=2)
    x = P.filled()
    q = P.normal(P.T, H, D_HEAD).cuda()
    ramp = torch.linspace(0, 3, 900, device="cuda")
    x.k_pe[:900] = (ramp[:, None] * torch.ones(D_ROPE, device="cuda")).bfloat16()
    lo = int(P.at[1])
    x.k_pe[lo:lo + 900] = (ramp.flip(0)[:, None] * torch.ones(D_ROPE, device="cuda")).bfloat16()
    q[..., 192:] = 4.0
    out = torch.empty((P.T, H, D_HEAD), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((P.T, H), device="cuda")
    dsa.prompt_mla_fwd(P.batch, q, x, SCALE, out, lse, ws=P.ws)
    for b in range(2):
        ref, z, big = attention_ref(P, q, x, b, [0, 5, 63])
        at = slice(int(P.off[b]), int(P.off[b]) + 900)
        # scores up to 48 + 10: their fp32 sums are off by 256 F32 (16 * 58)
        e = 256 * F32 * 58
        got, tol = out[at][:, [0, 5, 63]].cpu().double(), HALF * ref.abs() + (HALF * (1 + HALF) + 2 * e + 64 * F32) * big
        assert ((got - ref).abs() <= tol).all()
        assert ((lse[at][:, [0, 5, 63]].cpu().double() - z).abs() <= e + 16 * F32 * (1 + z.abs())).all()


@pytest.mark.parametrize("most", [128, 300])              # the bound on new rows chooses the kernel
@pytest.mark.parametrize("seed", range(5))
def test_random_batches(seed, most):
    rng = np.random.default_rng(200 + seed)
    n = int(rng.integers(1, 20))
    c = [int(x) for x in rng.choice([0, 0, 1, 5, 30, 63, 64, 100, 127, 128, 200, 500], n)]
    m = [int(x) for x in rng.choice([0, 1, 2, 5, 16, 17, 31, 32, 33, 48, 63, 64, 65, 90, 96, 97, 127, 128], n)]
    m[0] = max(m[0], 1)
    P = Prompts(c, m, seed=seed, gap=128, max_q=most, max_ctx=5000)
    x = P.filled()
    q = P.normal(P.T, H, D_HEAD).cuda()
    out = torch.empty((P.T, H, D_HEAD), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((P.T, H), device="cuda")
    dsa.prompt_mla_fwd(P.batch, q, x, SCALE, out, lse, ws=P.ws)
    assert dsa.read_device_status(P.ws) == 0
    check_attention(P, q, x, out, lse, heads=sorted(set(int(v) for v in rng.integers(0, H, 4))))


def test_many_items_of_few_rows():
    """More items than CTA pairs, of one to many tiles in turn, and rows at the ends of what a CTA and a warp hold."""
    c = [0, 900, 0, 64, 300, 0, 127, 40, 1500, 2, 250, 0, 129, 88]
    m = [64, 1, 65, 33, 97, 128, 1, 32, 31, 127, 96, 2, 63, 40]
    P = Prompts(c, m, seed=21, gap=128, pad=9, max_q=128)
    x = P.filled()
    q = P.normal(P.T + 9, H, D_HEAD).cuda()
    out = torch.full((P.T + 9, H, D_HEAD), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((P.T + 9, H), 9.0, device="cuda")
    dsa.prompt_mla_fwd(P.batch, q, x, SCALE, out, lse, ws=P.ws)
    assert dsa.read_device_status(P.ws) == 0
    check_attention(P, q, x, out, lse, heads=[0, 1, 29, 62, 63])
    assert (out[P.T:] == 9.0).all() and (lse[P.T:] == 9.0).all()
    for _ in range(20):                      # whatever order the pairs' parts come in
        again = torch.zeros_like(out)
        dsa.prompt_mla_fwd(P.batch, q, x, SCALE, again, None, ws=P.ws)
        assert torch.equal(out[:P.T], again[:P.T])


def test_moving_maxima_of_few_rows():
    """test_moving_maxima for at most 128 new rows."""
    P = Prompts([800, 803], [100, 97], seed=22, max_q=128)
    x = P.filled()
    q = P.normal(P.T, H, D_HEAD).cuda()
    ramp = torch.linspace(0, 3, 900, device="cuda")
    for b, r in ((0, ramp), (1, ramp.flip(0))):
        lo = int(P.at[b])
        x.k_pe[lo:lo + 900] = (r[:, None] * torch.ones(D_ROPE, device="cuda")).bfloat16()
    q[..., 192:] = 4.0
    out = torch.empty((P.T, H, D_HEAD), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((P.T, H), device="cuda")
    dsa.prompt_mla_fwd(P.batch, q, x, SCALE, out, lse, ws=P.ws)
    assert dsa.read_device_status(P.ws) == 0
    for b in range(2):
        ref, z, big = attention_ref(P, q, x, b, [0, 5, 63])
        at = slice(int(P.off[b]), int(P.off[b + 1]))
        e = 256 * F32 * 58                   # as there: the same scores
        got, tol = out[at][:, [0, 5, 63]].cpu().double(), HALF * ref.abs() + (HALF * (1 + HALF) + 2 * e + 64 * F32) * big
        assert ((got - ref).abs() <= tol).all()
        assert ((lse[at][:, [0, 5, 63]].cpu().double() - z).abs() <= e + 16 * F32 * (1 + z.abs())).all()


def test_masked_rows_do_not_leak_in_few_rows():
    """The same for the kernel of few rows over short contexts."""
    P = Prompts([5, 0, 0], [20, 9, 1], seed=16, gap=128, max_q=20, max_ctx=25)
    x = P.filled()
    q = P.normal(P.T, H, D_HEAD).cuda()
    out, out2 = (torch.empty((P.T, H, D_HEAD), dtype=torch.bfloat16, device="cuda") for _ in (0, 1))
    lse, lse2 = (torch.empty((P.T, H), device="cuda") for _ in (0, 1))
    dsa.prompt_mla_fwd(P.batch, q, x, SCALE, out, lse, ws=P.ws)
    x.k_pe[12] = float("nan")                # position 12: new row 7 of sequence 0 and later see it
    x.kv[15, 4, 192:] = float("inf")
    x.kv[int(P.at[1]) + 8] = float("nan")    # the last row of sequence 1
    q[3, 9] = float("-inf")
    dsa.prompt_mla_fwd(P.batch, q, x, SCALE, out2, lse2, ws=P.ws)
    assert dsa.read_device_status(P.ws) == 0
    hurt = torch.zeros(P.T, dtype=torch.bool)
    hurt[7:20] = True
    hurt[28] = True
    assert out2[hurt.cuda()].isnan().all() and lse2[hurt.cuda()].isnan().all()
    keep = ~hurt
    keep[3] = False
    keep = keep.cuda()
    assert torch.equal(out[keep], out2[keep]) and torch.equal(lse[keep], lse2[keep])
    heads = torch.arange(H, device="cuda") != 9
    assert torch.equal(out[3][heads], out2[3][heads]) and out2[3, 9].isnan().all()


def test_masked_rows_do_not_leak_in_short_items():
    """The same for items of at most 128 rows on the tensor cores, among others."""
    m = [20, 9, 1, 128, 70, 3] * 3
    P = Prompts([105, 0, 300] * 6, m, seed=23, gap=128, max_q=128)
    x = P.filled()
    q = P.normal(P.T, H, D_HEAD).cuda()
    out, out2 = (torch.empty((P.T, H, D_HEAD), dtype=torch.bfloat16, device="cuda") for _ in (0, 1))
    lse, lse2 = (torch.empty((P.T, H), device="cuda") for _ in (0, 1))
    dsa.prompt_mla_fwd(P.batch, q, x, SCALE, out, lse, ws=P.ws)
    x.k_pe[int(P.at[0]) + 112] = float("nan")            # new row 7 of sequence 0 and later see it
    x.kv[int(P.at[3]) + 200, 4, 192:] = torch.finfo(torch.bfloat16).max    # row 95 of sequence 3 and later
    x.k_pe[int(P.at[4]) + 69] = float("inf")             # sequence 4's last row
    q[int(P.off[6]) + 3, 9] = float("-inf")
    dsa.prompt_mla_fwd(P.batch, q, x, SCALE, out2, lse2, ws=P.ws)
    assert dsa.read_device_status(P.ws) == 0
    hurt = torch.zeros(P.T, H, dtype=torch.bool)
    hurt[7:20] = True
    hurt[int(P.off[5]) - 1] = True
    hurt[int(P.off[6]) + 3, 9] = True
    hurt = hurt.cuda()
    assert out2[hurt].isnan().all()
    moved = hurt.clone()
    moved[int(P.off[3]) + 95:int(P.off[4]), 4] = True
    assert torch.equal(out[~moved], out2[~moved]) and torch.equal(lse[~hurt], lse2[~hurt])


def test_masked_rows_do_not_leak():
    """Whatever later rows of the sequence, other sequences and the space between hold, a row gets what it sees."""
    P = Prompts([40, 0], [300, 100], seed=6, gap=256)
    x = P.filled()
    q = P.normal(P.T, H, D_HEAD).cuda()
    out, out2 = (torch.empty((P.T, H, D_HEAD), dtype=torch.bfloat16, device="cuda") for _ in (0, 1))
    lse, lse2 = (torch.empty((P.T, H), device="cuda") for _ in (0, 1))
    dsa.prompt_mla_fwd(P.batch, q, x, SCALE, out, lse, ws=P.ws)
    big = torch.finfo(torch.bfloat16).max
    x.k_pe[201] = float("nan")               # position 201: new row 161 of sequence 0 and later see it
    x.kv[260:340, :, 192:] = big             # later values at the type's end, seen by rows 220 and later
    q[161 + 30] = float("nan")
    q[50, 3] = float("inf")
    dsa.prompt_mla_fwd(P.batch, q, x, SCALE, out2, lse2, ws=P.ws)
    assert dsa.read_device_status(P.ws) == 0
    rows = torch.arange(P.T, device="cuda")
    hurt = (rows >= 161) & (rows < 300)
    assert out2[hurt].isnan().all() and lse2[hurt].isnan().all()
    keep = ~hurt
    keep[50] = False
    assert torch.equal(out[keep], out2[keep]) and torch.equal(lse[keep], lse2[keep])
    heads = torch.arange(H, device="cuda") != 3
    assert torch.equal(out[50][heads], out2[50][heads]) and out2[50, 3].isnan().all()


def test_bad_batches():
    P = Prompts([10, 0, 3], [20, 30, 40], seed=7)
    x = P.filled()
    q = P.normal(P.T, H, D_HEAD).cuda()
    ref = torch.empty((P.T, H, D_HEAD), dtype=torch.bfloat16, device="cuda")
    dsa.prompt_mla_fwd(P.batch, q, x, SCALE, ref, ws=P.ws)
    for off in ([0, 1, 128, 384], [0, 128, 128, 384], [0, -128, 256, 384], [0, 128, 1 << 30, 384], [128, 256, 384, 385]):
        y = dsa.make_expanded(P.i32(off), x.kv, x.k_pe)
        out = torch.full_like(ref, 3.0)
        dsa.prompt_mla_fwd(P.batch, q, y, SCALE, out, ws=P.ws)
        assert dsa.read_device_status(P.ws) == 6
        dsa.reset_device_status(P.ws)
        assert (out == 3.0).any()
    bad = dsa.Batch(P.i32([0, 20, 50, 90]), P.i32([30, 29, 43]), P.max_q, P.max_ctx, P.stride, total_q=90)
    out = torch.full_like(ref, 3.0)
    dsa.prompt_mla_fwd(bad, q, x, SCALE, out, ws=P.ws)
    assert dsa.read_device_status(P.ws) == 6
    assert torch.equal(out[:20], ref[:20]) and torch.equal(out[50:], ref[50:]) and (out[20:50] == 3.0).all()


def test_many_sequences():
    """65,535 sequences, few with rows."""
    B = 65535
    c, m = np.zeros(B, np.int64), np.zeros(B, np.int64)
    for b, (k, n) in {0: (3, 1), 77: (0, 200), 40000: (130, 2), B - 1: (0, 3)}.items():
        c[b], m[b] = k, n
    P = Prompts(c, m, seed=8)
    x = P.filled()
    q = P.normal(P.T, H, D_HEAD).cuda()
    out = torch.empty((P.T, H, D_HEAD), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((P.T, H), device="cuda")
    dsa.prompt_mla_fwd(P.batch, q, x, SCALE, out, lse, ws=P.ws)
    assert dsa.read_device_status(P.ws) == 0
    check_attention(P, q, x, out, lse, heads=[0, 13])


def test_empty_calls(weight):
    P = Prompts([0, 5], [0, 0], seed=8)
    x = P.filled()
    q = torch.empty((0, H, D_HEAD), dtype=torch.bfloat16, device="cuda")
    dsa.prompt_mla_fwd(P.batch, q, x, SCALE, q, ws=P.ws)
    none = dsa.make_expanded(P.i32([0, 0, 0]), x.kv[:0], x.k_pe[:0])
    z = dsa.make_batch(P.i32([0, 0, 0]), P.i32([0, 0]), 0, 0, 1, total_q=0)
    dsa.mla_expand(z, torch.empty((2, D_QK), dtype=torch.bfloat16, device="cuda"), weight.cuda(), none, ws=P.ws)
    assert dsa.read_device_status(P.ws) == 0


# ----------------------------------------------------------------- refusals --

def test_refusals(weight):
    P = Prompts([0], [20], seed=1)
    x = P.filled()
    q = P.normal(20, H, D_HEAD).cuda()
    out = torch.empty_like(q)
    kv, w = P.normal(P.cache_rows, D_QK).cuda(), weight.cuda()
    with pytest.raises(ValueError):
        dsa.make_expanded(P.x_off, x.kv, x.k_pe[:5])
    with pytest.raises(TypeError):
        dsa.make_expanded(P.x_off.long(), x.kv, x.k_pe)
    with pytest.raises(ValueError):
        dsa.prompt_mla_fwd(P.batch, q, dsa.make_expanded(P.x_off[:1], x.kv, x.k_pe), SCALE, out, ws=P.ws)
    for bad in (dict(q=q.float()), dict(q=q[:19]), dict(out=out.cpu()), dict(lse=torch.empty(5, device="cuda"))):
        a = dict(dict(q=q, out=out, lse=None), **bad)
        with pytest.raises((TypeError, ValueError)):
            dsa.prompt_mla_fwd(P.batch, a["q"], x, SCALE, a["out"], a["lse"], ws=P.ws)
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(dsa.DsaError):
            dsa.prompt_mla_fwd(P.batch, q, x, scale, out, ws=P.ws)
    for ws in (None, P.ws[:128]):
        with pytest.raises(dsa.DsaError):
            dsa.prompt_mla_fwd(P.batch, q, x, SCALE, out, ws=ws)
        with pytest.raises(dsa.DsaError):
            dsa.mla_expand(P.batch, kv, w, x, ws=ws)
    for bad in (dict(kv=kv[:5]), dict(w=w[:5]), dict(first=P.x_off.long()), dict(kv=kv.float())):
        a = dict(dict(kv=kv, w=w, first=None), **bad)
        with pytest.raises((TypeError, ValueError)):
            dsa.mla_expand(P.batch, a["kv"], a["w"], x, first=a["first"], ws=P.ws)


# ----------------------------------------------------------------- together --

def test_prompt_from_projections_to_output(weight):
    """Tables, rotation, latent rows, expansion, attention and o_proj of a prompt in two chunks over pages, captured
    and replayed: each step against its own inputs, and the expanded result against the absorbed one."""
    P = Prompts([0, 0], [200, 333], 64, seed=21)
    rows = [150, 170]                        # of the first chunk
    tws, mws = dsa.tree_workspace(), dsa.mla_workspace(P.T)
    w = weight.cuda()
    w_o = (torch.randn((6144, H * D_HEAD), generator=P.gen) / 128).bfloat16().cuda()
    cos, sin = (torch.empty((512, D_ROPE), device="cuda") for _ in (0, 1))
    gamma = torch.ones(D_LAT, device="cuda")
    kv = torch.zeros((P.cache_rows, D_QK), dtype=torch.bfloat16, device="cuda")
    x = P.buffers(0.0)
    hidden, q = torch.empty((P.T, D_QK), dtype=torch.bfloat16, device="cuda"), torch.empty((P.T, H, D_HEAD), dtype=torch.bfloat16, device="cuda")
    out, y = torch.empty_like(q), torch.empty((P.T, 6144), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((P.T, H), device="cuda")
    steps = []
    for lo, hi in (([0, 0], rows), (rows, P.L)):
        n = [b - a for a, b in zip(lo, hi)]
        pick = torch.cat([torch.arange(a, b) + int(P.off[i]) for i, (a, b) in enumerate(zip(lo, hi))]).cuda()
        batch = dsa.make_batch(P.i32([0, n[0], sum(n)]), P.i32(hi), max(n), P.max_ctx, P.stride, total_q=sum(n))
        pos = torch.cat([torch.arange(a, b) for a, b in zip(lo, hi)]).int().cuda()
        slots = torch.cat([P.slots(i, a, b) for i, (a, b) in enumerate(zip(lo, hi))]).int().cuda()
        steps.append((batch, P.i32(lo), pick, pos, slots))
    scratch = [(torch.empty((len(s[2]), H, D_HEAD), dtype=torch.bfloat16, device="cuda"), torch.empty((len(s[2]), H), device="cuda"))
               for s in steps]
    turned = torch.empty_like(q)

    def run():
        dsa.rope_table(cos, sin, 10000.0)
        for (batch, first, pick, pos, slots), (o, l) in zip(steps, scratch):
            part = q[pick]
            dsa.rope(part[..., 192:], cos, sin, pos, ws=tws)
            turned[pick] = part
            dsa.latent_append(hidden[pick], gamma, 1e-5, cos, sin, pos, slots, kv, ws=tws)
            dsa.mla_expand(batch, kv, w, x, first=first, pages=P.pages, ws=P.ws)
            dsa.prompt_mla_fwd(batch, part, x, SCALE, o, l, ws=P.ws)
            out[pick], lse[pick] = o, l
        dsa.mla_o_proj(out, w_o, y, mws)

    hidden.normal_()
    q.normal_()
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for seed in range(2):
        torch.cuda.manual_seed(seed)
        hidden.normal_()
        q.normal_()
        g.replay()
        torch.cuda.synchronize()
        assert [dsa.read_device_status(t) for t in (tws, mws, P.ws)] == [0, 0, 0]
        _check_expansion(P, x, kv.cpu(), weight, [0, 0], before=(x.kv.cpu(), x.k_pe.cpu()))
        check_attention(P, turned, x, out, lse, heads=[0, 31, 63])
        ref = out.view(P.T, -1).double().cpu()[:40] @ w_o.double().cpu().t()
        size = out.view(P.T, -1).double().cpu()[:40].abs() @ w_o.double().cpu().abs().t()
        assert ((y[:40].cpu().double() - ref).abs() <= HALF * ref.abs() + 16384 * F32 * (1 + HALF) * size).all()
        # the absorbed form of the same attention, head by head in 64 bits from the latent rows
        wd = weight.double().view(H, D_EXP, D_LAT)
        for b in range(2):
            c = kv.cpu()[P.slots(b, 0, P.L[b])].double()
            qd = turned[int(P.off[b]):int(P.off[b]) + P.m[b]].cpu().double()
            for h in (0, 40):
                qa = torch.cat([qd[:, h, :192] @ wd[h, :192], qd[:, h, 192:]], 1)
                s = (qa @ c.t() * SCALE).masked_fill(torch.ones(P.m[b], P.L[b], dtype=torch.bool).triu(1), float("-inf"))
                p = torch.softmax(s, -1)
                o = p @ c[:, :D_LAT] @ wd[h, 192:].t()
                # keys and values rounded to bf16: scores off by HALF |q| |k| at most, here under 0.04; three
                # roundings of HALF of values and weights
                got = out[int(P.off[b]):int(P.off[b]) + P.m[b], h].cpu().double()
                tol = 0.1 * (p @ (c[:, :D_LAT] @ wd[h, 192:].t()).abs()) + 1e-6
                assert ((got - o).abs() <= tol).all()


def test_two_streams():
    """Two calls at once, each with its own workspace."""
    P, Q = Prompts([0], [700], seed=31), Prompts([300], [500], seed=32)
    xs, qs = [P.filled(), Q.filled()], [p.normal(p.T, H, D_HEAD).cuda() for p in (P, Q)]
    outs = [torch.empty_like(q) for q in qs]
    refs = [torch.empty_like(q) for q in qs]
    for p, x, q, r in zip((P, Q), xs, qs, refs):
        dsa.prompt_mla_fwd(p.batch, q, x, SCALE, r, ws=p.ws)
    torch.cuda.synchronize()
    ss = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for p, x, q, o, s in zip((P, Q), xs, qs, outs, ss):
            dsa.prompt_mla_fwd(p.batch, q, x, SCALE, o, ws=p.ws, stream=s)
    torch.cuda.synchronize()
    for o, r in zip(outs, refs):
        assert torch.equal(o, r)

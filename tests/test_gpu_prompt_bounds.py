"""Calls for prompts and shared prefixes at the ends of what they take: workspaces of the size asked for, batches of
more sequences than a CTA plans, offsets past 32 bits, workspaces used again."""

import numpy as np
import pytest
import torch

import sparse_attention_gb300 as dsa
from prompt_case import D_EXP, D_HEAD, D_LAT, D_QK, D_ROPE, F32, H, HALF, SCALE, Prompts, check_attention, expand_ref
from test_gpu_prefix import Shared
from tree_case import check_attention as check_latent

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from sparse_attention_gb300 import build as B
    B.build()
    dsa.load_library()


@pytest.fixture(scope="module")
def weight():
    g = torch.Generator().manual_seed(6)
    return (torch.randn((H * D_EXP, D_LAT), generator=g) / D_LAT ** 0.5).bfloat16()


class Guarded:
    """A workspace of n bytes, the status word cleared, in front of bytes that nothing may write."""

    def __init__(self, n):
        self.all = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        self.ws = self.all[:n]
        dsa.reset_device_status(self.ws)

    def check(self, status=0):
        assert dsa.read_device_status(self.ws) == status
        assert (self.all[self.ws.numel():] == 0xA5).all()


@pytest.mark.parametrize("c,m", [([0], [70]), ([5] * 600, [1] * 600), ([0] * 384, [3] * 384), ([0] * 385, [3] * 385),
                                 ([0] * 512, [2] * 512), ([2] * 513, [2] * 513), ([130] * 3, [400] * 3)])
@pytest.mark.parametrize("max_ctx", [None, 3000])
def test_expanded_form(weight, c, m, max_ctx):
    """Up to 384 and 512 sequences the tensor kernels plan by themselves, above them a launch before."""
    P = Prompts(c, m, 16, seed=len(c), max_ctx=max_ctx)
    P.ws = (g := Guarded(P.ws.numel())).ws
    kv = P.normal(P.cache_rows, D_QK)
    x = P.buffers()
    for _ in range(2):
        dsa.mla_expand(P.batch, kv.cuda(), weight.cuda(), x, pages=P.pages, ws=P.ws)
    g.check()
    q = P.normal(P.T, H, D_HEAD).cuda()
    out, lse = torch.empty((P.T, H, D_HEAD), dtype=torch.bfloat16, device="cuda"), torch.empty((P.T, H), device="cuda")
    for _ in range(3):
        out.zero_()
        dsa.prompt_mla_fwd(P.batch, q, x, SCALE, out, lse, ws=P.ws)
    g.check()
    pick = [0, 1, P.B // 2, P.B - 1]
    for b in sorted(set(p for p in pick if p < P.B)):
        lo, n = int(P.at[b]), P.L[b]
        rows = kv[P.slots(b, 0, n)]
        ref, size = expand_ref(rows, weight)
        assert ((x.kv[lo:lo + n].cpu().double() - ref).abs() <= HALF * ref.abs() + 512 * F32 * (1 + HALF) * size).all()
        assert torch.equal(x.k_pe[lo:lo + n].cpu(), rows[:, D_LAT:])
    check_attention(P, q, x, out, lse, heads=[0, 29, 63])


@pytest.mark.parametrize("c,m,first,share,page", [
    ([1500] * 4, [8] * 4, [0, 4], [1408], 64), ([30000, 30010], [3, 1], [0, 2], [29952], 0),
    ([260] * 300, [1] * 300, [0, 100, 300], [256, 128], 16), ([130] * 1100, [1] * 1100, [0, 1100], [128], 16),
    ([128 + b % 3 for b in range(700)], [b % 3 for b in range(700)], list(range(0, 701, 2)), [128] * 350, 32),
])
def test_shared_prefixes(c, m, first, share, page):
    """Up to 1,024 groups and sequences are planned from shared memory, more from the workspace."""
    st = Shared(c, m, first, share, page, seed=len(c))
    q, kv = st.inputs()
    g = Guarded(st.ws.numel())
    st.ws = g.ws
    for _ in range(2):
        out, lse = st.prefix(q, kv)
    g.check()
    rng = np.random.default_rng(1)
    check_latent(st, q, kv, out, lse, rows=set(int(r) for r in rng.integers(0, st.T, 40)) | {0, st.T - 1})


def test_far_expanded_rows(weight):
    """A sequence whose expanded rows lie past 2^31 elements and 2^32 bytes of the buffer."""
    P = Prompts([0, 3], [140, 70], seed=2)
    far = 150016
    P.at = np.asarray([256, far, far + 128])
    P.rows_x = far + 128
    kv = P.normal(P.cache_rows, D_QK)
    x = dsa.make_expanded(P.i32(P.at), torch.zeros((P.rows_x, H, D_EXP), dtype=torch.bfloat16, device="cuda"),
                          torch.zeros((P.rows_x, D_ROPE), dtype=torch.bfloat16, device="cuda"))
    dsa.mla_expand(P.batch, kv.cuda(), weight.cuda(), x, first=P.i32([0, 1]), ws=P.ws)
    for b, f in ((0, 0), (1, 1)):
        lo, n = int(P.at[b]), P.L[b]
        ref, size = expand_ref(kv[P.slots(b, f, n)], weight)
        assert ((x.kv[lo + f:lo + n].cpu().double() - ref).abs() <= HALF * ref.abs() + 512 * F32 * (1 + HALF) * size).all()
    assert (x.kv[far] == 0).all() and (x.kv[:256] == 0).all()
    q = P.normal(P.T, H, D_HEAD).cuda()
    out = torch.empty((P.T, H, D_HEAD), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((P.T, H), device="cuda")
    dsa.prompt_mla_fwd(P.batch, q, x, SCALE, out, lse, ws=P.ws)
    assert dsa.read_device_status(P.ws) == 0
    check_attention(P, q, x, out, lse, heads=[0, 63])


@pytest.mark.parametrize("n", [9, 300])
def test_far_query_rows(n):
    """New rows past 2^31 elements of q and out."""
    P = Prompts([10], [n], seed=3)
    far = 140000
    batch = dsa.Batch(P.i32([far, far + n]), P.i32(P.L), n, P.max_ctx, P.stride, total_q=far + n)
    x = P.filled()
    q = torch.zeros((far + n, H, D_HEAD), dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 5.0)
    lse = torch.full((far + n, H), 5.0, device="cuda")
    q[far:] = P.normal(n, H, D_HEAD).cuda()
    ws = dsa.prompt_workspace(batch)
    dsa.prompt_mla_fwd(batch, q, x, SCALE, out, lse, ws=ws)
    assert dsa.read_device_status(ws) == 0
    check_attention(P, q[far:], x, out[far:], lse[far:], heads=[0, 63])
    assert (out[far - 1] == 5.0).all() and (lse[:far] == 5.0).all()


def test_far_rotated_rows():
    """Token strides whose offsets pass 32 bits."""
    ws = dsa.tree_workspace()
    cos, sin = (torch.empty((64, 64), device="cuda") for _ in (0, 1))
    dsa.rope_table(cos, sin, 10000.0)
    big = torch.zeros(300 * (1 << 24) // 2, dtype=torch.bfloat16, device="cuda")       # 5 GB
    x = torch.as_strided(big, (150, 2, 64), (1 << 24, 64, 1))
    x.copy_(torch.randn((150, 2, 64), device="cuda", dtype=torch.bfloat16))
    pos = torch.arange(150, device="cuda", dtype=torch.int32) % 64
    near = x.contiguous()
    dsa.rope(x, cos, sin, pos, ws=ws)
    dsa.rope(near, cos, sin, pos, ws=ws)
    assert torch.equal(x, near) and dsa.read_device_status(ws) == 0


def test_one_workspace_for_many_calls(weight):
    """Calls of different sizes that follow one another in one workspace, between them one whose sequences are all
    refused, and a cleared status word."""
    big = Prompts([0, 40, 900], [513, 300, 129], 16, seed=4)
    small = Prompts([10] * 20, [9] * 20, 16, seed=5)
    ws = dsa.prompt_workspace(small.batch if small.ws.numel() > big.ws.numel() else big.batch)
    done = []
    for P in (big, small, big, small, small, big):
        kv = P.normal(P.cache_rows, D_QK)
        x = P.buffers()
        dsa.mla_expand(P.batch, kv.cuda(), weight.cuda(), x, pages=P.pages, ws=ws)
        q = P.normal(P.T, H, D_HEAD).cuda()
        out = torch.empty((P.T, H, D_HEAD), dtype=torch.bfloat16, device="cuda")
        dsa.prompt_mla_fwd(P.batch, q, x, SCALE, out, ws=ws)
        done.append((P, q, x, out))
        wrong = dsa.make_expanded(x.off + 1, x.kv, x.k_pe)
        dsa.prompt_mla_fwd(P.batch, q, wrong, SCALE, torch.empty_like(out), ws=ws)
        dsa.reset_device_status(ws)
    assert dsa.read_device_status(ws) == 0
    for P, q, x, out in done:
        check_attention(P, q, x, out, None, heads=[7])


def test_captured_prompts_of_changing_lengths():
    """One graph of two calls over one workspace, replayed with other lengths and places."""
    P = Prompts([100, 0, 300], [200, 40, 150], seed=6, gap=256)
    x = P.filled()
    q = P.normal(P.T, H, D_HEAD).cuda()
    out, out2 = (torch.zeros((P.T, H, D_HEAD), dtype=torch.bfloat16, device="cuda") for _ in (0, 1))
    lse = torch.zeros((P.T, H), device="cuda")
    batch = dsa.Batch(P.i32(P.off), P.i32(P.L), 200, P.max_ctx, P.stride, total_q=P.T)

    def call():
        dsa.prompt_mla_fwd(batch, q, x, SCALE, out, lse, ws=P.ws)
        dsa.prompt_mla_fwd(batch, q, x, SCALE, out2, None, ws=P.ws)

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for m in ([200, 40, 150], [1, 0, 2], [0, 0, 150], [130, 7, 129]):
        P.m = m
        P.c = [n - k for n, k in zip((300, 40, 450), m)]
        P.L = [a + b for a, b in zip(P.c, P.m)]
        P.off = np.concatenate([[0], np.cumsum(m)]).astype(np.int64)
        batch.q_off.copy_(P.i32(P.off))
        batch.ctx_len.copy_(P.i32(P.L))
        out.fill_(3.0)
        out2.fill_(3.0)
        g.replay()
        torch.cuda.synchronize()
        assert dsa.read_device_status(P.ws) == 0 and torch.equal(out, out2)
        assert (out[int(P.off[-1]):] == 3.0).all()
        check_attention(P, q, x, out, lse, heads=[0, 50])

"""Expanded rows without a room for a sequence: which sequences are skipped, that they are reported, and that the
others get their results."""

import pytest
import torch

import sparse_attention_gb300 as dsa
from prompt_case import D_HEAD, D_ROPE, F32, H, HALF, SCALE, Prompts, check_attention, expand_ref, up

pytestmark = pytest.mark.gpu
BAD_BATCH = 6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from sparse_attention_gb300 import build as B
    B.build()
    dsa.load_library()


@pytest.mark.parametrize("max_q,max_ctx", [(20, 25), (20, 3000), (300, 3000), (1 << 19, 1 << 19)])      # each of the kernels
def test_no_rows_at_all(max_q, max_ctx):
    """Buffers of no rows: every sequence with new rows is left as it was, and reported."""
    P = Prompts([5, 0, 0, 3], [20, 0, 7, 1], max_q=max_q, max_ctx=max_ctx)
    q = P.normal(P.T, H, D_HEAD).cuda()
    none = dsa.make_expanded(P.i32([0] * 5), torch.empty((0, H, 448), dtype=torch.bfloat16, device="cuda"),
                             torch.empty((0, D_ROPE), dtype=torch.bfloat16, device="cuda"))
    out, lse = torch.full_like(q, 3.0), torch.full((P.T, H), 3.0, device="cuda")
    dsa.prompt_mla_fwd(P.batch, q, none, SCALE, out, lse, ws=P.ws)
    assert dsa.read_device_status(P.ws) == BAD_BATCH
    assert (out == 3.0).all() and (lse == 3.0).all()
    dsa.reset_device_status(P.ws)
    # bounds that leave room for rows, and lengths that have none: nothing is wrong
    P.batch.q_off.zero_()
    dsa.prompt_mla_fwd(P.batch, q, none, SCALE, out, lse, ws=P.ws)
    assert dsa.read_device_status(P.ws) == 0 and (out == 3.0).all() and (lse == 3.0).all()


BOUNDS = [(8, 13), (128, 3000), (300, 3000)]                  # each of the kernels


@pytest.mark.parametrize("idle", [0, 600])                    # (planned by a launch of their own)
@pytest.mark.parametrize("max_q,max_ctx", BOUNDS)
@pytest.mark.parametrize("off,good", [
    ([0, 128, 256, 384], [0, 1, 2]), ([0, 1, 128, 384], [2]), ([0, 128, 128, 384], [0, 2]), ([0, -128, 256, 384], [2]),
    ([0, 128, 1 << 30, 384], [0]), ([128, 256, 384, 385], [0, 1]), ([0, 128, 256, 383], [0, 1]), ([16, 144, 272, 384], []),
    ([0, 128, -2 ** 31, 2 ** 31 - 1], [0]), ([256, 384, 0, 128], [0, 2]),
])
def test_rooms(off, good, max_q, max_ctx, idle):
    """Sequences of rooms that are too small, unaligned, outside the buffers or upside down are skipped, all others computed."""
    P = Prompts([5, 0, 3] + [0] * idle, [8, 7, 6] + [0] * idle, max_q=max_q, max_ctx=max_ctx)
    gen = torch.Generator(device="cuda").manual_seed(1)
    kv = torch.randn((384, H, 448), generator=gen, device="cuda").bfloat16()
    k_pe = torch.randn((384, D_ROPE), generator=gen, device="cuda").bfloat16()
    x = dsa.make_expanded(P.i32(off + [off[-1]] * idle), kv, k_pe)
    q = P.normal(P.T, H, D_HEAD).cuda()
    out, lse = torch.full_like(q, 3.0), torch.full((P.T, H), 3.0, device="cuda")
    dsa.prompt_mla_fwd(P.batch, q, x, SCALE, out, lse, ws=P.ws)
    assert dsa.read_device_status(P.ws) == (0 if good == [0, 1, 2] else BAD_BATCH)
    skipped = torch.zeros(P.T, dtype=torch.bool)
    for b in range(3):
        if b not in good:
            skipped[int(P.off[b]):int(P.off[b + 1])] = True
            P.m[b] = 0                                        # (not checked below)
    skipped = skipped.cuda()
    assert (out[skipped] == 3.0).all() and (lse[skipped] == 3.0).all()
    P.at = off
    check_attention(P, q, x, out, lse)


@pytest.mark.parametrize("idle", [0, 400])
@pytest.mark.parametrize("off,good", [
    ([0, 128, 384, 768], [0, 1, 2]), ([0, 64, 512, 768], [2]), ([0, 256, 384, 10 ** 9], [0]), ([0, 512, 512, 768], [0, 2]),
    ([0, 128, 384, 769], [0, 1]), ([640, 768, 0, 128], [0, 2]), ([0, 128, -2 ** 31, 2 ** 31 - 1], [0]), ([16, 144, 400, 768], []),
])
def test_rooms_of_expansion(off, good, idle):
    P = Prompts([0, 0, 0] + [0] * idle, [40, 200, 10] + [0] * idle, 16, seed=4)
    gen = torch.Generator(device="cuda").manual_seed(2)
    kv = torch.randn((P.cache_rows, 576), generator=gen, device="cuda").bfloat16()
    w = (torch.randn((H * 448, 512), generator=gen, device="cuda") / 22).bfloat16()
    x = dsa.make_expanded(P.i32(off + [off[-1]] * idle), torch.full((768, H, 448), 5.0, dtype=torch.bfloat16, device="cuda"),
                          torch.full((768, D_ROPE), 5.0, dtype=torch.bfloat16, device="cuda"))
    dsa.mla_expand(P.batch, kv, w, x, pages=P.pages, ws=P.ws)
    assert dsa.read_device_status(P.ws) == (0 if good == [0, 1, 2] else BAD_BATCH)
    left = torch.ones(768, dtype=torch.bool, device="cuda")
    for b in good:
        lo, n = off[b], P.L[b]
        rows = kv[P.slots(b, 0, n).cuda()].cpu()
        ref, size = expand_ref(rows, w.cpu())
        err = (x.kv[lo:lo + n].cpu().double() - ref).abs()
        assert (err <= HALF * ref.abs() + 512 * F32 * (1 + HALF) * size).all(), b
        assert torch.equal(x.k_pe[lo:lo + n].cpu(), rows[:, 512:])
        assert (x.kv[lo + n:lo + up(n, 16)] == 0).all() and (x.k_pe[lo + n:lo + up(n, 16)] == 0).all()
        left[lo:lo + up(n, 16)] = False
    assert (x.kv[left] == 5.0).all() and (x.k_pe[left] == 5.0).all()

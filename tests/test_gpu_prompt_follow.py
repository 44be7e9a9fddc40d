"""Items of few new rows and very different lengths in turn: the softmax warps of one item follow the other ones' items."""

import pytest
import torch

import sparse_attention_gb300 as dsa
from prompt_case import D_HEAD, D_NOPE, F32, H, HALF, SCALE, Prompts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from sparse_attention_gb300 import build as B
    B.build()
    dsa.load_library()


def _filled(P):
    """Finite expanded rows throughout, made on the device."""
    gen = torch.Generator(device="cuda").manual_seed(P.T)
    x = P.buffers(0.0)
    x.kv.normal_(generator=gen)
    x.k_pe.normal_(generator=gen)
    return x


def _check(P, q, x, out, lse, heads):
    """In 64 bits on the device.  Scores and weights as in prompt_case.check_attention (an error e of the scores, HALF of a
    weight).  A tile adds 8 products of 16 positions to the results and 18 sums to a weight's, each with an fp32
    rounding, taken as a truncation (2 F32), of at most what the weights' sizes add up to."""
    for b in range(P.B):
        lo, n, L = int(P.at[b]), P.m[b], P.L[b]
        rows = slice(int(P.off[b]), int(P.off[b]) + n)
        seen = torch.arange(L, device="cuda")[None, :] <= (P.c[b] + torch.arange(n, device="cuda"))[:, None]
        e, steps = 256 * F32 * 20, (8 * 16 + 18) * (-(-L // 128)) * 2 * F32
        for h in heads:
            k = torch.cat([x.kv[lo:lo + L, h, :D_NOPE], x.k_pe[lo:lo + L]], 1).double()
            v = x.kv[lo:lo + L, h, D_NOPE:].double()
            s = torch.where(seen, q[rows, h].double() @ k.t() * SCALE, float("-inf"))
            z = torch.logsumexp(s, -1)
            p = torch.exp(s - z[:, None])
            ref, big = p @ v, p @ v.abs()
            tol = HALF * ref.abs() + (HALF * (1 + HALF) + 2 * e + steps) * big
            err = (out[rows, h].double() - ref).abs()
            assert (err <= tol).all(), (b, h, (err / tol).max())
            assert ((lse[rows, h].double() - z).abs() <= e + steps + 16 * F32 * (1 + z.abs())).all(), (b, h)


@pytest.mark.parametrize("c,m", [
    ([24000, 0, 31000, 3, 15000, 0, 2], [5, 60, 128, 1, 17, 128, 33]),       # long ones between those of one tile
    ([30000, 0], [3, 2]), ([0, 30000], [128, 1]), ([40000], [9]),            # one behind the other in each pair
    ([0] * 9 + [20000] + [0] * 9, [1, 128, 7] * 6 + [64]),                   # one among many
])
def test_long_items_between_short_ones(c, m):
    P = Prompts(c, m, seed=len(c), max_q=128)
    x = _filled(P)
    q = torch.randn((P.T, H, D_HEAD), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").bfloat16()
    out = torch.full((P.T, H, D_HEAD), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((P.T, H), 9.0, device="cuda")
    dsa.prompt_mla_fwd(P.batch, q, x, SCALE, out, lse, ws=P.ws)
    assert dsa.read_device_status(P.ws) == 0
    _check(P, q, x, out, lse, [0, 37, 63])
    for _ in range(10):
        again, lagain = torch.zeros_like(out), torch.zeros_like(lse)
        dsa.prompt_mla_fwd(P.batch, q, x, SCALE, again, lagain, ws=P.ws)
        assert torch.equal(out, again) and torch.equal(lse, lagain)
    assert dsa.read_device_status(P.ws) == 0

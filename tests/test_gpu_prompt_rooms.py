"""Expanded rows without a room for a sequence: which sequences are skipped, that they are reported, and that the
others get their results."""

import pytest
import torch

import sparse_attention_gb300 as dsa
from prompt_case import D_HEAD, D_ROPE, H, SCALE, Prompts

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

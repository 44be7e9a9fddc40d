"""Both forms of the kernels' bounded wait run out after their limit."""

import time

import pytest
import torch

import sparse_attention_gb300 as dsa

pytestmark = pytest.mark.gpu


def test_each_wait_takes_its_limit():
    from sparse_attention_gb300 import build as B
    B.build()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    limit = 0.1
    for _ in range(2):                                     # the first call loads the kernel
        dsa.reset_device_status(ws)
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        dsa.selftest_wait_timeout(ws, limit_us=int(limit * 1e6))
        assert dsa.read_device_status(ws) == 5             # DSA_ERR_TIMEOUT, from either
        took = time.perf_counter() - t0
    # one limit for each form (less the hundredth that clocks may differ by), and not many more polls
    assert 2 * limit * 0.99 <= took <= 2 * limit + 1.0, took

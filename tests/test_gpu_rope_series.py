"""Rotary tables against what their series and roundings allow, value by value."""

import numpy as np
import pytest
import torch

import sparse_attention_gb300 as dsa

pytestmark = pytest.mark.gpu
F32 = 2.0 ** -24             # half a step of fp32, relative


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from sparse_attention_gb300 import build as B
    B.build()
    dsa.load_library()


@pytest.mark.parametrize("rows,first,dim,base,mscale", [
    (200000, 0, 16, 1.0, None), (20000, 0, 256, 10000.0, None), (3000, 1000003, 64, 8e6, None), (20000, 0, 64, 8e6, 1.2079441),
])
def test_relative_error(rows, first, dim, base, mscale):
    """An angle is at most an eighth of a turn, x, from a quarter of one.  x is off by 3 F32 (the rest of the angle as a
    float, the factor to radians, their product), which moves sin x by at most 3 F32 of itself and cos x by
    x tan x <= pi / 4 of 3 F32, 2.4 F32.  The last fmaf rounds by F32.  The inner roundings are weighed by what their terms
    add: for the sine x^2 / 6 <= 0.11 of three roundings, with the series' rest of 1.8e-9 0.4 F32 in all; for the cosine
    x^2 / 2 <= 0.31 of two of at most cos x >= 0.7, 0.9 F32.  So 4.4 F32; mscale's rounding and product make it 6.4.
    The angle's own error, here and in the reference: f / (2 pi) and p f by a few roundings of 64 bits (8 allowed), and up to
    2^-64 turns a position for the bits of f behind the 64th."""
    cos, sin = (torch.empty((rows, dim), device="cuda") for _ in (0, 1))
    s = None if mscale is None else dsa.RopeScaling(1.0, 0, mscale=mscale)
    dsa.rope_table(cos, sin, base, first=first, scaling=s)
    p = np.arange(rows, dtype=np.float64)[:, None] + first
    ang = p * base ** (-2 * np.arange(dim // 2, dtype=np.float64) / dim)
    m, steps = (1.0, 4.4) if mscale is None else (mscale, 6.4)
    for got, ref in ((cos, np.cos(ang) * m), (sin, np.sin(ang) * m)):
        err = np.abs(got[:, :dim // 2].cpu().double().numpy() - ref)
        tol = steps * F32 * np.abs(ref) + m * (8 * 2.0 ** -53 * ang + 2 * np.pi * 2.0 ** -64 * p)
        assert np.all(err <= tol), (err / np.maximum(tol, 1e-300)).max()

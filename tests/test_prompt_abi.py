"""CPU-only host checks of the entry points for prompts and shared prefixes:
bad arguments are refused before any CUDA work."""

import ctypes
import math

import pytest

P, P2 = 0x7f0000100000, 0x7f0040000000
WS = 0x7f0000000000


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_gb300 import build as B
    B.build()
    import sparse_attention_gb300 as dsa
    return dsa.load_library()


def _table(lib, rows=4, first=0, dim=64, base=10000.0, scaling=None, cos=P, sin=P2):
    s = None
    if scaling is not None:
        import sparse_attention_gb300 as dsa
        s = ctypes.byref(dsa.DsaRopeScaling(*scaling))
    return lib.dsa_rope_table(rows, first, dim, ctypes.c_double(base), s, cos, sin, None)


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(first=-1), dict(rows=1 << 30, first=(1 << 30) + 1), dict(dim=0), dict(dim=24), dict(dim=272),
    dict(base=0.5), dict(base=math.inf), dict(base=math.nan), dict(cos=0), dict(sin=P2 + 4), dict(sin=P),
    dict(sin=P + 16), dict(scaling=(0.5, 0, 32, 1, 1)), dict(scaling=(math.nan, 0, 32, 1, 1)),
    dict(scaling=(2, -1, 32, 1, 1)), dict(scaling=(2, 0, 32, 1, 0)), dict(scaling=(2, 4096, 0, 1, 1)),
    dict(scaling=(2, 4096, 32, -1, 1)), dict(scaling=(2, 4096, 32, 1, math.inf)),
    dict(base=1.0, scaling=(2, 4096, 32, 1, 1)),
])
def test_table_refusals(lib, bad):
    assert _table(lib, **bad) == 1


def test_table_without_rows(lib):
    assert _table(lib, rows=0, cos=0, sin=0) == 0


def _rope(lib, t=4, heads=2, dim=64, x=P, xt=128, xh=64, cos=P, sin=P, rows=10, pos=P, flags=0, out=P2, ot=128, oh=64,
          ws=WS, n=256):
    return lib.dsa_rope(t, heads, dim, x, xt, xh, cos, sin, rows, pos, flags, out, ot, oh, ws, n, None)


@pytest.mark.parametrize("bad,code", [
    (dict(t=-1), 1), (dict(t=1 << 26), 1), (dict(heads=0), 1), (dict(dim=8), 1), (dict(dim=40), 1), (dict(rows=-1), 1),
    (dict(flags=4), 1), (dict(x=0), 1), (dict(x=P + 2), 1), (dict(out=0), 1), (dict(cos=0), 1), (dict(sin=P + 8), 1),
    (dict(pos=P + 2), 1), (dict(pos=0), 1), (dict(xt=-128), 1), (dict(xh=60), 1), (dict(ot=4), 1), (dict(oh=1 << 40), 1),
    (dict(ws=0), 3), (dict(ws=WS + 8), 3), (dict(n=255), 3),
    # out's rows share places: heads inside one another, tokens inside heads
    (dict(oh=32), 1), (dict(ot=64), 1), (dict(ot=0), 1), (dict(oh=0), 1), (dict(ot=64, oh=128), 1),
    # x and out overlap without being the same
    (dict(out=P + 128), 1), (dict(out=P, ot=256), 1), (dict(out=P, oh=72, ot=256), 1), (dict(x=P2 + 128), 1),
])
def test_rope_refusals(lib, bad, code):
    assert _rope(lib, **bad) == code


def test_rope_without_tokens(lib):
    assert _rope(lib, t=0, x=0, out=0, cos=0, sin=0, pos=0) == 0

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


def _batch(B=2, total_q=8, max_q=4, max_ctx=100, stride=100, q_off=0x10000, ctx=0x20000):
    import sparse_attention_gb300 as dsa
    return dsa.DsaBatch(B, total_q, max_q, max_ctx, stride, q_off, ctx)


def _pages(size=16, width=7, pool=20, table=0x30000):
    import sparse_attention_gb300 as dsa
    return dsa.DsaPages(size, width, pool, table)


def _expanded(rows=256, off=0x40000, kv=P, k_pe=P):
    import sparse_attention_gb300 as dsa
    return dsa.DsaExpanded(rows, off, kv, k_pe)


def _ws(lib, b):
    n = ctypes.c_size_t(0)
    assert lib.dsa_prompt_workspace_size(ctypes.byref(b), ctypes.byref(n)) == 0
    return n.value


def test_prompt_workspace(lib):
    n = ctypes.c_size_t(0)
    assert lib.dsa_prompt_workspace_size(None, ctypes.byref(n)) == 1
    assert lib.dsa_prompt_workspace_size(ctypes.byref(_batch()), None) == 1
    assert lib.dsa_prompt_workspace_size(ctypes.byref(_batch(B=0)), ctypes.byref(n)) == 1
    assert _ws(lib, _batch()) % 256 == 0 and _ws(lib, _batch(B=65535)) >= 256 + 4 * 65536      # an offset for each sequence and one behind them


def _call(lib, which, b, g, x, q=P, out=P, lse=None, scale=0.0625, first=None, w=P, ws=WS, n=None):
    n = _ws(lib, _batch()) if n is None else n
    b, x = (ctypes.byref(t) if t is not None else None for t in (b, x))
    if which == "prompt":
        return lib.dsa_prompt_mla_fwd(b, q, x, ctypes.c_float(scale), out, lse, ws, n, None)
    return lib.dsa_mla_expand(b, ctypes.byref(g) if g is not None else None, q, w, first, x, ws, n, None)


@pytest.mark.parametrize("which", ["prompt", "expand"])
@pytest.mark.parametrize("b,x,kw,code", [
    (None, {}, {}, 1), (dict(B=0), {}, {}, 1), (dict(B=65536), {}, {}, 1), (dict(total_q=-1), {}, {}, 1),
    (dict(stride=99), {}, {}, 1), (dict(q_off=0), {}, {}, 1), (dict(ctx=0x20002), {}, {}, 1),
    (dict(total_q=1 << 26), {}, {}, 2), (dict(max_q=(1 << 19) + 1), {}, {}, 2),
    ({}, None, {}, 1), ({}, dict(rows=-1), {}, 1), ({}, dict(off=0), {}, 1), ({}, dict(off=0x40002), {}, 1),
    ({}, dict(kv=0), {}, 1), ({}, dict(k_pe=P + 8), {}, 1), ({}, {}, dict(q=0), 1), ({}, {}, dict(q=P + 2), 1),
    ({}, {}, dict(ws=0), 3), ({}, {}, dict(ws=WS + 4), 3), ({}, {}, dict(n=256), 3),
])
def test_expanded_form_refusals(lib, which, b, x, kw, code):
    got = _call(lib, which, _batch(**b) if b is not None else None, None, _expanded(**x) if x is not None else None, **kw)
    assert got == code


@pytest.mark.parametrize("g,kw,code", [
    (dict(size=8), {}, 1), (dict(size=48), {}, 1), (dict(width=6), {}, 1), (dict(pool=0), {}, 1), (dict(table=0), {}, 1),
    (dict(pool=1 << 27), {}, 2), (None, dict(w=0), 1), (None, dict(first=0x50002), 1),
])
def test_expand_refusals(lib, g, kw, code):
    assert _call(lib, "expand", _batch(), _pages(**g) if g is not None else None, _expanded(), **kw) == code


@pytest.mark.parametrize("kw", [dict(scale=0.0), dict(scale=-1.0), dict(scale=math.inf), dict(scale=math.nan), dict(out=0),
                                dict(out=P + 4), dict(lse=P + 4)])
def test_prompt_refusals(lib, kw):
    assert _call(lib, "prompt", _batch(), None, _expanded(), **kw) == 1


def test_calls_without_rows(lib):
    assert _call(lib, "prompt", _batch(total_q=0), None, _expanded(), q=0, out=0) == 0
    assert _call(lib, "expand", _batch(max_ctx=0), None, _expanded(), q=0, w=0) == 0
    assert _call(lib, "expand", _batch(), None, _expanded(rows=0, kv=0, k_pe=0), q=0, w=0) == 0


@pytest.mark.parametrize("kw,code", [(dict(t=-1), 1), (dict(o=0), 1), (dict(w=P + 2), 1), (dict(y=0), 1), (dict(ws=0), 3),
                                     (dict(n=256), 3), (dict(t=0, o=0, w=0, y=0), 0)])
def test_o_proj_refusals(lib, kw, code):
    a = dict(dict(t=8, o=P, w=P, y=P, ws=WS, n=1 << 30), **kw)
    assert lib.dsa_mla_o_proj(a["t"], a["o"], a["w"], a["y"], a["ws"], a["n"], None) == code


def _groups(n=1, off=0x60000, shared=0x70000):
    import sparse_attention_gb300 as dsa
    return dsa.DsaGroups(n, off, shared)


def _prefix(lib, b, r, g=None, q=P, kv=P, mask=P, scale=0.0625, out=P, lse=None, ws=WS, n=1 << 40):
    b, r, g = (ctypes.byref(t) if t is not None else None for t in (b, r, g))
    return lib.dsa_prefix_mla_fwd(b, r, g, q, kv, mask, ctypes.c_float(scale), out, lse, ws, n, None)


def test_prefix_workspace(lib):
    n = ctypes.c_size_t(0)
    size = lambda b, r: lib.dsa_prefix_workspace_size(ctypes.byref(_batch(**b)), ctypes.byref(_groups(**r)),  # noqa: E731
                                                      ctypes.byref(n))
    assert size({}, {}) == 0 and n.value % 256 == 0
    assert [size(dict(B=0), {}), size({}, dict(n=0)), size({}, dict(n=3))] == [1, 1, 1]
    assert lib.dsa_prefix_workspace_size(ctypes.byref(_batch()), None, ctypes.byref(n)) == 1
    assert lib.dsa_prefix_workspace_size(ctypes.byref(_batch()), ctypes.byref(_groups()), None) == 1
    # two pieces of 128 rows for each of 76 CTA pairs, and two runs a sequence
    assert size(dict(B=64, total_q=64, max_q=1), {}) == 0 and n.value >= 2 * 76 * 4 * 128 * 513 + 64 * 128
    small = n.value
    assert size(dict(B=65535, total_q=65535, max_q=1), {}) == 0 and n.value >= small + (65535 - 64) * 128


@pytest.mark.parametrize("b,r,g,kw,code", [
    (None, {}, None, {}, 1), ({}, None, None, {}, 1), (dict(B=0), {}, None, {}, 1), (dict(max_q=65), {}, None, {}, 2),
    (dict(total_q=1 << 25), {}, None, {}, 2), (dict(stride=99), {}, None, {}, 1), (dict(stride=1 << 30), {}, None, {}, 2),
    ({}, dict(n=0), None, {}, 1), ({}, dict(n=3), None, {}, 1), ({}, dict(off=0), None, {}, 1),
    ({}, dict(shared=0x70002), None, {}, 1), ({}, {}, dict(size=24), {}, 1), ({}, {}, dict(width=6), {}, 1),
    ({}, {}, None, dict(q=0), 1), ({}, {}, None, dict(kv=P + 8), 1), ({}, {}, None, dict(mask=P + 4), 1),
    ({}, {}, None, dict(out=0), 1), ({}, {}, None, dict(lse=P + 4), 1), ({}, {}, None, dict(scale=0.0), 1),
    ({}, {}, None, dict(scale=math.nan), 1), ({}, {}, None, dict(ws=0), 3), ({}, {}, None, dict(n=4096), 3),
    (dict(total_q=0), {}, None, dict(q=0, kv=0, out=0), 0), (dict(max_ctx=0), {}, None, dict(q=0), 0),
])
def test_prefix_refusals(lib, b, r, g, kw, code):
    got = _prefix(lib, _batch(**b) if b is not None else None, _groups(**r) if r is not None else None,
                  _pages(**g) if g is not None else None, **kw)
    assert got == code

"""CPU-only host checks of the drafted-step entry points: bad arguments are
refused before any CUDA work."""

import ctypes

import pytest
import torch

P = 0x7f0000100000
WS = 0x7f0000000000


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_gb300 import build as B
    B.build()
    import sparse_attention_gb300 as dsa
    return dsa.load_library()


def _batch(B=2, total_q=8, max_q=4, max_ctx=100, stride=100, q_off=0x10000, ctx=0x20000):
    import sparse_attention_gb300 as dsa
    return dsa.DsaBatch(B, total_q, max_q, max_ctx, stride, q_off, ctx)


def _pages(size=16, width=7, pool=20, table=0x30000):
    import sparse_attention_gb300 as dsa
    return dsa.DsaPages(size, width, pool, table)


def _ws(lib, b):
    n = ctypes.c_size_t(0)
    assert lib.dsa_tree_workspace_size(ctypes.byref(b) if b is not None else None, ctypes.byref(n)) == 0
    return n.value


def _attn(lib, b, g=None, q=P, kv=P, mask=P, scale=0.0625, out=P, lse=None, ws=WS, n=None):
    return lib.dsa_tree_mla_fwd(ctypes.byref(b), ctypes.byref(g) if g is not None else None, q, kv, mask,
                                ctypes.c_float(scale), out, lse, ws, _ws(lib, _batch()) if n is None else n, None)


def test_workspace(lib):
    n = ctypes.c_size_t(0)
    assert lib.dsa_tree_workspace_size(None, ctypes.byref(n)) == 0 and n.value == 256
    assert lib.dsa_tree_workspace_size(None, None) == 1
    assert lib.dsa_tree_workspace_size(ctypes.byref(_batch(B=0)), ctypes.byref(n)) == 1
    assert _ws(lib, _batch()) % 256 == 0 and _ws(lib, _batch()) >= 256 + 4 * 6
    assert lib.dsa_status_string(9).startswith(b"DSA_ERR_NO_PAGES")


@pytest.mark.parametrize("b,g,code", [
    (dict(B=0), None, 1), (dict(B=65536), None, 1), (dict(total_q=-1), None, 1), (dict(max_q=65), None, 2),
    (dict(stride=99), None, 1), (dict(q_off=0), None, 1), (dict(ctx=0x20002), None, 1),
    (dict(stride=1 << 30), None, 2), (dict(total_q=1 << 26), None, 2), (dict(total_q=1 << 25), None, 2),
    ({}, dict(size=8), 1), ({}, dict(size=2048), 1), ({}, dict(size=48), 1), ({}, dict(width=6), 1),
    ({}, dict(pool=0), 1), ({}, dict(table=0), 1), ({}, dict(pool=1 << 27), 2),
])
def test_batches_and_pages(lib, b, g, code):
    assert _attn(lib, _batch(**b), _pages(**g) if g is not None else None) == code


def test_attention_arguments(lib):
    b = _batch()
    for kw in (dict(q=None), dict(kv=P + 8), dict(mask=None), dict(mask=P + 4), dict(out=None), dict(lse=P + 4),
               dict(scale=0.0), dict(scale=float("inf")), dict(scale=float("nan"))):
        assert _attn(lib, b, **kw) == 1, kw
    assert _attn(lib, b, ws=None) == 3 and _attn(lib, b, n=255) == 3 and _attn(lib, b, ws=WS + 8) == 3
    assert _attn(lib, _batch(total_q=0)) == 0 and _attn(lib, _batch(max_q=0)) == 0


def test_tables_arguments(lib):
    def call(b, g, n_new=P, ctx=P, parent=None, ho=P, hn=P, free=P, fr=P, fo=P, slots=P, pos=P, mask=None, n=None):
        return lib.dsa_step_tables(ctypes.byref(b), ctypes.byref(g) if g is not None else None, n_new, ctx, parent, ho,
                                   hn, free, fr, fo, slots, pos, mask, WS, _ws(lib, b) if n is None else n, None)
    b, g = _batch(), _pages()
    for kw in (dict(n_new=None), dict(ctx=P + 2), dict(ho=None), dict(hn=None), dict(free=None), dict(fr=None),
               dict(fo=None), dict(slots=None), dict(pos=None), dict(mask=P + 4), dict(parent=P + 1)):
        assert call(b, g, **kw) == 1, kw
    assert call(b, g, n=256) == 3


def test_append_arguments(lib):
    def call(T=4, x=P, xs=576, gamma=P, eps=1e-5, cos=P, sin=P, rows=9, pos=P, slots=P, cache=30, kv=P, ws=WS, n=256):
        return lib.dsa_latent_append(T, x, xs, gamma, ctypes.c_float(eps), cos, sin, rows, pos, slots, cache, kv, ws, n,
                                     None)
    for kw in (dict(T=-1), dict(T=1 << 26), dict(x=None), dict(x=P + 8), dict(xs=575), dict(xs=580), dict(gamma=None),
               dict(eps=0.0), dict(eps=float("inf")), dict(cos=None), dict(sin=P + 4), dict(rows=-1), dict(pos=None),
               dict(slots=None), dict(cache=-1), dict(kv=None)):
        assert call(**kw) == 1, kw
    assert call(ws=None) == 3 and call(n=255) == 3
    assert call(T=0, x=None) == 0


def test_topk_and_commit_arguments(lib):
    b = _batch()

    def topk(b=b, scores=P, ld=100, mask=P, k=8, idx=P, n=256):
        return lib.dsa_tree_topk(ctypes.byref(b), scores, ld, mask, k, idx, WS, n, None)
    for kw in (dict(scores=None), dict(ld=96), dict(ld=102), dict(mask=None), dict(k=0), dict(k=2049), dict(idx=P + 8)):
        assert topk(**kw) == 1, kw
    assert topk(b=_batch(max_q=65)) == 2 and topk(n=100) == 3 and topk(b=_batch(total_q=0)) == 0

    def commit(b=b, g=None, mask=P, acc=P, layers=1, rows=200, kv=P, ki=None, new=P, n=None):
        return lib.dsa_tree_commit(ctypes.byref(b), ctypes.byref(g) if g is not None else None, mask, acc, layers, rows,
                                   kv, ki, new, WS, _ws(lib, b) if n is None else n, None)
    for kw in (dict(mask=None), dict(acc=None), dict(layers=0), dict(layers=65536), dict(rows=199), dict(kv=P + 8),
               dict(ki=P + 4), dict(new=None), dict(g=_pages(), rows=321)):
        assert commit(**kw) == 1, kw
    assert commit(n=10) == 3


def test_binding_refuses_tensors(lib):
    import sparse_attention_gb300 as dsa
    ws = torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError):
        dsa.latent_append(torch.zeros((1, 576), dtype=torch.bfloat16), None, 1e-5, None, None, None, None, None, ws=ws)
    with pytest.raises(TypeError):
        dsa.make_pages(torch.zeros((2, 2), dtype=torch.int64), 16, 4)
    with pytest.raises(ValueError):
        dsa.make_pages(torch.zeros((2, 2), dtype=torch.int32), 16, 4)       # not on a device
    t = torch.zeros(4, dtype=torch.int32)
    cpu = -1
    with pytest.raises(TypeError):
        dsa._typed("t", t, torch.int64, 4, cpu)
    with pytest.raises(ValueError):
        dsa._typed("t", t, torch.int32, 5, cpu)
    with pytest.raises(ValueError):
        dsa._typed("t", t[::2], torch.int32, 2, cpu)
    assert dsa._typed("t", None, torch.int32, 5, cpu) is None


def test_topk_of_batches_whose_contiguous_cache_would_be_too_large(lib):
    """The call reads no cache: sequences times stride has no limit there, as in paged calls."""
    def topk(scores=P, **kw):
        b = _batch(B=16384, max_ctx=131072, stride=131072, **kw)
        return lib.dsa_tree_topk(ctypes.byref(b), scores, 131072, P, 8, P, WS, 256, None)
    g = _pages(width=8192)
    b = _batch(B=16384, max_ctx=131072, stride=131072, total_q=0)
    assert lib.dsa_tree_mla_fwd(ctypes.byref(b), ctypes.byref(g), P, P, P, ctypes.c_float(0.1), P, None, WS,
                                _ws(lib, b), None) == 0
    assert topk(total_q=0) == 0 and topk(scores=None) == 1
    assert topk(max_q=65) == 2 and topk(total_q=1 << 26) == 2
    # attention over contiguous caches of that size stays refused
    assert _attn(lib, b) == 2


def test_binding_without_a_workspace(lib):
    """DSA_ERR_WORKSPACE, as from the calls of the path."""
    import sparse_attention_gb300 as dsa
    calls = dict(step_tables=[None] * 5, latent_append=[None, None, 1e-5] + [None] * 5,
                 tree_mla_fwd=[None] * 4 + [0.1, None], tree_topk=[None, None, None, 8, None], tree_commit=[None] * 4)
    for name, args in calls.items():
        with pytest.raises(dsa.DsaError, match=f"dsa_{name}: DSA_ERR_WORKSPACE") as e:
            getattr(dsa, name)(*args, ws=None)
        assert e.value.code == 3


@pytest.mark.parametrize("B", [1, 2, 300])
def test_each_call_asks_for_its_own_workspace(lib, B):
    b, g = _batch(B=B), _pages()
    n = 264 + 8 * B
    assert n < _ws(lib, b)

    def tables(bytes_):
        return lib.dsa_step_tables(ctypes.byref(b), ctypes.byref(g), None, P, None, P, P, P, P, P, P, P, P, WS, bytes_, None)

    def commit(bytes_):
        return lib.dsa_tree_commit(ctypes.byref(b), ctypes.byref(g), P, None, 1, 320, P, None, P, WS, bytes_, None)
    for call in (tables, commit):
        assert call(n - 1) == 3 and call(n) == 1               # then refused for a missing array
    assert _attn(lib, b, g, q=None, n=n) == 3 and _attn(lib, b, g, q=None, n=_ws(lib, b)) == 1
    size = ctypes.c_size_t(0)
    assert lib.dsa_workspace_size(ctypes.byref(b), 1, ctypes.byref(size)) == 0 and size.value >= n


def test_attention_of_a_batch_without_context(lib):
    """No sequence can hold a row: nothing to do, as for max_q = 0, whatever the caches' size."""
    for g in (None, _pages()):
        assert _attn(lib, _batch(max_ctx=0, stride=0), g) == 0
    assert _attn(lib, _batch(max_ctx=0, stride=0), ws=None) == 3

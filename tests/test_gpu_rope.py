"""Rotary tables and rotation through the public entry points, against 64-bit
references."""

import math

import numpy as np
import pytest
import torch

import sparse_attention_gb300 as dsa

pytestmark = pytest.mark.gpu
HALF, F32 = 2.0 ** -8, 2.0 ** -24       # half a step of bf16 and of fp32, relative


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from sparse_attention_gb300 import build as B
    B.build()
    dsa.load_library()


@pytest.fixture(scope="module")
def ws():
    return dsa.tree_workspace()


def _freq(dim, base, scaling):
    i = np.arange(dim // 2, dtype=np.float64)
    f = base ** (-2 * i / dim)
    if scaling is None:
        return f, 1.0
    factor, ctx, fast, slow, m = scaling
    if ctx == 0:
        return f / factor, m
    e = [dim * math.log(ctx / (2 * math.pi * n)) / (2 * math.log(base)) for n in (fast, slow)]
    lo, hi = max(math.floor(e[0]), 0), min(math.ceil(e[1]), dim - 1)
    ramp = np.clip((i - lo) / max(hi - lo, 0.001), 0, 1)
    return f / factor * ramp + f * (1 - ramp), m


@pytest.mark.parametrize("rows,first,dim,base,scaling", [
    (1, 0, 64, 10000.0, None), (1, 1000003, 16, 10000.0, None), (3, 0, 16, 1.0, None), (70, 5, 256, 8e6, None),
    (5000, 0, 64, 10000.0, (4.0, 0, 32.0, 1.0, 1.0)), (257, 100000, 96, 5e5, (8.0, 4096, 32.0, 1.0, 1.2)),
    (33, 202719, 64, 8e6, (12.375, 16384, 32.0, 1.0, 1.25)), (9, 0, 64, 10000.0, (2.0, 1, 32.0, 1.0, 1.0)),
    (40, 2 ** 31 - 40, 64, 10000.0, None),
])
def test_table(rows, first, dim, base, scaling):
    cos = torch.full((rows + 1, dim), 7.0, device="cuda")
    sin = torch.full((rows + 1, dim), 7.0, device="cuda")
    s = dsa.RopeScaling(*scaling) if scaling else None
    dsa.rope_table(cos[:rows], sin[:rows], base, first=first, scaling=s)
    f, m = _freq(dim, base, scaling)
    ang = (np.arange(rows, dtype=np.float64) + first)[:, None] * f
    # sinpi and cospi are off by up to an ulp, and the corrections by half a
    # step each (of the rest's first-order term, of mscale, of mscale's own
    # rounding to fp32): 2 * 1 + 3 half steps; the angle, here and there, by
    # the frequency's power, its products and quotients: 8 half steps of 64 bits
    for got, ref in ((cos, np.cos(ang)), (sin, np.sin(ang))):
        g = got.cpu().double().numpy()
        assert np.all(g[rows] == 7.0)
        assert np.array_equal(g[:rows, :dim // 2], g[:rows, dim // 2:])
        err = np.abs(g[:rows, :dim // 2] - ref * m)
        assert np.all(err <= 7 * F32 * np.abs(ref * m) + 8 * 2.0 ** -53 * m * ang), err.max()


def test_table_refuses():
    a = torch.zeros((4, 64), device="cuda")
    with pytest.raises(dsa.DsaError):
        dsa.rope_table(a, a, 10000.0)
    with pytest.raises(ValueError):
        dsa.rope_table(a, torch.zeros((4, 32), device="cuda"), 10000.0)
    with pytest.raises(TypeError):
        dsa.rope_table(a, a.double(), 10000.0)
    with pytest.raises(ValueError):
        dsa.rope_table(a.t(), a.t().clone().t(), 10000.0)
    with pytest.raises(ValueError):
        dsa.rope_table(torch.zeros((4, 64)), torch.zeros((4, 64)), 10000.0)


def _tables(rows, dim, seed=0):
    """Any numbers: the rotation does not ask for cosines."""
    g = np.random.default_rng(seed)
    c, s = (torch.from_numpy(g.standard_normal((rows, dim // 2)).astype(np.float32)).cuda().repeat(1, 2) for _ in (0, 1))
    return c.contiguous(), s.contiguous()


def _ref(x, c, s, pos, neighbour, inverse):
    """In 64 bits, and the sum of the products' sizes."""
    x = x.double().cpu()
    r = x.shape[-1]
    p = pos.cpu().long().clamp(min=0)
    c, s = (t.cpu().double()[p, None, :r // 2] for t in (c, s))
    s = -s if inverse else s
    a, b = (x[..., 0::2], x[..., 1::2]) if neighbour else (x[..., :r // 2], x[..., r // 2:])
    y, z, u, v = a * c - b * s, b * c + a * s, (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
    if neighbour:
        return torch.stack([y, z], -1).flatten(-2), torch.stack([u, v], -1).flatten(-2)
    return torch.cat([y, z], -1), torch.cat([u, v], -1)


def _close(got, ref, size):
    # three fp32 roundings (two products, a sum), then one to bf16
    err = (got.cpu().double() - ref).abs()
    assert (err <= HALF * ref.abs() + 3 * F32 * size * (1 + HALF)).all(), err.max()


@pytest.mark.parametrize("t,heads,width,at,dim", [
    (1, 1, 64, 0, 64), (64, 64, 256, 192, 64), (7, 5, 128, 0, 64), (33, 32, 128, 64, 32), (300, 3, 256, 0, 256),
    (5, 64, 272, 8, 16), (1000, 64, 64, 0, 64), (2, 700, 96, 0, 96), (12000, 64, 256, 192, 64),
])
@pytest.mark.parametrize("neighbour,inverse", [(False, False), (True, False), (False, True), (True, True)])
def test_rotation(ws, t, heads, width, at, dim, neighbour, inverse):
    gen = torch.Generator(device="cuda").manual_seed(t * heads + dim)
    x = torch.randn((t, heads, width), generator=gen, device="cuda", dtype=torch.bfloat16)
    cos, sin = _tables(50, dim)
    pos = torch.randint(-1, 50, (t,), generator=gen, device="cuda", dtype=torch.int32)
    part = x[..., at:at + dim]
    ref, size = _ref(part, cos, sin, pos, neighbour, inverse)
    live = pos.cpu() >= 0
    out = torch.full((t, heads, dim), 3.0, device="cuda", dtype=torch.bfloat16)
    dsa.rope(part, cos, sin, pos, out, interleaved=neighbour, inverse=inverse, ws=ws)
    _close(out[live], ref[live], size[live])
    assert (out[~live.cuda()] == 3.0).all()
    # in place: the same bits, and nothing else touched
    y = x.clone()
    dsa.rope(y[..., at:at + dim], cos, sin, pos, interleaved=neighbour, inverse=inverse, ws=ws)
    z = x.clone()
    z[..., at:at + dim] = torch.where((pos >= 0)[:, None, None], out, part)
    assert torch.equal(y, z)
    assert dsa.read_device_status(ws) == 0


def test_layouts_of_strides(ws):
    """Heads outside tokens, a broadcast input, one token or head of any stride."""
    cos, sin = _tables(9, 32, 1)
    pos = torch.tensor([8, 0, 3, 3, 5], dtype=torch.int32, device="cuda")
    x = torch.randn((4, 5, 32), device="cuda", dtype=torch.bfloat16).transpose(0, 1)
    out = torch.zeros((4, 5, 32), device="cuda", dtype=torch.bfloat16).transpose(0, 1)
    dsa.rope(x, cos, sin, pos, out, ws=ws)
    _close(out, *_ref(x, cos, sin, pos, False, False))
    one = torch.randn((5, 1, 32), device="cuda", dtype=torch.bfloat16).expand(5, 4, 32)
    dsa.rope(one, cos, sin, pos, out, ws=ws)
    _close(out, *_ref(one, cos, sin, pos, False, False))
    with pytest.raises(dsa.DsaError):
        dsa.rope(one, cos, sin, pos, ws=ws)
    row = torch.randn((1, 1, 32), device="cuda", dtype=torch.bfloat16)
    ref = _ref(row, cos, sin, pos[:1], True, False)
    dsa.rope(row, cos, sin, pos[:1], interleaved=True, ws=ws)
    _close(row, *ref)
    assert dsa.rope(x[:0], cos, sin, pos[:0], out[:0], ws=ws).shape[0] == 0


def test_gradient(ws):
    """The inverse rotation of a gradient is the formula's, and undoes the rotation."""
    cos, sin = (torch.empty((64, 64), device="cuda") for _ in (0, 1))
    dsa.rope_table(cos, sin, 10000.0)
    pos = torch.arange(0, 60, dtype=torch.int32, device="cuda")
    g = torch.randn((60, 8, 64), device="cuda", dtype=torch.bfloat16)
    for neighbour in (False, True):
        x = torch.randn((60, 8, 64), dtype=torch.float64, requires_grad=True)
        y, _ = _ref(x, cos, sin, pos, neighbour, False)
        grad, = torch.autograd.grad((y * g.cpu().double()).sum(), x)
        out = torch.empty_like(g)
        dsa.rope(g, cos, sin, pos, out, interleaved=neighbour, inverse=True, ws=ws)
        _close(out, grad, _ref(g, cos, sin, pos, neighbour, True)[1])
        z = out.clone()
        dsa.rope(z, cos, sin, pos, interleaved=neighbour, ws=ws)
        # out's rounding turned with it (a vector of 2 keeps its length), then z's own
        pair = (g.double()[..., 0::2] ** 2 + g.double()[..., 1::2] ** 2).sqrt().repeat_interleave(2, -1) if neighbour else \
            (g.double()[..., :32] ** 2 + g.double()[..., 32:] ** 2).sqrt().repeat(1, 1, 2)
        assert ((z.double() - g.double()).abs() <= 2.02 * HALF * pair + 1e-30).all()


def test_bad_positions():
    ws = dsa.tree_workspace()
    cos, sin = _tables(4, 64, 2)
    x = torch.randn((3, 2, 64), device="cuda", dtype=torch.bfloat16)
    for bad in (4, -2, 2 ** 31 - 1):
        y = x.clone()
        pos = torch.tensor([1, bad, 2], dtype=torch.int32, device="cuda")
        dsa.rope(y, cos, sin, pos, ws=ws)
        assert dsa.read_device_status(ws) == 7 and torch.equal(y[1], x[1])
        keep = torch.tensor([0, 2])
        _close(y[keep], *(r[keep] for r in _ref(x, cos, sin, pos.clamp(0, 3), False, False)))
        dsa.reset_device_status(ws)


def test_special_values(ws):
    """Infinities and NaN stay in their pairs."""
    cos, sin = _tables(4, 64, 3)
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    x = torch.randn((2, 2, 64), device="cuda", dtype=torch.bfloat16)
    y = x.clone()
    y[0, 1, 3], y[1, 0, 40] = float("inf"), float("nan")
    a, b = x.clone(), y.clone()
    dsa.rope(a, cos, sin, pos, ws=ws)
    dsa.rope(b, cos, sin, pos, ws=ws)
    hit = torch.zeros_like(x, dtype=torch.bool)
    hit[0, 1, [3, 35]] = True
    hit[1, 0, [8, 40]] = True
    assert torch.equal(~torch.isfinite(b), hit) and torch.equal(a[~hit], b[~hit])


def test_refusals(ws):
    cos, sin = _tables(4, 64, 4)
    x = torch.zeros((3, 2, 64), device="cuda", dtype=torch.bfloat16)
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    for kw, err in ((dict(x=x.float()), TypeError), (dict(x=x.cpu()), TypeError), (dict(cos=cos[:, :32]), ValueError),
                    (dict(pos=pos[:2]), ValueError), (dict(pos=pos.long()), TypeError), (dict(out=x[:2]), ValueError),
                    (dict(x=x[..., ::2], cos=cos[:, :32], sin=sin[:, :32]), ValueError), (dict(ws=None), dsa.DsaError)):
        a = dict(dict(x=x, cos=cos, sin=sin, pos=pos, out=None, ws=ws), **kw)
        with pytest.raises(err):
            dsa.rope(a["x"], a["cos"], a["sin"], a["pos"], a["out"], ws=a["ws"])


def test_streams_and_graph():
    """A caller's stream, and a captured call replayed on new inputs."""
    ws = dsa.tree_workspace()
    cos, sin = (torch.empty((128, 64), device="cuda") for _ in (0, 1))
    x = torch.randn((40, 64, 256), device="cuda", dtype=torch.bfloat16)
    pos = torch.zeros(40, dtype=torch.int32, device="cuda")
    out = torch.zeros((40, 64, 64), device="cuda", dtype=torch.bfloat16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    dsa.rope_table(cos, sin, 10000.0, stream=s)
    dsa.rope(x[..., 192:], cos, sin, pos, out, ws=ws, stream=s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        dsa.rope_table(cos, sin, 10000.0)
        dsa.rope(x[..., 192:], cos, sin, pos, out, ws=ws)
    for k in range(3):
        x.normal_()
        pos.copy_(torch.randint(0, 128, (40,)))
        cos.zero_()
        sin.zero_()
        g.replay()
        torch.cuda.synchronize()
        _close(out, *_ref(x[..., 192:], cos, sin, pos, False, False))
    assert dsa.read_device_status(ws) == 0

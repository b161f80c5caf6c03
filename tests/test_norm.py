"""kda_rmsnorm and kda_rmsnorm_backward: host validation (CPU) and parity with
the formulas in 64 bits (GPU).

Tolerances. bf16 outputs: half a step of the result (2^-8 |y|) plus the fp32
arithmetic. Each factor of y = z s w sig carries a few fp32 roundings; the sum
of squares of n terms, added in at most 64 + log steps, is off by under
80 * 2^-24 of itself, so y by under 60 * 2^-24 |y| < 4e-6 |y|; hardware exp adds
2^-22 |gate| to the sigmoid. 2^-8 |y| + 2e-5 |y| + 1e-6 top covers it, `top` being the
row's largest value. fp8 outputs: half a step, 2^-4 |q|, or half the subnormal
spacing 2^-10 near zero, and the same again where fp32 tips a tie: the value then
still is one of the two neighbours, so 2^-4 * 1.001 |q| + 2^-10. dz cancels between
a and n mean(a n): its fp32 error scales with the row's largest |s a|. dweight
sums V vectors in fp32 over fewer than 1200 sequential steps: 1200 * 2^-24 = 7e-5
of the sum of magnitudes, in practice its root; 2e-5 of that sum.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np
import pytest
import torch

import gated_delta_rule_step_amd as kda

OK, NULLP, SHAPE, STRIDE, UNSUP, SEQ, WS = range(7)
BF = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(kda.LIB_PATH):
        from gated_delta_rule_step_amd import build
        build.build()
    return kda.lib()


# ---------------------------------------------------------------------------
# refusals: every call returns before anything is launched (made-up pointers)

def _fwd(lib, **kw):
    a = dict(rows=2, heads=3, width=128, x=4096, xs=384, r=0, rs=384, ro=0, ros=384, g=0, gs=384,
             w=4096, eps=1e-6, dt=0, o=4096, os=384, grp=0, sc=0, ss=3)
    a.update(kw)
    P = ctypes.c_void_p
    return lib.kda_rmsnorm(a["rows"], a["heads"], a["width"], P(a["x"]), a["xs"], P(a["r"]),
                           a["rs"], P(a["ro"]), a["ros"], P(a["g"]), a["gs"], P(a["w"]),
                           a["eps"], a["dt"], P(a["o"]), a["os"], a["grp"], P(a["sc"]), a["ss"],
                           P(0))


@pytest.mark.parametrize("want,kw", [
    (SHAPE, dict(rows=-1)), (SHAPE, dict(heads=0)), (SHAPE, dict(width=0)),
    (UNSUP, dict(width=16385)), (UNSUP, dict(heads=1 << 24)), (UNSUP, dict(rows=1 << 60)),
    (UNSUP, dict(eps=0.0)), (UNSUP, dict(eps=float("nan"))), (UNSUP, dict(eps=float("inf"))),
    (UNSUP, dict(dt=2)), (UNSUP, dict(ro=4096)), (UNSUP, dict(dt=1, sc=4096, grp=64)),
    (UNSUP, dict(dt=1, sc=4096, grp=128, width=200)),
    (NULLP, dict(x=0)), (NULLP, dict(w=0)), (NULLP, dict(o=0)), (NULLP, dict(dt=1)),
    (STRIDE, dict(xs=-1)), (STRIDE, dict(os=383)), (STRIDE, dict(r=4096, rs=-8)),
    (STRIDE, dict(r=4096, ro=4096, ros=100)), (STRIDE, dict(g=4096, gs=-1)),
    (STRIDE, dict(dt=1, sc=4096, ss=2)),
    (OK, dict(rows=0, x=0, w=0, o=0)),
])
def test_forward_refusals(lib, want, kw):
    assert _fwd(lib, **kw) == want


def _bwd(lib, **kw):
    a = dict(rows=2, heads=3, width=128, z=4096, zs=384, dy=4096, ys=384, g=0, gs=384, r=0,
             rs=384, w=4096, eps=1e-6, dz=4096, ds=384, dg=0, dgs=384, dw=0, ws=0, wb=0)
    a.update(kw)
    P = ctypes.c_void_p
    return lib.kda_rmsnorm_backward(a["rows"], a["heads"], a["width"], P(a["z"]), a["zs"],
                                    P(a["dy"]), a["ys"], P(a["g"]), a["gs"], P(a["r"]), a["rs"],
                                    P(a["w"]), a["eps"], P(a["dz"]), a["ds"], P(a["dg"]),
                                    a["dgs"], P(a["dw"]), P(a["ws"]), a["wb"], P(0))


@pytest.mark.parametrize("want,kw", [
    (SHAPE, dict(rows=-1)), (SHAPE, dict(heads=-2)), (UNSUP, dict(width=20000)),
    (UNSUP, dict(eps=-1.0)), (NULLP, dict(z=0)), (NULLP, dict(dy=0)), (NULLP, dict(dz=0)),
    (NULLP, dict(g=4096)), (NULLP, dict(dg=4096)), (STRIDE, dict(zs=-1)),
    (STRIDE, dict(ds=5)), (STRIDE, dict(g=4096, dg=4096, dgs=5)), (STRIDE, dict(r=4096, rs=-3)),
    (WS, dict(dw=4096, ws=4096, wb=3)), (NULLP, dict(dw=4096, wb=1 << 20)),
    (UNSUP, dict(dw=4096, ws=4100, wb=1 << 20)),
    (OK, dict(rows=0, z=0, dy=0, dz=0)),
])
def test_backward_refusals(lib, want, kw):
    assert _bwd(lib, **kw) == want


def test_workspace_size(lib):
    size = kda.kda_rmsnorm_backward_workspace_size
    assert size(1, 1, 100) == 400
    assert size(0, 1, 100) == 0 and size(5, 0, 100) == 0 and size(5, 1, 99999) == 0
    assert size(1 << 40, 1, 8192) == size(1 << 20, 1, 8192)  # bounded by the grid


@pytest.mark.parametrize("width", [1, 128, 200, 1024, 1536, 2560, 2561, 8192, 16384])
def test_workspace_grows_with_rows(lib, width):
    """One buffer made for the most rows serves every call with fewer: the shapes that hold
    a vector change with the row count."""
    size = kda.kda_rmsnorm_backward_workspace_size
    rows = [1, 2, 255, 256, 257, 511, 512, 513, 1000, 1024, 1025, 2100, 5000, 16384, 10 ** 6]
    for heads in (1, 3):
        got = [size(r, heads, width) for r in rows]
        assert got == sorted(got)


def test_binding_refuses(lib):
    x = torch.zeros(4, 128, dtype=BF)
    w = torch.ones(128)
    with pytest.raises(ValueError):
        kda.kda_rmsnorm(x, w, torch.empty_like(x))  # not on a GPU
    with pytest.raises(TypeError):
        kda.kda_rmsnorm(x.float(), w, torch.empty_like(x))


# ---------------------------------------------------------------------------
# GPU

def _rand(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(BF)


def _strided(t, pad, offset):
    """The same values on the GPU with `pad` more elements per row, starting `offset`
    elements into the allocation."""
    rows = t.shape[0]
    n = t[0].numel() if rows else 1
    buf = torch.full((offset + max(rows, 1) * (n + pad),), -7.0, dtype=t.dtype, device="cuda")
    view = buf[offset:].as_strided((rows,) + tuple(t.shape[1:]),
                                   (n + pad,) + tuple(t.stride()[1:]))
    view.copy_(t)
    return view, buf


def _ref(x, w, res, gate, eps):
    z = x.double() if res is None else x.double() + res.double()
    y = z / torch.sqrt(z.pow(2).mean(-1, keepdim=True) + eps) * w.double()
    if gate is not None:
        y = y * torch.sigmoid(gate.double())
    return z, y


# odd widths, one channel, the borders between the lane shapes, head vectors
SHAPES = [(1, 1, 1), (3, 1, 7), (5, 12, 128), (129, 3, 128), (2, 1, 129), (33, 1, 512),
          (7, 2, 513), (4, 1, 1001), (9, 1, 1024), (2, 1, 1025), (3, 1, 2048), (5, 1, 3000),
          (2, 1, 4096), (3, 1, 8192), (2, 1, 8193), (1, 1, 16384), (4100, 1, 1536)]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("res,gated,pad,off", [(False, False, 0, 0), (True, False, 0, 0),
                                               (False, True, 8, 8), (True, True, 3, 1)])
def test_forward_bf16(shape, res, gated, pad, off):
    rows, heads, width = shape
    x, w = _rand(shape, 1), 1 + 0.1 * _rand((width,), 2).float()
    r = _rand(shape, 3, 2.0) if res else None
    g = _rand(shape, 4) if gated else None
    z, y = _ref(x, w, r, g, 1e-6)
    xd = _strided(x, pad, off)[0]
    rd = _strided(r, pad, off)[0] if res else None
    gd = _strided(g, pad, off)[0] if gated else None
    out, obuf = _strided(torch.zeros(shape, dtype=BF), pad, off)
    zo, zbuf = _strided(torch.zeros(shape, dtype=BF), pad, off)
    kda.kda_rmsnorm(xd, w.cuda(), out, residual=rd, residual_out=zo if res else None, gate=gd)
    torch.cuda.synchronize()
    err = (out.double().cpu() - y).abs()
    top = y.abs().amax(-1, keepdim=True)
    assert (err <= (2.0 ** -8 + 2e-5) * y.abs() + 1e-6 * top).all()
    if res:  # the sum of two bf16 is rounded once: the nearest bf16 of it
        assert torch.equal(zo.cpu(), z.to(BF))
    # the padding between rows and before them stays
    for buf in (obuf, zbuf):
        n = heads * width
        gaps = torch.cat([buf[:off], buf[off:].reshape(-1, n + pad)[:, n:].reshape(-1)])
        assert (gaps == -7.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("shape,group", [((5, 12, 128), 0), ((5, 12, 128), 128), ((3, 1, 1001), 0),
                                         ((64, 1, 1536), 128), ((2, 4, 256), 128),
                                         ((2, 4, 256), 0), ((3, 1, 8192), 128),
                                         ((1, 1, 16384), 0), ((2, 1, 16384), 128)], ids=str)
@pytest.mark.parametrize("res,gated", [(True, False), (False, True)])
def test_forward_fp8(shape, group, res, gated):
    rows, heads, width = shape
    x, w = _rand(shape, 5, 30.0), 1 + 0.1 * _rand((width,), 6).float()
    x[0] = 0  # a row of zeros takes scale 1
    r = _rand(shape, 7) if res else None
    if res:
        r[0] = 0
    g = _rand(shape, 8) if gated else None
    _, y = _ref(x, w, r, g, 1e-6)
    cols = heads * (width // group if group else 1)
    out = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    sbuf = torch.full((rows, cols + 3), -1.0, device="cuda")
    sc = sbuf[:, :cols]
    kda.kda_rmsnorm(x.cuda(), w.cuda(), out, residual=r.cuda() if res else None,
                    gate=g.cuda() if gated else None, scales=sc)
    torch.cuda.synchronize()
    yg = y.reshape(rows, cols, -1)
    top = yg.abs().amax(-1)
    want = torch.where(top > 0, top / 448, 1.0)
    got = sc.double().cpu()
    assert ((got - want).abs() <= 1e-5 * want).all()
    assert (got[0] == 1).all() and (sbuf[:, cols:] == -1).all()
    q = out.float().double().cpu().reshape(yg.shape)
    exact = yg / got[..., None]
    assert ((q - exact).abs() <= 2.0 ** -4 * 1.001 * exact.abs() + 2.0 ** -10).all()
    assert (q.abs().amax(-1)[1:] == 448).all()  # the largest value uses the format's range


@pytest.mark.gpu
def test_forward_in_place_broadcast_and_specials():
    shape = (6, 1, 1000)
    x, r, w = _rand(shape, 9), _rand(shape, 10), torch.ones(1000)
    z, y = _ref(x, w, r, None, 1e-6)
    xd, rd = x.cuda(), r.cuda()
    kda.kda_rmsnorm(xd, w.cuda(), xd, residual=rd, residual_out=rd)  # both in place
    assert torch.equal(rd.cpu(), z.to(BF))
    assert ((xd.double().cpu() - y).abs() <= 2.0 ** -8 * 1.01 * y.abs() + 1e-5).all()
    # one residual row for all rows (stride 0)
    one = _rand((1, 1, 1000), 11)
    out = torch.empty(shape, dtype=BF, device="cuda")
    kda.kda_rmsnorm(x.cuda(), w.cuda(), out, residual=one.cuda().expand(shape))
    y = _ref(x, w, one.expand(shape), None, 1e-6)[1]
    assert ((out.double().cpu() - y).abs() <= 2.0 ** -8 * 1.01 * y.abs() + 1e-5).all()
    # a NaN spoils its row and no other; fp8 keeps it a NaN
    x[2, 0, 5] = float("nan")
    x[3] = 0
    o8 = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.empty(6, 1, device="cuda")
    kda.kda_rmsnorm(x.cuda(), w.cuda(), o8, scales=sc)
    bad = o8.float().cpu().isnan().all(-1)[:, 0]
    assert bad.tolist() == [False, False, True, False, False, False]
    assert (o8[3].float() == 0).all() and sc[3, 0] == 1
    # no rows
    kda.kda_rmsnorm(x[:0].cuda(), w.cuda(), out[:0])
    torch.cuda.synchronize()


def _ref_bwd(z, w, dy, gate, dres, eps):
    z = z.double().requires_grad_()
    w = w.double().requires_grad_()
    g = gate.double().requires_grad_() if gate is not None else None
    y = z / torch.sqrt(z.pow(2).mean(-1, keepdim=True) + eps) * w
    if g is not None:
        y = y * torch.sigmoid(g)
    y.backward(dy.double())
    dz = z.grad if dres is None else z.grad + dres.double()
    return dz, w.grad, None if g is None else g.grad


@pytest.mark.gpu
@pytest.mark.parametrize("shape", SHAPES + [(3000, 5, 128)], ids=str)
@pytest.mark.parametrize("res,gated,pad,off", [(False, False, 0, 0), (True, False, 8, 0),
                                               (False, True, 1, 3), (True, True, 0, 0)])
def test_backward(shape, res, gated, pad, off):
    rows, heads, width = shape
    z, dy, w = _rand(shape, 12), _rand(shape, 13), 1 + 0.1 * _rand((width,), 14).float()
    r = _rand(shape, 15) if res else None
    g = _rand(shape, 16) if gated else None
    dz, dw, dg = _ref_bwd(z, w, dy, g, r, 1e-6)
    zd, yd = _strided(z, pad, off)[0], _strided(dy, pad, off)[0]
    out, obuf = _strided(torch.zeros(shape, dtype=BF), pad, off)
    dgo = _strided(torch.zeros(shape, dtype=BF), pad, off)[0] if gated else None
    dwo = torch.empty(width, device="cuda")
    kw = dict(gate=_strided(g, pad, off)[0] if gated else None, dgate=dgo,
              d_residual=_strided(r, pad, off)[0] if res else None)
    kda.kda_rmsnorm_backward(zd, w.cuda(), yd, out, dwo, **kw)
    torch.cuda.synchronize()
    s = 1 / torch.sqrt(z.double().pow(2).mean(-1, keepdim=True) + 1e-6)
    big = (s * (dy.double() * w.double()).abs()).amax(-1, keepdim=True)
    err = (out.double().cpu() - dz).abs()
    assert (err <= 2.0 ** -8 * dz.abs() + 2e-5 * big).all()
    if gated:
        top = dg.abs().amax(-1, keepdim=True)
        assert ((dgo.double().cpu() - dg).abs() <= (2.0 ** -8 + 2e-5) * dg.abs() + 1e-6 * top).all()
    mags = (dy.double() * z.double() * s).abs().sum((0, 1))
    assert ((dwo.double().cpu() - dw).abs() <= 2e-5 * mags + 1e-12).all()
    if pad:
        assert (obuf[off:].reshape(-1, heads * width + pad)[:, heads * width:] == -7.0).all()
    # the same bits again, with a workspace of the caller's holding anything
    ws = torch.full((kda.kda_rmsnorm_backward_workspace_size(rows, heads, width),), 255,
                    dtype=torch.uint8, device="cuda")
    again = torch.empty_like(dwo)
    kda.kda_rmsnorm_backward(zd, w.cuda(), yd, torch.empty(shape, dtype=BF, device="cuda"), again,
                             workspace=ws, **kw)
    assert torch.equal(again, dwo)


# the last group of 8 holds 1 to 7 channels, next to another head's; below 8 it is the only one
@pytest.mark.gpu
@pytest.mark.parametrize("width", [2, 3, 5, 6] + list(range(9, 16)) + list(range(2049, 2056)) +
                         [8190, 16383])
def test_partial_groups(width):
    """Out of place, in place (the same bits) and fp8; gradients too."""
    shape = (5, 3, width)
    x, r, g, dy = (_rand(shape, 30 + i) for i in range(4))
    w = 1 + 0.1 * _rand((width,), 34).float()
    z, y = _ref(x, w, r, g, 1e-6)
    top = y.abs().amax(-1, keepdim=True)
    out, zo = torch.empty(shape, dtype=BF, device="cuda"), torch.empty(shape, dtype=BF, device="cuda")
    kda.kda_rmsnorm(x.cuda(), w.cuda(), out, residual=r.cuda(), residual_out=zo, gate=g.cuda())
    assert ((out.double().cpu() - y).abs() <= (2.0 ** -8 + 2e-5) * y.abs() + 1e-6 * top).all()
    assert torch.equal(zo.cpu(), z.to(BF))
    xi, ri = x.cuda(), r.cuda()
    kda.kda_rmsnorm(xi, w.cuda(), xi, residual=ri, residual_out=ri, gate=g.cuda())
    assert torch.equal(xi, out) and torch.equal(ri, zo)
    o8 = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.empty(5, 3, device="cuda")
    kda.kda_rmsnorm(x.cuda(), w.cuda(), o8, residual=r.cuda(), gate=g.cuda(), scales=sc)
    scd = sc.double().cpu()[..., None]
    assert ((scd * 448 - top).abs() <= 2e-5 * top).all()
    # half an e4m3 step: 2^-4 of the value, 2^-10 where the format is at its smallest
    assert ((o8.double().cpu() * scd - y).abs() <=
            (2.0 ** -4 + 1e-4) * y.abs() + (2.0 ** -10 + 1e-6) * scd).all()
    dz, dw, dg = _ref_bwd(x, w, dy, g, r, 1e-6)
    dzo, dgo = torch.empty_like(out), torch.empty_like(out)
    dwo = torch.empty(width, device="cuda")
    kda.kda_rmsnorm_backward(x.cuda(), w.cuda(), dy.cuda(), dzo, dwo, gate=g.cuda(), dgate=dgo,
                             d_residual=r.cuda())
    for got, ref in ((dzo, dz), (dgo, dg)):
        # half a bf16 step; what cancels in dz is as large as the row's largest
        big = (ref.abs() + r.double().abs()).amax(-1, keepdim=True)
        assert ((got.double().cpu() - ref).abs() <= (2.0 ** -8 + 2e-5) * ref.abs() + 2e-5 * big).all()
    mags = (dy.double().abs() * (x.double() / torch.sqrt(
        x.double().pow(2).mean(-1, keepdim=True) + 1e-6)).abs()).sum((0, 1))
    assert ((dwo.double().cpu() - dw).abs() <= 2e-5 * mags + 1e-12).all()
    di, gi = dy.cuda(), g.cuda()
    kda.kda_rmsnorm_backward(x.cuda(), w.cuda(), di, di, gate=gi, dgate=gi, d_residual=r.cuda())
    assert torch.equal(di, dzo) and torch.equal(gi, dgo)


@pytest.mark.gpu
def test_backward_against_differences():
    """dz, dgate and dweight against central differences of the forward formula."""
    shape, h = (2, 1, 40), 1e-5
    z, dy, g = _rand(shape, 20), _rand(shape, 21), _rand(shape, 22)
    w = 1 + 0.1 * _rand((40,), 23).float()
    dz = torch.empty(shape, dtype=BF, device="cuda")
    dg, dw = torch.empty_like(dz), torch.empty(40, device="cuda")
    kda.kda_rmsnorm_backward(z.cuda(), w.cuda(), dy.cuda(), dz, dw, gate=g.cuda(), dgate=dg)

    def loss(z, w, g):
        return (_ref(z, w, None, g, 1e-6)[1] * dy.double()).sum()

    args = [z.double(), w.double(), g.double()]
    for k, got in ((0, dz), (1, dw), (2, dg)):
        for i in (0, 17, 39):
            lo, hi = [a.clone() for a in args], [a.clone() for a in args]
            lo[k].view(-1)[i] -= h
            hi[k].view(-1)[i] += h
            diff = (loss(*hi) - loss(*lo)) / (2 * h)
            # half a bf16 step, and the difference's own error of about h^2 and 1e-16 / h
            assert abs(got.reshape(-1)[i].double().cpu() - diff) <= 2.0 ** -8 * abs(diff) + 1e-5


@pytest.mark.gpu
def test_backward_optional_parts():
    shape = (10, 2, 128)
    z, dy, w = _rand(shape, 24).cuda(), _rand(shape, 25).cuda(), torch.ones(128, device="cuda")
    dz, dw = torch.empty_like(z), torch.full((128,), -1.0, device="cuda")
    kda.kda_rmsnorm_backward(z, w, dy, dz, dw)
    only = torch.empty_like(z)
    kda.kda_rmsnorm_backward(z, w, dy, only)  # no weight gradient, no workspace
    assert torch.equal(only, dz)
    inplace = dy.clone()
    kda.kda_rmsnorm_backward(z, w, inplace, inplace)
    assert torch.equal(inplace, dz)
    kda.kda_rmsnorm_backward(z[:0], w, dy[:0], dz[:0], dw)  # no rows: zeros
    assert (dw == 0).all()


@pytest.mark.gpu
def test_captured_and_on_another_stream():
    """Both calls in one graph, replayed with changed inputs, next to eager calls
    between the replays on the default stream with a workspace of their own."""
    shape = (65, 1, 2000)
    w = 1 + 0.1 * _rand((2000,), 30).float().cuda()
    x, r, dy = (torch.zeros(shape, dtype=BF, device="cuda") for _ in range(3))
    ws = torch.empty(kda.kda_rmsnorm_backward_workspace_size(65, 1, 2000), dtype=torch.uint8,
                     device="cuda")

    def both(ws):
        out = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
        sc, zr = torch.empty(65, 1, device="cuda"), torch.empty_like(x)
        dz, dw = torch.empty_like(x), torch.empty(2000, device="cuda")
        kda.kda_rmsnorm(x, w, out, residual=r, residual_out=zr, scales=sc)
        kda.kda_rmsnorm_backward(zr, w, dy, dz, dw, workspace=ws)
        return out, sc, zr, dz, dw

    both(ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = both(ws)
    own = torch.empty_like(ws)
    for k in range(3):
        for t, s in ((x, 40), (r, 50), (dy, 60)):
            t.copy_(_rand(shape, s + k))
        graph.replay()
        eager = both(own)
        torch.cuda.synchronize()
        for a, b in zip(captured, eager):
            assert np.array_equal(a.view(torch.uint8).cpu().numpy(),
                                  b.view(torch.uint8).cpu().numpy())


# gate logits from where the sigmoid is 1e-13 to where 1 - sigmoid is; each vector holds one
# size of them, so that no other element sets its scale
@pytest.mark.gpu
@pytest.mark.parametrize("heads,width", [(3, 128), (1, 1001), (1, 2048)])
def test_backward_of_saturated_gates(heads, width):
    """dgate = dy n w sig (1 - sig), each element to half a bf16 step and the fp32 arithmetic:
    the exponential's argument is rounded to 2^-24 of itself, twice, so sig and 1 - sig are off
    by 2 * 2^-24 * 30 = 4e-6 at a logit of 30, and the other factors by a few roundings and
    the norm's 4e-6: 2e-5 covers it."""
    logits = torch.arange(-30.0, 31.0)
    shape = (len(logits), heads, width)
    z, dy, w = _rand(shape, 70), _rand(shape, 71), 1 + 0.1 * _rand((width,), 72).float()
    g = (logits[:, None, None] + 0.5 * _rand(shape, 73).float().clamp(-1, 1)).to(BF)
    dz, dw, _ = _ref_bwd(z, w, dy, g, None, 1e-6)
    x = g.double()
    n = z.double() / torch.sqrt(z.double().pow(2).mean(-1, keepdim=True) + 1e-6)
    dg = dy.double() * n * w.double() * torch.sigmoid(x) * torch.sigmoid(-x)
    dzo, dgo = (torch.empty(shape, dtype=BF, device="cuda") for _ in range(2))
    kda.kda_rmsnorm_backward(z.cuda(), w.cuda(), dy.cuda(), dzo, gate=g.cuda(), dgate=dgo)
    assert ((dgo.double().cpu() - dg).abs() <= (2.0 ** -8 + 2e-5) * dg.abs()).all()
    s = 1 / torch.sqrt(z.double().pow(2).mean(-1, keepdim=True) + 1e-6)
    big = (s * (dy.double() * w.double() * torch.sigmoid(g.double())).abs()).amax(-1, keepdim=True)
    assert ((dzo.double().cpu() - dz).abs() <= 2.0 ** -8 * dz.abs() + 2e-5 * big).all()


@pytest.mark.gpu
def test_backward_of_infinite_gates():
    """A gate of -inf or +inf, or one whose exponential overflows: sigmoid 0 or 1, no gradient
    at the gate, and nothing else disturbed."""
    shape = (4, 1, 256)
    z, dy, w = _rand(shape, 74), _rand(shape, 75), torch.ones(256)
    g = _rand(shape, 76)
    for i, x in enumerate((float("-inf"), float("inf"), -200.0, 200.0)):
        g[i, 0, ::3] = x
    dzo, dgo = (torch.empty(shape, dtype=BF, device="cuda") for _ in range(2))
    kda.kda_rmsnorm_backward(z.cuda(), w.cuda(), dy.cuda(), dzo, gate=g.cuda(), dgate=dgo)
    sig = torch.sigmoid(g.double())
    s = 1 / torch.sqrt(z.double().pow(2).mean(-1, keepdim=True) + 1e-6)
    n, a = z.double() * s, dy.double() * sig
    dz = s * (a - n * (a * n).mean(-1, keepdim=True))
    dg = dy.double() * n * sig * (1 - sig)
    dg[:, 0, ::3] = 0  # (e^-200 is 1e-87, below every bf16)
    got = dgo.double().cpu()
    assert (got[:, 0, ::3] == 0).all()
    assert ((got - dg).abs() <= (2.0 ** -8 + 2e-5) * dg.abs()).all()
    big = (s * a.abs()).amax(-1, keepdim=True)
    assert ((dzo.double().cpu() - dz).abs() <= 2.0 ** -8 * dz.abs() + 2e-5 * big).all()


# more than 512 vectors, where fewer lanes hold each: on both sides of every shape's border, with
# whole and partial last groups, and enough rows that workgroups walk (the gradient's from 513
# vectors on; the forward's from 2049 on where one vector fills a workgroup, so that with 4200
# some take a third)
MANY = [(512, 1, 1024), (513, 1, 513), (513, 1, 1001), (4200, 1, 1024), (700, 3, 640),
        (513, 1, 1025), (4200, 1, 2048), (513, 1, 2049), (4200, 1, 3000), (700, 2, 4096),
        (512, 1, 8192), (513, 1, 4097), (4200, 1, 8192), (600, 1, 8191), (513, 1, 8193),
        (2100, 1, 16384), (520, 1, 16383), (515, 1, 12160),
        # where the gradient takes more than two workgroups per CU, and its borders
        (16391, 1, 1536), (9001, 1, 2816), (16400, 1, 3200), (8500, 1, 3201)]


def _gpu(shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(BF)


def _padded(t, pad):
    """A copy with `pad` more elements between the rows (and so off 16 bytes)."""
    rows, n = t.shape[0], t[0].numel()
    buf = torch.full((rows, n + pad), -7.0, dtype=t.dtype, device="cuda")
    v = buf.as_strided(t.shape, (n + pad,) + tuple(t.stride()[1:]))
    v.copy_(t)
    return v, buf[:, n:]


def test_workspace_of_narrow_and_wide_rows(lib):
    """A partial row for each of four workgroups per CU up to 3200 channels, of two above."""
    size = kda.kda_rmsnorm_backward_workspace_size
    assert size(10 ** 6, 1, 1024) == 512 * 1024 * 4 and size(10 ** 6, 1, 1025) == 1024 * 1025 * 4
    assert size(10 ** 6, 1, 3200) == 1024 * 3200 * 4 and size(10 ** 6, 1, 3201) == 512 * 3201 * 4


@pytest.mark.gpu
@pytest.mark.parametrize("shape", MANY, ids=str)
@pytest.mark.parametrize("gated,pad", [(False, 0), (True, 3)])
def test_forward_of_many_rows(shape, gated, pad):
    """bf16 out of place and in place (the same bits), fp8 with a scale per vector and per
    group; the tolerances of the other tests."""
    rows, heads, width = shape
    x, r, w = _gpu(shape, 80), _gpu(shape, 81, 2.0), 1 + 0.1 * _gpu((width,), 82).float()
    g = _gpu(shape, 83) if gated else None
    z, y = _ref(x, w, r, g, 1e-6)
    top = y.abs().amax(-1, keepdim=True)
    (xp, _), (rp, _), (out, gap), (zo, zgap) = (_padded(t, pad) for t in (x, r, x * 0, x * 0))
    gp = _padded(g, pad)[0] if gated else None
    kda.kda_rmsnorm(xp, w, out, residual=rp, residual_out=zo, gate=gp)
    assert ((out.double() - y).abs() <= (2.0 ** -8 + 2e-5) * y.abs() + 1e-6 * top).all()
    assert torch.equal(zo, z.to(BF))
    assert (gap == -7.0).all() and (zgap == -7.0).all()
    kda.kda_rmsnorm(xp, w, xp, residual=rp, residual_out=rp, gate=gp)
    assert torch.equal(xp, out) and torch.equal(rp, zo)
    for group in (width, 128):
        if width % group:
            continue
        o8 = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
        sc = torch.empty(rows, heads * width // group, device="cuda")
        kda.kda_rmsnorm(x, w, o8, residual=r, gate=g, scales=sc)
        yg = y.reshape(rows, -1, group)
        scd, most = sc.double()[..., None], yg.abs().amax(-1, keepdim=True)
        assert ((scd * 448 - most).abs() <= 2e-5 * most).all()
        assert ((o8.double().reshape(yg.shape) * scd - yg).abs() <=
                (2.0 ** -4 + 1e-4) * yg.abs() + (2.0 ** -10 + 1e-6) * scd).all()


@pytest.mark.gpu
@pytest.mark.parametrize("shape", MANY, ids=str)
@pytest.mark.parametrize("res,gated,pad", [(True, False, 0), (False, True, 3)])
def test_backward_of_many_rows(shape, res, gated, pad):
    rows, heads, width = shape
    z, dy, w = _gpu(shape, 84), _gpu(shape, 85), 1 + 0.1 * _gpu((width,), 86).float()
    r = _gpu(shape, 87) if res else None
    g = _gpu(shape, 88) if gated else None
    dz, dw, dg = _ref_bwd(z, w, dy, g, r, 1e-6)
    (zp, _), (dp, _), (out, gap) = (_padded(t, pad) for t in (z, dy, z * 0))
    kw = dict(gate=_padded(g, pad)[0] if gated else None, d_residual=r)
    dgo = _padded(z, pad)[0] if gated else None
    dwo = torch.empty(width, device="cuda")
    kda.kda_rmsnorm_backward(zp, w, dp, out, dwo, dgate=dgo, **kw)
    assert (gap == -7.0).all()
    s = 1 / torch.sqrt(z.double().pow(2).mean(-1, keepdim=True) + 1e-6)
    big = (s * (dy.double() * w.double()).abs()).amax(-1, keepdim=True)
    if res:
        big = big + r.double().abs().amax(-1, keepdim=True)
    assert ((out.double() - dz).abs() <= 2.0 ** -8 * dz.abs() + 2e-5 * big).all()
    if gated:
        assert ((dgo.double() - dg).abs() <= (2.0 ** -8 + 2e-5) * dg.abs()).all()
    mags = (dy.double() * z.double() * s).abs().sum((0, 1))
    assert ((dwo.double() - dw).abs() <= 2e-5 * mags + 1e-12).all()
    again, ws = torch.empty_like(dwo), torch.full(
        (kda.kda_rmsnorm_backward_workspace_size(rows, heads, width),), 255, dtype=torch.uint8,
        device="cuda")
    gi = kw.pop("gate")
    kda.kda_rmsnorm_backward(zp, w, dp, dp, again, gate=gi, dgate=gi, workspace=ws, **kw)
    assert torch.equal(again, dwo) and torch.equal(dp, out)  # in place
    assert gi is None or torch.equal(gi, dgo)


@pytest.mark.gpu
def test_strides_past_32_bits():
    """Rows 2^21 elements apart: 1100 of them span 2.3e9 elements. The same bits as from packed
    rows, forward (bf16 and fp8, with its scales) and gradient."""
    shape, stride = (1100, 2, 200), 1 << 21
    rows, n = shape[0], shape[1] * shape[2]
    x, r, g, dy = (_gpu(shape, 90 + i) for i in range(4))
    w = 1 + 0.1 * _gpu((200,), 94).float()

    def calls(place, o8, sc):
        xs, rs, gs, ys = (place(t, i) for i, t in enumerate((x, r, g, dy)))
        outs = [place(torch.zeros_like(x), 4 + i) for i in range(4)]
        dw = torch.empty(200, device="cuda")
        kda.kda_rmsnorm(xs, w, outs[0], residual=rs, residual_out=outs[1], gate=gs)
        kda.kda_rmsnorm(xs, w, o8, residual=rs, gate=gs, scales=sc)
        kda.kda_rmsnorm_backward(xs, w, ys, outs[2], dw, gate=gs, dgate=outs[3], d_residual=rs)
        torch.cuda.synchronize()
        return outs + [o8.view(torch.uint8), sc, dw]

    e4m3 = torch.float8_e4m3fn
    want = calls(lambda t, i: t, torch.empty(shape, dtype=e4m3, device="cuda"),
                 torch.empty(rows, 2, device="cuda"))
    buf = torch.empty(rows * stride, dtype=BF, device="cuda")
    far = torch.empty(rows * stride, dtype=torch.uint8, device="cuda")

    def place(t, i):
        v = buf[stride - 1 - (i + 1) * n:].as_strided(shape, (stride, 200, 1))
        v.copy_(t)
        return v

    got = calls(place, far.view(e4m3).as_strided(shape, (stride, 200, 1), 3),
                torch.empty(rows * stride, device="cuda").as_strided((rows, 2), (stride, 1)))
    for a, b in zip(got, want):
        assert torch.equal(a, b)

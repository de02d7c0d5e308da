"""Layer norm and RMS norm on the device (gift_norm_*) against fp64.

Tolerances, with u = 2^-24 and d the row length (rows R for the weight's
gradient).  A sum of d terms is off by at most d u times the sum of their
magnitudes, in any order.
"""

import numpy as np
import pytest
import torch

import fac_whitening_gift_amd as fg
from oracle import layer as ol
from gpu_util import DEV, host, say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
KINDS = [fg.NORM_LAYER, fg.NORM_RMS]
DTYPES = [torch.float32, torch.bfloat16]
SIZES = [(1, 1), (1, 4096), (2, 64), (3, 7), (5, 513), (9, 1000), (33, 1024), (7, 1025), (4, 2050), (6, 4096), (2, 8192),
         (3, 11008), (2, 16384), (2, 16385), (1, 40000), (1000, 96)]


def _draw(rows, d, seed, dtype, mean=0.1):
    rng = np.random.default_rng(seed)
    return torch.from_numpy((rng.standard_normal((rows, d)) + mean).astype(np.float32)).to(dtype)


def _half_step(dtype):
    return torch.finfo(dtype).eps / 2


def _inputs(rows, d, dtype):
    x, dy = _draw(rows, d, rows + d, dtype), _draw(rows, d, 7 * rows + d, dtype, 0.0)
    w, b = 1 + 0.2 * _draw(1, d, 3, torch.float32)[0], _draw(1, d, 4, torch.float32)[0]
    return x, dy, w, b


def _np(t):
    return None if t is None else t.detach().cpu().double().numpy()


def _check_forward(x, w, b, eps, kind, got):
    y, mean, rstd = got
    layer = kind == fg.NORM_LAYER
    d = x.shape[1]
    ry, rm, rr = ol.norm_forward(_np(x), _np(w), _np(b), eps, layer)
    xa = np.abs(_np(x))
    em = (d + 1) * U * xa.mean(1) if layer else np.zeros(x.shape[0])   # of the mean
    if layer:
        assert np.all(np.abs(_np(mean) - rm) <= em + 1e-300)
    else:
        assert mean is None
    # centred values off by em and a rounding: the mean square by 2 |c| e + e^2,
    # and (d + 2) u of itself; the root halves the relative error, and adds 2 u
    c = _np(x) - rm[:, None]
    e = em[:, None] + U * (np.abs(c) + em[:, None])
    var = (c * c).mean(1) + eps
    ev = (2 * np.abs(c) * e + e * e).mean(1) + (d + 2) * U * var
    er = rr * (0.5 * ev / var * (1 + ev / var) + 3 * U)
    assert np.all(np.abs(_np(rstd) - rr) <= er)
    wa = 1.0 if w is None else np.abs(_np(w))
    ba = 0.0 if b is None else np.abs(_np(b))
    ey = wa * (e * rr[:, None] + np.abs(c) * er[:, None]) * 1.01 + 3 * U * (wa * np.abs(c) * rr[:, None] + ba)
    ey = ey + _half_step(x.dtype) * (np.abs(ry) + ey)
    assert np.all(np.abs(_np(y) - ry) <= ey)


def _check_backward(dy, x, w, mean, rstd, kind, got):
    layer = kind == fg.NORM_LAYER
    rows, d = x.shape
    dx, dw, db = got
    rx, rw, rb = ol.norm_backward(_np(dy), _np(x), _np(w), _np(mean), _np(rstd), layer)
    r = _np(rstd)[:, None]
    c = _np(x) - (_np(mean)[:, None] if layer else 0.0)
    h, dya = np.abs(c * r), np.abs(_np(dy))
    g = dya * (1.0 if w is None else np.abs(_np(w)))
    if dx is not None:
        # h 2 u, g 1 u; the means (d + 3) u of the means of magnitudes; the rest 4 u
        along = (g * h).mean(1, keepdims=True)
        level = g.mean(1, keepdims=True) if layer else 0.0
        ex = r * ((d + 8) * U * (h * along + level) + 8 * U * (g + h * along + level))
        ex = ex + _half_step(x.dtype) * (np.abs(rx) + ex)
        assert np.all(np.abs(_np(dx) - rx) <= ex)
    if dw is not None:
        assert np.all(np.abs(_np(dw) - rw) <= (rows + 4) * U * (dya * h).sum(0) + 1e-300)
    if db is not None:
        assert np.all(np.abs(_np(db) - rb) <= (rows + 2) * U * dya.sum(0) + 1e-300)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,d", SIZES)
def test_forward_and_backward(rows, d, dtype, kind):
    say("norm %dx%d %s kind %d" % (rows, d, dtype, kind))
    x, dy, w, b = _inputs(rows, d, dtype)
    X, DY, W, B = (t.to(DEV) for t in (x, dy, w, b))
    eps = 1e-5
    got = fg.gift_norm_forward(X, W, B, eps=eps, kind=kind)
    assert got[0].dtype == dtype
    _check_forward(x, w, b, eps, kind, got)
    _check_forward(x, None, None, eps, kind, fg.gift_norm_forward(X, eps=eps, kind=kind))
    _, mean, rstd = got
    db = torch.empty(d, device=DEV)
    grads = fg.gift_norm_backward(DY, X, W, mean, rstd, kind=kind, dbias=db)
    _check_backward(dy, x, w, mean, rstd, kind, grads)
    _check_backward(dy, x, None, mean, rstd, kind, fg.gift_norm_backward(DY, X, None, mean, rstd, kind=kind))
    # one output at a time: the same bits
    dx1, n1, n2 = fg.gift_norm_backward(DY, X, W, mean, rstd, kind=kind, dweight=False, dbias=False)
    assert n1 is None and n2 is None and torch.equal(dx1, grads[0])
    n0, dw1, n2 = fg.gift_norm_backward(DY, X, W, mean, rstd, kind=kind, dx=False, dbias=False)
    assert n0 is None and n2 is None and torch.equal(dw1, grads[1])
    n0, n1, db1 = fg.gift_norm_backward(DY, X, W, mean, rstd, kind=kind, dx=False, dweight=False,
                                        dbias=torch.empty(d, device=DEV))
    assert n0 is None and n1 is None and torch.equal(db1, grads[2])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d", [96, 100, 4096, 9001, 17000])
def test_unaligned_and_in_place(d, kind):
    """Rows that start anywhere; Y over X, dX over dY; nothing written beside."""
    say("norm unaligned d=%d kind %d" % (d, kind))
    rows = 9
    for dtype in DTYPES:
        x, dy, w, b = _inputs(rows, d, dtype)
        W, B = w.to(DEV), b.to(DEV)
        want = fg.gift_norm_forward(x.to(DEV), W, B, kind=kind)
        flat = torch.full((rows * d + 3,), 5.0, dtype=dtype, device=DEV)
        view = flat[1:1 + rows * d].view(rows, d)
        view.copy_(x)
        y, mean, rstd = fg.gift_norm_forward(view, W, B, kind=kind, out=view)
        assert float(flat[0]) == 5.0 and float(flat[-2]) == 5.0 and float(flat[-1]) == 5.0
        _check_forward(x, w, b, 1e-5, kind, (y, mean, rstd))
        X = x.to(DEV)
        ref = fg.gift_norm_backward(dy.to(DEV), X, W, want[1], want[2], kind=kind)
        view.copy_(dy)
        got = fg.gift_norm_backward(view, X, W, want[1], want[2], kind=kind, dx=view)
        assert float(flat[0]) == 5.0 and float(flat[-2]) == 5.0
        _check_backward(dy, x, w, want[1], want[2], kind, (got[0], got[1], got[2]))
        D = dy.to(DEV)
        got = fg.gift_norm_backward(D, X, W, want[1], want[2], kind=kind, dx=D)
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_rows_of_one_value_and_far_means():
    """A constant row has variance 0: y = bias.  A mean far above the spread
    loses only what the mean's own rounding costs (the second pass)."""
    say("norm constant rows and far means")
    d = 4096
    x = torch.full((3, d), 3.0)
    b = _draw(1, d, 1, torch.float32)[0]
    y, mean, rstd = fg.gift_norm_forward(x.to(DEV), None, b.to(DEV))
    assert torch.equal(y.cpu(), b.expand(3, d)) and bool((mean == 3.0).all())
    x = _draw(4, d, 2, torch.float32, 1000.0)
    _check_forward(x, None, None, 1e-5, fg.NORM_LAYER, fg.gift_norm_forward(x.to(DEV)))


@pytest.mark.parametrize("kind", KINDS)
def test_nan_rows_stay_alone(kind):
    say("norm nan rows kind %d" % kind)
    x, dy, w, b = _inputs(20, 200, torch.float32)
    clean = fg.gift_norm_forward(x.to(DEV), w.to(DEV), b.to(DEV), kind=kind)
    x[3, 5], x[7, 0] = float("nan"), float("inf")
    y, mean, rstd = fg.gift_norm_forward(x.to(DEV), w.to(DEV), b.to(DEV), kind=kind)
    keep = [i for i in range(20) if i not in (3, 7)]
    assert torch.equal(y[keep], clean[0][keep]) and torch.equal(rstd[keep], clean[2][keep])
    assert bool(torch.isnan(y[3]).all()) and bool(torch.isnan(y[7]).any())
    dx, _, _ = fg.gift_norm_backward(dy.to(DEV), x.to(DEV), w.to(DEV), mean, rstd, kind=kind)
    assert bool(torch.isfinite(dx[keep]).all()) and bool(torch.isnan(dx[3]).all())


@pytest.mark.parametrize("rows,d", [(5, 40), (3000, 256), (700, 4096), (3, 20000)])
def test_accumulate_and_repeat(rows, d):
    say("norm accumulate %dx%d" % (rows, d))
    x, dy, w, _ = _inputs(rows, d, torch.float32)
    X, DY, W = x.to(DEV), dy.to(DEV), w.to(DEV)
    _, mean, rstd = fg.gift_norm_forward(X, W)
    dx, dw, db = fg.gift_norm_backward(DY, X, W, mean, rstd)
    _check_backward(dy, x, w, mean, rstd, fg.NORM_LAYER, (dx, dw, db))
    aw, ab = torch.ones(d, device=DEV), torch.full((d,), -2.0, device=DEV)
    fg.gift_norm_backward(DY, X, W, mean, rstd, dweight=aw, dbias=ab, accumulate=True)
    assert torch.equal(aw, dw + 1.0) and torch.equal(ab, db - 2.0)
    for _ in range(2):
        again = fg.gift_norm_backward(DY, X, W, mean, rstd)
        assert all(torch.equal(p, q) for p, q in zip(again, (dx, dw, db)))


def test_refuses():
    x = torch.zeros(4, 64, device=DEV)
    for bad in (x[:, ::2], x.half(), x[0], x.t()):
        with pytest.raises(ValueError):
            fg.gift_norm_forward(bad)
    with pytest.raises(ValueError):
        fg.gift_norm_forward(x, torch.ones(63, device=DEV))
    with pytest.raises(ValueError):
        fg.gift_norm_forward(x, kind=fg.NORM_RMS, mean=torch.ones(4, device=DEV))
    with pytest.raises(ValueError):
        fg.gift_norm_backward(x.bfloat16(), x, None, x[:, 0].contiguous(), x[:, 0].contiguous())
    with pytest.raises(ValueError):
        fg.gift_norm_backward(x, x, None, None, x[:, 0].contiguous(), accumulate=True)
    with pytest.raises(fg.GiftError):
        fg.gift_norm_backward(x, x, None, None, x[:, 0].contiguous())


@pytest.mark.parametrize("kind", KINDS)
def test_offsets_past_32_bits(kind):
    """2.4 G elements: the first and last rows equal those rows alone, and the
    gradients of the weight count every row."""
    say("norm large offsets kind %d" % kind)
    rows, d = 600001, 4096
    x = torch.empty(rows, d, dtype=torch.bfloat16, device=DEV).normal_()
    w = torch.ones(d, device=DEV)
    y, mean, rstd = fg.gift_norm_forward(x, w, kind=kind)
    pick = torch.tensor([0, rows // 2, rows - 1], device=DEV)
    alone = fg.gift_norm_forward(x[pick].contiguous(), w, kind=kind)
    assert torch.equal(y[pick], alone[0]) and torch.equal(rstd[pick], alone[2])
    # dY = 1: d bias is the number of rows, exactly; dX in place of dY
    dy = y.fill_(1.0)
    m = None if mean is None else mean[pick].contiguous()
    part = fg.gift_norm_backward(dy[pick].contiguous(), x[pick].contiguous(), w, m, rstd[pick].contiguous(),
                                 kind=kind)
    dx, dw, db = fg.gift_norm_backward(dy, x, w, mean, rstd, kind=kind, dx=dy, dbias=torch.empty(d, device=DEV))
    assert torch.equal(dx[pick], part[0]) and bool((db == rows).all()) and bool(torch.isfinite(dw).all())


@pytest.mark.parametrize("kind", KINDS)
def test_many_short_rows(kind):
    """5 M rows shorter than a vector, and the most rows there may be."""
    say("norm many short rows kind %d" % kind)
    rows, d = 5000001, 3
    x, dy, w, b = _inputs(rows, d, torch.float32)
    X, DY, W, B = (t.to(DEV) for t in (x, dy, w, b))
    got = fg.gift_norm_forward(X, W, B, kind=kind)
    _check_forward(x, w, b, 1e-5, kind, got)
    grads = fg.gift_norm_backward(DY, X, W, got[1], got[2], kind=kind, dbias=torch.empty(d, device=DEV))
    _check_backward(dy, x, w, got[1], got[2], kind, grads)
    X = torch.full((2 ** 24, 1), 2.0, device=DEV)
    y, mean, rstd = fg.gift_norm_forward(X, eps=0.0 if kind == fg.NORM_RMS else 1.0, kind=kind)
    assert bool((y == (1.0 if kind == fg.NORM_RMS else 0.0)).all())
    dx, dw, db = fg.gift_norm_backward(torch.ones_like(X), X, None, mean, rstd, kind=kind,
                                       dbias=torch.empty(1, device=DEV))
    assert bool((dx == 0.0).all()) and float(db) == 2 ** 24
    assert float(dw) == (2 ** 24 if kind == fg.NORM_RMS else 0.0)


@pytest.mark.parametrize("rows,d", [(70, 1000), (5, 20000)])
def test_side_stream_and_graph(rows, d):
    """The calls on another stream, and captured: replays equal eager calls,
    with eager work between them, and read the live inputs."""
    say("norm stream and graph %dx%d" % (rows, d))
    x, dy, w, b = (t.to(DEV) for t in _inputs(rows, d, torch.bfloat16))

    def step(stream=None):
        y, mean, rstd = fg.gift_norm_forward(x, w, b, stream=stream)
        return (y, mean, rstd) + fg.gift_norm_backward(dy, x, w, mean, rstd, stream=stream)
    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for rep in range(3):
        for t in got:
            t.fill_(float("nan"))
        step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want)), rep
    dy.mul_(2.0)   # a power of two: every gradient doubles, exactly
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and all(torch.equal(p, 2 * q) for p, q in zip(got[3:], want[3:]))

"""Softmax cross entropy over a vocabulary on the device (gift_xent_*) against
fp64.

Tolerances, with u = 2^-24.  A logit is a sum of d exact products: off by at
most es = 2 d 2^-23 sum |x w| (any order, any grouping).  The sum of
exponentials is joined from parts, each join and exponential adding a few u:
fewer than 50 + V / 2048 of them, 4 u each (V / 128 of up to 64 rows, whose
parts are of 128 columns and joined eight at a time: V / 1024); an exponential
exp2((s - m) log2 e) is off by 4 u and 3 u |s - m|, and |s - m| e^(s - m) <
0.37, of a sum that is at least 1: V terms of them, each with its own weight,
are held by 2 u (1 + ln V) of the sum.
D = exp(s - lse) - [target] for the lse given is off by exp(s - lse) (es + 3 u
|s - lse| + 4 u) and u; it is rounded to bf16 (a half step: 2^-8 relative),
twice for an fp32 dW (2^-16).
"""

import numpy as np
import pytest
import torch

import fac_whitening_gift_amd as fg
from oracle import step as os_
from gpu_util import DEV, host, say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16 = torch.bfloat16
HALF = 2.0 ** -8


def _draw(rows, d, vocab, seed=0, out=0.1):
    rng = np.random.default_rng(seed + rows + d + vocab)

    def normal(*shape):
        return torch.from_numpy(rng.standard_normal(shape).astype(np.float32))
    w = (normal(vocab, d) * 2 * d ** -0.5).to(BF16)
    t = torch.from_numpy(rng.integers(0, vocab, rows))
    toward = w[t].float()
    x = (normal(rows, d) + torch.from_numpy(rng.uniform(0, 15, (rows, 1)).astype(np.float32)) * toward /
         (toward.square().sum(1, keepdim=True) + 1e-3)).to(BF16)
    t[torch.from_numpy(rng.uniform(size=rows) < out)] = -100
    g = torch.from_numpy(rng.uniform(0.5, 1.5, rows).astype(np.float32)) / rows
    return x, w, t, g


def _np(t):
    return t.detach().cpu().double().numpy()


def _logit_error(x, w):
    return 2 * x.shape[1] * 2.0 ** -23 * (np.abs(_np(x)) @ np.abs(_np(w)).T)


def _check_forward(x, w, t, got):
    loss, lse = _np(got[0]), _np(got[1])
    vocab = w.shape[0]
    rl, rz, s = os_.xent_forward(_np(x), _np(w), t.numpy())
    es = _logit_error(x, w).max(axis=1)
    e = es + 4 * (50 + vocab / 1024) * U + 2 * U * (1 + np.log(vocab)) * 4
    assert np.all(np.abs(lse - rz) <= e + 3 * U * (np.abs(rz) + np.abs(s).max(axis=1)))
    live = os_.counts(t.numpy(), vocab)
    assert np.all(loss[~live] == 0)
    tol = (e + es + 4 * U * (np.abs(rz) + np.abs(s).max(axis=1)))
    assert np.all(np.abs(loss - rl)[live] <= tol[live])


def _check_backward(x, w, t, lse, g, dx, dw):
    X, W, z = _np(x), _np(w), _np(lse)
    live = os_.counts(t.numpy(), w.shape[0])
    X = np.where(live[:, None], X, 0.0)
    s = X @ W.T
    gl = np.where(live, 1.0 if g is None else _np(g), 0.0)
    rx, rw = os_.xent_backward(_np(x), W, t.numpy(), z, gl)
    D = os_.xent_residual(s, z, t.numpy())
    a = np.where(live[:, None], s - z[:, None], -np.inf)
    p = np.exp(a)
    ed = np.where(live[:, None], p * (_logit_error(torch.from_numpy(X), w) + 3 * U * np.abs(s - z[:, None]) + 4 * U) + U, 0.0)
    ga = np.abs(gl)[:, None]
    if dx is not None:
        sums = 2 * w.shape[0] * 2.0 ** -23
        e = ga * ((ed + (HALF + sums) * (np.abs(D) + ed)) @ np.abs(W))
        e = e + (HALF + U) * (np.abs(rx) + e)
        assert np.all(np.abs(_np(dx) - rx) <= e)
        assert not _np(dx)[~live].any()
    if dw is not None:
        part = HALF if dw.dtype == BF16 else HALF * HALF
        sums = 4 * x.shape[0] * 2.0 ** -23
        e = (ga * (ed + (part + sums + 3 * U) * (np.abs(D) + ed))).T @ np.abs(X)
        e = e + (HALF if dw.dtype == BF16 else 3 * U) * (np.abs(rw) + e)
        assert np.all(np.abs(_np(dw) - rw) <= e)


SIZES = [(1, 1, 1), (1, 64, 100), (3, 7, 5), (16, 96, 33), (17, 100, 257), (33, 40, 1000), (64, 130, 128), (65, 64, 256),
         (65, 33, 1), (70, 32, 300), (128, 128, 256), (129, 96, 511), (200, 1000, 777), (300, 257, 1500), (1000, 64, 2000)]


@pytest.mark.parametrize("rows,d,vocab", SIZES)
def test_forward_and_backward(rows, d, vocab):
    say("xent %d x %d over %d" % (rows, d, vocab))
    x, w, t, g = _draw(rows, d, vocab)
    X, W, T, G = x.to(DEV), w.to(DEV), t.to(DEV), g.to(DEV)
    loss, lse = fg.gift_xent_forward(X, W, T)
    torch.cuda.synchronize()
    _check_forward(x, w, t, (loss, lse))
    for gl, gd in ((g, G), (None, None)):
        for dtype in (torch.float32, BF16):
            dx, dw = fg.gift_xent_backward(X, W, T, lse, gd, dtype=dtype)
            torch.cuda.synchronize()
            assert dx.dtype == BF16 and dw.dtype == dtype
            _check_backward(x, w, t, lse, gl, dx, dw)
            # one output at a time: the same bits
            dx1, none = fg.gift_xent_backward(X, W, T, lse, gd, dw=False, dtype=dtype)
            assert none is None and torch.equal(dx1, dx)
            none, dw1 = fg.gift_xent_backward(X, W, T, lse, gd, dx=False, dtype=dtype)
            assert none is None and torch.equal(dw1, dw)


@pytest.mark.parametrize("rows", [5, 40, 150])
@pytest.mark.parametrize("d", [64, 100, 97])
def test_strides_and_alignment(rows, d):
    """Rows that lie apart and start anywhere, in X, W, dX and dW; nothing
    written between them."""
    say("xent strides rows=%d d=%d" % (rows, d))
    vocab = 300
    x, w, t, g = _draw(rows, d, vocab)
    T, G = t.to(DEV), g.to(DEV)
    want = fg.gift_xent_forward(x.to(DEV), w.to(DEV), T)
    ref = fg.gift_xent_backward(x.to(DEV), w.to(DEV), T, want[1], G)
    for pad, skip in ((3, 1), (8, 8)):
        X = torch.full((rows, d + pad), float("nan"), dtype=BF16, device=DEV)[:, :d]
        W = torch.full((vocab * (d + pad) + skip,), float("nan"), dtype=BF16, device=DEV)[skip:].view(vocab, d + pad)[:, :d]
        X.copy_(x)
        W.copy_(w)
        loss, lse = fg.gift_xent_forward(X, W, T)
        _check_forward(x, w, t, (loss, lse))
        assert torch.equal(lse, want[1]) and torch.equal(loss, want[0])
        dxf = torch.full((rows, d + pad), 7.0, dtype=BF16, device=DEV)
        dwf = torch.full((vocab, d + pad), 7.0, device=DEV)
        fg.gift_xent_backward(X, W, T, lse, G, dx=dxf[:, :d], dw=dwf[:, :d])
        assert torch.equal(dxf[:, :d], ref[0]) and torch.equal(dwf[:, :d], ref[1])
        assert bool((dxf[:, d:] == 7.0).all()) and bool((dwf[:, d:] == 7.0).all())


@pytest.mark.parametrize("rows", [7, 100])
def test_rows_left_out(rows):
    """Every row, or what counts for nothing holding NaN and infinities; targets
    past the vocabulary are left out and flagged."""
    say("xent rows left out rows=%d" % rows)
    d, vocab = 96, 333
    x, w, t, g = _draw(rows, d, vocab, out=0.0)
    t[1::3] = -1
    t[2::3] = vocab
    X, W, T, G = x.to(DEV), w.to(DEV), t.to(DEV), g.to(DEV)
    flags = torch.zeros(1, dtype=torch.int32, device=DEV)
    loss, lse = fg.gift_xent_forward(X, W, T, flags=flags)
    assert int(flags) == fg.FLAG_TARGET
    dx, dw = fg.gift_xent_backward(X, W, T, lse, G)
    _check_forward(x, w, t, (loss, lse))
    _check_backward(x, w, t, lse, g, dx, dw)
    X[1::3], X[2::3] = float("nan"), float("inf")
    G[1::3] = float("nan")
    flags.zero_()
    loss2, lse2 = fg.gift_xent_forward(X, W, T, flags=flags)
    assert torch.equal(loss2, loss) and int(flags) == fg.FLAG_TARGET
    dx2, dw2 = fg.gift_xent_backward(X, W, T, lse2, G)
    assert torch.equal(dx2, dx) and torch.equal(dw2, dw)
    # none counts
    T.fill_(-100)
    flags.zero_()
    loss, lse = fg.gift_xent_forward(X, W, T, flags=flags)
    assert int(flags) == 0 and not bool(loss.any())
    for dtype in (BF16, torch.float32):
        dx, dw = fg.gift_xent_backward(X, W, T, lse, G, dtype=dtype)
        assert not bool(dx.any()) and not bool(dw.any())


@pytest.mark.parametrize("rows", [4, 130])
def test_far_logits_and_nonfinite(rows):
    """Logits far apart (a certain token, -inf beside it), NaN in one row."""
    say("xent far logits rows=%d" % rows)
    d, vocab = 32, 300
    w = torch.zeros(vocab, d, dtype=BF16)
    w[:, 0] = torch.arange(vocab).to(BF16) * -1e4   # logits 0, -1e4, ...
    x = torch.zeros(rows, d, dtype=BF16)
    x[:, 0] = 1.0
    t = torch.zeros(rows, dtype=torch.int64)
    X, W, T = x.to(DEV), w.to(DEV), t.to(DEV)
    loss, lse = fg.gift_xent_forward(X, W, T)
    assert not bool(loss.any()) and not bool(lse.any())
    dx, dw = fg.gift_xent_backward(X, W, T, lse)
    assert not bool(dx.any()) and not bool(dw.any())
    W[5, 0] = float("-inf")   # a logit of -inf counts nothing
    flags = torch.zeros(1, dtype=torch.int32, device=DEV)
    loss, lse = fg.gift_xent_forward(X, W, T, flags=flags)
    assert not bool(loss.any()) and not bool(lse.any()) and int(flags) == 0
    W[5, 0] = 0.0
    clean = fg.gift_xent_forward(X, W, T)
    X[2, 3] = float("nan")
    loss, lse = fg.gift_xent_forward(X, W, T, flags=flags)
    keep = [i for i in range(rows) if i != 2]
    assert bool(torch.isnan(loss[2])) and bool(torch.isnan(lse[2])) and int(flags) == fg.FLAG_NONFINITE
    assert torch.equal(loss[keep], clean[0][keep]) and torch.equal(lse[keep], clean[1][keep])


@pytest.mark.parametrize("rows,d,vocab", [(40, 64, 500), (300, 100, 3000)])
def test_accumulate_repeat_stream_and_graph(rows, d, vocab):
    """dW added to; the same bits again; on another stream; captured, replays
    with eager work between them equal to the eager calls, reading live inputs."""
    say("xent accumulate, stream, graph %d x %d over %d" % (rows, d, vocab))
    x, w, t, g = (v.to(DEV) for v in _draw(rows, d, vocab))

    def step(stream=None):
        loss, lse = fg.gift_xent_forward(x, w, t, stream=stream)
        return (loss, lse) + fg.gift_xent_backward(x, w, t, lse, g, stream=stream)
    want = [v.clone() for v in step()]
    assert all(torch.equal(a, b) for a, b in zip(step(), want))
    acc = torch.full_like(want[3], 0.5)
    fg.gift_xent_backward(x, w, t, want[1], g, dx=False, dw=acc, accumulate=True)
    assert torch.equal(acc, want[3] + 0.5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for rep in range(3):
        for v in got:
            v.fill_(float("nan"))
        step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), rep
    g.mul_(2.0)   # a power of two: both gradients double, exactly
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], 2 * want[2]) and torch.equal(got[3], 2 * want[3])


def test_refuses():
    x, w = torch.zeros(4, 64, dtype=BF16, device=DEV), torch.zeros(9, 64, dtype=BF16, device=DEV)
    t, lse = torch.zeros(4, dtype=torch.int64, device=DEV), torch.zeros(4, device=DEV)
    for bad in (x.float(), x.half(), x[:, ::2], x[0], x.t(), x[:, :32]):
        with pytest.raises(ValueError):
            fg.gift_xent_forward(bad, w, t)
    for bad in (t.int(), t[:3], t.cpu(), t.view(2, 2)):
        with pytest.raises(ValueError):
            fg.gift_xent_forward(x, w, bad)
    with pytest.raises(ValueError):
        fg.gift_xent_forward(x, w, t, loss=lse[:2])
    with pytest.raises(ValueError):
        fg.gift_xent_backward(x, w, t, lse, accumulate=True)
    with pytest.raises(ValueError):
        fg.gift_xent_backward(x, w, t, lse, dtype=torch.float16)
    with pytest.raises(ValueError):
        fg.gift_xent_backward(x, w, t, lse, dx=torch.zeros(4, 64, device=DEV))
    with pytest.raises(fg.GiftError):
        fg.gift_xent_backward(x, w, t, lse, dx=False, dw=False)

"""CPU checks of the gift_mx_* and gift_norm_* entry points: sizes, and bad
arguments refused synchronously (before any HIP call, so no GPU is needed)."""

import ctypes

import pytest

import fac_whitening_gift_amd as fg
from fac_whitening_gift_amd import _lib

X, Y, W, WS = 0x10000, 0x20000, 0x30000, 0x100000
BF, F32 = fg.DTYPE_BF16, fg.DTYPE_F32
INVALID, SHAPE, SMALL = 1, 2, 3


def mx(rows=64, k=128, data=0x40000):
    return ctypes.pointer(_lib._Mx(rows, k, data))


def refused(status, want):
    assert status == want
    assert fg.load().gift_last_error()


def test_sizes():
    assert fg.gift_mx_bytes(64, 128) == 4352
    assert fg.gift_mx_bytes(1, 1) == 4352
    assert fg.gift_mx_bytes(65, 129) == 4 * 4352
    for rows, k in [(0, 1), (1, 0), (-1, 5), ((1 << 24) + 1, 1), (1 << 24, 1 << 13)]:
        assert fg.gift_mx_bytes(rows, k) == 0
    # a narrow operand whose padding takes it out of range
    assert fg.gift_mx_bytes(1 << 24, 4096) > 0
    assert fg.gift_mx_bytes(1 << 24, 4097) == 0
    assert fg.gift_mx_matmul_workspace_bytes(0, 5, 5) == 0
    assert fg.gift_mx_linear_workspace_bytes(1, 4096, 4096) == 0
    assert fg.gift_mx_linear_workspace_bytes(100, 4096, 4096) >= fg.gift_mx_bytes(100, 4096)
    assert fg.gift_norm_backward_workspace_bytes(0, 8) == 0
    assert fg.gift_norm_backward_workspace_bytes(1000, 64) > 0


@pytest.mark.parametrize("want,case", [
    (INVALID, dict(x=None)), (INVALID, dict(x=0x10001)), (INVALID, dict(dt=2)), (INVALID, dict(dt=-1)),
    (INVALID, dict(dt=F32, x=0x10002)),
    (SHAPE, dict(rows=0)), (SHAPE, dict(cols=0)), (SHAPE, dict(ld=127)), (SHAPE, dict(rows=1 << 25)),
    (INVALID, dict(row=None, col=None)),
    (INVALID, dict(row=mx(63))), (INVALID, dict(row=mx(64, 129))), (INVALID, dict(col=mx(64, 128))),
    (INVALID, dict(row=mx(data=None))), (INVALID, dict(row=mx(data=0x40008))),
    (INVALID, dict(flags=0x50002)),
    (INVALID, dict(rows=128, row=mx(128, 128), col=mx(128, 128))),
])
def test_quantize_refuses(want, case):
    a = dict(x=X, dt=BF, rows=64, cols=128, ld=128, row=mx(), col=mx(128, 64, 0x50000), flags=None)
    a.update(case)
    refused(fg.load().gift_mx_quantize(a["x"], a["dt"], a["rows"], a["cols"], a["ld"], a["row"], a["col"],
                                       a["flags"], None), want)


@pytest.mark.parametrize("want,case", [
    (INVALID, dict(a=None)), (INVALID, dict(out=None)), (INVALID, dict(dt=7)), (SHAPE, dict(ld=100)),
    (SHAPE, dict(a=mx(0))), (INVALID, dict(out=0x20001)),
])
def test_dequantize_refuses(want, case):
    a = dict(a=mx(), out=Y, dt=BF, ld=128)
    a.update(case)
    refused(fg.load().gift_mx_dequantize(a["a"], a["out"], a["dt"], a["ld"], None), want)


@pytest.mark.parametrize("want,case", [
    (INVALID, dict(a=None)), (INVALID, dict(b=None)), (INVALID, dict(b=mx(64, 256))), (INVALID, dict(c=None)),
    (INVALID, dict(dt=5)), (SHAPE, dict(ldc=63)), (INVALID, dict(bias=0x60002)),
    (INVALID, dict(acc=1)), (INVALID, dict(acc=1, dt=F32, bias=0x60000)),
    (SHAPE, dict(a=mx(1 << 23, 128), b=mx(1 << 14, 128), ldc=1 << 14)),
])
def test_matmul_refuses(want, case):
    a = dict(a=mx(), b=mx(), bias=None, c=Y, dt=BF, ldc=64, acc=0, ws=WS, n=1 << 30)
    a.update(case)
    refused(fg.load().gift_mx_matmul(a["a"], a["b"], a["bias"], a["c"], a["dt"], a["ldc"], a["acc"], a["ws"],
                                     a["n"], None), want)


def test_matmul_refuses_a_bad_workspace():
    lib = fg.load()
    m, n, k = 1024, 1024, 16384   # few tiles, a long sum: split over k
    need = fg.gift_mx_matmul_workspace_bytes(m, n, k)
    assert need >= 2 * m * n * 4

    def call(ws, nbytes):
        return lib.gift_mx_matmul(mx(m, k), mx(n, k), None, Y, F32, n, 0, ws, nbytes, None)
    refused(call(WS, need - 1), SMALL)
    refused(call(None, need), INVALID)
    refused(call(WS + 16, need), INVALID)


@pytest.mark.parametrize("want,case", [
    (INVALID, dict(x=None)), (INVALID, dict(dt=3)), (SHAPE, dict(rows=0)), (SHAPE, dict(ldx=4095)),
    (INVALID, dict(w=None)), (INVALID, dict(y=None)), (INVALID, dict(ydt=9)), (SHAPE, dict(ldy=4)),
    (INVALID, dict(flags=0x50001)), (SMALL, dict(rows=100, n=0)), (INVALID, dict(rows=100, ws=None)),
])
def test_linear_refuses(want, case):
    a = dict(x=X, dt=BF, rows=1, ldx=4096, w=mx(64, 4096), bias=None, y=Y, ydt=BF, ldy=64, flags=None, ws=WS,
             n=1 << 30)
    a.update(case)
    refused(fg.load().gift_mx_linear(a["x"], a["dt"], a["rows"], a["ldx"], a["w"], a["bias"], a["y"], a["ydt"],
                                     a["ldy"], a["flags"], a["ws"], a["n"], None), want)


@pytest.mark.parametrize("want,case", [
    (INVALID, dict(x=None)), (INVALID, dict(y=None)), (INVALID, dict(dt=4)), (SHAPE, dict(rows=0)),
    (SHAPE, dict(d=0)), (SHAPE, dict(d=1 << 25)), (INVALID, dict(kind=2)), (INVALID, dict(eps=-1.0)),
    (INVALID, dict(eps=float("nan"))), (INVALID, dict(eps=float("inf"))), (INVALID, dict(w=0x30001)),
    (INVALID, dict(mean=0x50002)), (INVALID, dict(x=0x10001)),
])
def test_norm_forward_refuses(want, case):
    a = dict(x=X, dt=BF, rows=4, d=64, kind=0, w=W, b=None, eps=1e-5, y=Y, mean=0x50000, rstd=0x60000)
    a.update(case)
    refused(fg.load().gift_norm_forward(a["x"], a["dt"], a["rows"], a["d"], a["kind"], a["w"], a["b"], a["eps"],
                                        a["y"], a["mean"], a["rstd"], None), want)


@pytest.mark.parametrize("want,case", [
    (INVALID, dict(x=None)), (INVALID, dict(dy=None)), (INVALID, dict(dt=4)), (SHAPE, dict(d=0)),
    (INVALID, dict(kind=5)), (INVALID, dict(dx=None, dw=None, db=None)), (INVALID, dict(mean=None)),
    (INVALID, dict(rstd=None)), (INVALID, dict(dx=0x70001)), (INVALID, dict(dw=0x70002)),
    (SMALL, dict(n=16)), (INVALID, dict(ws=None)), (INVALID, dict(ws=WS + 8)),
])
def test_norm_backward_refuses(want, case):
    a = dict(dy=Y, x=X, dt=BF, rows=4, d=64, kind=0, w=W, mean=0x50000, rstd=0x60000, dx=0x70000, dw=0x80000,
             db=0x90000, acc=0, ws=WS, n=1 << 30)
    a.update(case)
    refused(fg.load().gift_norm_backward(a["dy"], a["x"], a["dt"], a["rows"], a["d"], a["kind"], a["w"],
                                         a["mean"], a["rstd"], a["dx"], a["dw"], a["db"], a["acc"], a["ws"],
                                         a["n"], None), want)


def test_python_refuses_host_tensors():
    import torch
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        fg.gift_mx_quantize(x, by_row=True)
    with pytest.raises(ValueError):
        fg.gift_norm_forward(x)
    with pytest.raises(ValueError):
        fg.gift_mx_matmul(x, x)


def test_norm_refuses_one_buffer_for_two_results():
    lib = fg.load()
    refused(lib.gift_norm_forward(X, BF, 4, 64, 0, W, None, 1e-5, Y, 0x50000, 0x50000, None), INVALID)
    refused(lib.gift_norm_backward(Y, X, BF, 4, 64, 0, W, 0x50000, 0x60000, 0x70000, 0x80000, 0x80000, 0, WS,
                                   1 << 30, None), INVALID)

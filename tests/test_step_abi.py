"""CPU checks of the entry points of a training step around its layers: sizes,
and bad arguments refused synchronously (before any HIP call, so no GPU is
needed)."""

import pytest
import torch

import fac_whitening_gift_amd as fg

X, W, T, LOSS, LSE, DX, DW, WS = (0x100000 * i for i in range(1, 9))
BF, F32 = fg.DTYPE_BF16, fg.DTYPE_F32
INVALID, SHAPE, SMALL = 1, 2, 3


def refused(status, want):
    assert status == want
    assert fg.load().gift_last_error()


def test_xent_sizes():
    for rows, d, vocab in [(0, 64, 100), (1, 0, 100), (1, 64, 0), (-1, 64, 100), ((1 << 20) + 1, 64, 100),
                           (1, (1 << 16) + 1, 100), (1, 64, (1 << 20) + 1)]:
        assert fg.gift_xent_forward_workspace_bytes(rows, d, vocab) == 0
        assert fg.gift_xent_backward_workspace_bytes(rows, d, vocab) == 0
    assert fg.gift_xent_forward_workspace_bytes(1, 64, 100) > 0
    assert fg.gift_xent_backward_workspace_bytes(5, 64, 100, dx=False, dw=False) == 0
    both = fg.gift_xent_backward_workspace_bytes(5000, 640, 10000)
    for other in (dict(dx=False), dict(dw=False), dict(dtype=torch.bfloat16)):
        assert 0 < fg.gift_xent_backward_workspace_bytes(5000, 640, 10000, **other) < both
    # far less than the logits
    n, v = 1 << 17, 131072
    assert fg.gift_xent_forward_workspace_bytes(n, 4096, v) < 4 * n * v / 16
    assert fg.gift_xent_backward_workspace_bytes(n, 4096, v) < 4 * n * v / 4


@pytest.mark.parametrize("want,case", [
    (INVALID, dict(x=None)), (INVALID, dict(x=X + 1)), (INVALID, dict(w=None)), (INVALID, dict(w=W + 1)),
    (SHAPE, dict(rows=0)), (SHAPE, dict(d=0)), (SHAPE, dict(vocab=0)), (SHAPE, dict(rows=1 << 21)),
    (SHAPE, dict(d=1 << 17)), (SHAPE, dict(vocab=1 << 21)), (SHAPE, dict(ldx=63)), (SHAPE, dict(ldw=10)),
    (INVALID, dict(t=None)), (INVALID, dict(t=T + 4)), (INVALID, dict(loss=None, lse=None)),
    (INVALID, dict(loss=LSE)), (INVALID, dict(loss=LOSS + 2)), (INVALID, dict(flags=0x50001)),
    (SMALL, dict(n=0)), (INVALID, dict(ws=None)), (INVALID, dict(ws=WS + 16)),
])
def test_xent_forward_refuses(want, case):
    a = dict(x=X, rows=4, d=64, ldx=64, w=W, vocab=100, ldw=64, t=T, loss=LOSS, lse=LSE, flags=None, ws=WS, n=1 << 30)
    a.update(case)
    refused(fg.load().gift_xent_forward(a["x"], a["rows"], a["d"], a["ldx"], a["w"], a["vocab"], a["ldw"], a["t"],
                                        a["loss"], a["lse"], a["flags"], a["ws"], a["n"], None), want)


@pytest.mark.parametrize("want,case", [
    (INVALID, dict(x=None)), (INVALID, dict(w=None)), (INVALID, dict(t=None)), (INVALID, dict(lse=None)),
    (INVALID, dict(lse=LSE + 1)), (INVALID, dict(g=LOSS + 2)), (INVALID, dict(dx=None, dw=None)),
    (INVALID, dict(dt=5)), (SHAPE, dict(lddx=63)), (SHAPE, dict(lddw=63)), (INVALID, dict(dx=DX + 1)),
    (INVALID, dict(dw=DW + 2)), (INVALID, dict(dx=DW)), (INVALID, dict(dt=BF, acc=1)), (INVALID, dict(dw=None, acc=1)),
    (SHAPE, dict(rows=0)), (SMALL, dict(n=100)), (INVALID, dict(ws=None)), (INVALID, dict(ws=WS + 8)),
])
def test_xent_backward_refuses(want, case):
    a = dict(x=X, rows=4, d=64, ldx=64, w=W, vocab=100, ldw=64, t=T, lse=LSE, g=LOSS, dx=DX, lddx=64, dw=DW, dt=F32,
             lddw=64, acc=0, ws=WS, n=1 << 30)
    a.update(case)
    refused(fg.load().gift_xent_backward(a["x"], a["rows"], a["d"], a["ldx"], a["w"], a["vocab"], a["ldw"], a["t"],
                                         a["lse"], a["g"], a["dx"], a["lddx"], a["dw"], a["dt"], a["lddw"], a["acc"],
                                         a["ws"], a["n"], None), want)


def test_python_refuses_host_tensors_and_types():
    x, w, t = torch.zeros(4, 64), torch.zeros(9, 64), torch.zeros(4, dtype=torch.int64)
    for bad in (x, x.bfloat16()):
        with pytest.raises(ValueError):
            fg.gift_xent_forward(bad, w.bfloat16(), t)
        with pytest.raises(ValueError):
            fg.gift_xent_backward(bad, w.bfloat16(), t, x[:, 0].contiguous())

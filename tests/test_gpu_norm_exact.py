"""The norm's weight and bias gradients on rows of +-1, where they are whole
numbers: with eps = 0 (and, for layer norm, as many +1 as -1 in a row) h = x
and rstd = 1 exactly, so for dY = c_i x_i of row i
  dweight = sum c_i,  dbias_j = sum c_i x_ij,  dX = 0,
all exact in fp32 while they stay below 2^24.  Every row has to be counted
once: a rounding bound over millions of rows would let lost ones pass."""

import pytest
import torch

import fac_whitening_gift_amd as fg
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

KINDS = [fg.NORM_LAYER, fg.NORM_RMS]


def _signs(rows, d, dtype, balanced, g):
    if not balanced:
        return (torch.randint(0, 2, (rows, d), generator=g, device=DEV, dtype=torch.int8) * 2 - 1).to(dtype)
    half = _signs(rows, d // 2, dtype, False, g)
    return torch.cat([half, -half], 1)[:, torch.randperm(d, generator=g, device=DEV)].contiguous()


def _check(rows, d, dtype, kind):
    g = torch.Generator(device=DEV).manual_seed(rows + d)
    x = _signs(rows, d, dtype, kind == fg.NORM_LAYER, g)
    y, mean, rstd = fg.gift_norm_forward(x, eps=0.0, kind=kind)
    assert torch.equal(y, x) and bool((rstd == 1).all()) and (mean is None or bool((mean == 0).all()))
    c = torch.randint(-1, 4, (rows, 1), generator=g, device=DEV, dtype=torch.int8)
    c[rows // 2:] = 2   # no run of rows sums to what another does
    dy = x * c.to(dtype)
    total = c.sum(dtype=torch.float64)
    assert float(c.double().abs().sum()) + 7 < 2 ** 24
    level = torch.zeros(d, dtype=torch.float64, device=DEV)
    for i in range(0, rows, 100000):
        level += dy[i:i + 100000].double().sum(0)
    db = torch.empty(d, device=DEV)
    dx, dw, db = fg.gift_norm_backward(dy, x, None, mean, rstd, kind=kind, dbias=db)
    assert bool((dx == 0).all())
    assert bool((dw.double() == total).all()) and torch.equal(db.double(), level)
    aw, ab = torch.full((d,), 7.0, device=DEV), torch.full((d,), -7.0, device=DEV)
    fg.gift_norm_backward(dy, x, None, mean, rstd, kind=kind, dx=dy, dweight=aw, dbias=ab, accumulate=True)
    assert bool((aw.double() == total + 7).all()) and torch.equal(ab.double(), level - 7)
    assert bool((dy == 0).all())


# every width class of the register form, whole vectors and not; rows shorter
# than a vector, and wider than the register form (an odd row of +-1 has no
# zero mean)
WIDTHS = [1, 2, 3, 6, 8, 100, 128, 250, 256, 500, 512, 1000, 1001, 1024, 2000, 2050, 4095, 4096, 6002, 6144, 8190,
          8192, 9001, 12288, 16382, 16384, 17000, 20001]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d,kind", [(d, kind) for d in WIDTHS for kind in KINDS
                                    if kind == fg.NORM_RMS or d % 2 == 0])
def test_gradients_count_every_row(d, kind, dtype):
    for rows in (1, 7, 1003, 5000):
        say("norm exact %dx%d %s kind %d" % (rows, d, dtype, kind))
        _check(rows, d, dtype, kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,d,dtype", [(600001, 4096, torch.bfloat16), (300001, 8190, torch.float32),
                                          (150001, 17000, torch.bfloat16), (5000001, 2, torch.float32),
                                          (5000001, 6, torch.bfloat16)])
def test_gradients_count_millions_of_rows(rows, d, dtype, kind):
    """Register form and wide form past 2^31 elements, and 5 M short rows."""
    say("norm exact %dx%d %s kind %d" % (rows, d, dtype, kind))
    _check(rows, d, dtype, kind)


@pytest.mark.parametrize("d", [200, 4096, 17000])
def test_rows_that_overflow(d):
    """Squares past fp32: rstd 0, Y the bias; layer norm's sum past it too: NaN."""
    say("norm overflow d=%d" % d)
    x = torch.full((3, d), 1e25, device=DEV)
    x[:, ::2] = -2e25
    x[1] = 1.0
    b = torch.randn(d, device=DEV)
    for kind in KINDS:
        y, _, rstd = fg.gift_norm_forward(x, None, b, kind=kind)
        assert float(rstd[0]) == 0 and float(rstd[2]) == 0 and bool(torch.isfinite(y).all())
        assert torch.equal(y[0], b) and torch.equal(y[2], b)
    x[0] = 3e38
    y, mean, rstd = fg.gift_norm_forward(x, None, b)
    assert float(rstd[0]) == 0 and float(mean[0]) == float("inf") and bool(torch.isnan(y[0]).all())
    assert bool(torch.isfinite(y[1:]).all())
    y, _, rstd = fg.gift_norm_forward(x, None, b, kind=fg.NORM_RMS)
    assert float(rstd[0]) == 0 and torch.equal(y[0], b)

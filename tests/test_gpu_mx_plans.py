"""Every instance of the MXFP4 product on the device (the shapes of
mx_plans.py: tiles with rows of C on 128-byte lines and not, split sums, the
small form by rows and columns, the one-launch linear), on operands whose
products are exact in fp32: whole results have to be equal to the fp64
product, in both types, with a bias and accumulated."""

import pytest
import torch

import fac_whitening_gift_amd as fg
import mx_plans as mp
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _operands(m, n, k):
    """-> the two operands and their exact fp64 product"""
    g = _gen(m + 3 * n + 7 * k)
    a, ra = mp.exact_values(m, k, g, DEV)
    b, rb = mp.exact_values(n, k, g, DEV)
    qa, qb = (fg.gift_mx_quantize(t, by_row=True)[0] for t in (a, b))
    assert torch.equal(fg.gift_mx_dequantize(qa), a) and torch.equal(fg.gift_mx_dequantize(qb), b)
    return qa, qb, mp.exact_product(a, ra, b, rb)


def _rounded(c, dtype):
    return c.float().to(dtype)


@pytest.mark.parametrize("shape", mp.PRODUCTS)
def test_product_is_exact(shape):
    say("mx exact product %dx%dx%d" % shape)
    m, n, k = shape
    assert mp.plan(*shape) == mp.PRODUCTS[shape]
    qa, qb, want = _operands(m, n, k)
    for dtype in (torch.float32, BF16):
        assert torch.equal(fg.gift_mx_matmul(qa, qb, dtype=dtype), _rounded(want, dtype)), dtype
    bias = torch.randn(n, generator=_gen(1), device=DEV)
    # one fp32 addition to the exact sum
    with_bias = want.float() + bias
    for dtype in (torch.float32, BF16):
        got = fg.gift_mx_matmul(qa, qb, bias=bias, dtype=dtype)
        assert torch.equal(got, with_bias.to(dtype)), dtype
    acc = torch.randn(m, n, generator=_gen(2), device=DEV)
    before = acc.clone()
    fg.gift_mx_matmul(qa, qb, out=acc, accumulate=True)
    assert torch.equal(acc, before + want.float())


@pytest.mark.parametrize("shape", mp.PRODUCTS)
def test_product_into_a_slice(shape):
    """Rows of a wider C: at a line, and off it; what lies beside stays."""
    say("mx exact product %dx%dx%d into a slice" % shape)
    m, n, k = shape
    qa, qb, want = _operands(m, n, k)
    bias = torch.randn(n, generator=_gen(3), device=DEV)
    for dtype in (torch.float32, BF16):
        for ld, off in ((-(-(n + 64) // 64) * 64, 64), (n + 7, 3)):
            flat = torch.full(((m + 2) * ld + 64,), -7.0, dtype=dtype, device=DEV)
            view = flat[:(m + 2) * ld].view(m + 2, ld)[1:-1, off:off + n]
            fg.gift_mx_matmul(qa, qb, bias=bias, out=view)
            assert torch.equal(view, (want.float() + bias).to(dtype))
            if dtype == torch.float32:
                fg.gift_mx_matmul(qa, qb, out=view, accumulate=True)
                assert torch.equal(view, (want.float() + bias) + want.float())
            view.fill_(-7.0)
            assert bool((flat == -7.0).all())


@pytest.mark.parametrize("x_dtype", [torch.float32, BF16])
@pytest.mark.parametrize("shape", mp.LINEARS)
def test_linear_is_exact(shape, x_dtype):
    say("mx exact linear %dx%dx%d %s" % (shape + (x_dtype,)))
    rows, n, k = shape
    assert mp.linear_cols(*shape) == mp.LINEARS[shape]
    g = _gen(rows + n + k)
    x, rx = mp.exact_values(rows, k, g, DEV)
    w, rw = mp.exact_values(n, k, g, DEV)
    want = mp.exact_product(x, rx, w, rw)
    qw, _ = fg.gift_mx_quantize(w, by_row=True)
    bias = torch.randn(n, generator=g, device=DEV)
    x = x.to(x_dtype)   # exact: at most 3 bits and a sign
    for dtype in (torch.float32, BF16):
        assert torch.equal(fg.gift_mx_linear(x, qw, dtype=dtype), _rounded(want, dtype))
        assert torch.equal(fg.gift_mx_linear(x, qw, bias=bias, dtype=dtype), (want.float() + bias).to(dtype))
    wide = torch.full((rows, k + 9), float("nan"), dtype=x_dtype, device=DEV)
    wide[:, 5:5 + k] = x
    assert torch.equal(fg.gift_mx_linear(wide[:, 5:5 + k], qw, dtype=torch.float32), want.float())

"""Every instance of the MXFP4 product on the device (the shapes of
mx_plans.py: tiles with rows of C on 128-byte lines and not, split sums, the
small form by rows and columns, the one-launch linear), on operands whose
products are exact in fp32: whole results have to be equal to the fp64
product, in both types, with a bias and accumulated; and operands and results
past 32-bit offsets."""

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


@pytest.mark.parametrize("n", [16, 700])
def test_operands_past_32_bits(n):
    """An operand of 4.5 GB as A and as B.  Its rows are 97 rows over and
    over, each time times another power of two, so the whole result is known;
    no offset that loses its upper bits meets an equal row (2^31 and 2^32
    bytes are no whole multiples of 97 rows)."""
    say("mx exact operands past 32 bits n=%d" % n)
    rows, k = 70000, 122000
    g = _gen(n)
    base, rb = mp.exact_values(97, k, g, DEV)
    w, rw = mp.exact_values(n, k, g, DEV)
    small = mp.exact_product(base, rb, w, rw)
    at = torch.arange(rows, device=DEV)
    power = torch.exp2((at // 97 % 5 - 2).float())[:, None]
    x = torch.empty(rows, k, dtype=BF16, device=DEV)
    for i in range(0, rows, 10000):   # (in parts: less memory on the way)
        x[i:i + 10000] = (base.to(BF16)[at[i:i + 10000] % 97] * power[i:i + 10000].to(BF16))
    q, _ = fg.gift_mx_quantize(x, by_row=True)
    del x
    assert q.data.numel() > 2 ** 32
    for wrap in (2 ** 31, 2 ** 32):
        assert wrap * 64 // (-(-k // 128) * 4352) % 97 != 0
    qw, _ = fg.gift_mx_quantize(w, by_row=True)
    want = (small[at % 97] * power.double()).float()
    assert torch.equal(fg.gift_mx_matmul(q, qw, dtype=torch.float32), want)
    assert torch.equal(fg.gift_mx_matmul(qw, q, dtype=torch.float32), want.t().contiguous())


@pytest.mark.parametrize("shape", [(5, 300, 600), (40, 300, 600), (300, 1083, 300), (1999, 4064, 300)])
def test_rows_far_apart(shape):
    """Rows of X and of C whose offsets pass 2^32 bytes in small matrices."""
    say("mx rows far apart %dx%dx%d" % shape)
    m, n, k = shape
    ld = 2 ** 33 // m // 64 * 64 + 64   # 16 GB of bf16 from the first row to the last
    g = _gen(m)
    a, ra = mp.exact_values(m, k, g, DEV)
    b, rb = mp.exact_values(n, k, g, DEV)
    want = mp.exact_product(a, ra, b, rb)
    wide = torch.zeros(m, ld, dtype=BF16, device=DEV)
    wide[:, 64:64 + k] = a.to(BF16)
    x = wide[:, 64:64 + k]
    qa, _ = fg.gift_mx_quantize(x, by_row=True)
    qb, _ = fg.gift_mx_quantize(b, by_row=True)
    assert torch.equal(fg.gift_mx_dequantize(qa), a)
    assert torch.equal(fg.gift_mx_linear(x, qb, dtype=torch.float32), want.float())
    view = wide[:, 128:128 + n]
    fg.gift_mx_matmul(qa, qb, out=view)
    assert torch.equal(view, _rounded(want, BF16))
    view = wide[:, 64:64 + k]
    fg.gift_mx_dequantize(qa, out=view)
    assert torch.equal(view, a.to(BF16))


@pytest.mark.parametrize("shape", [(7, 100, 500), (300, 2100, 900), (1999, 4064, 300), (349, 33, 26797)])
def test_operands_at_any_16_bytes(shape):
    """Operands that start 16 bytes past a larger alignment; nothing beside
    them is written."""
    say("mx operands at 16 bytes %dx%dx%d" % shape)
    g = _gen(sum(shape))
    m, n, k = shape
    want, ops = [], []
    for rows in (m, n):
        v, r = mp.exact_values(rows, k, g, DEV)
        size = fg.gift_mx_bytes(rows, k)
        buf = torch.full((size + 48,), 171, dtype=torch.uint8, device=DEV)
        op = fg.MxOperand(rows, k, data=buf[16:16 + size])
        fg.gift_mx_quantize(v, by_row=op)
        assert bool((buf[:16] == 171).all()) and bool((buf[16 + size:] == 171).all())
        assert torch.equal(fg.gift_mx_dequantize(op), v)
        want += [v, r]
        ops.append(op)
    assert torch.equal(fg.gift_mx_matmul(*ops, dtype=torch.float32), mp.exact_product(*want).float())
    assert torch.equal(fg.gift_mx_linear(want[0], ops[1], dtype=torch.float32), mp.exact_product(*want).float())

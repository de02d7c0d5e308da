"""CPU check that the shapes of tests/mx_plans.py still reach the kernel
instances that they are there for, and that between them they reach all."""

import pytest

import mx_plans as mp


@pytest.mark.parametrize("shape", mp.PRODUCTS)
def test_products(shape):
    assert mp.plan(*shape) == mp.PRODUCTS[shape]


@pytest.mark.parametrize("shape", mp.LINEARS)
def test_linears(shape):
    assert mp.linear_cols(*shape) == mp.LINEARS[shape]


def test_every_instance_is_there():
    tiles, few, split = set(), set(), set()
    for (m, n, _), (rows, cols, splits) in mp.PRODUCTS.items():
        if rows == 64:
            few.add((16 if m <= 16 else 32 if m <= 32 else 64, cols))
        elif splits > 1:
            split.add((splits, n % 32 == 0))
        else:
            tiles |= {(cols, "bf16", n % 64 == 0), (cols, "f32", n % 32 == 0)}
    assert tiles == {(c, t, w) for c in (128, 256) for t in ("bf16", "f32") for w in (False, True)}
    assert few == {(r, c) for r in (16, 32, 64) for c in (16, 32, 64)}
    assert {s for s, _ in split} == {2, 4, 8, 15, 16} and {w for _, w in split} == {False, True}
    assert set(mp.LINEARS.values()) == {0, 16, 32, 64}


def test_exact_values_are_exact():
    """The oracle's quantization gives the values back, and fp32 sums them
    exactly in either direction."""
    import numpy as np
    import torch
    from oracle import layer as ol
    g = torch.Generator().manual_seed(1)
    a, ra = mp.exact_values(9, 333, g, "cpu")
    b, rb = mp.exact_values(7, 333, g, "cpu")
    for v in (a, b):
        codes, scales, _ = ol.quantize(v.numpy())
        assert np.array_equal(ol.values(codes, scales, 333), v.double().numpy())
    want = mp.exact_product(a, ra, b, rb)
    for order in (range(333), reversed(range(333))):
        s = torch.zeros(9, 7)
        for i in order:
            s = s + a[:, i:i + 1] * b[:, i]
        assert torch.equal(s.double(), want)


def test_lds_of_the_one_launch_linear():
    """Rows quantized in front of a product take 68 bytes per row and 128 k
    elements; the cut keeps them under 32.5 KB."""
    most = 0
    for rows in range(1, 17):
        for steps in list(range(400 // rows, 520 // rows + 2)) + [600, 2000]:
            for n in (16, 1000, 4096, 8000, 11008, 20000, 100000):
                if mp.linear_cols(rows, n, 128 * steps):
                    most = max(most, rows * steps * 68)
    assert 30000 < most < 32500

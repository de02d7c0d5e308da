"""How products of the tests are cut (csrc/mx.hip, mx_plan and
mx_linear_cols), and operands whose products are exact in fp32.

PRODUCTS: (M, N, k) -> (rows, columns of a workgroup, k splits): 64 rows is
the small form (k_mx_few, 16 / 32 / 64 columns), 128 the tiles (k_mx_gemm).
LINEARS: (rows, n, k) -> columns of the one-launch form, 0 for two launches.
"""

import ctypes

import torch

import fac_whitening_gift_amd as fg

PRODUCTS = {
    # tiles; rows of C start on 128-byte lines in both types, in fp32 only, in neither
    (1999, 4096, 1100): (128, 128, 1),
    (1999, 4064, 300): (128, 128, 1),
    (2816, 1024, 1000): (128, 128, 1),
    (1000, 2816, 1024): (128, 128, 1),
    (1999, 4090, 1100): (128, 128, 1),
    (1999, 4096, 4100): (128, 256, 1),
    (4100, 4032, 4200): (128, 256, 1),
    (4100, 4064, 4100): (128, 256, 1),
    (4100, 4030, 4100): (128, 256, 1),
    # split sums: the partials' rows start on 128-byte lines, or not
    (570, 1920, 13104): (128, 128, 2),
    (1000, 1088, 16000): (128, 128, 4),
    (1067, 160, 14185): (128, 128, 8),
    (1067, 42, 14185): (128, 128, 8),
    (349, 33, 26797): (128, 128, 15),
    (300, 320, 40000): (128, 128, 16),
    # small: 16, 32 and more rows, by 16, 32 and 64 columns
    (7, 100, 500): (64, 16, 1),
    (1, 6500, 5946): (64, 32, 1),
    (2, 11062, 1899): (64, 64, 1),
    (24, 4090, 11000): (64, 16, 1),
    (20, 6870, 2193): (64, 32, 1),
    (20, 15400, 551): (64, 64, 1),
    (100, 99, 26797): (64, 16, 1),
    (300, 1083, 16000): (64, 32, 1),
    (1000, 1024, 2816): (64, 64, 1),
    (1109, 2279, 181): (64, 64, 1),
    (300, 2100, 900): (64, 64, 1),
}

LINEARS = {
    (1, 4096, 4096): 16,
    (3, 1001, 20352): 16,
    (3, 8000, 2000): 32,
    (9, 8000, 6784): 32,
    (16, 8100, 300): 32,
    (1, 11008, 4096): 64,
    (1, 11001, 4090): 64,
    (9, 11008, 6784): 64,   # the most LDS that rows quantized in front take
    (16, 11008, 1000): 64,
    (5, 20001, 500): 64,
    (16, 4096, 11008): 0,
    (24, 4096, 11008): 0,
    (1, 40, 180000): 0,
    (2, 24, 90001): 0,
}


class _Plan(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int), ("cols", ctypes.c_int), ("n_split", ctypes.c_int),
                ("per_split", ctypes.c_int)]


def _planner(name, restype):
    fn = fg.load()[name]
    fn.restype, fn.argtypes = restype, [ctypes.c_int64] * 3
    return fn


def plan(m, n, k):
    """-> (rows, columns of a workgroup, k splits) of a product"""
    p = _planner("_ZN4gift7mx_planElll", _Plan)(m, n, k)
    return p.rows, p.cols, p.n_split


def linear_cols(rows, n, k):
    """-> columns of a workgroup of the one-launch form, 0: two launches"""
    return _planner("_ZN4gift14mx_linear_colsElll", ctypes.c_int)(rows, n, k)


def exact_values(rows, k, g, device, powers=(-3, 4)):
    """rows x k values that MXFP4 holds exactly: random E2M1 values with a 4
    or 6 in every block of 32, a power of two per block (1 or 2) and one per
    row.  Over the row's power they are multiples of 1/2 up to 12, so with two
    such matrices every product is a multiple of 1/4 and every sum exact in
    fp32, in any order, while sum |a b| < 2^22 (see exact_product)."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=device)
    blocks = -(-k // 32)
    v = grid[torch.randint(0, 8, (rows, k), generator=g, device=device)]
    at = torch.arange(blocks, device=device) * 32
    v[:, at] = 4.0 + 2.0 * torch.randint(0, 2, (rows, blocks), generator=g, device=device)
    v *= torch.randint(0, 2, (rows, k), generator=g, device=device) * 2.0 - 1.0
    v *= torch.exp2(torch.randint(0, 2, (rows, blocks), generator=g,
                                  device=device).float()).repeat_interleave(32, 1)[:, :k]
    row = torch.exp2(torch.randint(*powers, (rows, 1), generator=g, device=device).float())
    return v * row, row


def exact_product(a, row_a, b, row_b):
    """fp64 a b^T, exact, and exact in fp32 in any order of its sums"""
    most = ((a / row_a).double().abs() @ (b / row_b).double().abs().t()).max()
    assert float(most) < 2.0 ** 22
    return a.double() @ b.double().t()

"""CPU pins of the layer oracle (oracle/layer.py): the block quantizer against
the payload oracle, the operand layout byte by byte from its definition, and
the norm's gradients against central differences."""

import numpy as np
import pytest

from oracle import layer, mxfp4


def test_quantize_equals_the_payload_oracle():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((7, 96)) * np.exp2(rng.integers(-30, 30, (7, 1)))).astype(np.float32)
    x[2, 32:64] = 0.0
    x[3, 5] = np.inf
    codes, scales, flags = layer.quantize(x)
    pc, ps, pf = mxfp4.quantize(x)
    assert np.array_equal(codes, mxfp4.unpack(pc)) and np.array_equal(scales, ps) and flags == pf


def test_quantize_fills_a_short_block_with_zeros():
    x = np.arange(1, 41, dtype=np.float32).reshape(1, 40)
    codes, scales, flags = layer.quantize(x)
    full = np.zeros((1, 64), dtype=np.float32)
    full[:, :40] = x
    c2, s2, _ = layer.quantize(full)
    assert np.array_equal(codes, c2) and np.array_equal(scales, s2) and flags == 0


@pytest.mark.parametrize("rows,k", [(1, 32), (70, 160), (128, 300)])
def test_pack_follows_the_layout(rows, k):
    rng = np.random.default_rng(rows)
    codes, scales, _ = layer.quantize(rng.standard_normal((rows, k)).astype(np.float32))
    data = layer.pack(codes, scales)
    steps = -(-k // 128)
    assert data.size == -(-rows // 64) * steps * 4352
    for _ in range(200):
        i, e = int(rng.integers(rows)), int(rng.integers(k))
        base = ((i // 64) * steps + e // 128) * 4352
        r, j = i % 64, e % 128
        byte = data[base + 1024 * (r // 16) + 16 * (16 * (j // 32) + r % 16) + (j % 32) // 2]
        assert (byte >> (4 * (j % 2))) & 0xF == codes[i, e]
        assert data[base + 4096 + 4 * (16 * (j // 32) + r % 16) + r // 16] == scales[i, e // 32]


@pytest.mark.parametrize("is_layer", [True, False])
def test_norm_gradients_match_differences(is_layer):
    """d/dt of sum(dy * y) along random directions, central differences with
    step h: error h^2 f'''/6 + eps/h, both below 1e-8 at h = 1e-5 here."""
    rng = np.random.default_rng(1)
    x, dy = rng.standard_normal((5, 12)), rng.standard_normal((5, 12))
    w, b = 1 + 0.3 * rng.standard_normal(12), rng.standard_normal(12)

    def f(x, w, b):
        return (dy * layer.norm_forward(x, w, b, 1e-5, is_layer)[0]).sum()
    _, mu, r = layer.norm_forward(x, w, b, 1e-5, is_layer)
    dx, dw, db = layer.norm_backward(dy, x, w, mu, r, is_layer)
    h = 1e-5
    for _ in range(5):
        vx, vw, vb = rng.standard_normal(x.shape), rng.standard_normal(12), rng.standard_normal(12)
        num = (f(x + h * vx, w + h * vw, b + h * vb) - f(x - h * vx, w - h * vw, b - h * vb)) / (2 * h)
        assert abs(num - ((dx * vx).sum() + (dw * vw).sum() + (db * vb).sum())) < 1e-7

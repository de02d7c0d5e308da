"""MXFP4 operands of a layer's products, and layer / RMS norm (oracle; test
infrastructure only).

The block rules are those of ``mxfp4`` (OCP Microscaling Formats v1.0):
blocks of 32 along the axis a product sums over, a block cut short by the
matrix's edge quantized as if filled with zeros.  The operand layout
restates the one of include/gift.h: 64-row panels x 128-element k steps of
4352 bytes, four 1 KB fragments of 16 rows, then 256 scale bytes.  Norms are
fp64 formulas.
"""

import numpy as np

from . import mxfp4

PANEL_ROWS, STEP, PANEL_BYTES = 64, 128, 4352


def quantize(x):
    """fp32 rows x k -> (codes rows x K (0..15), scales rows x K/32 E8M0,
    flags), K = k rounded up to whole blocks."""
    x = np.asarray(x, dtype=np.float32)
    rows, k = x.shape
    nb = -(-k // 32)
    full = np.zeros((rows, nb * 32), dtype=np.float32)
    full[:, :k] = x
    blocks = full.reshape(rows, nb, 32)
    amax = (blocks.view(np.uint32) & np.uint32(0x7FFFFFFF)).max(axis=2).view(np.float32)
    scales = np.empty((rows, nb), dtype=np.uint8)
    flags = 0
    known = {}
    for i in range(rows):
        for b in range(nb):
            key = amax[i, b].tobytes()
            if key not in known:
                known[key] = mxfp4.scale_exponent(amax[i, b])
            scales[i, b], f = known[key]
            flags |= f
    e = np.where(scales == mxfp4.SCALE_NAN, 0, scales.astype(np.int64) - mxfp4.SCALE_BIAS)
    y = np.ldexp(blocks.astype(np.float64), -e[:, :, None])
    return mxfp4.encode_elements(y.astype(np.float32)).reshape(rows, nb * 32), scales, flags


def values(codes, scales, k=None):
    """fp64 values of (codes, scales), the first k columns."""
    sc = np.where(scales == mxfp4.SCALE_NAN, np.nan,
                  np.ldexp(1.0, scales.astype(np.int64) - mxfp4.SCALE_BIAS))
    v = mxfp4.decode_elements(codes) * np.repeat(sc, 32, axis=1)
    return v if k is None else v[:, :k]


def pack(codes, scales):
    """(codes, scales) -> the bytes of the device operand."""
    rows, kk = codes.shape
    panels, steps = -(-rows // PANEL_ROWS), -(-kk // STEP)
    c = np.zeros((panels * PANEL_ROWS, steps * STEP), dtype=np.uint8)
    c[:rows, :kk] = codes
    s = np.full((panels * PANEL_ROWS, steps * 4), 127, dtype=np.uint8)
    s[:rows, :kk // 32] = scales
    out = np.empty((panels, steps, PANEL_BYTES), dtype=np.uint8)
    two = c[:, 0::2] | (c[:, 1::2] << 4)
    # panel, fragment, row, step, block, byte -> panel, step, fragment, block, row, byte
    out[:, :, :4096] = two.reshape(panels, 4, 16, steps, 4, 16).transpose(0, 3, 1, 4, 2, 5).reshape(
        panels, steps, 4096)
    # panel, fragment, row, step, block -> panel, step, block, row, fragment
    out[:, :, 4096:] = s.reshape(panels, 4, 16, steps, 4).transpose(0, 3, 4, 2, 1).reshape(
        panels, steps, 256)
    return out.reshape(-1)


def norm_forward(x, weight=None, bias=None, eps=1e-5, layer=True):
    """-> (y, mean, rstd) in fp64 (mean zero for RMS)."""
    x = np.asarray(x, dtype=np.float64)
    mu = x.mean(axis=1) if layer else np.zeros(x.shape[0])
    c = x - mu[:, None]
    r = 1.0 / np.sqrt((c * c).mean(axis=1) + eps)
    y = c * r[:, None]
    if weight is not None:
        y = y * weight
    if bias is not None:
        y = y + bias
    return y, mu, r


def norm_backward(dy, x, weight, mean, rstd, layer=True):
    """-> (dx, dweight, dbias) in fp64 for the given statistics."""
    dy, x = np.asarray(dy, dtype=np.float64), np.asarray(x, dtype=np.float64)
    r = np.asarray(rstd, dtype=np.float64)[:, None]
    h = (x - (np.asarray(mean, dtype=np.float64)[:, None] if layer else 0.0)) * r
    g = dy if weight is None else dy * weight
    dx = g - h * (g * h).mean(axis=1, keepdims=True)
    if layer:
        dx = dx - g.mean(axis=1, keepdims=True)
    return dx * r, (dy * h).sum(axis=0), dy.sum(axis=0)

"""A layer's training step run as it is used: norm, refresh of the factor on
its output, the three MXFP4 products, G accumulated over micro-batches, the
norm's backward pass, and the round trip of G and of the norm's weight
gradient -- each stage checked against the oracle on what the stage before it
left."""

import argparse

import numpy as np
import pytest
import torch

import fac_whitening_gift_amd as fg
from oracle import gift as og, layer as ol
from gpu_util import DEV, factor_host, host, rel_fro, say
from test_gpu_norm import _check_backward, _check_forward

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def _values(t):
    """fp64 values of the oracle's operand of a tensor"""
    codes, scales, _ = ol.quantize(t.float().cpu().numpy())
    return ol.values(codes, scales, t.shape[1])


def _near(got, va, vb, half_step):
    """|got - va vb^T| <= 2 k 2^-23 sum |a b|, and half a step of the type"""
    c, s = va @ vb.T, np.abs(va) @ np.abs(vb).T
    tol = 2 * va.shape[1] * 2.0 ** -23 * s
    err = np.abs(got.double().cpu().numpy() - c)
    assert np.all(err <= tol + half_step * (np.abs(c) + tol))
    return tol


@pytest.mark.parametrize("tokens", [300, 1])
@pytest.mark.parametrize("kind", [fg.NORM_LAYER, fg.NORM_RMS])
def test_step_into_the_round_trip(tokens, kind):
    say("layer step tokens=%d kind=%d" % (tokens, kind))
    d_in, d_out, micro = 128, 224, 2
    is_layer = kind == fg.NORM_LAYER
    rng = np.random.default_rng(tokens + kind)

    def draw(*shape):
        return torch.from_numpy(rng.standard_normal(shape).astype(np.float32))
    W, weight = (draw(d_out, d_in) * d_in ** -0.5).to(DEV), (1 + 0.1 * draw(d_in)).to(DEV)
    bias = (0.1 * draw(d_in)).to(DEV) if is_layer else None
    wr, wc = fg.gift_mx_quantize(W, by_row=True, by_col=True)
    vw, vwt = _values(W), _values(W.t())
    G = torch.zeros(d_out, d_in, device=DEV)
    dweight, dbias = torch.zeros(d_in, device=DEV), torch.zeros(d_in, device=DEV)
    want_g, tol_g, want_w = 0.0, 0.0, 0.0
    for m in range(micro):
        H = (draw(tokens, d_in) * 2 + 0.3).to(BF16).to(DEV)
        dY = (draw(tokens, d_out) * 1e-2).to(BF16).to(DEV)
        X, mean, rstd = fg.gift_norm_forward(H, weight, bias, kind=kind)
        _check_forward(H, weight, bias, 1e-5, kind, (X, mean, rstd))
        xr, xc = fg.gift_mx_quantize(X, by_row=True, by_col=True)
        gr, gc = fg.gift_mx_quantize(dY, by_row=True, by_col=True)
        vx, vxt, vg, vgt = _values(X), _values(X.t()), _values(dY), _values(dY.t())
        Y = fg.gift_mx_matmul(xr, wr)
        _near(Y, vx, vw, 2.0 ** -8)
        dX = fg.gift_mx_matmul(gr, wc)
        _near(dX, vg, vwt, 2.0 ** -8)
        fg.gift_mx_matmul(gc, xc, out=G, accumulate=True)
        want_g = want_g + vgt @ vxt.T
        tol_g = tol_g + 2 * tokens * 2.0 ** -23 * (np.abs(vgt) @ np.abs(vxt).T)
        dH, _, _ = fg.gift_norm_backward(dX, H, weight, mean, rstd, kind=kind, dweight=dweight,
                                         dbias=dbias, accumulate=True)
        alone = fg.gift_norm_backward(dX, H, weight, mean, rstd, kind=kind)
        _check_backward(dX, H, weight, mean, rstd, kind, (dH, alone[1], alone[2]))
        want_w = want_w + alone[1]   # in the order the calls add
        # one token alone: the serving form
        y1 = fg.gift_mx_linear(X[:1], wr)
        _near(y1, vx[:1], vw, 2.0 ** -8)
    err = np.abs(host(G).astype(np.float64) - want_g)
    assert np.all(err <= tol_g + 2.0 ** -24 * micro * (np.abs(want_g) + tol_g))
    assert torch.equal(dweight, want_w)
    # the round trip takes G whitened with the factor of the X it came with
    factor = fg.Factor(d_in)
    fg.gift_refresh_factor(X, factor, seed=5)
    layers = [fg.Layer(G, factor=factor, W_out=torch.empty_like(G)), fg.Layer(dweight.view(1, -1))]
    fg.gift_whiten_quantize(layers)
    fg.gift_dequant_unwhiten(layers)
    U, alpha, beta, d_w, d_u = factor_host(factor)
    Wd = host(layers[0].W_out)
    assert rel_fro(Wd, og.whiten_with(host(G).astype(np.float64), U, alpha, d_w)) <= 1e-5
    codes, inv, _ = og.quantize_tensor(Wd)
    assert np.array_equal(host(layers[0].q), codes)
    assert rel_fro(host(layers[0].G_hat), og.unwhiten_with(og.dequantize_tensor(codes, inv), U, beta, d_u)) <= 1e-5
    codes, inv, _ = og.quantize_tensor(host(dweight).reshape(1, -1))
    assert np.array_equal(host(layers[1].q), codes)
    assert np.array_equal(host(layers[1].G_hat), og.dequantize_tensor(codes, inv).astype(np.float32))


def test_mx_payload_of_the_mx_gradient():
    """G from the MXFP4 product through the MXFP4 payload: the payload's
    reconstruction is what quantizing G along its rows gives."""
    say("layer mx payload")
    x, dy = torch.randn(200, 96, device=DEV), torch.randn(200, 64, device=DEV)
    _, xc = fg.gift_mx_quantize(x, by_col=True)
    _, gc = fg.gift_mx_quantize(dy, by_col=True)
    G = fg.gift_mx_matmul(gc, xc, dtype=torch.float32)
    L = fg.Layer(G, mxfp4=True)
    fg.gift_euclid_fp8_roundtrip([L], scaling=fg.SCALE_MXFP4)
    gr, _ = fg.gift_mx_quantize(G, by_row=True)
    assert torch.equal(fg.gift_mx_dequantize(gr), L.G_hat)


def test_layer_study_small():
    """bench.py --study layer on a small shape runs and reports finite errors
    and a time for every call."""
    import bench
    say("layer study 128,256,1024")
    res = bench.layer_study(argparse.Namespace(ref_shape="128,256,1024"))
    for key in ("norm_forward", "quantize_x", "quantize_w", "y", "quantize_dy", "dx", "g", "norm_backward"):
        assert res["ms"][key] > 0
    nums = list(res["m1"].values()) + [res["g_m2"]]
    for fmt in ("e4m3_tensor", "mxfp4"):
        for method in ("gift", "euclid"):
            nums += list(res[fmt][method].values())
    assert all(np.isfinite(v) and v > 0 for v in nums)

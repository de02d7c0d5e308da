"""A training step run as it is used: two residual blocks whose products are
MXFP4, the norms between them, the loss over a vocabulary, the way back through
all of it with gradients summed over micro-batches, clipping of every gradient
together, and the round trip of the clipped head and block gradients -- each
stage checked against the oracle on what the stage before it left."""

import numpy as np
import pytest
import torch

import fac_whitening_gift_amd as fg
from oracle import gift as og
from gpu_util import DEV, factor_host, host, rel_fro, say
from test_gpu_block_norm import _check_backward as block_backward, _check_forward as block_forward
from test_gpu_grad_clip import _check as check_clip
from test_gpu_layer import _near, _values
from test_gpu_xent import _check_backward as xent_backward, _check_forward as xent_forward

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.mark.parametrize("sequences,tokens", [(3, 50), (1, 1), (2, 97)])
@pytest.mark.parametrize("kind", [fg.NORM_RMS, fg.NORM_LAYER])
def test_step(kind, sequences, tokens):
    say("step kind=%d %d x %d" % (kind, sequences, tokens))
    d, vocab, blocks, micro = 128, 500, 2, 2
    n = sequences * tokens
    rng = np.random.default_rng(n + kind)
    layer = kind == fg.NORM_LAYER

    def draw(*shape):
        return torch.from_numpy(rng.standard_normal(shape).astype(np.float32))
    W = [(draw(d, d) * d ** -0.5).to(DEV) for _ in range(blocks)]
    ops = [fg.gift_mx_quantize(w, by_row=True, by_col=True) for w in W]
    head = (2 * draw(vocab, d) * d ** -0.5).to(BF16)
    first = (1 + 0.1 * draw(d)).to(DEV)
    vectors = [{"weight": 1 + 0.1 * draw(d), "post_weight": 1 + 0.1 * draw(d), "gate": 0.5 + 0.1 * draw(sequences, d),
                **({"bias": 0.1 * draw(d), "post_bias": 0.1 * draw(d)} if layer else {})} for _ in range(blocks)]
    on_dev = [{k: t.to(DEV) for k, t in v.items()} for v in vectors]
    how = dict(kind=kind, scale=0.9)
    G = [torch.zeros(d, d, device=DEV) for _ in range(blocks)]
    G_head = torch.zeros(vocab, d, device=DEV)
    dv = [{"d" + k: torch.zeros_like(t) for k, t in v.items()} for v in on_dev]
    d_first = torch.zeros(d, device=DEV)
    sums = [{k: torch.zeros_like(t) for k, t in v.items()} for v in dv]
    head_sum = torch.zeros_like(G_head)
    for _ in range(micro):
        h0 = draw(n, d).to(DEV)
        t = torch.from_numpy(rng.integers(0, vocab, n))
        t[n // 2:n // 2 + n // 8] = -100
        T = t.to(DEV)
        dloss = torch.full((n,), 1.0 / n, device=DEV)
        # forward: an fp32 stream beside bf16 block inputs and outputs
        x, mean, rstd = fg.gift_norm_forward(h0.to(BF16), first, kind=kind)
        h, kept = h0, []
        for b in range(blocks):
            xr, xc = fg.gift_mx_quantize(x, by_row=True, by_col=True)
            y = fg.gift_mx_matmul(xr, ops[b][0])
            _near(y, _values(x), _values(W[b]), 2.0 ** -8)
            got = fg.gift_block_norm_forward(y, h, **on_dev[b], **how)
            block_forward(y.cpu(), h.cpu(), vectors[b], how, got)
            kept.append((x, xc, y, got[1], got[2]))
            x, h = got[0], got[1]
        loss, lse = fg.gift_xent_forward(x, head.to(DEV), T)
        xent_forward(x.cpu(), head, t, (loss, lse))
        # and back
        before = G_head.clone()
        dx, _ = fg.gift_xent_backward(x, head.to(DEV), T, lse, dloss, dw=G_head, accumulate=True)
        alone = fg.gift_xent_backward(x, head.to(DEV), T, lse, dloss)
        xent_backward(x.cpu(), head, t, lse, dloss.cpu(), dx, alone[1])
        assert torch.equal(dx, alone[0]) and torch.equal(G_head, before + alone[1])
        dh = None
        for b in reversed(range(blocks)):
            x_in, xc, y, h2, stats = kept[b]
            g = fg.gift_block_norm_backward(dx, dh, y, h2, stats, **on_dev[b], **how, grads=dict(dv[b]), accumulate=True)
            one = fg.gift_block_norm_backward(dx, dh, y, h2, stats, **on_dev[b], **how)
            block_backward(dx.cpu(), None if dh is None else dh.cpu(), y.cpu(), h2, stats, vectors[b], how, one)
            for k in sums[b]:
                sums[b][k] += one[k]
                assert torch.equal(dv[b][k], sums[b][k])
            gr, gc = fg.gift_mx_quantize(g["dy"], by_row=True, by_col=True)
            dx = fg.gift_mx_matmul(gr, ops[b][1])
            _near(dx, _values(g["dy"]), _values(W[b].t()), 2.0 ** -8)
            fg.gift_mx_matmul(gc, xc, out=G[b], accumulate=True)
            dh = g["dh"]
        fg.gift_norm_backward(dx, h0.to(BF16), first, mean, rstd, kind=kind, dx=False, dweight=d_first, dbias=False,
                              accumulate=True)
    # every gradient clipped by the norm of all, in place
    grads = G + [G_head, d_first] + [t for v in dv for t in v.values()]
    was = [t.cpu().clone() for t in grads]
    total = sum(float((t.double() ** 2).sum()) for t in was) ** 0.5
    norm = fg.gift_grad_clip(fg.TensorGroup(grads), 0.25 * total)
    check_clip(was, np.float32(0.25 * total), np.float32(1e-6), norm, grads)
    assert abs(float(fg.gift_grad_norm(grads)) - 0.25 * total) <= 1e-5 * total
    # the round trip: the last block's gradient whitened with the factor of its
    # input, the head's Euclidean
    factor = fg.Factor(d)
    fg.gift_refresh_factor(kept[-1][0], factor, seed=5)
    layers = [fg.Layer(G[-1], factor=factor, W_out=torch.empty_like(G[-1])), fg.Layer(G_head)]
    fg.gift_whiten_quantize(layers)
    fg.gift_dequant_unwhiten(layers)
    U, alpha, beta, d_w, d_u = factor_host(factor)
    Wd = host(layers[0].W_out)
    assert rel_fro(Wd, og.whiten_with(host(G[-1]).astype(np.float64), U, alpha, d_w)) <= 1e-5
    codes, inv, _ = og.quantize_tensor(Wd)
    assert np.array_equal(host(layers[0].q), codes)
    assert rel_fro(host(layers[0].G_hat), og.unwhiten_with(og.dequantize_tensor(codes, inv), U, beta, d_u)) <= 1e-5
    codes, inv, _ = og.quantize_tensor(host(G_head))
    assert np.array_equal(host(layers[1].q), codes)

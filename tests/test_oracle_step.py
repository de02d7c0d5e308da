"""CPU pins of the step oracle (oracle/step.py): gradients against central
differences, and rows left out."""

import numpy as np
import pytest

from oracle import step


def test_xent_gradients_match_differences():
    """Central differences with step h along random directions: error h^2 f'''/6
    + eps / h, both below 1e-8 at h = 1e-5 here."""
    rng = np.random.default_rng(0)
    x, w = rng.standard_normal((6, 9)), rng.standard_normal((11, 9))
    t = np.array([3, -100, 10, 0, 11, 5])
    g = rng.standard_normal(6)
    _, lse, _ = step.xent_forward(x, w, t)
    dx, dw = step.xent_backward(x, w, t, lse, g)
    h = 1e-5
    for _ in range(5):
        vx, vw = rng.standard_normal(x.shape), rng.standard_normal(w.shape)
        num = ((g * step.xent_forward(x + h * vx, w + h * vw, t)[0]).sum() -
               (g * step.xent_forward(x - h * vx, w - h * vw, t)[0]).sum()) / (2 * h)
        assert abs(num - (dx * vx).sum() - (dw * vw).sum()) < 1e-7


def test_rows_left_out_count_for_nothing():
    rng = np.random.default_rng(1)
    x, w = rng.standard_normal((4, 5)), rng.standard_normal((7, 5))
    t = np.array([2, -1, 7, 6])
    loss, lse, _ = step.xent_forward(x, w, t)
    assert loss[1] == 0 and loss[2] == 0 and loss[0] > 0
    dx, dw = step.xent_backward(x, w, t, lse, np.ones(4))
    keep = [0, 3]
    dx2, dw2 = step.xent_backward(x[keep], w, t[keep], lse[keep], np.ones(2))
    assert np.array_equal(dx[keep], dx2) and np.allclose(dw, dw2, atol=1e-15) and not dx[1:3].any()
    x[1] = np.nan
    assert np.array_equal(step.xent_backward(x, w, t, lse, np.ones(4))[1], dw)


@pytest.mark.parametrize("groups", [0, 1, 3])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("is_layer", [True, False])
def test_block_norm_gradients_match_differences(is_layer, post, groups):
    """As above, along random directions of every input and vector at once."""
    rng = np.random.default_rng(2)
    rows, d = 6, 10
    v = {"y": rng.standard_normal((rows, d)), "h": rng.standard_normal((rows, d)),
         "weight": 1 + 0.3 * rng.standard_normal(d), "bias": rng.standard_normal(d)}
    if post:
        v["post_weight"], v["post_bias"] = 1 + 0.3 * rng.standard_normal(d), rng.standard_normal(d)
    if groups:
        v["gate"] = rng.standard_normal((groups, d))
    dx, dh = rng.standard_normal((rows, d)), rng.standard_normal((rows, d))
    how = dict(post=post, scale=0.7, layer=is_layer)

    def f(v):
        x, h2, _ = step.block_norm_forward(**v, **how)
        return (dx * x).sum() + (dh * h2).sum()
    _, h2, stats = step.block_norm_forward(**v, **how)
    vec = {k: v.get(k) for k in ("weight", "post_weight", "post_bias", "gate")}
    g = step.block_norm_backward(dx, dh, v["y"], h2, stats, **vec, **how)
    h = 1e-5
    for _ in range(5):
        to = {k: rng.standard_normal(a.shape) for k, a in v.items()}
        num = (f({k: a + h * to[k] for k, a in v.items()}) - f({k: a - h * to[k] for k, a in v.items()})) / (2 * h)
        assert abs(num - sum((g["d" + k] * to[k]).sum() for k in v)) < 1e-7


def test_grad_clip():
    rng = np.random.default_rng(3)
    t = [rng.standard_normal((3, 4)), np.zeros((0, 5)), rng.standard_normal(7)]
    flat = np.concatenate([v.ravel() for v in t])
    q, norm, out = step.grad_clip(t, 0.5, 0.0)
    assert np.isclose(q, flat @ flat) and np.isclose(norm, np.linalg.norm(flat))
    assert np.isclose(np.sqrt(sum((v * v).sum() for v in out)), 0.5)
    assert all(np.array_equal(a, b) for a, b in zip(step.grad_clip(t, 100.0)[2], t))
    assert not step.grad_clip([np.zeros(3)], 0.0, 0.0)[2][0].any()

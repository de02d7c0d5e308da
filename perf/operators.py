"""What the operators around the gradient round trip are measured on.

A layer's training step in MXFP4 (OCP Microscaling Formats v1.0: E2M1
elements, one E8M0 scale per 32 consecutive elements along the contraction)
and the norm in front of it:

  quantize       X -> its MXFP4 operands along the rows and along the columns
  linear         Y = Q(X) Q(W)^T + b, W quantized before (serving, one token up)
  step           Y = Q(X) Q(W)^T, dX = Q(dY) Q(W), dW = Q(dY)^T Q(X), each
                 operand quantized along the axis its product sums over
  norm_forward   layer norm / RMS norm of every row
  norm_backward  its gradients: dX, and d weight, d bias summed over the rows

`own` False computes them in elementary torch operations, True with the
calls of fac_whitening_gift_amd.  Sizes are those of the benchmark's and the
tests' layers: hidden 1024 / 1536 / 4096, MLP 2816 / 4096 / 11008, up to
16384 tokens.
"""

import math

import torch

own = False

EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # the weight of a hidden-1024 block's gate, fp32 master, once per optimizer step
        {"name": "quantize_weight_2816x1024", "op": "quantize", "rows": 2816, "cols": 1024, "dtype": "f32"},
        # the layer input of one hidden-4096 block over a training batch
        {"name": "quantize_input_16384x4096", "op": "quantize", "rows": 16384, "cols": 4096, "dtype": "bf16"},
        # generation, one sequence: one token through the gate of a 4096 / 11008 block
        {"name": "linear_1x4096_11008", "op": "linear", "rows": 1, "d_in": 4096, "d_out": 11008, "bias": False},
        # generation, a small batch of sequences; the wide contraction of the down projection
        {"name": "linear_24x11008_4096", "op": "linear", "rows": 24, "d_in": 11008, "d_out": 4096, "bias": True},
        # a prompt of ragged length through an attention projection
        {"name": "linear_1999x4096_4096", "op": "linear", "rows": 1999, "d_in": 4096, "d_out": 4096, "bias": False},
        # training step of a layer: a short ragged batch on the hidden-1024 block
        {"name": "step_1000x1024_2816", "op": "step", "rows": 1000, "d_in": 1024, "d_out": 2816},
        # the 600M stack's up projection over its 16384 tokens
        {"name": "step_16384x1536_4096", "op": "step", "rows": 16384, "d_in": 1536, "d_out": 4096},
        # the default benchmark's gate over its 16384 tokens
        {"name": "step_16384x4096_11008", "op": "step", "rows": 16384, "d_in": 4096, "d_out": 11008},
        # generation: the norm of one token
        {"name": "norm_forward_1x4096", "op": "norm_forward", "rows": 1, "d": 4096, "dtype": "bf16", "kind": "rms"},
        # the norm in front of a 4096-wide layer over a training batch
        {"name": "norm_forward_16384x4096", "op": "norm_forward", "rows": 16384, "d": 4096, "dtype": "bf16", "kind": "layer"},
        # backward over a ragged batch in fp32
        {"name": "norm_backward_1000x1536", "op": "norm_backward", "rows": 1000, "d": 1536, "dtype": "f32", "kind": "layer"},
        # backward over a training batch
        {"name": "norm_backward_16384x4096", "op": "norm_backward", "rows": 16384, "d": 4096, "dtype": "bf16", "kind": "rms"},
    ]


def _size(rng, lo, hi):
    """Log-uniform in [lo, hi]; half of them whole multiples of 32."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if n >= 64 and rng.random() < 0.5:
        n -= n % 32
    return max(lo, min(hi, n))


def draw(rng):
    op = rng.choice(["quantize", "linear", "step", "norm_forward", "norm_backward"])
    if op == "quantize":
        return {"op": op, "rows": _size(rng, 1, 16384), "cols": _size(rng, 64, 11008), "dtype": rng.choice(["bf16", "f32"])}
    if op == "linear":
        return {"op": op, "rows": _size(rng, 1, 16384), "d_in": _size(rng, 64, 11008), "d_out": _size(rng, 64, 4096),
                "bias": rng.random() < 0.5}
    if op == "step":
        return {"op": op, "rows": _size(rng, 32, 16384), "d_in": _size(rng, 64, 4096), "d_out": _size(rng, 64, 11008)}
    return {"op": op, "rows": _size(rng, 1, 16384), "d": _size(rng, 64, 11008), "dtype": rng.choice(["bf16", "f32"]),
            "kind": rng.choice(["layer", "rms"])}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _activations(rows, d, g, dtype=torch.bfloat16):
    """Tokens whose features have a power-law spectrum, a few of them outliers."""
    s = torch.arange(1, d + 1, device="cuda", dtype=torch.float32).pow(-0.25)
    s = s[torch.randperm(d, generator=g, device="cuda")]
    s[torch.randint(0, d, (max(1, d // 256),), generator=g, device="cuda")] *= 12.0
    x = torch.randn(rows, d, generator=g, device="cuda") * s
    return (x + 0.1).to(dtype)


def _gradients(rows, d, g, dtype=torch.bfloat16):
    """Output gradients: Gaussian with a lognormal size per token."""
    s = torch.randn(rows, 1, generator=g, device="cuda").exp() * 1e-3
    return (torch.randn(rows, d, generator=g, device="cuda") * s).to(dtype)


def _weights(d_out, d_in, g):
    return torch.randn(d_out, d_in, generator=g, device="cuda") * (d_in ** -0.5)


def _inputs(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "quantize":
        dt = DTYPES[case["dtype"]]
        return {"x": _activations(case["rows"], case["cols"], g, dt)}
    if op in ("linear", "step"):
        n, d_in, d_out = case["rows"], case["d_in"], case["d_out"]
        s = {"x": _activations(n, d_in, g), "w": _weights(d_out, d_in, g)}
        if op == "linear":
            s["bias"] = torch.randn(d_out, generator=g, device="cuda") if case["bias"] else None
        else:
            s["dy"] = _gradients(n, d_out, g)
        return s
    n, d, dt = case["rows"], case["d"], DTYPES[case["dtype"]]
    layer = case["kind"] == "layer"
    x = _activations(n, d, g, dt)
    s = {"x": x, "weight": 1 + 0.1 * torch.randn(d, generator=g, device="cuda"),
         "bias": 0.1 * torch.randn(d, generator=g, device="cuda") if layer else None}
    if op == "norm_backward":
        # dY, and the statistics that the forward pass left
        s["dy"] = _gradients(n, d, g, dt)
        mean = x.float().mean(1) if layer else None
        c = x.float() - mean[:, None] if layer else x.float()
        s["mean"], s["rstd"] = mean, (c.square().mean(1) + EPS).rsqrt()
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["op"], s["kind"] = case["op"], case.get("kind")
    if case["op"] == "linear":
        # a serving program quantizes its weights once; the plain form keeps
        # them as the values they stand for
        if own:
            import fac_whitening_gift_amd as fg
            s["wq"], _ = fg.gift_mx_quantize(s.pop("w"), by_row=True)
        else:
            s["wq"] = _mx(s.pop("w"))
    return s


# --------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------

def _mx(x):
    """fp32 values of the MXFP4 quantization of x along its last axis: per 32
    elements (the last block shorter, as if filled with zeros) the scale
    2^(floor(log2 amax) - 2), elements to the nearest of 0, .5, 1, 1.5, 2, 3,
    4, 6 (ties to the even code, larger ones to 6)."""
    rows, k = x.shape
    pad = -k % 32
    v = x.float()
    if pad:
        v = torch.cat([v, v.new_zeros(rows, pad)], 1)
    v = v.view(rows, -1, 32)
    amax = v.abs().amax(2, keepdim=True)
    e = (torch.frexp(amax).exponent - 3).clamp(-127, 127)
    e = torch.where(amax == 0, torch.zeros_like(e), e)
    u = torch.ldexp(v, -e)
    a = u.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = ((a / step).round() * step).clamp(max=6.0)
    q = torch.ldexp(torch.copysign(q, u), e)
    return q.view(rows, -1)[:, :k]


def _run_plain(s):
    op = s["op"]
    if op == "quantize":
        x = s["x"]
        return {"by_row": _mx(x).to(torch.bfloat16), "by_col": _mx(x.t()).to(torch.bfloat16)}
    if op == "linear":
        y = _mx(s["x"]) @ s["wq"].t()
        if s["bias"] is not None:
            y = y + s["bias"]
        return {"y": y.to(torch.bfloat16)}
    if op == "step":
        x, w, dy = s["x"], s["w"], s["dy"]
        return {"y": (_mx(x) @ _mx(w).t()).to(torch.bfloat16),
                "dx": (_mx(dy) @ _mx(w.t()).t()).to(torch.bfloat16),
                "dw": _mx(dy.t()) @ _mx(x.t()).t()}
    layer = s["kind"] == "layer"
    x, w = s["x"].float(), s["weight"]
    if op == "norm_forward":
        mean = x.mean(1) if layer else None
        c = x - mean[:, None] if layer else x
        rstd = 1.0 / (c.square().mean(1) + EPS).sqrt()
        y = c * rstd[:, None] * w
        if s["bias"] is not None:
            y = y + s["bias"]
        return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}
    dy = s["dy"].float()
    c = x - s["mean"][:, None] if layer else x
    xhat = c * s["rstd"][:, None]
    g = dy * w
    dx = g - xhat * (g * xhat).mean(1, keepdim=True)
    if layer:
        dx = dx - g.mean(1, keepdim=True)
    return {"dx": (dx * s["rstd"][:, None]).to(s["x"].dtype),
            "dweight": (dy * xhat).sum(0, dtype=torch.float64).float(),
            "dbias": dy.sum(0, dtype=torch.float64).float() if layer else None}


# --------------------------------------------------------------------------
# the framework's calls
# --------------------------------------------------------------------------

def _run_own(s):
    import fac_whitening_gift_amd as fg
    op = s["op"]
    if op == "quantize":
        r, c = fg.gift_mx_quantize(s["x"], by_row=True, by_col=True)
        return {"by_row": fg.gift_mx_dequantize(r, dtype=torch.bfloat16),
                "by_col": fg.gift_mx_dequantize(c, dtype=torch.bfloat16)}
    if op == "linear":
        return {"y": fg.gift_mx_linear(s["x"], s["wq"], bias=s["bias"])}
    if op == "step":
        xr, xc = fg.gift_mx_quantize(s["x"], by_row=True, by_col=True)
        wr, wc = fg.gift_mx_quantize(s["w"], by_row=True, by_col=True)
        y = fg.gift_mx_matmul(xr, wr, dtype=torch.bfloat16)
        gr, gc = fg.gift_mx_quantize(s["dy"], by_row=True, by_col=True)
        dx = fg.gift_mx_matmul(gr, wc, dtype=torch.bfloat16)
        dw = fg.gift_mx_matmul(gc, xc, dtype=torch.float32)
        return {"y": y, "dx": dx, "dw": dw}
    kind = fg.NORM_LAYER if s["kind"] == "layer" else fg.NORM_RMS
    if op == "norm_forward":
        y, mean, rstd = fg.gift_norm_forward(s["x"], s["weight"], s["bias"], eps=EPS, kind=kind)
        return {"y": y, "mean": mean, "rstd": rstd}
    dx, dw, db = fg.gift_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], kind=kind)
    return {"dx": dx, "dweight": dw, "dbias": db}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (2 if case["dtype"] == "bf16" else 4) + 2 * 2 * n, "flops": 0}
    if op in ("linear", "step"):
        n, k, m = case["rows"], case["d_in"], case["d_out"]
        if op == "linear":
            # W as 4-bit codes with a scale byte per 32
            b = 2 * n * k + m * k * 17 / 32 + 2 * n * m + (4 * m if case["bias"] else 0)
            return {"bytes": b, "flops": 2 * n * k * m}
        b = 2 * n * k + 4 * m * k + 2 * n * m + 2 * n * m + 2 * n * k + 4 * m * k
        return {"bytes": b, "flops": 6 * n * k * m}
    n, d, size = case["rows"], case["d"], 2 if case["dtype"] == "bf16" else 4
    layer = case["kind"] == "layer"
    stats = 4 * n * (2 if layer else 1)
    if op == "norm_forward":
        return {"bytes": 2 * n * d * size + 4 * d * (2 if layer else 1) + stats, "flops": 8 * n * d}
    return {"bytes": 3 * n * d * size + 4 * d * (3 if layer else 2) + stats, "flops": 14 * n * d}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _blocks64(x):
    """MXFP4 values of x along its last axis, by the list of representable
    magnitudes: an element passes from code i to i + 1 above their midpoint,
    and at it where i + 1 is even."""
    rows, k = x.shape
    out = torch.zeros(rows, (k + 31) // 32 * 32, dtype=torch.float64, device=x.device)
    out[:, :k] = x
    b = out.view(rows, -1, 32)
    top = b.abs().max(2, keepdim=True).values
    # the power of two at or below the block's largest magnitude, through the
    # exponent field of the 64-bit number (an fp32 input is never subnormal there)
    field = (top.view(torch.int64) >> 52) & 0x7FF
    e = torch.where(top > 0, field - 1023 - 2, torch.zeros_like(field)).clamp(-127, 127)
    scale = torch.exp2(e.double())
    mag = b.abs() / scale
    code = torch.zeros_like(mag)
    for i in range(7):
        mid = (_GRID[i] + _GRID[i + 1]) / 2
        code += (mag >= mid) if i % 2 else (mag > mid)
    val = torch.tensor(_GRID, dtype=torch.float64, device=x.device)[code.long()]
    return (val * b.sign() * scale).view(rows, -1)[:, :k]


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "quantize":
        return {"by_row": _blocks64(s["x"]), "by_col": _blocks64(s["x"].t())}
    if op == "linear":
        y = torch.matmul(_blocks64(s["x"]), _blocks64(s["w"]).t())
        return {"y": y if s["bias"] is None else y + s["bias"].double()}
    if op == "step":
        return {"y": torch.matmul(_blocks64(s["x"]), _blocks64(s["w"]).t()),
                "dx": torch.matmul(_blocks64(s["dy"]), _blocks64(s["w"].t()).t()),
                "dw": torch.matmul(_blocks64(s["dy"].t()), _blocks64(s["x"].t()).t())}
    x = s["x"].double()
    w = s["weight"].double()
    layer = case["kind"] == "layer"
    if op == "norm_forward":
        mu = x.sum(1) / x.shape[1] if layer else torch.zeros(x.shape[0], dtype=torch.float64, device=x.device)
        var = ((x - mu.unsqueeze(1)) ** 2).sum(1) / x.shape[1]
        r = (var + EPS) ** -0.5
        y = (x - mu.unsqueeze(1)) * r.unsqueeze(1) * w
        return {"y": y + s["bias"].double() if layer else y, "mean": mu if layer else None, "rstd": r}
    # d/dx of sum(dy * y) with y = w (x - mu) r, for the statistics given
    dy, r = s["dy"].double(), s["rstd"].double().unsqueeze(1)
    h = (x - s["mean"].double().unsqueeze(1)) * r if layer else x * r
    n = x.shape[1]
    along = (dy * w * h).sum(1, keepdim=True) / n
    level = (dy * w).sum(1, keepdim=True) / n if layer else 0.0
    return {"dx": r * (dy * w - level - h * along), "dweight": (dy * h).sum(0),
            "dbias": dy.sum(0) if layer else None}

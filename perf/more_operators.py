"""What the operators of a training step around the layers are measured on.

  score           logits S = X W^T of a vocabulary, never stored: per row
                  lse = log sum exp S and loss = lse - S[target]
  loss            the same and its gradients: dS = dloss (exp(S - lse) -
                  [target]), dX = dS W, dW = dS^T X
  block_forward   the norm after a block, its gate and the residual scale, and
                  the norm in front of the next block in one pass:
                  h' = scale h + gate norm(y), x = norm(h')
  block_backward  its gradients for dx and dh'
  clip            the norm of all gradients of a model together, and the
                  gradients scaled to at most max_norm

`own` False computes them in elementary torch operations, True with the
calls of fac_whitening_gift_amd.  Sizes are those of the benchmark's stacks
(hidden 1024 / 1536 / 4096, MLP 2816 / 4096, vocabulary 32000, up to 16384
tokens) and ragged ones beside them.
"""

import math

import torch

own = False

EPS = 1e-5
CLIP_EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # generation: the log-probability of one sequence's next token
        {"name": "score_1x4096_32000", "op": "score", "rows": 1, "d": 4096, "vocab": 32000},
        # scoring a few ragged continuations against a vocabulary of odd size
        {"name": "score_777x1536_50257", "op": "score", "rows": 777, "d": 1536, "vocab": 50257},
        # training, a short ragged batch on the hidden-1024 stack, the head's gradient in fp32 for the round trip
        {"name": "loss_1000x1024_32000", "op": "loss", "rows": 1000, "d": 1024, "vocab": 32000, "dw": "f32", "weights": False},
        # an odd hidden size and vocabulary, a weight per token, the head's gradient in the weights' type
        {"name": "loss_2047x1000_50257", "op": "loss", "rows": 2047, "d": 1000, "vocab": 50257, "dw": "bf16", "weights": True},
        # training, the head of the hidden-4096 stack over its 16384 tokens
        {"name": "loss_16384x4096_32000", "op": "loss", "rows": 16384, "d": 4096, "vocab": 32000, "dw": "f32", "weights": False},
        # generation: the norms between two blocks for one token
        {"name": "block_forward_1x4096", "op": "block_forward", "groups": 1, "per": 1, "d": 4096, "dtype": "bf16", "kind": "rms",
         "post": True, "gate": True, "scale": 1.0},
        # training batch of the hidden-4096 stack, a gate per channel
        {"name": "block_forward_16384x4096", "op": "block_forward", "groups": 1, "per": 16384, "d": 4096, "dtype": "bf16", "kind": "rms",
         "post": True, "gate": True, "scale": 1.0},
        # a short ragged batch in fp32, layer norms, a gate per sequence
        {"name": "block_backward_1000x1536", "op": "block_backward", "groups": 4, "per": 250, "d": 1536, "dtype": "f32", "kind": "layer",
         "post": True, "gate": True, "scale": 0.7},
        # backward over a training batch of the hidden-4096 stack
        {"name": "block_backward_16384x4096", "op": "block_backward", "groups": 1, "per": 16384, "d": 4096, "dtype": "bf16", "kind": "rms",
         "post": True, "gate": True, "scale": 1.0},
        # the gradients of one hidden-1024 block
        {"name": "clip_block_1024", "op": "clip", "blocks": 1, "hidden": 1024, "mlp": 2816, "vocab": 0, "dtype": "f32", "over": 3.0},
        # bf16 gradients of four blocks of odd width, their tensors one behind the other at any element
        {"name": "clip_4_blocks_1333", "op": "clip", "blocks": 4, "hidden": 1333, "mlp": 4001, "vocab": 0, "dtype": "bf16", "over": 20.0},
        # the 600M stack with its embedding and head, fp32
        {"name": "clip_24_blocks_1536_32000", "op": "clip", "blocks": 24, "hidden": 1536, "mlp": 4096, "vocab": 32000, "dtype": "f32",
         "over": 3.0},
    ]


def _size(rng, lo, hi):
    """Log-uniform in [lo, hi]; half of them whole multiples of 32."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if n >= 64 and rng.random() < 0.5:
        n -= n % 32
    return max(lo, min(hi, n))


def draw(rng):
    op = rng.choice(["score", "loss", "block_forward", "block_backward", "clip"])
    if op in ("score", "loss"):
        d, vocab = _size(rng, 64, 4096), _size(rng, 1000, 131072)
        most = min(16384, (1 << 29) // vocab, 16384 * 4096 * 32000 // (d * vocab))
        case = {"op": op, "rows": _size(rng, 1, most), "d": d, "vocab": vocab}
        if op == "loss":
            case["dw"], case["weights"] = rng.choice(["f32", "bf16"]), rng.random() < 0.5
        return case
    if op == "clip":
        hidden = _size(rng, 64, 1536)
        return {"op": op, "blocks": rng.randint(1, 24), "hidden": hidden, "mlp": _size(rng, hidden, 4096),
                "vocab": rng.choice([0, _size(rng, 1000, 32000)]), "dtype": rng.choice(["bf16", "f32"]),
                "over": rng.choice([0.5, 3.0, 20.0])}
    groups = rng.choice([1, 1, _size(rng, 2, 64)])
    return {"op": op, "groups": groups, "per": _size(rng, 1, 16384 // groups), "d": _size(rng, 64, 4096),
            "dtype": rng.choice(["bf16", "f32", "mixed"]), "kind": rng.choice(["layer", "rms"]), "post": rng.random() < 0.75,
            "gate": rng.random() < 0.75, "scale": rng.choice([1.0, 0.7, 2.5])}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _head(case, g):
    """Normed tokens, a head whose logits spread by about 2, and targets that
    the model finds anywhere from unlikely to certain; of more than one token
    about a tenth are left out, as padding is."""
    n, d, v = case["rows"], case["d"], case["vocab"]
    w = (torch.randn(v, d, generator=g, device="cuda") * (2.0 * d ** -0.5)).to(torch.bfloat16)
    t = torch.randint(0, v, (n,), generator=g, device="cuda")
    toward = w[t].float()
    boost = torch.rand(n, 1, generator=g, device="cuda") * 15.0 / toward.square().sum(1, keepdim=True)
    x = (torch.randn(n, d, generator=g, device="cuda") + boost * toward).to(torch.bfloat16)
    if n > 1:
        t = torch.where(torch.rand(n, generator=g, device="cuda") < 0.1, torch.full_like(t, -100), t)
    return x, w, t


def _shapes(case):
    """Tensors of the model: per block q, k, v, o, gate, up, down and two norms."""
    h, m, v = case["hidden"], case["mlp"], case["vocab"]
    block = [(h, h)] * 4 + [(m, h)] * 2 + [(h, m)] + [(h,)] * 2
    return block * case["blocks"] + [(h,)] + ([(v, h)] * 2 if v else [])


def _views(flat, shapes):
    """The tensors one behind the other in a flat buffer."""
    parts = flat.split([math.prod(s) for s in shapes])
    return [p.view(s) for p, s in zip(parts, shapes)]


def _norm_stats(x, layer):
    mean = x.mean(1) if layer else x.new_zeros(x.shape[0])
    c = x - mean[:, None]
    return mean, 1.0 / (c.square().mean(1) + EPS).sqrt()


def _inputs(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op in ("score", "loss"):
        x, w, t = _head(case, g)
        s = {"x": x, "w": w, "targets": t}
        if op == "loss":
            live = (t >= 0).float()
            weight = live * (torch.rand(case["rows"], generator=g, device="cuda") + 0.5 if case["weights"] else 1.0)
            s["dloss"] = weight / weight.sum().clamp(min=1e-3)
            s["dw_type"] = DTYPES[case["dw"]]
        return s
    if op == "clip":
        shapes = _shapes(case)
        n = sum(math.prod(sh) for sh in shapes)
        flat = (torch.randn(n, generator=g, device="cuda") * 1e-3).to(DTYPES[case["dtype"]])
        return {"flat": flat, "shapes": shapes, "max_norm": 1e-3 * math.sqrt(n) / case["over"]}
    n, d = case["groups"] * case["per"], case["d"]
    layer = case["kind"] == "layer"
    yt = DTYPES["f32" if case["dtype"] == "f32" else "bf16"]
    ht = DTYPES["bf16" if case["dtype"] == "bf16" else "f32"]

    def vec(mean, spread):
        return mean + spread * torch.randn(d, generator=g, device="cuda")

    y = (torch.randn(n, d, generator=g, device="cuda") * 0.5 + 0.05).to(yt)
    h = (torch.randn(n, d, generator=g, device="cuda") * vec(1.0, 0.5)).to(ht)
    s = {"y": y, "h": h, "weight": vec(1.0, 0.1), "bias": vec(0.0, 0.1) if layer else None,
         "post": case["post"], "scale": case["scale"],
         "post_weight": vec(1.0, 0.1) if case["post"] else None,
         "post_bias": vec(0.0, 0.1) if case["post"] and layer else None, "gate": None}
    if case["gate"]:
        s["gate"] = 0.3 + 0.2 * torch.randn(case["groups"], d, generator=g, device="cuda")
    if op == "block_backward":
        # what the forward pass left, and the gradients that come back
        x, h2, stats = _block_forward(s, layer)
        s["h"], s["stats"] = h2, stats
        s["dx"] = (torch.randn(n, d, generator=g, device="cuda") * 1e-3).to(yt)
        s["dh"] = (torch.randn(n, d, generator=g, device="cuda") * 1e-3).to(ht)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["op"], s["kind"] = case["op"], case.get("kind")
    if case["op"] == "clip":
        # a program's gradients stay where they are from step to step
        s["grads"] = _views(s["flat"], s["shapes"])
        if own:
            import fac_whitening_gift_amd as fg
            s["clipped"] = torch.empty_like(s["flat"])
            s["group"], s["into"] = fg.TensorGroup(s["grads"]), fg.TensorGroup(_views(s["clipped"], s["shapes"]))
    return s


# --------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------

def _score(x, w, t):
    """-> logits, lse, rows that count, loss"""
    s = x.float() @ w.float().t()
    m = s.amax(1, keepdim=True)
    lse = (m + (s - m).exp().sum(1, keepdim=True).log())[:, 0]
    live = (t >= 0) & (t < w.shape[0])
    at = torch.where(live, t, torch.zeros_like(t))
    picked = s.gather(1, at[:, None])[:, 0]
    return s, lse, live, at, torch.where(live, lse - picked, torch.zeros_like(lse))


def _gate_rows(s, v):
    """The gate of every row of v, and v's rows by gate."""
    gate = s["gate"]
    return gate.repeat_interleave(v.shape[0] // gate.shape[0], 0) if gate is not None else 1.0


def _block_forward(s, layer):
    y, h = s["y"].float(), s["h"].float()
    rows = y.shape[0]
    pm, pr = y.new_zeros(rows), y.new_ones(rows)
    n = y
    if s["post"]:
        pm, pr = _norm_stats(y, layer)
        n = (y - pm[:, None]) * pr[:, None] * s["post_weight"]
        if s["post_bias"] is not None:
            n = n + s["post_bias"]
    h2 = s["scale"] * h + _gate_rows(s, n) * n
    m, r = _norm_stats(h2, layer)
    x = (h2 - m[:, None]) * r[:, None] * s["weight"]
    if s["bias"] is not None:
        x = x + s["bias"]
    return x.to(s["y"].dtype), h2.to(s["h"].dtype), torch.stack([pm, pr, m, r])


def _norm_grad(g, xhat, r, layer):
    d = g - xhat * (g * xhat).mean(1, keepdim=True)
    if layer:
        d = d - g.mean(1, keepdim=True)
    return d * r


def _block_backward(s, layer):
    pm, pr, m, r = s["stats"].unbind(0)
    dx = s["dx"].float()
    xhat = (s["h"].float() - m[:, None]) * r[:, None]
    t = s["dh"].float() + _norm_grad(dx * s["weight"], xhat, r[:, None], layer)
    y = s["y"].float()
    yhat = (y - pm[:, None]) * pr[:, None]
    dn = _gate_rows(s, t) * t
    n = yhat
    dy = dn
    post_w = post_b = gate = None
    if s["post"]:
        n = yhat * s["post_weight"]
        if s["post_bias"] is not None:
            n = n + s["post_bias"]
            post_b = dn.sum(0, dtype=torch.float64).float()
        post_w = (dn * yhat).sum(0, dtype=torch.float64).float()
        dy = _norm_grad(dn * s["post_weight"], yhat, pr[:, None], layer)
    if s["gate"] is not None:
        groups = s["gate"].shape[0]
        gate = (t * n).view(groups, -1, n.shape[1]).sum(1, dtype=torch.float64).float()
    return {"dy": dy.to(s["y"].dtype), "dh": (s["scale"] * t).to(s["h"].dtype),
            "dweight": (dx * xhat).sum(0, dtype=torch.float64).float(),
            "dbias": dx.sum(0, dtype=torch.float64).float() if s["bias"] is not None else None,
            "dpost_weight": post_w, "dpost_bias": post_b, "dgate": gate}


def _run_plain(s):
    op = s["op"]
    if op == "score":
        _, lse, _, _, loss = _score(s["x"], s["w"], s["targets"])
        return {"loss": loss, "lse": lse}
    if op == "loss":
        x, w = s["x"], s["w"]
        logits, lse, live, at, loss = _score(x, w, s["targets"])
        ds = (logits - lse[:, None]).exp()
        ds.scatter_add_(1, at[:, None], torch.full_like(lse, -1.0)[:, None])
        ds = ds * torch.where(live, s["dloss"], torch.zeros_like(lse))[:, None]
        return {"loss": loss, "lse": lse, "dx": (ds @ w.float()).to(x.dtype), "dw": (ds.t() @ x.float()).to(s["dw_type"])}
    if op == "clip":
        total = torch.stack([t.float().square().sum(dtype=torch.float64) for t in s["grads"]]).sum()
        norm = total.sqrt().float()
        c = (s["max_norm"] / (norm + CLIP_EPS)).clamp(max=1.0)
        return {"norm": norm.view(1), "clipped": torch.cat([(t.float() * c).to(t.dtype).view(-1) for t in s["grads"]])}
    layer = s["kind"] == "layer"
    if op == "block_forward":
        x, h, stats = _block_forward(s, layer)
        return {"x": x, "h": h, "stats": stats}
    return _block_backward(s, layer)


# --------------------------------------------------------------------------
# the framework's calls
# --------------------------------------------------------------------------

def _run_own(s):
    import fac_whitening_gift_amd as fg
    op = s["op"]
    if op == "score":
        loss, lse = fg.gift_xent_forward(s["x"], s["w"], s["targets"])
        return {"loss": loss, "lse": lse}
    if op == "loss":
        x, w, t = s["x"], s["w"], s["targets"]
        loss, lse = fg.gift_xent_forward(x, w, t)
        dx, dw = fg.gift_xent_backward(x, w, t, lse, s["dloss"], dtype=s["dw_type"])
        return {"loss": loss, "lse": lse, "dx": dx, "dw": dw}
    if op == "clip":
        norm = fg.gift_grad_clip(s["group"], s["max_norm"], eps=CLIP_EPS, out=s["into"])
        return {"norm": norm, "clipped": s["clipped"]}
    kind = fg.NORM_LAYER if s["kind"] == "layer" else fg.NORM_RMS
    how = dict(post=s["post"], post_weight=s["post_weight"], post_bias=s["post_bias"], gate=s["gate"], scale=s["scale"], kind=kind)
    if op == "block_forward":
        x, h, stats = fg.gift_block_norm_forward(s["y"], s["h"], s["weight"], s["bias"], eps=EPS, **how)
        return {"x": x, "h": h, "stats": stats}
    return fg.gift_block_norm_backward(s["dx"], s["dh"], s["y"], s["h"], s["stats"], s["weight"], s["bias"], **how)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("score", "loss"):
        n, d, v = case["rows"], case["d"], case["vocab"]
        b = 2 * (n + v) * d + 8 * n + 8 * n
        if op == "score":
            return {"bytes": b, "flops": 2 * n * d * v}
        return {"bytes": b + 4 * n + 2 * n * d + (4 if case["dw"] == "f32" else 2) * v * d, "flops": 6 * n * d * v}
    if op == "clip":
        n = sum(math.prod(sh) for sh in _shapes(case))
        return {"bytes": 2 * n * (2 if case["dtype"] == "bf16" else 4), "flops": 3 * n}
    n, d = case["groups"] * case["per"], case["d"]
    layer = case["kind"] == "layer"
    a, b = 4 if case["dtype"] == "f32" else 2, 2 if case["dtype"] == "bf16" else 4
    vectors = (2 if layer else 1) * (2 if case["post"] else 1) + (case["groups"] if case["gate"] else 0)
    if op == "block_forward":
        return {"bytes": n * d * (2 * a + 2 * b) + 4 * d * vectors + 16 * n, "flops": 16 * n * d}
    return {"bytes": n * d * (3 * a + 3 * b) + 8 * d * vectors + 16 * n, "flops": 36 * n * d}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def _exact_loss(case, s):
    x, w, t = s["x"].double(), s["w"].double(), s["targets"]
    logits = torch.mm(x, w.t())
    lse = torch.logsumexp(logits, 1)
    counted = torch.nonzero((t >= 0) & (t < w.shape[0]))[:, 0]
    loss = torch.zeros_like(lse)
    loss[counted] = lse[counted] - logits[counted, t[counted]]
    if case["op"] == "score":
        return {"loss": loss, "lse": lse}
    weight = torch.zeros_like(lse)
    weight[counted] = s["dloss"][counted].double()
    ds = logits.sub_(lse.unsqueeze(1)).exp_()
    ds[counted, t[counted]] -= 1.0
    ds.mul_(weight.unsqueeze(1))
    return {"loss": loss, "lse": lse, "dx": torch.mm(ds, w), "dw": torch.mm(ds.t(), x)}


def _exact_norm(v, layer):
    mu = v.sum(1) / v.shape[1] if layer else torch.zeros(v.shape[0], dtype=torch.float64, device=v.device)
    c = v - mu.unsqueeze(1)
    return mu, ((c * c).sum(1) / v.shape[1] + EPS) ** -0.5


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op in ("score", "loss"):
        return _exact_loss(case, s)
    if op == "clip":
        v = s["flat"].double()
        norm = torch.dot(v, v) ** 0.5
        return {"norm": norm.view(1), "clipped": v * torch.clamp(s["max_norm"] / (norm + CLIP_EPS), max=1.0)}
    layer = case["kind"] == "layer"
    y, h = s["y"].double(), s["h"].double()
    one = torch.ones(case["d"], dtype=torch.float64, device=y.device)
    zero = torch.zeros_like(one)
    w = s["weight"].double()
    b = s["bias"].double() if s["bias"] is not None else zero
    pw = s["post_weight"].double() if s["post_weight"] is not None else one
    pb = s["post_bias"].double() if s["post_bias"] is not None else zero
    gate = s["gate"].double() if s["gate"] is not None else one.unsqueeze(0)
    which = torch.arange(y.shape[0], device=y.device) // (y.shape[0] // gate.shape[0])
    if op == "block_forward":
        pm, pr = torch.zeros_like(y[:, 0]), torch.ones_like(y[:, 0])
        if case["post"]:
            pm, pr = _exact_norm(y, layer)
        after = torch.addcmul(pb, (y - pm.unsqueeze(1)) * pr.unsqueeze(1), pw)
        h2 = case["scale"] * h + gate[which] * after
        m, r = _exact_norm(h2, layer)
        return {"x": torch.addcmul(b, (h2 - m.unsqueeze(1)) * r.unsqueeze(1), w), "h": h2, "stats": torch.stack([pm, pr, m, r])}
    # the gradients of sum(dx x) + sum(dh' h') for the statistics given
    pm, pr, m, r = [v.double().unsqueeze(1) for v in s["stats"]]
    dx, dh, d = s["dx"].double(), s["dh"].double(), case["d"]
    u = (h - m) * r
    a = dx * w
    t = dh + r * (a - u * ((a * u).sum(1, keepdim=True) / d) - ((a.sum(1, keepdim=True) / d) if layer else 0.0))
    v = (y - pm) * pr
    e = gate[which] * t
    if case["post"]:
        f = e * pw
        dy = pr * (f - v * ((f * v).sum(1, keepdim=True) / d) - ((f.sum(1, keepdim=True) / d) if layer else 0.0))
    else:
        dy = e
    per_gate = torch.zeros_like(gate).index_add_(0, which, t * (v * pw + pb)) if case["gate"] else None
    return {"dy": dy, "dh": case["scale"] * t, "dweight": (dx * u).sum(0), "dbias": dx.sum(0) if s["bias"] is not None else None,
            "dpost_weight": (e * v).sum(0) if case["post"] else None,
            "dpost_bias": e.sum(0) if s["post_bias"] is not None else None, "dgate": per_gate}

"""Benchmark of the GIFT FP8 gradient round trip on one MI355X.

Default workload: a synthetic stack of 32 Llama-style blocks at hidden 4096,
MLP 11008 -- per block q, k, v, o (4096 x 4096), gate and up (11008 x 4096),
down (4096 x 11008) fp32 weight gradients, 224 layers and 6.48 G elements
(25.9 GB) resident in HBM -- with 16384 bf16 activation tokens per distinct
input (4 per block, 128 in all: attention in, o in, MLP in at width 4096,
down in at width 11008), power-law spectrum of exponent 1.5, rank-32 factors,
every layer whitened, per-tensor E4M3.

One step = the per-step path of GIFT over the whole stack: the grouped
whiten + quantize of every gradient and the grouped dequantize + un-whiten
(prepared once and captured in one HIP graph, one replay per step), plus the
step's share of the factor refresh (the paper refreshes every factor every 50
steps): step s refreshes the inputs i with floor(50 i / n_inputs) ==
s mod 50, so any 50 consecutive steps refresh every input exactly once and
each timed step carries 1/50 of the refresh work whatever --steps is.  The
gradients (25.9 GB) are a hundred times the 256 MB Infinity Cache, so every
step reads them from HBM.  Inputs are resident before the timed region.  One
JSON line on stdout.

    python bench.py [--gpus 1] [--steps 50] [--warmup 5]
    python bench.py --workload stack600m     # 24 blocks at 1536/4096, 16384 tokens
    python bench.py --workload stack300m     # 24 blocks at 1024/2816 + embed/head, top-8 by rho
    python bench.py --workload block1024     # one block at hidden 1024
    python bench.py --study staleness [--blocks 1 --hidden 4096 --mlp 11008]
    python bench.py --study interval [--intervals 10,25,50,100]   # refresh-interval ablation
    python bench.py --study rank [--rank-list 8,16,32,64,b32,b64]  # rank / block-A sweep
    python bench.py --study reference     # full-rank, Cholesky-form and two-sided references
    python bench.py --study reduce [--ranks 8]   # simulated data-parallel reduction
    python bench.py --study matrixfree    # refresh power steps with A Q = X^T (X Q) / N
    python bench.py --study stream        # HBM rates of the round trip's access patterns
    python bench.py --study layer [--ref-shape 1024,2816,8192]   # a layer's MXFP4 step into the round trip
"""

import argparse
import json
import math
import os
import sys
import time

METRIC = ("GB/s of fp32 gradient through whiten→FP8→unwhiten (% HBM peak); "
          "rel. error vs Euclid")
HBM_PEAK_GBS = 8000.0
MFMA_BF16_PEAK_TFLOPS = 2500.0
REFRESH_EVERY = 50
HERE = os.path.dirname(os.path.abspath(__file__))


def parse():
    p = argparse.ArgumentParser()
    p.add_argument("--gpus", type=int, default=1)
    p.add_argument("--steps", type=int, default=50)
    p.add_argument("--warmup", type=int, default=5)
    p.add_argument("--workload", default="stack4096",
                   choices=["stack4096", "stack600m", "stack300m", "block1024"])
    p.add_argument("--ring", type=int, default=None,
                   help="resident gradient sets (default: 4 for block1024, else 1)")
    p.add_argument("--no-cpu-baseline", action="store_true")
    p.add_argument("--cpu-seconds", type=float, default=15.0)
    p.add_argument("--no-quality", action="store_true")
    p.add_argument("--serial-refresh", action="store_true",
                   help="run each step's refresh share before its round trip on the same stream "
                        "(default: on a second stream into the next interval's factor set)")
    p.add_argument("--quiet", action="store_true")
    p.add_argument("--counters", action="store_true",
                   help="for runs under hardware-counter collection: axis-aligned spectra "
                        "(no device QR or eigendecomposition), no quality report")
    p.add_argument("--study", default=None,
                   choices=["staleness", "interval", "rank", "reference", "copy", "reduce",
                            "matrixfree", "stream", "layer"])
    p.add_argument("--ref-shape", default="1024,2816,8192",
                   help="hidden,mlp,tokens of the block of the reference and layer studies")
    p.add_argument("--rank-list", default="8,16,32,64,b32,b64",
                   help="factor ranks, and bN for block-diagonal N x N blocks (rank study)")
    p.add_argument("--intervals", default="10,25,50,100", help="refresh intervals (interval study)")
    p.add_argument("--ranks", type=int, default=8, help="ranks of the reduce study")
    p.add_argument("--blocks", type=int, default=1)
    p.add_argument("--hidden", type=int, default=4096)
    p.add_argument("--mlp", type=int, default=11008)
    p.add_argument("--tokens", type=int, default=16384)
    p.add_argument("--angle", type=float, default=0.02)
    p.add_argument("--study-steps", type=int, default=None,
                   help="horizon of the staleness (default 50) and interval (default max K) studies")
    return p.parse_args()


def log(args, msg):
    if not args.quiet:
        print("[bench] " + msg, file=sys.stderr, flush=True)


def kernel_source_hash():
    """Hash of the kernel sources of the loaded library; warns when the
    sources on disk differ from what the library was built from."""
    import fac_whitening_gift_amd as fg
    from fac_whitening_gift_amd.build import source_hash
    built, disk = fg.build_hash(), source_hash()
    if built != disk:
        print("[bench] warning: libgift.so was built from other sources (%s) than the ones on "
              "disk (%s); rebuild it" % (built, disk), file=sys.stderr, flush=True)
    return built


def load_traffic(kernel, src_hash, elems):
    """HBM bytes per launch from the committed rocprofv3 counter summaries
    (their "traffic:" lines), if taken on the current kernel sources and the
    same number of elements; else None."""
    pdir = os.path.join(HERE, "profiles")
    if not os.path.isdir(pdir):
        return None
    for name in sorted(os.listdir(pdir)):
        if not name.startswith("hbm_traffic"):
            continue
        with open(os.path.join(pdir, name)) as fh:
            for line in fh:
                if not line.startswith("traffic:"):
                    continue
                kv = dict(f.split("=", 1) for f in line.split()[1:])
                if (kv.get("kernel") == kernel and kv.get("source_hash") == src_hash
                        and int(kv.get("elements", -1)) == elems):
                    return int(kv["hbm_bytes_per_launch"])
    return None


# ---------------------------------------------------------------------------
# workloads
# ---------------------------------------------------------------------------

def build_workload(args):
    """-> (workload, top-k selection or None for all, ring sets)."""
    import synth
    ring = args.ring
    if args.workload == "block1024":
        w = synth.llama_block(hidden=1024, mlp=2816, tokens=8192, exponent=1.5)
        return w, None, ring or 4
    if args.workload == "stack300m":
        w = synth.llama_stack(24, 1024, 2816, 8192, exponent_range=(1.0, 2.0), vocab=32000)
        return w, 8, ring or 1
    if args.workload == "stack600m":
        return synth.llama_stack(24, 1536, 4096, 16384, exponent=1.5), None, ring or 1
    return synth.llama_stack(32, 4096, 11008, 16384, exponent=1.5), None, ring or 1


def describe(args, w, select_k, ring):
    refresh = ("the refresh staggered over the %d-step interval (step s refreshes the inputs i with "
               "floor(%d i / %d) == s mod %d)" % (REFRESH_EVERY, REFRESH_EVERY, len(w.inputs),
                                                  REFRESH_EVERY))
    if args.workload == "block1024":
        return ("%s: q,k,v,o 1024x1024, gate/up 2816x1024, down 1024x2816 fp32 gradients; 8192 "
                "bf16 tokens per input, spectrum i^-1.5; rank 32; per-tensor E4M3; %s; ring of %d "
                "gradient sets" % (w.name, refresh, ring))
    if args.workload == "stack300m":
        return ("%s: 24 Llama blocks (hidden 1024, MLP 2816) + 32000x1024 embedding and head "
                "(Euclidean); 8192 bf16 tokens per input, per-input spectrum exponent ~U[1,2]; "
                "GIFT on the top-%d layers by theta_1/tr(A), the rest Euclidean; per-tensor E4M3; "
                "%s" % (w.name, select_k, refresh))
    if args.workload == "stack600m":
        return ("%s: 24 Llama blocks (hidden 1536, MLP 4096); 16384 bf16 tokens per input, "
                "spectrum i^-1.5; all 168 layers whitened; per-tensor E4M3; %s"
                % (w.name, refresh))
    return ("%s: 32 Llama blocks (hidden 4096, MLP 11008), 224 fp32 gradients (25.9 GB resident); "
            "16384 bf16 tokens per input (128 inputs), spectrum i^-1.5; rank 32; all layers "
            "whitened; per-tensor E4M3; %s" % (w.name, refresh))


def draw_all(args, w, dev, ring_n):
    """Activations of every input (bf16) and ring_n gradient sets, drawn input
    by input so only one eigenbasis is held at a time."""
    import synth
    inputs, grads = {}, [dict() for _ in range(ring_n)]
    by_input = {}
    for i, l in enumerate(w.layers):
        by_input.setdefault(l.input, []).append(i)
    for k, spec in enumerate(w.inputs):
        inp = synth.draw_input(spec, seed=1000 + k, device=dev, as_bf16=True,
                               axis_aligned=args.counters)
        for r in range(ring_n):
            for i in by_input.get(spec.name, []):
                grads[r][i] = synth.draw_gradient(w.layers[i].d_out, inp["Q"], inp["ev"],
                                                  seed=5000 + 1000 * r + i, device=dev)
        inputs[spec.name] = {"X": inp["X"], "ev": inp["ev"]}
        del inp
    for r in range(ring_n):
        for i in by_input.get(None, []):
            l = w.layers[i]
            grads[r][i] = synth.draw_isotropic_gradient(l.d_out, l.d_in, seed=5000 + 1000 * r + i,
                                                        device=dev)
    return inputs, [[g[i] for i in range(len(w.layers))] for g in grads]


def refresh_shares(n):
    """Inputs refreshed at each step of a REFRESH_EVERY-step window."""
    shares = [[] for _ in range(REFRESH_EVERY)]
    for i in range(n):
        shares[i * REFRESH_EVERY // n].append(i)
    return shares


def refresh_macs(specs):
    """Algorithmic multiply-adds of the covariances: N d (d + 1) / 2 per input
    (one triangle of the symmetric X^T X)."""
    return sum(s.tokens * s.d_in * (s.d_in + 1) / 2 for s in specs)


def main():
    args = parse()
    if args.gpus != 1:
        print("bench.py measures one GPU: the GIFT path here has no inter-GPU part "
              "(the collective is out of scope); run with --gpus 1", file=sys.stderr)
        sys.exit(2)
    studies = {"staleness": staleness_study, "interval": interval_study, "rank": rank_study,
               "reference": reference_study, "reduce": reduce_study,
               "matrixfree": matrixfree_study, "stream": stream_study, "layer": layer_study}
    if args.study == "copy":
        print(json.dumps(copy_calibration()), flush=True)
        return
    if args.study is not None:
        print(json.dumps(studies[args.study](args)), flush=True)
        return

    import torch

    import fac_whitening_gift_amd as fg
    from fac_whitening_gift_amd.select import select_layers

    fg.load()
    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    w, select_k, ring_n = build_workload(args)
    elems = w.gradient_elements
    grad_bytes = 4 * elems
    log(args, "workload %s: %d layers, %d inputs, %.1f M gradient elements (%.2f GB fp32)" %
        (w.name, len(w.layers), len(w.inputs), elems / 1e6, grad_bytes / 1e9))

    # ---- resident inputs ---------------------------------------------------
    t0 = time.perf_counter()
    inputs, ring_grads = draw_all(args, w, dev, ring_n)
    torch.cuda.synchronize()
    log(args, "inputs drawn in %.1f s" % (time.perf_counter() - t0))
    factors = {s.name: fg.Factor(s.d_in, device=dev) for s in w.inputs}
    items = [dict(X=inputs[s.name]["X"], factor=factors[s.name], seed=k)
             for k, s in enumerate(w.inputs)]
    ws_all = torch.empty(max(fg.gift_refresh_group_workspace_bytes(items), 256),
                         dtype=torch.uint8, device=dev)
    rflags = torch.zeros(1, dtype=torch.int32, device=dev)
    fg.gift_refresh_factors(items, flags=rflags, ws=ws_all)
    torch.cuda.synchronize()
    if int(rflags.item()):
        raise RuntimeError("refresh flagged non-finite activations")
    shares = [[items[i] for i in sh] for sh in refresh_shares(len(items))]
    ws_share = torch.empty(max(max(fg.gift_refresh_group_workspace_bytes(sh) for sh in shares if sh),
                               256), dtype=torch.uint8, device=dev)
    # Overlapped refresh: a second factor set, so the shares of one 50-step
    # interval build the factors of the next while the round trip reads the
    # current ones.
    overlap = not args.serial_refresh
    if overlap:
        factors_b = {s.name: fg.Factor(s.d_in, device=dev) for s in w.inputs}
        items_b = [dict(X=it["X"], factor=factors_b[s.name], seed=it["seed"])
                   for it, s in zip(items, w.inputs)]
        fg.gift_refresh_factors(items_b, ws=ws_all)
        shares_b = [[items_b[i] for i in sh] for sh in refresh_shares(len(items_b))]

    layer_factor = [factors[l.input] if l.input is not None else None for l in w.layers]
    selected = ([i for i, f in enumerate(layer_factor) if f is not None] if select_k is None
                else select_layers(layer_factor, select_k))
    sel = set(selected)
    log(args, "whitened layers: %d of %d" % (len(selected), len(w.layers)))
    ring = []
    for grads in ring_grads:
        gl = [fg.Layer(G, factor=layer_factor[i]) for i, G in enumerate(grads) if i in sel]
        el = [fg.Layer(G) for i, G in enumerate(grads) if i not in sel]
        ring.append((gl, el))
    gl0, el0 = ring[0]
    if overlap:  # the same gradients and payload buffers, whitened with the second set
        ring_b = [([fg.Layer(L.G, factor=factors_b[w.layers[i].input], q=L.q, G_hat=L.G_hat)
                    for L, i in zip(gl, sorted(sel))], el) for gl, el in ring]

    def ws_for(op, layers, scaling=fg.SCALE_TENSOR):
        nb = fg.gift_group_workspace_bytes(op, layers, scaling) if layers else 0
        return torch.empty(max(nb, 256), dtype=torch.uint8, device=dev)

    ws_w, ws_d, ws_e = ws_for(0, gl0), ws_for(1, gl0), ws_for(2, el0)
    flags = torch.zeros(1, dtype=torch.int32, device=dev)
    ev = lambda: torch.cuda.Event(enable_timing=True)  # noqa: E731

    def capture(calls):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for c in calls:
                c()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for c in calls:
                c()
        return graph, calls         # the calls own the workspaces the graph writes

    # Per ring slot the per-step round trip -- grouped whiten + quantize,
    # grouped dequantize + un-whiten, Euclidean round trip of the other layers
    # -- as prepared calls captured in one HIP graph, and each entry point in a
    # graph of its own for the per-call timings below.
    def entry_calls(gl, el):
        calls = []
        if gl:
            calls.append(("whiten_quantize",
                          fg.GroupCall(fg.OP_WHITEN_QUANTIZE, gl, flags=flags, ws=ws_w)))
            calls.append(("dequant_unwhiten", fg.GroupCall(fg.OP_DEQUANT_UNWHITEN, gl, ws=ws_d)))
        if el:
            calls.append(("euclid_rest",
                          fg.GroupCall(fg.OP_EUCLID_ROUNDTRIP, el, flags=flags, ws=ws_e)))
        return calls

    slot_graphs, entry_graphs = [], {}
    for gl, el in ring:
        calls = entry_calls(gl, el)
        slot_graphs.append(capture([c for _, c in calls]))
        for name, c in calls:
            entry_graphs.setdefault(name, []).append(capture([c]))
    slot_graphs_b = [capture([c for _, c in entry_calls(gl, el)]) for gl, el in ring_b] \
        if overlap else None
    torch.cuda.synchronize()
    main_stream = torch.cuda.current_stream()
    side_stream = torch.cuda.Stream() if overlap else None

    def step(s):
        k, ph = divmod(s, REFRESH_EVERY)
        if not overlap:
            if shares[ph]:
                fg.gift_refresh_factors(shares[ph], ws=ws_share)
            slot_graphs[s % len(ring)][0].replay()
            return
        # interval k whitens with set k % 2 and refreshes the other one on the
        # side stream; at an interval's first step the round trip waits for
        # the shares that built its set, and the shares wait for the round
        # trips that read the set they overwrite
        cur = k % 2
        if ph == 0 and s > 0:
            main_stream.wait_stream(side_stream)
            side_stream.wait_stream(main_stream)
        share = (shares_b if cur == 0 else shares)[ph]
        if share:
            with torch.cuda.stream(side_stream):
                fg.gift_refresh_factors(share, ws=ws_share)
        (slot_graphs_b if cur == 1 else slot_graphs)[s % len(ring)][0].replay()

    for s in range(args.warmup):
        step(s)
    torch.cuda.synchronize()
    log(args, "timing %d steps" % args.steps)
    t0 = time.perf_counter()
    for s in range(args.warmup, args.warmup + args.steps):
        step(s)
    torch.cuda.synchronize()
    elapsed = time.perf_counter() - t0
    value = grad_bytes * args.steps / elapsed / 1e9
    ms_per_step = elapsed / args.steps * 1e3
    refreshed = sum(len(shares[s % REFRESH_EVERY])
                    for s in range(args.warmup, args.warmup + args.steps))

    # ---- the pieces on their own (graph replays between events) --------------
    def timed(fn, n=10):
        a, b = ev(), ev()
        fn()
        torch.cuda.synchronize()
        a.record()
        for i in range(n):
            fn()
        b.record()
        torch.cuda.synchronize()
        return a.elapsed_time(b) / n * 1e-3

    def timed_graph(calls, n=10):
        if not calls:
            return 0.0
        held = [capture(c) for c in calls]
        torch.cuda.synchronize()
        return timed(lambda: [g.replay() for g, _ in held], n) / len(held)

    # Each entry point on its own: its graph for every ring slot replayed in
    # turn, back to back between two events on the launch stream (torch's
    # current stream, where the graphs replay), right after the timed steps.
    def entry_time(name, n=20):
        held = entry_graphs.get(name)
        if not held:
            return 0.0
        return timed(lambda: [g.replay() for g, _ in held], n) / len(held)

    t_whiten = entry_time("whiten_quantize")
    t_dq = entry_time("dequant_unwhiten")
    t_eu = entry_time("euclid_rest")
    refresh_s = timed(lambda: fg.gift_refresh_factors(items, ws=ws_all), 3)
    share_s = sorted(timed(lambda: fg.gift_refresh_factors(sh, ws=ws_share), 3)
                     for sh in shares[:5] if sh)
    gift_elems = sum(L.d_out * L.d_in for L in gl0)
    # the other payloads, reusing the codes and reconstruction buffers
    all_eu = [fg.Layer(L.G, q=L.q, G_hat=L.G_hat) for L in gl0 + el0]
    t_eu_all = timed_graph([[fg.GroupCall(fg.OP_EUCLID_ROUNDTRIP, all_eu)]])
    blk = [fg.Layer(L.G, factor=L.factor, q=L.q, G_hat=L.G_hat, block128=True) for L in gl0]
    t_b = timed_graph([[fg.GroupCall(fg.OP_WHITEN_QUANTIZE, blk, fg.SCALE_BLOCK128),
                        fg.GroupCall(fg.OP_DEQUANT_UNWHITEN, blk, fg.SCALE_BLOCK128)]]) \
        if blk else 0.0
    mxl = [fg.Layer(L.G, factor=L.factor, q=L.q.view(-1)[:L.q.numel() // 2].view(L.d_out, -1),
                    G_hat=L.G_hat, mxfp4=True) for L in gl0]
    t_mx = timed_graph([[fg.GroupCall(fg.OP_WHITEN_QUANTIZE, mxl, fg.SCALE_MXFP4),
                         fg.GroupCall(fg.OP_DEQUANT_UNWHITEN, mxl, fg.SCALE_MXFP4)]]) \
        if mxl else 0.0
    del all_eu, blk, mxl
    torch.cuda.synchronize()

    # ---- quality: relative error vs Euclidean FP8 on the whitened layers -----
    quality = None
    if gl0 and not args.counters and not args.no_quality:
        log(args, "quality")
        quality = quality_report(w, selected, gl0, inputs, items, ws_all, ws_w, ws_d, dev)

    # ---- roofline of the dominant launch -------------------------------------
    src = kernel_source_hash()
    if t_dq >= t_whiten:
        kname, t_k = "dequant_unwhiten", t_dq
    else:
        kname, t_k = "whiten_quantize", t_whiten
    alg_bytes = 5.0 * gift_elems                 # 4 B of fp32 + 1 B of code per element
    gbs = alg_bytes / t_k / 1e9 if t_k > 0 else 0.0
    roof = {"bound": "hbm", "achieved": round(gbs, 1), "peak": HBM_PEAK_GBS, "unit": "GB/s",
            "frac": round(gbs / HBM_PEAK_GBS, 4),
            "traffic": load_traffic(kname, src, gift_elems), "kernel": kname,
            "launch_ms": round(t_k * 1e3, 4), "alg_bytes_per_launch": int(alg_bytes),
            "source_hash": src}
    macs = refresh_macs(w.inputs)
    refresh = {"bound": "mfma", "ms": round(refresh_s * 1e3, 3), "inputs": len(w.inputs),
               "alg_tflop": round(2 * macs / 1e12, 3),
               "achieved_tflops": round(2 * macs / refresh_s / 1e12, 1),
               "peak_tflops": MFMA_BF16_PEAK_TFLOPS,
               "frac": round(2 * macs / refresh_s / 1e12 / MFMA_BF16_PEAK_TFLOPS, 4),
               "work": "covariance triangles N d (d + 1) / 2 multiply-adds per input over the "
                       "whole grouped refresh (covariance, subspace iteration, Rayleigh-Ritz)",
               "share_ms_min_max": [round(share_s[0] * 1e3, 3), round(share_s[-1] * 1e3, 3)]
               if share_s else None,
               "per_step_ms": round(refresh_s * 1e3 / REFRESH_EVERY, 3)}

    cpu = None
    if not args.no_cpu_baseline:
        cpu = cpu_baseline(gl0, args)

    rt = t_whiten + t_dq
    out = {
        "metric": METRIC, "value": round(value, 2), "unit": "GB/s", "n_gpus": 1,
        "steps": args.steps, "warmup": args.warmup, "ms_per_step": round(ms_per_step, 4),
        "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": "f32",
        "data": "synthetic",
        "config": {"workload": describe(args, w, select_k, ring_n), "layers": len(w.layers),
                   "whitened_layers": len(gl0), "inputs": len(w.inputs),
                   "gradient_elements": elems,
                   "refresh_charge": "%d input refreshes in the %d timed steps (%.3f of all "
                                     "inputs per step), %s" % (
                                         refreshed, args.steps, refreshed / args.steps / len(w.inputs),
                                         "on a second stream, overlapping the round trip, into the "
                                         "factor set of the next 50-step interval" if overlap else
                                         "before each step's round trip on the same stream")},
        "hbm_frac_of_value": round(value / HBM_PEAK_GBS, 4),
        "roundtrip_only_gbps": round(4 * gift_elems / rt / 1e9, 2) if rt > 0 else None,
        "roundtrip_hbm_frac": round(10 * gift_elems / rt / 1e9 / HBM_PEAK_GBS, 4) if rt > 0 else None,
        "whiten_quantize_ms": round(t_whiten * 1e3, 4), "dequant_unwhiten_ms": round(t_dq * 1e3, 4),
        "euclid_rest_ms": round(t_eu * 1e3, 4),
        "layers_per_s": round(len(w.layers) * args.steps / elapsed, 1),
        "refresh": refresh,
        "euclid_all_layers_gbps": round(grad_bytes / t_eu_all / 1e9, 2),
        "block128_roundtrip_gbps": round(4 * gift_elems / t_b / 1e9, 2) if t_b > 0 else None,
        "mxfp4_roundtrip_gbps": round(4 * gift_elems / t_mx / 1e9, 2) if t_mx > 0 else None,
        "quality": quality,
        "roofline": roof,
        "cpu_baseline": cpu,
    }
    print(json.dumps(out), flush=True)


# ---------------------------------------------------------------------------
# quality
# ---------------------------------------------------------------------------

def kfac_metric(X, eps=1e-3):
    """S = (A + lambda_floor I)^-1/2 of A = X^T X / N from the exact fp64
    eigendecomposition (measurement harness, on the device)."""
    import torch
    X = X.double()
    A = X.T @ X / X.shape[0]
    lam = eps * torch.trace(A) / A.shape[0]
    ev_, V = torch.linalg.eigh(A)
    return (V * (ev_.clamp_min(0) + lam).rsqrt()) @ V.T


def m2_parts(G, G_hat, S):
    """(||(G^ - G) S||_F^2, ||G S||_F^2) in fp64: the terms of the K-FAC metric
    error M2 of one layer."""
    G = G.double()
    return (float(((G_hat.double() - G) @ S).pow(2).sum()), float((G @ S).pow(2).sum()))


def quality_report(w, selected, gl, inputs, items, ws_all, ws_w, ws_d, dev):
    """Relative reconstruction error of GIFT and of Euclidean quantization of
    the same gradients, for both damping readings (floor+tail, the default
    factors; floor, factors refreshed again with GIFT_DAMP_FLOOR) and for the
    per-tensor E4M3 and MXFP4 payloads.  M1 (plain relative Frobenius) over
    every whitened layer from the device error sums; M2 (error in the K-FAC
    metric of the exact damped sample covariance, fp64 torch on the device as
    measurement harness) over the layers of the first block (the first 7
    whitened layers), whose inputs' exact eigendecompositions it needs."""
    import numpy as np
    import torch

    import fac_whitening_gift_amd as fg

    m2_layers = list(range(min(7, len(gl))))
    S = {}
    for j in m2_layers:
        name = w.layers[selected[j]].input
        if name not in S:
            S[name] = kfac_metric(inputs[name]["X"])
    den2 = sum(m2_parts(gl[j].G, gl[j].G, S[w.layers[selected[j]].input])[1] for j in m2_layers)

    def measure(layers, run, scaling=fg.SCALE_TENSOR):
        run(layers, scaling)
        err = fg.gift_roundtrip_error(layers).cpu().numpy()
        m1 = float(np.sqrt(err[:, 0].sum() / err[:, 1].sum()))
        num = sum(m2_parts(layers[j].G, layers[j].G_hat, S[w.layers[selected[j]].input])[0]
                  for j in m2_layers)
        return m1, float(np.sqrt(num / den2))

    def gift(layers, sc):
        fg.gift_whiten_quantize(layers, scaling=sc, ws=ws_w if sc == fg.SCALE_TENSOR else None)
        fg.gift_dequant_unwhiten(layers, scaling=sc, ws=ws_d if sc == fg.SCALE_TENSOR else None)

    def euclid(layers, sc):
        fg.gift_euclid_fp8_roundtrip(layers, scaling=sc)

    res = {}
    eu = [fg.Layer(L.G, q=L.q, G_hat=L.G_hat) for L in gl]
    res["euclid"] = measure(eu, euclid)
    res["gift_floor+tail"] = measure(gl, gift)
    mx_q = lambda L: L.q.view(-1)[:L.q.numel() // 2].view(L.d_out, -1)  # noqa: E731
    gm = [fg.Layer(L.G, factor=L.factor, q=mx_q(L), G_hat=L.G_hat, mxfp4=True) for L in gl]
    res["gift_mxfp4"] = measure(gm, gift, fg.SCALE_MXFP4)
    em = [fg.Layer(L.G, q=mx_q(L), G_hat=L.G_hat, mxfp4=True) for L in gl]
    res["euclid_mxfp4"] = measure(em, euclid, fg.SCALE_MXFP4)
    del gm, em
    # the literal damping reading: every input refreshed again with the floor only
    floor = {}
    for it in items:
        f = it["factor"]
        floor[f.U.data_ptr()] = fg.Factor(f.d_in, device=dev)
    fitems = [dict(X=it["X"], factor=floor[it["factor"].U.data_ptr()], seed=it["seed"])
              for it in items]
    fg.gift_refresh_factors(fitems, damping_mode=fg.DAMP_FLOOR, ws=ws_all)
    gf = [fg.Layer(L.G, factor=floor[L.factor.U.data_ptr()], q=L.q, G_hat=L.G_hat) for L in gl]
    res["gift_floor"] = measure(gf, gift)
    del gf, floor, fitems
    torch.cuda.synchronize()

    def row(g, e):
        return {"m1_gift": round(res[g][0], 5), "m1_euclid": round(res[e][0], 5),
                "m1_ratio": round(res[g][0] / res[e][0], 4),
                "m2_gift": round(res[g][1], 5), "m2_euclid": round(res[e][1], 5),
                "m2_ratio": round(res[g][1] / res[e][1], 4),
                "m2_reduction": round(1 - res[g][1] / res[e][1], 4)}

    return {"e4m3_floor+tail": row("gift_floor+tail", "euclid"),
            "e4m3_floor": row("gift_floor", "euclid"),
            "mxfp4_floor+tail": row("gift_mxfp4", "euclid_mxfp4"),
            "m1_layers": len(gl), "m2_layers": [w.layers[selected[j]].name for j in m2_layers],
            "m2_metric": "(A + 1e-3 tr(A)/d_in I)^-1/2 of the sample A, exact fp64 eigh"}


def cpu_baseline(layers, args):
    """The oracle (fp64 numpy, as it stands) on the host: the same round trip
    (whiten, E4M3, dequantize, un-whiten) on the workload's first gradients,
    layer after layer, until about cpu_seconds of work; GB/s of fp32 gradient."""
    from threadpoolctl import threadpool_info

    from oracle import gift as og

    log(args, "cpu baseline (oracle)")
    done_bytes, t0 = 0, time.perf_counter()
    n_layers = 0
    shapes = []
    facs = {}
    for L in layers:
        key = L.factor.U.data_ptr()
        if key not in facs:
            c = L.factor.coef.cpu().numpy().astype("float64")
            facs[key] = og.factor_from_parts(L.factor.U.cpu().numpy(), L.factor.theta.cpu().numpy(),
                                             c[2], c[3], c[4], c[5])
        G = L.G.cpu().numpy()
        og.gift_roundtrip(G, facs[key])
        done_bytes += G.nbytes
        n_layers += 1
        shapes.append("%dx%d" % G.shape)
        del G
        if time.perf_counter() - t0 >= args.cpu_seconds:
            break
    el = time.perf_counter() - t0
    threads = max([t.get("num_threads", 1) for t in threadpool_info()] or [1])
    return {"value": round(done_bytes / el / 1e9, 4), "unit": "GB/s", "cores": int(threads),
            "kind": "oracle",
            "sample": "the first %d gradients of the workload (%s; %.2f GB fp32) through the "
                      "oracle's fp64 round trip, %.1f s (including the host copies), BLAS threads "
                      "%d, host CPUs %d" % (n_layers, ", ".join(shapes), done_bytes / 1e9, el,
                                            threads, len(os.sched_getaffinity(0)))}


# ---------------------------------------------------------------------------
# copy calibration
# ---------------------------------------------------------------------------

def copy_calibration(mib=1024, reps=5, device="cuda:0"):
    """A plain device-to-device copy of a known size (torch's copy kernel),
    for scaling the FETCH_SIZE / WRITE_SIZE counters of a profiler run: the
    counters' reading for this kernel divided by the bytes it must move."""
    import torch

    n = mib * 2 ** 20 // 4
    a = torch.randn(n, device=device)
    b = torch.empty_like(a)
    b.copy_(a)
    torch.cuda.synchronize()
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    e0.record()
    for _ in range(reps):
        b.copy_(a)
    e1.record()
    torch.cuda.synchronize()
    t = e0.elapsed_time(e1) / reps * 1e-3
    return {"study": "copy", "bytes_read": 4 * n, "bytes_written": 4 * n, "launches": reps + 1,
            "us_per_copy": round(t * 1e6, 2), "GBps": round(8 * n / t / 1e9, 1)}


def stream_study(args, mib=1024, reps=20, device="cuda:0"):
    """HBM rates of the access patterns the round-trip kernels use, from the
    probe kernels of libgift_probe.so (include/gift_probe.h) on one 1 GiB
    buffer (a 65536 x 4096 fp32 matrix for the tile and slab patterns):
    float4 read, write and copy streams with plain and nontemporal accesses,
    the 64 x 256 tiles read in one load round and written in the un-whiten
    pass's store pattern, and the 64-row slabs walked 32 columns at a time.  GB/s counts the bytes each kernel must move."""
    import ctypes

    import torch

    from fac_whitening_gift_amd import build as fb

    if not os.path.exists(fb.PROBE_LIB):
        raise RuntimeError("libgift_probe.so is not built: python -m fac_whitening_gift_amd.build")
    lib = ctypes.CDLL(fb.PROBE_LIB)
    vp, sz, i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64
    for name, types in (("gift_probe_read", [vp, sz, ctypes.c_int, vp]),
                        ("gift_probe_write", [vp, sz, ctypes.c_int, vp]),
                        ("gift_probe_copy", [vp, vp, sz, ctypes.c_int, vp]),
                        ("gift_probe_tile_read", [vp, i64, i64, vp]),
                        ("gift_probe_tile_write", [vp, i64, i64, ctypes.c_int, vp]),
                        ("gift_probe_slab_read", [vp, i64, i64, vp])):
        getattr(lib, name).argtypes = types
        getattr(lib, name).restype = ctypes.c_int
    dev = torch.device(device)
    torch.cuda.set_device(dev)
    nbytes = mib * 2 ** 20
    a = torch.randn(nbytes // 4, device=dev)
    b = torch.empty_like(a)
    rows, cols = nbytes // 4 // 4096, 4096
    st = torch.cuda.current_stream().cuda_stream
    pa, pb = a.data_ptr(), b.data_ptr()
    cases = [
        ("read", nbytes, lambda: lib.gift_probe_read(pa, nbytes, 0, st)),
        ("read_nt", nbytes, lambda: lib.gift_probe_read(pa, nbytes, 1, st)),
        ("write", nbytes, lambda: lib.gift_probe_write(pb, nbytes, 0, st)),
        ("write_nt", nbytes, lambda: lib.gift_probe_write(pb, nbytes, 1, st)),
        ("copy", 2 * nbytes, lambda: lib.gift_probe_copy(pa, pb, nbytes, 0, st)),
        ("copy_nt", 2 * nbytes, lambda: lib.gift_probe_copy(pa, pb, nbytes, 1, st)),
        ("tile_read_64x256", nbytes, lambda: lib.gift_probe_tile_read(pa, rows, cols, st)),
        ("tile_write_64x256", nbytes, lambda: lib.gift_probe_tile_write(pb, rows, cols, 0, st)),
        ("tile_write_64x256_nt", nbytes, lambda: lib.gift_probe_tile_write(pb, rows, cols, 1, st)),
        ("slab_read_64_rows", nbytes, lambda: lib.gift_probe_slab_read(pa, rows, cols, st)),
    ]
    out = {}
    for name, moved, fn in cases:
        for _ in range(3):
            if fn() != 0:
                raise RuntimeError("probe %s failed" % name)
        torch.cuda.synchronize()
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        e0.record()
        for _ in range(reps):
            fn()
        e1.record()
        torch.cuda.synchronize()
        t = e0.elapsed_time(e1) / reps * 1e-3
        out[name] = {"us": round(t * 1e6, 1), "GBps": round(moved / t / 1e9, 1)}
    return {"study": "stream", "bytes": nbytes, "reps": reps, "hbm_peak_GBps": 8000.0,
            "patterns": out}


# ---------------------------------------------------------------------------
# staleness study
# ---------------------------------------------------------------------------

def _rotating_block(args, dev):
    """Workload of the staleness and interval studies: its inputs, a Haar basis
    per input and the rotation each input's eigenbasis follows."""
    import torch

    import synth

    w = synth.llama_stack(args.blocks, args.hidden, args.mlp, args.tokens, exponent=1.5)
    base, rots = {}, {}
    for k, spec in enumerate(w.inputs):
        g = torch.Generator(device=dev).manual_seed(3000 + k)
        base[spec.name] = synth.haar(spec.d_in, g, dev)
        rots[spec.name] = synth.rotation_pair(spec.d_in, 4000 + k, dev)
    return w, base, rots


def _inputs_at(w, base, rots, t, angle, dev):
    """Rotated bases and fresh bf16 activations of every input at step t."""
    import synth

    Qt, X = {}, {}
    for k, spec in enumerate(w.inputs):
        Qt[spec.name] = synth.rotate_input(base[spec.name], rots[spec.name], t * angle) \
            if t else base[spec.name]
        X[spec.name] = synth.draw_input(spec, seed=7000 + 100 * t + k, device=dev,
                                        Q=Qt[spec.name], as_bf16=True)
    return Qt, X


def _step_errors(w, X, Qt, t, methods, block, dev):
    """M1 and M2 of the round trip of every layer's gradient at step t for each
    method (name -> factor, None = Euclidean), summed over the layers.  M2 is
    taken in the metric of the population covariance C_t, whose damped inverse
    square root is known in closed form for the generator."""
    import synth
    import fac_whitening_gift_amd as fg

    sc = fg.SCALE_BLOCK128 if block else fg.SCALE_TENSOR
    acc = {m: [0.0, 0.0, 0.0] for m in methods}
    den1 = 0.0
    for i, l in enumerate(w.layers):
        inp = X[l.input]
        G = synth.draw_gradient(l.d_out, Qt[l.input], inp["ev"], seed=9000 + 100 * t + i,
                                device=dev)
        lam = 1e-3 * float(inp["ev"].double().sum()) / l.d_in
        Sdiag = (inp["ev"].double() + lam).rsqrt().float()
        GS = (G @ Qt[l.input]) * Sdiag
        den2 = float(GS.double().pow(2).sum())
        for m, fac in methods.items():
            L = fg.Layer(G, factor=None if fac is None else fac[l.input], block128=block)
            if fac is None:
                fg.gift_euclid_fp8_roundtrip([L], scaling=sc)
            else:
                fg.gift_whiten_quantize([L], scaling=sc)
                fg.gift_dequant_unwhiten([L], scaling=sc)
            e = fg.gift_roundtrip_error([L]).cpu().numpy()[0]
            ES = ((L.G_hat - G) @ Qt[l.input]) * Sdiag
            acc[m][0] += float(e[0])
            acc[m][1] += float(ES.double().pow(2).sum())
            acc[m][2] += den2
        den1 += float(e[1])
    return {m: (math.sqrt(e1 / den1), math.sqrt(e2 / d2)) for m, (e1, e2, d2) in acc.items()}


def _refresh(w, X, factors):
    import fac_whitening_gift_amd as fg

    fg.gift_refresh_factors([dict(X=X[s.name]["X"], factor=factors[s.name], seed=s_i)
                             for s_i, s in enumerate(w.inputs)])


def staleness_study(args, device="cuda:0"):
    """Error of the round trip as a function of steps since the last factor
    refresh (the falsifier the GIFT review proposes: if at step 49 the stale
    factor's error reaches Euclidean FP8's, the refresh interval is too long).

    Every input's eigenbasis rotates by R(t) = V B(t*angle) V^T (all principal
    angles exactly t*angle); at step t fresh activations X_t and gradients G_t
    are drawn from the rotated covariance.  Methods per step: Euclidean, GIFT
    with the factor refreshed at t = 0 (stale), GIFT refreshed at t (fresh),
    each with per-tensor and 1x128 scaling.  M1 from the device error sums; M2
    in the metric of the population covariance C_t (C_t^-1/2 is known in
    closed form for the generator, so no eigensolve is needed)."""
    import torch

    import fac_whitening_gift_amd as fg

    dev = torch.device(device)
    w, base, rots = _rotating_block(args, dev)
    stale = {s.name: fg.Factor(s.d_in, device=dev) for s in w.inputs}
    fresh = {s.name: fg.Factor(s.d_in, device=dev) for s in w.inputs}
    steps = args.study_steps if args.study_steps is not None else 50
    rows = []
    for t in range(steps):
        Qt, X = _inputs_at(w, base, rots, t, args.angle, dev)
        if t == 0:
            _refresh(w, X, stale)
        _refresh(w, X, fresh)
        res = {"step": t}
        for block in (False, True):
            err = _step_errors(w, X, Qt, t, {"euclid": None, "stale": stale, "fresh": fresh},
                               block, dev)
            tag = "b128" if block else "tensor"
            for m, (m1, m2) in err.items():
                res["m1_%s_%s" % (m, tag)] = m1
                res["m2_%s_%s" % (m, tag)] = m2
        rows.append(res)
        if not args.quiet:
            print("[staleness] %s" % json.dumps({k: (round(v, 5) if isinstance(v, float) else v)
                                                for k, v in res.items()}),
                  file=sys.stderr, flush=True)
    last = rows[-1]
    return {"study": "staleness", "workload": w.name, "angle_rad_per_step": args.angle,
            "steps": len(rows), "refresh_at": 0,
            "falsified_at_last_step_m2": bool(last["m2_stale_tensor"] >= last["m2_euclid_tensor"]),
            "falsified_at_last_step_m1": bool(last["m1_stale_tensor"] >= last["m1_euclid_tensor"]),
            "rows": [{k: (round(v, 6) if isinstance(v, float) else v) for k, v in r.items()}
                     for r in rows]}


def interval_study(args, device="cuda:0"):
    """Ablation over the refresh interval K (the GIFT referee report asks for
    K in {10, 25, 50, 100}, measuring the round-trip error and the cost-quality
    trade-off).  On the rotating workload of the staleness study, one factor
    set per K is refreshed at every step t with t % K == 0 and used at every
    step in between; per-tensor E4M3.  Reported per K: M1 and M2 averaged over
    the horizon, M2 at the stalest step, and the grouped refresh's time
    amortized over K steps; the Euclidean round trip alongside."""
    import torch

    import fac_whitening_gift_amd as fg

    dev = torch.device(device)
    w, base, rots = _rotating_block(args, dev)
    intervals = [int(k) for k in args.intervals.split(",")]
    facs = {k: {s.name: fg.Factor(s.d_in, device=dev) for s in w.inputs} for k in intervals}
    steps = args.study_steps if args.study_steps is not None else max(intervals)
    sums = {m: [0.0, 0.0, 0.0] for m in ["euclid"] + intervals}   # m1, m2, worst m2
    refresh_ms = []
    for t in range(steps):
        Qt, X = _inputs_at(w, base, rots, t, args.angle, dev)
        for k in intervals:
            if t % k == 0:
                e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
                e0.record()
                _refresh(w, X, facs[k])
                e1.record()
                torch.cuda.synchronize()
                refresh_ms.append(e0.elapsed_time(e1))
        methods = {"euclid": None}
        methods.update({k: facs[k] for k in intervals})
        err = _step_errors(w, X, Qt, t, methods, False, dev)
        for m, (m1, m2) in err.items():
            sums[m][0] += m1
            sums[m][1] += m2
            sums[m][2] = max(sums[m][2], m2)
        if not args.quiet:
            print("[interval] step %d %s" % (t, json.dumps({str(m): round(v[1], 5)
                                                             for m, v in err.items()})),
                  file=sys.stderr, flush=True)
    # the first refresh of a run carries one-time set-up; the median of the rest
    rms = sorted(refresh_ms[1:] or refresh_ms)[len(refresh_ms[1:] or refresh_ms) // 2]
    rows = []
    for k in intervals:
        rows.append({"K": k, "m1_mean": round(sums[k][0] / steps, 6),
                     "m2_mean": round(sums[k][1] / steps, 6), "m2_worst": round(sums[k][2], 6),
                     "m2_reduction_vs_euclid": round(1 - sums[k][1] / sums["euclid"][1], 4),
                     "refreshes": -(-steps // k),
                     "refresh_ms_per_step": round(rms / k, 5)})
    return {"study": "interval", "workload": w.name, "angle_rad_per_step": args.angle,
            "steps": steps, "refresh_ms": round(rms, 4),
            "euclid": {"m1_mean": round(sums["euclid"][0] / steps, 6),
                       "m2_mean": round(sums["euclid"][1] / steps, 6)},
            "rows": rows}


# ---------------------------------------------------------------------------
# rank study
# ---------------------------------------------------------------------------

def rank_study(args, device="cuda:0"):
    """Round-trip error as a function of the factor's structure (the review
    chose rank 32 from a round-trip error table over ranks, with block-A-32
    and block-A-64 beside them).  On the hidden-1024 block (4 inputs, 7
    gradients): for each rank r, the grouped refresh keeps the top r Ritz
    pairs of a subspace iteration of sketch width r + 32 rounded to the
    factor's storage (64 up to rank 32, 96 for rank 64) and damps with the
    mean of the d_in - r discarded eigenvalues; an entry "bN" is the
    block-diagonal factor with N x N blocks, damped by lambda_floor; then the
    grouped per-tensor E4M3 round trip of all 7 gradients.  M1 from the
    device error sums, M2 in the metric of the exact damped sample
    covariance (fp64 eigendecomposition on the device, measurement harness);
    the Euclidean round trip of the same gradients alongside."""
    import numpy as np
    import torch

    import synth
    import fac_whitening_gift_amd as fg

    dev = torch.device(device)
    w = synth.llama_block(hidden=1024, mlp=2816, tokens=8192, exponent=1.5)
    inputs = {s.name: synth.draw_input(s, seed=1000 + k, device=dev, as_bf16=True)
              for k, s in enumerate(w.inputs)}
    grads = [synth.draw_gradient(l.d_out, inputs[l.input]["Q"], inputs[l.input]["ev"],
                                 seed=5000 + i, device=dev) for i, l in enumerate(w.layers)]
    S = {}
    for name, inp in inputs.items():
        X = inp["X"].double()
        A = X.T @ X / X.shape[0]
        lam = 1e-3 * torch.trace(A) / A.shape[0]
        ev_, V = torch.linalg.eigh(A)
        S[name] = (V * (ev_.clamp_min(0) + lam).rsqrt()) @ V.T
    den2 = sum(float(torch.linalg.norm(G.double() @ S[l.input]) ** 2)
               for G, l in zip(grads, w.layers))

    def errors(layers):
        err = fg.gift_roundtrip_error(layers).cpu().numpy()
        m1 = float(np.sqrt(err[:, 0].sum() / err[:, 1].sum()))
        num = sum(float(torch.linalg.norm((L.G_hat.double() - L.G.double()) @ S[l.input]) ** 2)
                  for L, l in zip(layers, w.layers))
        return m1, float(np.sqrt(num / den2))

    elems = sum(G.numel() for G in grads)

    def roundtrip_gbps(layers, n=20):
        """fp32 gradient GB/s of the grouped whiten + quantize and dequantize +
        un-whiten calls, back to back on the stream (prepared calls)."""
        cw = fg.GroupCall(fg.OP_WHITEN_QUANTIZE, layers)
        cd = fg.GroupCall(fg.OP_DEQUANT_UNWHITEN, layers)
        for _ in range(3):
            cw()
            cd()
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        e0.record()
        for _ in range(n):
            cw()
            cd()
        e1.record()
        torch.cuda.synchronize()
        return 4 * elems / (e0.elapsed_time(e1) / n * 1e-3) / 1e9

    eu = [fg.Layer(G) for G in grads]
    fg.gift_euclid_fp8_roundtrip(eu)
    m1_e, m2_e = errors(eu)
    rows = []
    for entry in args.rank_list.split(","):
        blk = int(entry[1:]) if entry.startswith("b") else 0
        r = 0 if blk else int(entry)
        facs = {s.name: fg.Factor(s.d_in, device=dev, rank=r or 32, block=blk) for s in w.inputs}
        items = [dict(X=inputs[s.name]["X"], factor=facs[s.name], seed=k)
                 for k, s in enumerate(w.inputs)]
        fg.gift_refresh_factors(items)
        gl = [fg.Layer(G, factor=facs[l.input]) for G, l in zip(grads, w.layers)]
        fg.gift_whiten_quantize(gl)
        fg.gift_dequant_unwhiten(gl)
        m1, m2 = errors(gl)
        lam = [float(facs[s.name].coef[fg.COEF_LAMBDA_ISO]) for s in w.inputs]
        gbps = roundtrip_gbps(gl)
        rows.append({"factor": "block-A-%d" % blk if blk else "rank %d" % r,
                     "m1": round(m1, 5), "m2": round(m2, 5),
                     "m1_ratio_vs_euclid": round(m1 / m1_e, 4),
                     "m2_reduction_vs_euclid": round(1 - m2 / m2_e, 4),
                     "roundtrip_GBps": round(gbps, 1),
                     "lambda_iso": [float("%.4g" % x) for x in lam]})
        if not args.quiet:
            print("[rank] %s" % json.dumps(rows[-1]), file=sys.stderr, flush=True)
    return {"study": "rank", "workload": w.name, "scaling": "per-tensor E4M3",
            "damping": "floor+tail", "euclid": {"m1": round(m1_e, 5), "m2": round(m2_e, 5)},
            "rows": rows}


# ---------------------------------------------------------------------------
# full-rank and two-sided references
# ---------------------------------------------------------------------------

def reference_factors(A, dev):
    """The harness's fp64 transforms of one input: (S, S^-1) = ((A + lam I)^-1/2,
    (A + lam I)^1/2) by eigh, and the Cholesky pair (L^-T, L^T) of A + lam I,
    lam = 1e-3 tr(A) / d_in."""
    import torch

    def sym_pair(M):
        lam = 1e-3 * torch.trace(M) / M.shape[0]
        ev_, V = torch.linalg.eigh(M + lam * torch.eye(M.shape[0], dtype=M.dtype, device=dev))
        ev_ = ev_.clamp_min(0)
        return (V * ev_.rsqrt()) @ V.T, (V * ev_.sqrt()) @ V.T

    S, Si = sym_pair(A)
    lam = 1e-3 * torch.trace(A) / A.shape[0]
    eye = torch.eye(A.shape[0], dtype=A.dtype, device=dev)
    L = torch.linalg.cholesky(A + lam * eye)
    Linv = torch.linalg.solve_triangular(L, eye, upper=False)
    return {"S": S, "Si": Si, "Lt_inv": Linv.T.contiguous(), "Lt": L.T.contiguous(),
            "sym_pair": sym_pair}


def reference_outputs(G, rf, factor):
    """Round trips of one gradient G (fp32, device) under every method of the
    reference study.  Returns {method: (W32, codes, inv, G^ fp64)}; W32 is
    None for the library's own paths (Euclid, GIFT rank 32).  The reference
    transforms are fp64 torch (harness); each whitened tensor is rounded to
    fp32 and quantized by the library's per-tensor E4M3 kernels."""
    import fac_whitening_gift_amd as fg

    G64 = G.double()
    SB, SBi = rf["sym_pair"](G64 @ G64.T / G64.shape[1])
    outs = {}
    eu = fg.Layer(G)
    fg.gift_euclid_fp8_roundtrip([eu])
    outs["euclid"] = (None, eu.q, eu.inv_scale, eu.G_hat.double())
    gl = fg.Layer(G, factor=factor)
    fg.gift_whiten_quantize([gl])
    fg.gift_dequant_unwhiten([gl])
    outs["gift_rank32"] = (None, gl.q, gl.inv_scale, gl.G_hat.double())
    for name, (lt, rt, lti, rti) in (("input_full", (None, rf["S"], None, rf["Si"])),
                                      ("input_cholesky", (None, rf["Lt_inv"], None, rf["Lt"])),
                                      ("two_sided", (SB, rf["S"], SBi, rf["Si"]))):
        W = G64 if lt is None else lt @ G64
        W32 = (W @ rt).float().contiguous()
        q = fg.Layer(W32)
        fg.gift_euclid_fp8_roundtrip([q])
        Wh = q.G_hat.double()
        outs[name] = (W32, q.q, q.inv_scale, (Wh if lti is None else lti @ Wh) @ rti)
    return outs


def reference_study(args, device="cuda:0"):
    """Where the rank-32 input-side factor stands against the transforms it
    simplifies (the review: the input-side factor alone matches the full
    two-sided K-FAC transform almost exactly; its Eq. 14 Cholesky form).
    On a Llama-style block (default hidden 1024, MLP 2816, 8192 tokens), per
    gradient: Euclidean FP8; GIFT with the rank-32 factor (the library's
    path end to end); full-rank input-side W = G (A + lam I)^-1/2; its
    Cholesky form W = G L^-T (L L^T = A + lam I); two-sided
    W = (B + mu I)^-1/2 G (A + lam I)^-1/2 with the output-side factor read as
    B = G G^T / d_in.  The reference transforms and their inverses are fp64
    torch on the device (measurement harness, from the exact sample A); the
    whitened tensors are quantized by the library's per-tensor E4M3 kernels.
    M1 and M2 (input-side K-FAC metric) summed over the block's gradients."""
    import numpy as np
    import torch

    import synth
    import fac_whitening_gift_amd as fg

    dev = torch.device(device)
    h, m, n = (int(x) for x in args.ref_shape.split(","))
    w = synth.llama_block(hidden=h, mlp=m, tokens=n, exponent=1.5)
    inputs = {s.name: synth.draw_input(s, seed=1000 + k, device=dev, as_bf16=True)
              for k, s in enumerate(w.inputs)}
    facs = {s.name: fg.Factor(s.d_in, device=dev) for s in w.inputs}
    fg.gift_refresh_factors([dict(X=inputs[s.name]["X"], factor=facs[s.name], seed=k)
                             for k, s in enumerate(w.inputs)])
    methods = ["euclid", "gift_rank32", "input_full", "input_cholesky", "two_sided"]
    num1 = {k: 0.0 for k in methods}
    num2 = {k: 0.0 for k in methods}
    den1 = den2 = 0.0
    cache = {}
    for i, l in enumerate(w.layers):
        inp = inputs[l.input]
        if l.input not in cache:
            X = inp["X"].double()
            cache[l.input] = reference_factors(X.T @ X / X.shape[0], dev)
        rf = cache[l.input]
        G = synth.draw_gradient(l.d_out, inp["Q"], inp["ev"], seed=5000 + i, device=dev)
        outs = reference_outputs(G, rf, facs[l.input])
        G64 = G.double()
        for k in methods:
            e2, g2 = m2_parts(G64, outs[k][3], rf["S"])
            num1[k] += float((outs[k][3] - G64).pow(2).sum())
            num2[k] += e2
        den1 += float(G64.pow(2).sum())
        den2 += g2
    rows = {k: {"m1": round(float(np.sqrt(num1[k] / den1)), 5),
                "m2": round(float(np.sqrt(num2[k] / den2)), 5),
                "m2_reduction_vs_euclid": round(1 - float(np.sqrt(num2[k] / num2["euclid"])), 4)}
            for k in methods}
    return {"study": "reference", "workload": w.name, "scaling": "per-tensor E4M3",
            "output_factor": "G G^T / d_in", "rows": rows}


# ---------------------------------------------------------------------------
# reduce study
# ---------------------------------------------------------------------------

def reduce_study(args, device="cuda:0"):
    """A data-parallel step on one GPU: `ranks` ranks hold independent
    gradients of the hidden-1024 block (drawn from the same input
    covariances), each quantizes its own (GIFT: whitened with the shared
    factors; Euclidean: as is), and the receive side sums the dequantized
    payloads in fp32 rank by rank and un-whitens the sum once.  Error of the
    reduced gradient against the exact sum of the ranks' gradients: M1 and M2
    (the K-FAC metric of the exact sample covariance), per-tensor E4M3 and
    MXFP4; and the rates of the accumulate and un-whiten calls."""
    import numpy as np
    import torch

    import synth
    import fac_whitening_gift_amd as fg

    dev = torch.device(device)
    R = args.ranks
    w = synth.llama_block(hidden=1024, mlp=2816, tokens=8192, exponent=1.5)
    inputs, factors = {}, {}
    for k, spec in enumerate(w.inputs):
        inputs[spec.name] = synth.draw_input(spec, seed=1000 + k, device=dev, as_bf16=True)
        factors[spec.name] = fg.Factor(spec.d_in, device=dev)
    fg.gift_refresh_factors([dict(X=inputs[s.name]["X"], factor=factors[s.name], seed=k)
                             for k, s in enumerate(w.inputs)])
    grads = [[synth.draw_gradient(l.d_out, inputs[l.input]["Q"], inputs[l.input]["ev"],
                                  seed=20000 + 1000 * r + i, device=dev)
              for i, l in enumerate(w.layers)] for r in range(R)]
    exact = [sum(grads[r][i].double() for r in range(R)) for i in range(len(w.layers))]
    S_metric = {}
    for spec in w.inputs:
        X = inputs[spec.name]["X"].double()
        A = X.T @ X / X.shape[0]
        lam = 1e-3 * torch.trace(A) / A.shape[0]
        ev_, V = torch.linalg.eigh(A)
        S_metric[spec.name] = (V * (ev_.clamp_min(0) + lam).rsqrt()) @ V.T
    ev = lambda: torch.cuda.Event(enable_timing=True)  # noqa: E731
    out = {"study": "reduce", "workload": w.name, "ranks": R,
           "gradient_elements": w.gradient_elements}
    for fmt, sc in (("e4m3_tensor", fg.SCALE_TENSOR), ("mxfp4", fg.SCALE_MXFP4)):
        mx_ = sc == fg.SCALE_MXFP4
        res = {}
        for method in ("gift", "euclid"):
            ranks = []
            for r in range(R):
                layers = [fg.Layer(grads[r][i], mxfp4=mx_,
                                   factor=factors[l.input] if method == "gift" else None)
                          for i, l in enumerate(w.layers)]
                fg.gift_whiten_quantize(layers, scaling=sc)
                ranks.append(layers)
            acc = [torch.empty_like(grads[0][i]) for i in range(len(w.layers))]
            views = [[fg.Layer(None, factor=L.factor, q=L.q, inv_scale=L.inv_scale, G_hat=a,
                               d_out=L.d_out, d_in=L.d_in, allocate=False, mxfp4=mx_)
                      for L, a in zip(ranks[r], acc)] for r in range(R)]
            torch.cuda.synchronize()
            t0, t1, t2 = ev(), ev(), ev()
            t0.record()
            for r in range(R):
                fg.gift_dequant_accumulate(views[r], scaling=sc, first=r == 0)
            t1.record()
            if method == "gift":
                fg.gift_unwhiten_f32(views[0])
            t2.record()
            torch.cuda.synchronize()
            num1 = den1 = num2 = den2 = 0.0
            for i, l in enumerate(w.layers):
                E = acc[i].double() - exact[i]
                S = S_metric[l.input]
                num1 += float(E.pow(2).sum())
                den1 += float(exact[i].pow(2).sum())
                num2 += float((E @ S).pow(2).sum())
                den2 += float((exact[i] @ S).pow(2).sum())
            res[method] = {"m1": round(math.sqrt(num1 / den1), 5),
                           "m2": round(math.sqrt(num2 / den2), 5),
                           "accumulate_ms_per_rank": round(t0.elapsed_time(t1) / R, 4)}
            if method == "gift":
                res[method]["unwhiten_ms"] = round(t1.elapsed_time(t2), 4)
        res["m2_reduction"] = round(1 - res["gift"]["m2"] / res["euclid"]["m2"], 4)
        out[fmt] = res
    return out


# ---------------------------------------------------------------------------
# layer study
# ---------------------------------------------------------------------------

def layer_study(args, device="cuda:0"):
    """A gate layer's training step with its products in MXFP4, from the
    residual stream to the round trip of its gradient: RMS norm, refresh of
    the factor on the norm's output X, Y = X W^T, dX = dY W and G = dY^T X on
    operands quantized along the summed axis, the norm's backward pass, and
    the round trip of G (GIFT and Euclidean; per-tensor E4M3 and MXFP4).
    Errors against fp64 products of the unquantized tensors (torch, as
    measurement harness): M1 of Y, dX and G, and M1 and M2 of the
    reconstructed G, so that the payload's error can be read beside the
    product's own."""
    import torch

    import synth
    import fac_whitening_gift_amd as fg

    dev = torch.device(device)
    hidden, mlp, tokens = (int(v) for v in args.ref_shape.split(","))
    g = torch.Generator(device=dev).manual_seed(7)
    spec = synth.InputSpec("residual", hidden, tokens, 1.5)
    H = synth.draw_input(spec, seed=1000, device=dev, as_bf16=True)["X"]
    weight = torch.ones(hidden, device=dev)
    W = torch.randn(mlp, hidden, generator=g, device=dev) * hidden ** -0.5
    dY = (torch.randn(tokens, mlp, generator=g, device=dev)
          * torch.randn(tokens, 1, generator=g, device=dev).exp() * 1e-3).bfloat16()
    factor = fg.Factor(hidden, device=dev)
    ev = lambda: torch.cuda.Event(enable_timing=True)  # noqa: E731
    ms, marks = {}, []

    def timed(name, fn):
        fn()  # warm-up
        a, b = ev(), ev()
        a.record()
        res = fn()
        b.record()
        marks.append((name, a, b))
        return res

    X, _, rstd = timed("norm_forward", lambda: fg.gift_norm_forward(H, weight, kind=fg.NORM_RMS))
    fg.gift_refresh_factor(X, factor, seed=3)
    xr, xc = timed("quantize_x", lambda: fg.gift_mx_quantize(X, by_row=True, by_col=True))
    wr, wc = timed("quantize_w", lambda: fg.gift_mx_quantize(W, by_row=True, by_col=True))
    Y = timed("y", lambda: fg.gift_mx_matmul(xr, wr))
    gr, gc = timed("quantize_dy", lambda: fg.gift_mx_quantize(dY, by_row=True, by_col=True))
    dX = timed("dx", lambda: fg.gift_mx_matmul(gr, wc))
    G = timed("g", lambda: fg.gift_mx_matmul(gc, xc, dtype=torch.float32))
    timed("norm_backward", lambda: fg.gift_norm_backward(dX, H, weight, None, rstd, kind=fg.NORM_RMS))
    torch.cuda.synchronize()
    for name, a, b in marks:
        ms[name] = round(a.elapsed_time(b), 4)

    def m1(got, want):
        return round(float((got.double() - want).norm() / want.norm()), 5)

    X64, W64, dY64 = X.double(), W.double(), dY.double()
    G64 = dY64.T @ X64
    out = {"study": "layer", "hidden": hidden, "mlp": mlp, "tokens": tokens, "ms": ms,
           "m1": {"y": m1(Y, X64 @ W64.T), "dx": m1(dX, dY64 @ W64), "g": m1(G, G64)}}
    S = kfac_metric(X)
    num, den = m2_parts(G64, G, S)
    out["g_m2"] = round(math.sqrt(num / den), 5)
    for fmt, sc in (("e4m3_tensor", fg.SCALE_TENSOR), ("mxfp4", fg.SCALE_MXFP4)):
        out[fmt] = {}
        for method in ("gift", "euclid"):
            L = fg.Layer(G, factor=factor if method == "gift" else None, mxfp4=sc == fg.SCALE_MXFP4)
            fg.gift_whiten_quantize([L], scaling=sc)
            fg.gift_dequant_unwhiten([L], scaling=sc)
            total, own = m2_parts(G64, L.G_hat, S)[0], m2_parts(G, L.G_hat, S)
            out[fmt][method] = {"m1_total": m1(L.G_hat, G64), "m1_payload": m1(L.G_hat, G.double()),
                                "m2_total": round(math.sqrt(total / den), 5),
                                "m2_payload": round(math.sqrt(own[0] / own[1]), 5)}
    return out


# ---------------------------------------------------------------------------
# matrix-free refresh study
# ---------------------------------------------------------------------------

def matrixfree_study(args, device="cuda:0"):
    """Would the matrix-free form of the refresh's products, A Q = X^T (X Q) / N,
    pay on these shapes?  It skips the covariance but reads X twice per
    product.  On the 600M stack's 96 inputs (72 of width 1536, 24 of width
    4096, 16384 bf16 tokens each): the library's grouped refresh (covariance
    on bf16 MFMA, then six products with A on split-bf16 MFMA, CholeskyQR and
    Rayleigh-Ritz) against the six products alone in matrix-free form as
    plain fp32 library GEMMs (torch on the device; the products need fp32
    accuracy, and X is exact in fp32).  If the products alone take longer
    than the whole library refresh, the matrix-free form cannot win.  The
    matrix-free product is checked against A Q on one input (fp64)."""
    import torch

    import synth
    import fac_whitening_gift_amd as fg

    dev = torch.device(device)
    w = synth.llama_stack(24, 1536, 4096, 16384, exponent=1.5)
    inputs = [synth.draw_input(s, seed=1000 + k, device=dev, as_bf16=True, axis_aligned=True)
              for k, s in enumerate(w.inputs)]
    facs = [fg.Factor(s.d_in, device=dev) for s in w.inputs]
    items = [dict(X=inp["X"], factor=f, seed=k) for k, (inp, f) in enumerate(zip(inputs, facs))]
    ws = torch.empty(fg.gift_refresh_group_workspace_bytes(items), dtype=torch.uint8, device=dev)
    ev = lambda: torch.cuda.Event(enable_timing=True)  # noqa: E731

    def timed(fn, n=3):
        fn()
        torch.cuda.synchronize()
        a, b = ev(), ev()
        a.record()
        for _ in range(n):
            fn()
        b.record()
        torch.cuda.synchronize()
        return a.elapsed_time(b) / n

    t_lib = timed(lambda: fg.gift_refresh_factors(items, ws=ws))
    Xf = [inp["X"].float() for inp in inputs]
    Qs = [torch.linalg.qr(torch.randn(s.d_in, 64, device=dev))[0] for s in w.inputs]

    def products():
        for X, Q in zip(Xf, Qs):
            for _ in range(6):
                (X.T @ (X @ Q)) / X.shape[0]

    t_mf = timed(products)
    X64 = Xf[-1].double()
    A = X64.T @ X64 / X64.shape[0]
    Q = Qs[-1]
    ref = A @ Q.double()
    got = (Xf[-1].T @ (Xf[-1] @ Q)) / Xf[-1].shape[0]
    rel = float(torch.linalg.norm(got.double() - ref) / torch.linalg.norm(ref))
    flops = sum(6 * 2 * 2 * s.tokens * s.d_in * 64 for s in w.inputs)
    return {"study": "matrixfree", "workload": w.name, "inputs": len(w.inputs),
            "library_refresh_ms": round(t_lib, 3),
            "matrix_free_six_products_ms": round(t_mf, 3),
            "matrix_free_tflop": round(flops / 1e12, 3),
            "matrix_free_tflops": round(flops / t_mf / 1e9, 1),
            "matrix_free_rel_err_vs_fp64": rel,
            "ratio_products_over_library_refresh": round(t_mf / t_lib, 3)}


if __name__ == "__main__":
    main()

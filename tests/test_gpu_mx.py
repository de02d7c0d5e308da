"""MXFP4 operands and products on the device (gift_mx_*) against the oracle.

Operands: every byte equal to the oracle's (codes, scales, padding).
Products: C[i, j] = sum_k a b over the exact operand values in fp64.  Each of
the at most k additions of the fp32 sum, and each of the terms it aligns, is
off by at most one unit in the last place of a partial sum, which is at most
S = sum_k |a b|: bound 2 k 2^-23 S.  A bf16 result adds half a step,
2^-8 |C|.
"""

import numpy as np
import pytest
import torch

import fac_whitening_gift_amd as fg
from oracle import layer as ol
from gpu_util import DEV, host, say

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def _draw(rows, cols, seed, dtype=torch.float32, spread=8):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-spread, spread + 1, (rows, 1)))
    return torch.from_numpy(x.astype(np.float32)).to(dtype)


def _f32(t):
    return t.float().numpy()


def _operand(x):
    """oracle operand values (fp64) and bytes of a CPU tensor"""
    codes, scales, flags = ol.quantize(_f32(x))
    return ol.values(codes, scales, x.shape[1]), ol.pack(codes, scales), flags


SIZES = [(1, 1), (1, 4096), (3, 31), (16, 32), (17, 33), (64, 128), (65, 129), (127, 127), (128, 256),
         (200, 511), (300, 130), (257, 1025)]


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_quantize_bytes(rows, cols, dtype):
    say("mx quantize %dx%d %s" % (rows, cols, dtype))
    x = _draw(rows, cols, rows * 7 + cols, dtype)
    flags = torch.zeros(1, dtype=torch.int32, device=DEV)
    r, c = fg.gift_mx_quantize(x.to(DEV), by_row=True, by_col=True, flags=flags)
    vr, br, fr = _operand(x)
    vc, bc, fc = _operand(x.t().contiguous())
    assert np.array_equal(host(r.data), br)
    assert np.array_equal(host(c.data), bc)
    assert int(host(flags)[0]) == fr | fc
    assert np.array_equal(host(fg.gift_mx_dequantize(r)).astype(np.float64), vr)
    got = fg.gift_mx_dequantize(c, dtype=BF16)
    assert got.dtype == BF16 and np.array_equal(_f32(got.cpu()).astype(np.float64), vc)
    # either one alone
    r1, none = fg.gift_mx_quantize(x.to(DEV), by_row=True)
    none2, c1 = fg.gift_mx_quantize(x.to(DEV), by_col=True)
    assert none is None and none2 is None
    assert torch.equal(r1.data, r.data) and torch.equal(c1.data, c.data)


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("ld,offset", [(200, 0), (200, 3), (136, 8), (131, 1)])
def test_quantize_slices(ld, offset, dtype):
    """A slice of a wider matrix: any leading dimension, any start."""
    say("mx quantize slice ld %d offset %d %s" % (ld, offset, dtype))
    wide = _draw(130, ld, ld + offset, dtype)
    x = wide[:, offset:offset + 128]
    r, c = fg.gift_mx_quantize(wide.to(DEV)[:, offset:offset + 128], by_row=True, by_col=True)
    assert np.array_equal(host(r.data), _operand(x)[1])
    assert np.array_equal(host(c.data), _operand(x.t().contiguous())[1])


def test_quantize_special_blocks():
    """NaN, infinities, zeros, signed zeros, subnormal and the largest values:
    bytes and flags of the oracle."""
    say("mx quantize specials")
    x = torch.zeros(64, 96)
    x[0, :32] = float("nan")
    x[1, 3] = float("inf")
    x[1, 4] = 1.0
    x[2, 40] = -float("inf")
    x[3, 41] = float("nan")
    x[4, :] = -0.0
    x[5, :32] = 2.0 ** -140
    x[6, :32] = torch.finfo(torch.float32).max
    x[7, :] = torch.linspace(-7.9, 7.9, 96)
    x[8, :32] = 2.0 ** -149
    x[9, ::3] = -3.5
    for part, want in ((x, 3), (x[7:8], 0), (x[4:5], 2), (x[1:2, :32], 1)):
        flags = torch.zeros(1, dtype=torch.int32, device=DEV)
        r, _ = fg.gift_mx_quantize(part.contiguous().to(DEV), by_row=True, flags=flags)
        v, b, f = _operand(part)
        assert np.array_equal(host(r.data), b)
        assert f == want and int(host(flags)[0]) == want
        got = host(fg.gift_mx_dequantize(r)).astype(np.float64)
        assert np.array_equal(np.isnan(got), np.isnan(v))
        assert np.array_equal(got[~np.isnan(v)], v[~np.isnan(v)])


def test_quantize_equals_the_payload():
    """The round trip's MXFP4 reconstruction of the same gradient."""
    say("mx quantize vs payload")
    G = _draw(77, 256, 5).to(DEV)
    L = fg.Layer(G, mxfp4=True)
    fg.gift_euclid_fp8_roundtrip([L], scaling=fg.SCALE_MXFP4)
    r, _ = fg.gift_mx_quantize(G, by_row=True)
    assert torch.equal(fg.gift_mx_dequantize(r), L.G_hat)


def _check_product(got, va, vb, bias=None, add=None, bf16=False):
    c = va @ vb.T
    s = np.abs(va) @ np.abs(vb).T
    tol = 2 * va.shape[1] * 2.0 ** -23 * s
    if bias is not None:
        c, tol = c + bias, tol + 2.0 ** -24 * (np.abs(c) + np.abs(bias))
    if add is not None:
        c, tol = c + add, tol + 2.0 ** -24 * (np.abs(c) + np.abs(add))
    if bf16:
        tol = tol + 2.0 ** -8 * np.abs(c) + 2.0 ** -133
    err = np.abs(got.astype(np.float64) - c)
    assert np.all(err <= tol), (err - tol).max()


PRODUCTS = [(1, 1, 1), (1, 300, 4096), (2, 64, 33), (16, 48, 128), (17, 100, 500), (33, 16, 1024), (64, 1000, 257),
            (65, 65, 65), (100, 128, 1280), (128, 128, 512), (130, 300, 700), (256, 512, 128), (300, 200, 4000),
            (513, 257, 129), (1000, 1030, 260)]


@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_matmul(m, n, k):
    say("mx matmul %dx%dx%d" % (m, n, k))
    a, b = _draw(m, k, m + k, BF16, 3), _draw(n, k, n + k + 1, torch.float32, 3)
    ra, _ = fg.gift_mx_quantize(a.to(DEV), by_row=True)
    rb, _ = fg.gift_mx_quantize(b.to(DEV), by_row=True)
    va, vb = _operand(a)[0], _operand(b)[0]
    f = fg.gift_mx_matmul(ra, rb, dtype=torch.float32)
    _check_product(host(f), va, vb)
    h = fg.gift_mx_matmul(ra, rb)
    assert torch.equal(h, f.to(BF16))          # rounded once from the same sums
    bias = torch.from_numpy(np.random.default_rng(1).standard_normal(n).astype(np.float32))
    _check_product(host(fg.gift_mx_matmul(ra, rb, bias=bias.to(DEV), dtype=torch.float32)), va, vb,
                   bias=bias.numpy().astype(np.float64))
    acc = torch.from_numpy(np.random.default_rng(2).standard_normal((m, n)).astype(np.float32)).to(DEV)
    before = host(acc).astype(np.float64)
    assert fg.gift_mx_matmul(ra, rb, out=acc, accumulate=True) is acc
    _check_product(host(acc), va, vb, add=before)
    assert torch.equal(fg.gift_mx_matmul(ra, rb, dtype=torch.float32), f)   # the same bits again


# (cut into: 256-tiles, several and one a workgroup; 128-tiles, one, several and split
# four ways; small products of 64 and 16 columns a workgroup)
LARGE = [(8100, 8180, 4100), (4000, 4090, 4200), (1100, 3001, 1100), (4100, 4030, 2100), (1000, 1101, 16000),
         (1030, 2050, 1100), (3000, 9, 300)]


@pytest.mark.parametrize("m,n,k", LARGE)
def test_matmul_large(m, n, k):
    """Whole outputs against fp64 products, on the device, of the operands'
    decoded values; accumulation over 3 micro-batches; the last panels and
    k steps ragged."""
    say("mx matmul large %dx%dx%d" % (m, n, k))
    g = torch.Generator(device=DEV).manual_seed(m + n)
    a, b = torch.randn(m, k, generator=g, device=DEV), torch.randn(n, k, generator=g, device=DEV)
    a *= torch.exp2(torch.randint(-6, 7, (m, 1), generator=g, device=DEV).float())
    ra, _ = fg.gift_mx_quantize(a, by_row=True)
    rb, _ = fg.gift_mx_quantize(b, by_row=True)
    va, vb = (fg.gift_mx_dequantize(r).double() for r in (ra, rb))
    c, s = va @ vb.t(), va.abs() @ vb.abs().t()
    tol = 2 * k * 2.0 ** -23 * s
    f = fg.gift_mx_matmul(ra, rb, dtype=torch.float32)
    assert bool(((f.double() - c).abs() <= tol).all())
    bias = torch.randn(n, generator=g, device=DEV)
    h = fg.gift_mx_matmul(ra, rb, bias=bias)
    ref = c + bias.double()
    # the fp32 sum, the bias' rounding, the rounding to bf16
    t = tol + 2.0 ** -24 * (ref.abs() + tol)
    assert bool(((h.double() - ref).abs() <= t + 2.0 ** -8 * (ref.abs() + t)).all())
    assert torch.equal(fg.gift_mx_matmul(ra, rb), f.to(BF16))
    acc = torch.zeros(m, n, device=DEV)
    for _ in range(3):
        fg.gift_mx_matmul(ra, rb, out=acc, accumulate=True)
    assert bool(((acc.double() - 3 * c).abs() <= 3 * tol + 3 * 2.0 ** -24 * (3 * c.abs() + 3 * tol)).all())
    assert torch.equal(fg.gift_mx_matmul(ra, rb, dtype=torch.float32), f)


@pytest.mark.parametrize("m,n,k", [(20, 70, 200), (200, 150, 300), (600, 2000, 128), (1100, 3001, 1100)])
@pytest.mark.parametrize("dtype", [torch.float32, BF16])
def test_matmul_into_a_slice(m, n, k, dtype):
    """Rows of a wider C: what lies beside the product stays as it was."""
    say("mx matmul slice %dx%dx%d %s" % (m, n, k, dtype))
    a, b = _draw(m, k, 1, BF16, 2), _draw(n, k, 2, BF16, 2)
    ra, _ = fg.gift_mx_quantize(a.to(DEV), by_row=True)
    rb, _ = fg.gift_mx_quantize(b.to(DEV), by_row=True)
    want = fg.gift_mx_matmul(ra, rb, dtype=dtype)
    for pad, off in ((8, 4), (5, 3)):
        wide = torch.full((m + 2, n + pad), -7.0, dtype=dtype, device=DEV)
        view = wide[1:-1, off:off + n]
        fg.gift_mx_matmul(ra, rb, out=view)
        assert torch.equal(view, want)
        view.fill_(-7.0)
        assert bool((wide == -7.0).all())


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("m,n,k", [(1, 40, 64), (1, 1000, 4096), (5, 129, 1000), (16, 64, 2048), (16, 32, 8192),
                                   (24, 100, 600), (70, 90, 260), (2, 9000, 300), (16, 5000, 513),
                                   (1, 40, 180000), (2, 24, 90001)])
def test_linear(m, n, k, dtype):
    say("mx linear %dx%dx%d %s" % (m, n, k, dtype))
    x, w = _draw(m, k, m + n, dtype, 3), _draw(n, k, k, torch.float32, 3)
    bias = torch.from_numpy(np.random.default_rng(3).standard_normal(n).astype(np.float32))
    rw, _ = fg.gift_mx_quantize(w.to(DEV), by_row=True)
    vx, vw = _operand(x)[0], _operand(w)[0]
    y = fg.gift_mx_linear(x.to(DEV), rw, dtype=torch.float32)
    _check_product(host(y), vx, vw)
    y = fg.gift_mx_linear(x.to(DEV), rw, bias=bias.to(DEV), dtype=BF16)
    _check_product(_f32(y.cpu()), vx, vw, bias=bias.numpy().astype(np.float64), bf16=True)
    wide = torch.zeros(m, k + 9, dtype=dtype, device=DEV)
    wide[:, 5:5 + k] = x.to(DEV)
    assert torch.equal(fg.gift_mx_linear(wide[:, 5:5 + k], rw, bias=bias.to(DEV), dtype=BF16), y)


def test_linear_flags():
    say("mx linear flags")
    rw, _ = fg.gift_mx_quantize(_draw(40, 256, 1).to(DEV), by_row=True)
    for m in (1, 40):
        for bad, want in ((None, 0), (0.0, 2), (float("nan"), 1)):
            x = torch.ones(m, 256)
            if bad is not None:
                x[m - 1, 32:64] = bad
            flags = torch.zeros(1, dtype=torch.int32, device=DEV)
            y = fg.gift_mx_linear(x.to(DEV), rw, flags=flags)
            assert int(host(flags)[0]) == want
            nan = host(torch.isnan(y))
            assert nan[m - 1].all() == (want == 1) and not nan[:m - 1].any()


@pytest.mark.parametrize("m", [1, 40, 200])
def test_nan_scales_reach_their_rows_and_columns_only(m):
    """A block with a NaN scale makes its row (of A) or column (of B) NaN, the
    zero codes beside it included, and nothing else."""
    say("mx nan scales m=%d" % m)
    a, b = _draw(m, 300, 1), _draw(150, 300, 2)
    a[m - 1, 290] = float("inf")
    b[7, 0] = float("nan")
    ra, _ = fg.gift_mx_quantize(a.to(DEV), by_row=True)
    rb, _ = fg.gift_mx_quantize(b.to(DEV), by_row=True)
    c = host(fg.gift_mx_matmul(ra, rb, dtype=torch.float32))
    want = np.zeros((m, 150), dtype=bool)
    want[m - 1] = True
    want[:, 7] = True
    assert np.array_equal(np.isnan(c), want)


@pytest.mark.parametrize("m", [3, 100])
def test_scale_range(m):
    """Scales far apart: products from 2^-120 to 2^120, exact in fp32."""
    say("mx scale range m=%d" % m)
    k = 128
    for ea, eb in ((-60, -60), (60, 60), (-120, 118), (120, -118), (0, -100)):
        a = torch.zeros(m, k)
        a[:, ::7] = 3.0 * 2.0 ** ea
        b = torch.zeros(70, k)
        b[:, ::7] = -1.5 * 2.0 ** eb
        ra, _ = fg.gift_mx_quantize(a.to(DEV), by_row=True)
        rb, _ = fg.gift_mx_quantize(b.to(DEV), by_row=True)
        c = host(fg.gift_mx_matmul(ra, rb, dtype=torch.float32)).astype(np.float64)
        assert np.all(c == -4.5 * len(range(0, k, 7)) * 2.0 ** (ea + eb))


def test_side_stream_and_graph():
    """The calls on another stream, and captured: replays equal eager calls,
    with eager work between them, and read the live inputs."""
    say("mx stream and graph")
    x, w, dy = (_draw(*s, dtype=BF16).to(DEV) for s in ((200, 384, 1), (320, 384, 2), (200, 320, 3)))

    def step(buf=None):
        xr, xc = fg.gift_mx_quantize(x, by_row=True, by_col=True)
        wr, wc = fg.gift_mx_quantize(w, by_row=True, by_col=True)
        gr, gc = fg.gift_mx_quantize(dy, by_row=True, by_col=True)
        return (fg.gift_mx_matmul(xr, wr), fg.gift_mx_matmul(gr, wc),
                fg.gift_mx_matmul(gc, xc, dtype=torch.float32), fg.gift_mx_linear(x[:4], wr))
    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    xr, _ = fg.gift_mx_quantize(x, by_row=True, stream=side)
    wr, _ = fg.gift_mx_quantize(w, by_row=True, stream=side)
    y = fg.gift_mx_matmul(xr, wr, stream=side)
    side.synchronize()
    assert torch.equal(y, want[0])
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for rep in range(3):
        for t in got:
            t.fill_(float("nan"))
        step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), rep
    x.mul_(2.0)   # a power of two: the same codes, scales one step up
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0] * 2) and torch.equal(got[1], want[1])
    assert torch.equal(got[2], want[2] * 2)


def _rows_near(c, a, b, rows, half_step):
    """Rows of c against fp64 products of the decoded rows of a and all of b."""
    va = fg.gift_mx_dequantize(fg.gift_mx_quantize(a[rows].contiguous(), by_row=True)[0]).double()
    vb = fg.gift_mx_dequantize(fg.gift_mx_quantize(b, by_row=True)[0]).double()
    want, tol = va @ vb.t(), 2 * a.shape[1] * 2.0 ** -23 * (va.abs() @ vb.abs().t())
    return bool(((c[rows].double() - want).abs() <= tol + half_step * (want.abs() + tol)).all())


def test_offsets_past_32_bits():
    """An X of 4.9 G elements and its operands of 2.6 GB, and a C of 4.9 G
    elements: rows at both ends and in the middle."""
    say("mx large offsets")
    rows, cols = 40000, 122000
    x = torch.empty(rows, cols, dtype=BF16, device=DEV).normal_()
    r, c = fg.gift_mx_quantize(x, by_row=True, by_col=True)
    assert r.data.numel() > 2 ** 31 and c.data.numel() > 2 ** 31
    pick = torch.tensor([0, 1, rows // 2, rows - 65, rows - 1], device=DEV)
    back = fg.gift_mx_dequantize(r, dtype=BF16)
    few, _ = fg.gift_mx_quantize(x[pick].contiguous(), by_row=True)
    assert torch.equal(back[pick], fg.gift_mx_dequantize(few, dtype=BF16))
    del back
    back = fg.gift_mx_dequantize(c, dtype=BF16)
    edge = x[:, cols - 200:].t().contiguous()
    last, _ = fg.gift_mx_quantize(edge, by_row=True)
    assert torch.equal(back[cols - 200:], fg.gift_mx_dequantize(last, dtype=BF16))
    del back, c
    for n in (16, 700):   # small products, and tiles
        w = torch.randn(n, cols, device=DEV)
        wr, _ = fg.gift_mx_quantize(w, by_row=True)
        y = fg.gift_mx_matmul(r, wr, dtype=torch.float32)
        assert _rows_near(y, x, w, pick, 0.0)
    del x, r, y
    a, b = torch.randn(70000, 96, device=DEV), torch.randn(70001, 96, device=DEV)
    ra, rb = (fg.gift_mx_quantize(t, by_row=True)[0] for t in (a, b))
    out = fg.gift_mx_matmul(ra, rb)
    assert _rows_near(out, a, b, torch.tensor([0, 35000, 69999], device=DEV), 2.0 ** -8)


@pytest.mark.parametrize("m,n,k", [(1100, 3001, 1100), (4000, 4090, 300), (1000, 1101, 16000)])
def test_nan_scales_and_far_scales_in_tiles(m, n, k):
    """As the two tests above for products cut into tiles and split sums."""
    say("mx nan and far scales %dx%dx%d" % (m, n, k))
    a, b = torch.zeros(m, k, device=DEV), torch.zeros(n, k, device=DEV)
    a[:, ::7], b[:, ::7] = 3.0 * 2.0 ** -120, -1.5 * 2.0 ** 118
    a[m // 2, k - 1], b[7, 0] = float("inf"), float("nan")
    ra, _ = fg.gift_mx_quantize(a, by_row=True)
    rb, _ = fg.gift_mx_quantize(b, by_row=True)
    c = fg.gift_mx_matmul(ra, rb, dtype=torch.float32)
    want = torch.full_like(c, -4.5 * len(range(0, k, 7)) * 2.0 ** -2)
    want[m // 2], want[:, 7] = float("nan"), float("nan")
    assert torch.equal(torch.isnan(c), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(c), torch.nan_to_num(want))


def test_tiles_on_two_streams_and_in_two_graphs():
    """Products that need a workspace, two at once on two streams, and in two
    captured graphs that share one workspace and run one after the other."""
    say("mx two streams, two graphs")
    ops = [fg.gift_mx_quantize(_draw(*s).to(DEV), by_row=True)[0] for s in
           ((1000, 16000, 1), (1101, 16000, 2), (1000, 16000, 3))]
    need = fg.gift_mx_matmul_workspace_bytes(1000, 1101, 16000)
    assert need > 0
    want = [fg.gift_mx_matmul(ops[i], ops[1], dtype=torch.float32) for i in (0, 2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(3):
        for i, s in enumerate(streams):
            got[i].append(fg.gift_mx_matmul(ops[2 * i], ops[1], dtype=torch.float32, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i]) for i in range(2) for g in got[i])
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    graphs, outs = [], []
    for i in range(2):
        out = torch.empty(1000, 1101, device=DEV)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            fg.gift_mx_matmul(ops[2 * i], ops[1], out=out, ws=ws)
        graphs.append(graph)
        outs.append(out)
    for rep in range(3):
        for out in outs:
            out.fill_(float("nan"))
        ws.fill_(255)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), rep


def test_quantize_of_very_many_tiles():
    """34 G elements: rows at both ends and in the middle of both operands."""
    say("mx very many tiles")
    rows, cols = 2 ** 23 + 70, 4100
    x = torch.ones(1, dtype=BF16, device=DEV).expand(rows, cols).contiguous()
    pick = torch.tensor([0, 1, rows // 2, rows - 71, rows - 1], device=DEV)
    x[pick] = _draw(5, cols, 1, BF16).to(DEV)
    r, _ = fg.gift_mx_quantize(x, by_row=True)
    few, _ = fg.gift_mx_quantize(x[pick].contiguous(), by_row=True)
    want = fg.gift_mx_dequantize(few, dtype=BF16)
    for i, row in enumerate(pick.tolist()):   # the operand's panel of that row
        step = r.data.numel() // -(-rows // 64)
        panel = fg.MxOperand(64, cols, data=r.data[row // 64 * step:][:step])
        assert torch.equal(fg.gift_mx_dequantize(panel, dtype=BF16)[row % 64], want[i])
    del r
    _, c = fg.gift_mx_quantize(x, by_col=True)
    edge = x[-(rows % 128) - 128:].t().contiguous()   # whole steps to the end
    last = fg.gift_mx_quantize(edge, by_row=True)[0].data.view(-1, 2, 4352)
    assert torch.equal(c.data.view(-1, -(-rows // 128), 4352)[:, -2:], last)

"""GPU parity of the products of microscaled matrices against their float64
definitions: formats, shapes, epilogues, microscaled outputs, every way of a product."""
import pytest
import torch

from tests import dense_ref as R
from tests import mx_ref as X

pytestmark = pytest.mark.gpu
rvq = pytest.importorskip("moe_expert_ffn_router_gb300")
DEV = "cuda"
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
F8, F4 = X.F8, X.F4
U = R.U32
FORMATS = [(F8, F8), (F4, F4), (F8, F4), (F4, F8)]


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(shape, g, std=1.0, dtype=F32):
    return (torch.randn(shape, device=DEV, generator=g) * std).to(dtype)


def workspace(n, rows, cols, gated=False):
    f = rvq.moe_mx_gated_linear_workspace_bytes if gated else rvq.moe_mx_linear_workspace_bytes
    ws = torch.zeros(f(n, rows, cols), dtype=torch.uint8, device=DEV)
    assert ws.numel() >= 256
    return ws


def product(x, w):
    """x w^T and the bound of its fp32 sums: products of codes and scales are exact, and
    each of the depth / 16 accumulations, and of the few joins of split sums, is off by
    at most two units of the last place (2^-22) of the sum of magnitudes."""
    return x @ w.t(), (x.shape[1] / 16 + 16) * 2.0 ** -22 * (x.abs() @ w.abs().t())


def want_linear(x, w, bias, name, alpha, residual, dtype):
    p, ep = product(x, w)
    if bias is not None:
        p = p + bias.double()
    ep = ep + 2 * U * p.abs()
    v = alpha * R.act(name, p)
    # every activation's slope is within [-0.2, 1.2]; its evaluation is good to a few
    # units of fp32 of max(|v|, |p|)
    ev = abs(alpha) * (1.2 * ep + 16 * U * p.abs()) + 4 * U * v.abs()
    if residual is not None:
        v = v + residual.double()
    return v, ev + (R.half_step(dtype) + 2 * U) * v.abs() + R.tiny(dtype)


def want_gated(x, wg, wu, bg, bu, name):
    (g, eg), (u, eu) = product(x, wg), product(x, wu)
    if bg is not None:
        g = g + bg.double()
    if bu is not None:
        u = u + bu.double()
    eg, eu = eg + 2 * U * g.abs(), eu + 2 * U * u.abs()
    a = R.act(name, g)
    ea = 1.2 * eg + 16 * U * g.abs()
    v = a * u
    return v, ea * u.abs() + a.abs() * eu + ea * eu + 2 * U * v.abs()


def run_linear(n, rows, cols, xf, wf, act="none", alpha=1.0, bias=False, res=None, out=F32, seed=0):
    g = gen(seed + n * 31 + rows * 7 + cols)
    x, xs, vx = X.random_mx(n, cols, xf, g)
    w, ws_, vw = X.random_mx(rows, cols, wf, g, std=cols ** -0.5)
    b = normal((rows,), g, 0.5) if bias else None
    r = None if res is None else normal((n, rows), g, 1.0, res)
    o = torch.full((n, rows), 99.0, dtype=out, device=DEV)
    ws = workspace(n, rows, cols)
    rvq.moe_mx_linear(x, xs, w, ws_, n, rows, cols, o, ws, xfmt=xf, wfmt=wf, bias=b,
                      act=rvq.MOE_ACTS[act], alpha=alpha, residual=r)
    assert rvq.rvq_ws_status(ws) == (0, 0)
    R.check(o, want_linear(vx, vw, b, act, alpha, r, out), f"{n} {rows} {cols}")


def run_gated(n, rows, cols, xf, wf, act="silu", bias=False, out=BF, ofmt=None, seed=0):
    g = gen(seed + n * 31 + rows * 7 + cols)
    x, xs, vx = X.random_mx(n, cols, xf, g)
    wg, wgs, vg = X.random_mx(rows, cols, wf, g, std=cols ** -0.5)
    wu, wus, vu = X.random_mx(rows, cols, wf, g, std=cols ** -0.5)
    bg = normal((rows,), g, 0.5) if bias else None
    bu = normal((rows,), g, 0.5) if bias else None
    ws = workspace(n, rows, cols, True)
    kw = dict(xfmt=xf, wfmt=wf, bg=bg, bu=bu, act=rvq.MOE_ACTS[act])
    v, e = want_gated(vx, vg, vu, bg, bu, act)
    if ofmt is None:
        o = torch.full((n, rows), 99.0, dtype=out, device=DEV)
        rvq.moe_mx_gated_linear(x, xs, wg, wgs, wu, wus, n, rows, cols, o, ws, **kw)
        R.check(o, (v, e + R.half_step(out) * 1.001 * v.abs() + R.tiny(out)), f"{n} {rows} {cols}")
    else:
        c = torch.full((rvq.moe_mx_code_bytes(ofmt, n, rows),), 0xEE, dtype=torch.uint8, device=DEV)
        s = torch.full((rvq.moe_mx_scale_bytes(n, rows),), 0xEE, dtype=torch.uint8, device=DEV)
        rvq.moe_mx_gated_linear(x, xs, wg, wgs, wu, wus, n, rows, cols, c, ws, out_scales=s,
                                ofmt=ofmt, **kw)
        X.check_quantized(c, s, n, rows, ofmt, v, e, f"{n} {rows} {cols}")
        blocks = X.from_tiles(s, X.up(n, 128), rows)
        assert (blocks[n:] == 0xEE).all()
        assert (blocks[:n, X.up(rows, 32) // 32:] == 0).all()
    assert rvq.rvq_ws_status(ws) == (0, 0)


@pytest.mark.parametrize("xf,wf", FORMATS)
@pytest.mark.parametrize("n,rows,cols", [(16, 128, 128), (1, 128, 256), (1, 8, 8), (3, 40, 136),
                                         (17, 264, 520), (64, 136, 2048), (100, 1000, 328),
                                         (128, 384, 1024), (129, 256, 256), (300, 520, 904)])
def test_linear(n, rows, cols, xf, wf):
    run_linear(n, rows, cols, xf, wf)


@pytest.mark.parametrize("xf,wf", FORMATS)
@pytest.mark.parametrize("n,rows,cols", [(1, 128, 512), (2, 8, 8), (5, 72, 264), (64, 256, 2048),
                                         (33, 520, 1736), (200, 136, 392)])
def test_gated(n, rows, cols, xf, wf):
    run_gated(n, rows, cols, xf, wf)


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("n", [7, 260])
def test_linear_epilogue(n, act):
    run_linear(n, 264, 392, F8, F4, act=act, alpha=0.5, bias=True, res=F32, out=BF)
    run_linear(n, 264, 392, F4, F4, act=act, bias=True, res=BF, out=F32)
    run_linear(n, 136, 392, F4, F4, act=act, alpha=-2.0, res=HF, out=HF)


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("n,rows,cols", [(3, 72, 264), (130, 200, 520), (517, 384, 256)])
def test_gated_epilogue(n, rows, cols, act):
    run_gated(n, rows, cols, F8, F4, act=act, bias=True, out=HF)
    run_gated(n, rows, cols, F4, F4, act=act, out=F32)
    for ofmt in (F8, F4):
        run_gated(n, rows, cols, F4, F4, act=act, bias=True, ofmt=ofmt)
        run_gated(n, rows, cols, F8, F4, act=act, ofmt=ofmt)


@pytest.mark.parametrize("ofmt", [F8, F4])
@pytest.mark.parametrize("n,rows,cols", [(1, 8, 8), (1, 2048, 1024), (64, 1000, 512),
                                         (300, 136, 264)])
def test_gated_into_microscaled(n, rows, cols, ofmt):
    run_gated(n, rows, cols, F8, F4, ofmt=ofmt)
    run_gated(n, rows, cols, F4, F4, ofmt=ofmt)


def test_strides_and_residual_in_place():
    """Outputs and residuals that are columns of wider matrices; the residual's place."""
    n, rows, cols = 70, 136, 264
    g = gen(11)
    x, xs, vx = X.random_mx(n, cols, F8, g)
    w, ws_, vw = X.random_mx(rows, cols, F4, g, std=cols ** -0.5)
    for m in (n, 1):
        xm = x.view(n, -1)[:m].contiguous()
        xsm = X.to_tiles(X.from_tiles(xs, n, cols)[:m])
        ws = workspace(m, rows, cols)
        wide = normal((m, 512), g, 1.0, BF)
        keep = wide.clone()
        o = wide[:, 64:64 + rows]
        rvq.moe_mx_linear(xm, xsm, w, ws_, m, rows, cols, o, ws, residual=o)
        R.check(o, want_linear(vx[:m], vw, None, "none", 1.0, keep[:, 64:64 + rows], BF), "in place")
        assert torch.equal(wide[:, :64], keep[:, :64])
        assert torch.equal(wide[:, 64 + rows:], keep[:, 64 + rows:])
    res = normal((n, 2 * rows), g, 1.0, F32)
    o = torch.zeros((n, rows + 8), dtype=HF, device=DEV)
    ws = workspace(n, rows, cols)
    rvq.moe_mx_linear(x, xs, w, ws_, n, rows, cols, o[:, :rows], ws, residual=res[:, rows:])
    R.check(o[:, :rows], want_linear(vx, vw, None, "none", 1.0, res[:, rows:], HF), "strided")
    assert (o[:, rows:] == 0).all()


@pytest.mark.parametrize("n", [3, 400])
def test_nan_blocks(n):
    """A block of NaN spoils its token's outputs (or its weight row's) and no other."""
    rows, cols = 136, 520
    g = gen(5)
    for xf in (F8, F4):
        x, xs, vx = X.random_mx(n, cols, xf, g)
        w, ws_, vw = X.random_mx(rows, cols, F4, g, std=cols ** -0.5)
        bx, bw = X.from_tiles(xs, n, cols), X.from_tiles(ws_, rows, cols)
        bx[n // 2, 7] = 255
        bw[77, 3] = 255
        o = torch.zeros((n, rows), device=DEV)
        ws = workspace(n, rows, cols)
        rvq.moe_mx_linear(x, X.to_tiles(bx), w, X.to_tiles(bw), n, rows, cols, o, ws, xfmt=xf)
        bad = torch.zeros((n, rows), dtype=torch.bool, device=DEV)
        bad[n // 2], bad[:, 77] = True, True
        assert torch.equal(o.isnan(), bad)
        v, e = want_linear(vx, vw, None, "none", 1.0, None, F32)
        assert ((o.double() - v).abs() <= e)[~bad].all()


def test_scales_far_apart():
    """Scales from the smallest to large ones in one row: the sums keep the large."""
    n, rows, cols = 20, 40, 256
    g = gen(8)
    for xf, wf in FORMATS:
        x, xs, _ = X.random_mx(n, cols, xf, g)
        w, ws_, _ = X.random_mx(rows, cols, wf, g)
        bx, bw = X.from_tiles(xs, n, cols), X.from_tiles(ws_, rows, cols)
        bx[:, 1], bx[:, 2], bx[3] = 0, 160, 20
        bw[:, 5], bw[:, 6] = 30, 0
        xs, ws_ = X.to_tiles(bx), X.to_tiles(bw)
        vx = X.dequantize(x.view(-1), xs, n, cols, xf)
        vw = X.dequantize(w.view(-1), ws_, rows, cols, wf)
        o = torch.zeros((n, rows), device=DEV)
        ws = workspace(n, rows, cols)
        rvq.moe_mx_linear(x, xs, w, ws_, n, rows, cols, o, ws, xfmt=xf, wfmt=wf)
        R.check(o, want_linear(vx, vw, None, "none", 1.0, None, F32), f"{xf} {wf}")


def test_streams_and_graph():
    """Two calls at once on two streams (own workspaces), and a captured call replayed
    on new inputs."""
    rows, cols = 520, 1040
    g = gen(21)
    w, ws_, vw = X.random_mx(rows, cols, F4, g, std=cols ** -0.5)
    for n in (9, 333):
        ins = [X.random_mx(n, cols, F8, g) for _ in range(3)]
        outs = [torch.zeros((n, rows), device=DEV) for _ in range(3)]
        wss = [workspace(n, rows, cols) for _ in range(3)]
        streams = [torch.cuda.Stream() for _ in range(2)]
        torch.cuda.synchronize()
        for _ in range(5):
            for i, s in enumerate(streams):
                rvq.moe_mx_linear(ins[i][0], ins[i][1], w, ws_, n, rows, cols, outs[i], wss[i],
                                  stream=s)
        torch.cuda.synchronize()
        for i in range(2):
            R.check(outs[i], want_linear(ins[i][2], vw, None, "none", 1.0, None, F32), f"stream {i}")
        x, xs = ins[2][0].clone(), ins[2][1].clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            rvq.moe_mx_linear(x, xs, w, ws_, n, rows, cols, outs[2], wss[2])
        for i in range(3):
            x.copy_(ins[i][0])
            xs.copy_(ins[i][1])
            outs[2].zero_()
            graph.replay()
            torch.cuda.synchronize()
            R.check(outs[2], want_linear(ins[i][2], vw, None, "none", 1.0, None, F32), "graph")
            if i < 2:
                assert torch.equal(outs[2], outs[i])
        assert all(rvq.rvq_ws_status(s) == (0, 0) for s in wss)


def test_together():
    """A block's chain: norm join -> gated -> linear, against the chain in float64 of the
    values that each call was given."""
    n, d, f = 37, 520, 264
    g = gen(31)
    y, h = normal((n, d), g, 0.5, BF), normal((n, d), g, 2.0)
    wg, wgs, vg = X.random_mx(f, d, F4, g, std=d ** -0.5)
    wu, wus, vu = X.random_mx(f, d, F4, g, std=d ** -0.5)
    wd, wds, vd = X.random_mx(d, f, F4, g, std=f ** -0.5)

    def new(rows, cols):
        return (torch.zeros(rvq.moe_mx_code_bytes(F8, rows, cols), dtype=torch.uint8, device=DEV),
                torch.zeros(rvq.moe_mx_scale_bytes(rows, cols), dtype=torch.uint8, device=DEV))

    (xc, xs), (hc, hs) = new(n, d), new(n, f)
    ho, out = torch.zeros((n, d), device=DEV), torch.zeros((n, d), device=DEV)
    ws = workspace(n, max(d, f), max(d, f), True)
    rvq.moe_norm_join_mx(y, n, d, ho, xc, xs, h=h, post_norm=False)
    rvq.moe_mx_gated_linear(xc, xs, wg, wgs, wu, wus, n, f, d, hc, ws, out_scales=hs)
    rvq.moe_mx_linear(hc, hs, wd, wds, n, d, f, out, ws, residual=ho)
    vx = X.dequantize(xc, xs, n, d, F8)
    v, e = want_gated(vx, vg, vu, None, None, "silu")
    X.check_quantized(hc, hs, n, f, F8, v, e, "hidden")
    vh = X.dequantize(hc, hs, n, f, F8)
    R.check(out, want_linear(vh, vd, None, "none", 1.0, ho, F32), "out")
    assert rvq.rvq_ws_status(ws) == (0, 0)


@pytest.mark.parametrize("xf,wf", FORMATS)
@pytest.mark.parametrize("n,rows,cols", [(257, 8, 8), (512, 256, 256), (1025, 520, 2056),
                                         (4100, 1304, 264)])
def test_many_tokens(n, rows, cols, xf, wf):
    """Tiles of CTA pairs: one, several per pair (102 of the last), ragged in every way."""
    run_linear(n, rows, cols, xf, wf)
    run_gated(n, rows, cols, xf, wf)


@pytest.mark.parametrize("n,rows,cols", [(513, 264, 520), (4100, 712, 136)])
def test_many_tokens_epilogue(n, rows, cols):
    run_linear(n, rows, cols, F8, F4, act="gelu", alpha=0.5, bias=True, res=F32, out=BF)
    run_linear(n, rows, cols, F4, F4, act="silu", res=BF, out=F32)
    run_linear(n, rows, cols, F4, F4, bias=True, out=HF)
    run_gated(n, rows, cols, F8, F4, bias=True, out=F32)
    for ofmt in (F8, F4):
        run_gated(n, rows, cols, F8, F4, bias=True, ofmt=ofmt)
        run_gated(n, rows, cols, F4, F4, act="gelu_tanh", ofmt=ofmt)


# one shape for every way of a product: (gated, formats, n, rows, cols)
WAYS = {("stream", 1): (False, F8, F4, 5, 136, 264), ("stream", 2): (False, F8, F4, 9, 264, 520),
        ("stream", 4): (True, F8, F4, 40, 136, 1040), ("stream", 8): (True, F4, F4, 3, 264, 4360),
        ("tiles", 1): (False, F8, F4, 2040, 2040, 1032)}
MORE_WAYS = [(("stream", 1), (True, F4, F4, 20, 136, 520)),
             (("stream", 4), (True, F8, F4, 200, 1032, 2056)),
             (("stream", 8), (False, F8, F8, 128, 1000, 2056)),
             (("tiles", 1), (True, F4, F4, 1100, 1032, 520))]


@pytest.mark.parametrize("way,case", list(WAYS.items()) + MORE_WAYS)
def test_ways(way, case):
    """Streams whole and split among two, four and eight CTAs, and tiles: the shapes take
    the way they are meant for."""
    gated, xf, wf, n, rows, cols = case
    assert rvq.rvq_selftest_mx_plan(gated, xf, wf, n, rows, cols) == way
    if gated:
        run_gated(n, rows, cols, xf, wf, bias=True)
        run_gated(n, rows, cols, xf, wf, ofmt=F8)
    else:
        run_linear(n, rows, cols, xf, wf, bias=True, act="silu", res=F32)


@pytest.mark.parametrize("xf,wf", [(F8, F4), (F4, F4)])
def test_partial_tiles_that_fit_an_sm_once(xf, wf):
    """Gated products of 111 and 112 tokens: their partial tile is longer than the ring and
    does not fit an SM twice, so the depth is split as for 113 to 128 tokens, which take an
    SM alone too; and the outputs around that border."""
    alone = rvq.rvq_selftest_mx_plan(True, xf, wf, 128, 2048, 7168)
    for n in (111, 112, 113):
        assert rvq.rvq_selftest_mx_plan(True, xf, wf, n, 2048, 7168) == alone
    for n in (110, 111, 112, 113):
        run_gated(n, 264, 1024, xf, wf, out=F32)
        run_gated(n, 264, 1024, xf, wf, ofmt=F8)
    run_gated(112, 2048, 1024, xf, wf)

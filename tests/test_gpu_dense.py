"""GPU parity of moe_linear, moe_gated_linear and their gradients against the
float64 definitions, at sizes around every tile edge, with row pitches, partly
filled tiles, NaN beside the matrices, side streams and CUDA graphs."""
import pytest
import torch

from tests import dense_ref as R

pytestmark = pytest.mark.gpu
rvq = pytest.importorskip("moe_expert_ffn_router_gb300")
DEV = "cuda"
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, device=DEV, generator=g) * std).to(dtype)


def padded(t, extra):
    """The same values as a view of a wider tensor whose padding is NaN, with a
    NaN row before and after."""
    if extra == 0:
        return t
    r, c = t.shape
    big = torch.full((r + 2, c + extra), float("nan"), dtype=t.dtype, device=t.device)
    v = big[1:1 + r, :c]
    v.copy_(t)
    return v


def hole(shape, dtype, extra):
    """An output as a view of a tensor filled with a marker, and the tensor."""
    r, c = shape
    big = torch.full((r + 2, c + extra), -77.0, dtype=dtype, device=DEV)
    return big[1:1 + r, :c], big


def untouched(big, view):
    """Only the view's elements were written."""
    v = view.clone()
    view.fill_(-77.0)
    ok = bool((big == -77.0).all())
    view.copy_(v)
    return ok


def workspace(n, rows, cols, gated=False):
    f = rvq.moe_gated_linear_workspace_bytes if gated else rvq.moe_linear_workspace_bytes
    ws = torch.empty(f(n, rows, cols, True), dtype=torch.uint8, device=DEV)
    rvq.rvq_ws_clear(ws)
    return ws


# tokens around the tile edges; features from one group of eight to several
# tiles, with odd multiples of eight
SIZES = [(1, 8, 8), (1, 256, 512), (2, 136, 72), (7, 256, 512), (8, 1000, 1736), (9, 264, 4104),
         (16, 2048, 1024), (31, 72, 1000), (33, 520, 264), (64, 2056, 520), (65, 128, 64),
         (127, 136, 200), (128, 1024, 2048), (129, 264, 136), (200, 1000, 648), (256, 512, 256),
         (257, 2008, 1096), (300, 8, 2048), (511, 384, 1160), (1333, 1000, 2048),
         (2049, 3000, 328)]


@pytest.mark.parametrize("n,rows,cols", SIZES)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_linear_forward(n, rows, cols, dtype):
    g = gen(n * 7 + rows)
    extra = 8 * (n % 3)
    x, w = padded(normal(g, (n, cols), dtype), extra), padded(
        normal(g, (rows, cols), dtype, cols ** -0.5), 2 * extra)
    out, big = hole((n, rows), dtype, extra)
    ws = workspace(n, rows, cols)
    rvq.moe_linear(x, w, n, rows, cols, out, ws)
    want, _ = R.linear(x, w, None, "none", 1.0, None, dtype)
    R.check(out, want, "out", 1.0)
    assert untouched(big, out)
    assert rvq.rvq_ws_status(ws) == (0, 0)


@pytest.mark.parametrize("act", R.ACTS)
@pytest.mark.parametrize("n,rows,cols", [(1, 264, 520), (5, 1000, 328), (70, 136, 1032),
                                         (300, 520, 264)])
def test_linear_epilogue(act, n, rows, cols):
    """Bias, activation, scale and residual of every type mix, and pre."""
    g = gen(rows + n)
    x, w = normal(g, (n, cols), BF), normal(g, (rows, cols), BF, cols ** -0.5)
    bias = normal(g, (rows,), BF)
    ws = workspace(n, rows, cols)
    code = rvq.MOE_ACTS[act]
    for rdt, odt, alpha in ((BF, BF, 1.0), (F32, F32, -0.5), (HF, F32, 2.0), (F32, BF, 0.25),
                            (None, F32, 1.0), (None, HF, 1.5)):
        res = None if rdt is None else padded(normal(g, (n, rows), rdt), 8)
        out, big = hole((n, rows), odt, 16)
        pre = torch.empty((n, rows), dtype=F32, device=DEV)
        rvq.moe_linear(x, w, n, rows, cols, out, ws, bias=bias, act=code, alpha=alpha,
                       residual=res, pre=pre)
        want, wpre = R.linear(x, w, bias, act, alpha, res, odt)
        R.check(out, want, f"out {rdt} {odt}")
        R.check(pre, wpre, "pre")
        assert untouched(big, out)
        if res is not None and rdt == odt:   # in place over the residual
            inplace = res.clone()
            rvq.moe_linear(x, w, n, rows, cols, inplace, ws, bias=bias, act=code, alpha=alpha,
                           residual=inplace)
            assert torch.equal(inplace, out)


@pytest.mark.parametrize("n,rows,cols", SIZES)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_gated_forward(n, rows, cols, dtype):
    g = gen(n * 5 + rows)
    extra = 8 * (n % 2)
    x = padded(normal(g, (n, cols), dtype), extra)
    wg = padded(normal(g, (rows, cols), dtype, cols ** -0.5), extra)
    wu = padded(normal(g, (rows, cols), dtype, cols ** -0.5), extra)
    act = R.ACTS[(n + rows // 8) % 5]
    bg = normal(g, (rows,), dtype) if n % 2 else None
    bu = normal(g, (rows,), dtype) if n % 4 > 1 else None
    out, big = hole((n, rows), dtype, extra)
    pre = torch.empty((2, n, rows), dtype=F32, device=DEV)
    ws = workspace(n, rows, cols, True)
    rvq.moe_gated_linear(x, wg, wu, n, rows, cols, out, ws, bg=bg, bu=bu,
                         act=rvq.MOE_ACTS[act], pre=pre)
    want, wg_, wu_ = R.gated(x, wg, wu, bg, bu, act)
    R.check(out, want, "out", 1.05)
    R.check(pre[0], wg_, "pre g")
    R.check(pre[1], wu_, "pre u")
    assert untouched(big, out)
    again = torch.empty((n, rows), dtype=dtype, device=DEV)   # without pre: the same values
    rvq.moe_gated_linear(x, wg, wu, n, rows, cols, again, ws, bg=bg, bu=bu,
                         act=rvq.MOE_ACTS[act])
    assert torch.equal(again, out)
    assert rvq.rvq_ws_status(ws) == (0, 0)


@pytest.mark.parametrize("n,rows,cols", [(193, 256, 1024), (257, 520, 4096), (112, 7168, 1024),
                                         (113, 512, 1024), (65, 512, 2048), (600, 1000, 2048)])
def test_every_way_of_a_product(n, rows, cols):
    """Tokens at the ends of the stream of weights and of tiles cut by slices:
    the same epilogue in each (bias, activation, scale, residual, pre)."""
    g = gen(n)
    x, w, w2 = normal(g, (n, cols), BF), normal(g, (rows, cols), BF, cols ** -0.5), \
        normal(g, (rows, cols), BF, cols ** -0.5)
    bias, bias2, res = normal(g, (rows,), BF), normal(g, (rows,), BF), normal(g, (n, rows), F32)
    ws = workspace(n, rows, cols)
    out, big = hole((n, rows), BF, 8)
    pre = torch.empty((n, rows), dtype=F32, device=DEV)
    rvq.moe_linear(x, w, n, rows, cols, out, ws, bias=bias, act=rvq.MOE_ACT_GELU, alpha=0.5,
                   residual=res, pre=pre)
    want, wpre = R.linear(x, w, bias, "gelu", 0.5, res, BF)
    R.check(out, want, "out")
    R.check(pre, wpre, "pre")
    assert untouched(big, out)
    ws2 = workspace(n, rows, cols, True)
    gout, gbig = hole((n, rows), BF, 8)
    pre2 = torch.empty((2, n, rows), dtype=F32, device=DEV)
    rvq.moe_gated_linear(x, w, w2, n, rows, cols, gout, ws2, bg=bias, bu=bias2,
                         act=rvq.MOE_ACT_GELU_TANH, pre=pre2)
    wg, (g0, e0), (g1, e1) = R.gated(x, w, w2, bias, bias2, "gelu_tanh")
    R.check(gout, wg, "gated out")
    R.check(pre2[0], (g0, e0), "g")
    R.check(pre2[1], (g1, e1), "u")
    assert untouched(gbig, gout)
    assert rvq.rvq_ws_status(ws) == (0, 0) and rvq.rvq_ws_status(ws2) == (0, 0)


def linear_train(n, rows, cols, dtype, act, bias, alpha=1.0, seed=0, extra=0):
    g = gen(seed)
    x = padded(normal(g, (n, cols), dtype), extra)
    w = padded(normal(g, (rows, cols), dtype, cols ** -0.5), extra)
    b = normal(g, (rows,), dtype) if bias else None
    dout = padded(normal(g, (n, rows), dtype, 0.5), extra)
    ws = workspace(n, rows, cols)
    out = torch.empty((n, rows), dtype=dtype, device=DEV)
    pre = torch.empty((n, rows), dtype=F32, device=DEV) if act != "none" else None
    dx, bx = hole((n, cols), dtype, extra)
    dw, bw = hole((rows, cols), dtype, extra)
    db = torch.empty(rows, dtype=dtype, device=DEV) if bias else None
    code = rvq.MOE_ACTS[act]
    rvq.moe_linear(x, w, n, rows, cols, out, ws, bias=b, act=code, alpha=alpha, pre=pre)
    rvq.moe_linear_backward(dout, x, w, n, rows, cols, ws, dx=dx, dw=dw, dbias=db, pre=pre,
                            act=code, alpha=alpha)
    assert rvq.rvq_ws_status(ws) == (0, 0)
    assert untouched(bx, dx) and untouched(bw, dw)
    p, ep = R.product(R.d(x), R.d(w))
    if b is not None:
        p = p + R.d(b)
    ep = ep + 2 * R.U32 * p.abs()
    s = R.slope(act, p)
    dp = alpha * R.d(dout) * s
    edp = abs(alpha) * R.d(dout).abs() * (R.slope_err(p, ep) if act != "none" else 0) \
        + 4 * R.U32 * dp.abs()
    edp = edp + R.near_step(act, p, ep) * abs(alpha) * R.d(dout).abs()
    wdx, outs = R.grads([dp], [edp], x, [w], dtype, act != "none")
    f = 1.05 if act == "none" else 1.25
    R.check(dx, wdx, "dx", f)
    R.check(dw, outs[0][0], "dw", f)
    if bias:
        R.check(db, outs[0][1], "dbias")


@pytest.mark.parametrize("n,rows,cols", SIZES)
def test_linear_gradients(n, rows, cols):
    act = R.ACTS[(n + rows // 8) % 5]
    linear_train(n, rows, cols, BF if n % 2 else HF, act, n % 3 != 0, extra=8 * (n % 2), seed=n)


@pytest.mark.parametrize("act", R.ACTS)
@pytest.mark.parametrize("alpha", [1.0, -1.75])
def test_linear_gradients_scale(act, alpha):
    linear_train(150, 264, 200, BF, act, True, alpha=alpha, seed=3)


def gated_dp(x, wg, wu, bg, bu, dout, act):
    g, eg = R.product(R.d(x), R.d(wg))
    u, eu = R.product(R.d(x), R.d(wu))
    if bg is not None:
        g = g + R.d(bg)
    if bu is not None:
        u = u + R.d(bu)
    eg, eu = eg + 2 * R.U32 * g.abs(), eu + 2 * R.U32 * u.abs()
    do = R.d(dout)
    s, a = R.slope(act, g), R.act(act, g)
    es = R.slope_err(g, eg) + R.near_step(act, g, eg)
    if act == "none":
        es = torch.zeros_like(g)
    ea = 1.2 * eg + 16 * R.U32 * g.abs()
    dg, du = do * u * s, do * a
    edg = do.abs() * (u.abs() * es + eu * s.abs() + eu * es) + 4 * R.U32 * dg.abs()
    return dg, edg, du, do.abs() * ea + 4 * R.U32 * du.abs()


@pytest.mark.parametrize("n,rows,cols", SIZES)
def test_gated_gradients(n, rows, cols):
    dtype = HF if n % 2 else BF
    act = R.ACTS[(n + rows // 8) % 5]
    g = gen(n + 1)
    extra = 8 * (n % 2)
    x = padded(normal(g, (n, cols), dtype), extra)
    wg, wu = (padded(normal(g, (rows, cols), dtype, cols ** -0.5), extra) for _ in range(2))
    bg, bu = ((normal(g, (rows,), dtype), normal(g, (rows,), dtype)) if n % 3 else (None, None))
    dout = padded(normal(g, (n, rows), dtype, 0.5), extra)
    ws = workspace(n, rows, cols, True)
    out = torch.empty((n, rows), dtype=dtype, device=DEV)
    pre = torch.empty((2, n, rows), dtype=F32, device=DEV)
    dx, bx = hole((n, cols), dtype, extra)
    dwg, b1 = hole((rows, cols), dtype, extra)
    dwu, b2 = hole((rows, cols), dtype, extra)
    dbg = torch.empty(rows, dtype=dtype, device=DEV) if bg is not None else None
    dbu = torch.empty(rows, dtype=dtype, device=DEV) if bg is not None else None
    code = rvq.MOE_ACTS[act]
    rvq.moe_gated_linear(x, wg, wu, n, rows, cols, out, ws, bg=bg, bu=bu, act=code, pre=pre)
    rvq.moe_gated_linear_backward(dout, x, wg, wu, pre, n, rows, cols, ws, dx=dx, dwg=dwg, dwu=dwu,
                                  dbg=dbg, dbu=dbu, act=code)
    assert rvq.rvq_ws_status(ws) == (0, 0)
    assert untouched(bx, dx) and untouched(b1, dwg) and untouched(b2, dwu)
    dg, edg, du, edu = gated_dp(x, wg, wu, bg, bu, dout, act)
    wdx, outs = R.grads([dg, du], [edg, edu], x, [wg, wu], dtype)
    R.check(dx, wdx, "dx", 1.25)
    for got, want, what in ((dwg, outs[0][0], "dwg"), (dwu, outs[1][0], "dwu")):
        R.check(got, want, what, 1.25)
    if bg is not None:
        R.check(dbg, outs[0][1], "dbg")
        R.check(dbu, outs[1][1], "dbu")
    # each gradient alone is the same
    only = torch.empty((n, cols), dtype=dtype, device=DEV)
    rvq.moe_gated_linear_backward(dout, x, wg, wu, pre, n, rows, cols, ws, dx=only, act=code)
    assert torch.equal(only, dx)


def test_gated_gradients_against_differences():
    """<gradient, direction> equals central differences of the float64 loss
    sum(dout * out) along random directions, to the gradients' rounding."""
    n, rows, cols, act = 24, 136, 72, "silu"
    g = gen(5)
    x, wg, wu = (normal(g, s, BF, v) for s, v in (((n, cols), 1.0), ((rows, cols), 0.15),
                                                  ((rows, cols), 0.15)))
    dout = normal(g, (n, rows), BF)
    ws = workspace(n, rows, cols, True)
    out = torch.empty((n, rows), dtype=BF, device=DEV)
    pre = torch.empty((2, n, rows), dtype=F32, device=DEV)
    rvq.moe_gated_linear(x, wg, wu, n, rows, cols, out, ws, pre=pre)
    grad = [torch.empty_like(t) for t in (x, wg, wu)]
    rvq.moe_gated_linear_backward(dout, x, wg, wu, pre, n, rows, cols, ws, dx=grad[0], dwg=grad[1],
                                  dwu=grad[2])

    def loss(a, b, c):
        return (dout.double() * R.act(act, a @ b.t()) * (a @ c.t())).sum().item()

    base = [t.double() for t in (x, wg, wu)]
    for i in range(3):
        v = torch.randn(base[i].shape, device=DEV, generator=g, dtype=torch.float64)
        eps = 1e-4
        hi, lo = list(base), list(base)
        hi[i], lo[i] = base[i] + eps * v, base[i] - eps * v
        diff = (loss(*hi) - loss(*lo)) / (2 * eps)
        got = (grad[i].double() * v).sum().item()
        # dp and the result are each rounded to bf16: errors of independent
        # signs, half a step each, over the terms of the sum; 8 deviations
        scale = (grad[i].double().square() * v.square()).sum().sqrt().item()
        assert abs(got - diff) <= 8 * 2 * R.half_step(BF) * scale, (i, got, diff)


@pytest.mark.parametrize("n", [3, 40, 300])
def test_nan_and_inf_stay_in_their_rows(n):
    """A NaN token spoils its own row, a NaN or infinite weight row its own
    column, in the forward and in dx/dw; nothing leaks through tile tails."""
    rows, cols = 200, 136
    g = gen(9)
    x, w = normal(g, (n, cols), BF), normal(g, (rows, cols), BF, 0.1)
    ws = workspace(n, rows, cols)
    clean = torch.empty((n, rows), dtype=BF, device=DEV)
    rvq.moe_linear(x, w, n, rows, cols, clean, ws)
    x2, w2 = x.clone(), w.clone()
    x2[n // 2, 5] = float("nan")
    w2[77, 3] = float("inf")
    out = torch.empty_like(clean)
    rvq.moe_linear(x2, w2, n, rows, cols, out, ws)
    keep_r = torch.arange(n, device=DEV) != n // 2
    keep_c = torch.arange(rows, device=DEV) != 77
    assert torch.equal(out[keep_r][:, keep_c], clean[keep_r][:, keep_c])
    assert torch.isnan(out[n // 2]).all()
    assert not torch.isfinite(out[:, 77]).any()
    dw = torch.empty((rows, cols), dtype=BF, device=DEV)
    dx = torch.empty((n, cols), dtype=BF, device=DEV)
    dout = normal(g, (n, rows), BF)
    rvq.moe_linear_backward(dout, x2, w, n, rows, cols, ws, dx=dx, dw=dw)
    assert torch.isfinite(dx).all()
    bad = torch.isnan(dw)
    assert bad[:, 5].all() and bad.sum() == rows
    do2 = dout.clone()
    do2[n // 2, 11] = float("nan")
    rvq.moe_linear_backward(do2, x, w, n, rows, cols, ws, dx=dx, dw=dw)
    assert torch.isnan(dx[n // 2]).all() and torch.isnan(dx).sum() == cols
    assert torch.isnan(dw[11]).all() and torch.isnan(dw).sum() == cols


def test_results_repeat_and_streams_and_graphs():
    """Bit-equal on repeated calls, on a side stream, and replayed from a CUDA
    graph of forward and backward while the eager buffers live."""
    for n, rows, cols in ((1, 512, 1024), (48, 1000, 520), (777, 648, 1096)):
        g = gen(n)
        x, dout = normal(g, (n, cols), BF), normal(g, (n, rows), BF)
        wg, wu = normal(g, (rows, cols), BF, 0.05), normal(g, (rows, cols), BF, 0.05)
        ws = workspace(n, rows, cols, True)

        def buffers():
            return dict(out=torch.zeros((n, rows), dtype=BF, device=DEV),
                        pre=torch.zeros((2, n, rows), dtype=F32, device=DEV),
                        dx=torch.zeros((n, cols), dtype=BF, device=DEV),
                        dwg=torch.zeros((rows, cols), dtype=BF, device=DEV),
                        dwu=torch.zeros((rows, cols), dtype=BF, device=DEV))

        def step(b, stream=None):
            rvq.moe_gated_linear(x, wg, wu, n, rows, cols, b["out"], ws, pre=b["pre"],
                                 stream=stream)
            rvq.moe_gated_linear_backward(dout, x, wg, wu, b["pre"], n, rows, cols, ws,
                                          dx=b["dx"], dwg=b["dwg"], dwu=b["dwu"], stream=stream)

        first, second, third = buffers(), buffers(), buffers()
        step(first)
        step(second)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        step(third, side)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        for k in first:
            assert torch.equal(first[k], second[k]) and torch.equal(first[k], third[k]), (n, k)
        cap = buffers()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(cap)
        x.copy_(normal(g, (n, cols), BF))
        step(first)
        graph.replay()
        torch.cuda.synchronize()
        for k in first:
            assert torch.equal(first[k], cap[k]), (n, k)
        assert rvq.rvq_ws_status(ws) == (0, 0)


def test_offsets_beyond_32_bits():
    """A view whose last rows lie more than 2^32 elements in, as a slice of a
    large buffer has it: reads and writes land where the pitch says."""
    n, rows, cols = 129, 72, 64
    ld = (1 << 32) // 120 // 8 * 8
    big = torch.zeros(ld * (n - 1) + rows, dtype=BF, device=DEV)   # 9.2 GB
    g = gen(2)
    x, w = normal(g, (n, cols), BF), normal(g, (rows, cols), BF, 0.1)
    res = normal(g, (n, rows), BF)
    strided = big.as_strided((n, rows), (ld, 1))
    strided.copy_(res)
    ws = workspace(n, rows, cols)
    rvq.moe_linear(x, w, n, rows, cols, strided, ws, residual=strided)
    plain = torch.empty((n, rows), dtype=BF, device=DEV)
    rvq.moe_linear(x, w, n, rows, cols, plain, ws, residual=res)
    assert torch.equal(strided, plain)
    dx = torch.empty((n, cols), dtype=BF, device=DEV)
    dx2 = torch.empty_like(dx)
    rvq.moe_linear_backward(strided, x, w, n, rows, cols, ws, dx=dx)
    rvq.moe_linear_backward(plain, x, w, n, rows, cols, ws, dx=dx2)
    assert torch.equal(dx, dx2)


@pytest.mark.parametrize("n,rows,cols", [(3, 264, 200), (300, 1000, 136), (5000, 8, 72),
                                         (700, 4104, 264)])
def test_bias_gradients_beside_any_product(n, rows, cols):
    """The sums of a bias gradient are the same with both products, one or none,
    and with the other bias left out."""
    g = gen(n)
    x, wg, wu = (normal(g, s, BF, v) for s, v in (((n, cols), 1.0), ((rows, cols), cols ** -0.5),
                                                  ((rows, cols), cols ** -0.5)))
    bg, bu = normal(g, (rows,), BF), normal(g, (rows,), BF)
    dout = normal(g, (n, rows), BF, 0.5)
    ws = workspace(n, rows, cols, True)
    out = torch.empty((n, rows), dtype=BF, device=DEV)
    pre = torch.empty((2, n, rows), dtype=F32, device=DEV)
    rvq.moe_gated_linear(x, wg, wu, n, rows, cols, out, ws, bg=bg, bu=bu, pre=pre)
    dg, edg, du, edu = gated_dp(x, wg, wu, bg, bu, dout, "silu")
    _, outs = R.grads([dg, du], [edg, edu], x, [wg, wu], BF)
    first = None
    for products in (("dx", "dwg", "dwu"), ("dx",), ("dwg", "dwu"), ()):
        for biases in (("dbg", "dbu"), ("dbg",), ("dbu",)):
            kw = {k: torch.full((n if k == "dx" else rows, cols), float("nan"), dtype=BF, device=DEV)
                  for k in products}
            kw.update({k: torch.full((rows,), float("nan"), dtype=BF, device=DEV) for k in biases})
            rvq.moe_gated_linear_backward(dout, x, wg, wu, pre, n, rows, cols, ws, **kw)
            assert rvq.rvq_ws_status(ws) == (0, 0)
            if first is None:
                first = kw
                R.check(kw["dbg"], outs[0][1], "dbg")
                R.check(kw["dbu"], outs[1][1], "dbu")
            for k in biases:
                assert torch.equal(kw[k], first[k]), (products, k)


# tiles split among the pairs of a cluster (two or four), ragged and whole
SPLITS = [(250, 856, 1240), (512, 2048, 2048), (1000, 1000, 2040), (385, 712, 2048),
          (129, 520, 3000)]


@pytest.mark.parametrize("n,rows,cols", SPLITS)
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_linear_split_tiles(n, rows, cols, act):
    g = gen(n)
    x, w = normal(g, (n, cols), BF), normal(g, (rows, cols), BF, cols ** -0.5)
    b, res = normal(g, (rows,), BF), normal(g, (n, rows), F32)
    ws = workspace(n, rows, cols)
    out, bo = hole((n, rows), F32 if act == "none" else BF, 8)
    pre = torch.empty((n, rows), dtype=F32, device=DEV)
    rvq.moe_linear(x, w, n, rows, cols, out, ws, bias=b, act=rvq.MOE_ACTS[act], alpha=-0.5,
                   residual=res, pre=pre)
    assert rvq.rvq_ws_status(ws) == (0, 0) and untouched(bo, out)
    p, ep = R.product(R.d(x), R.d(w))
    p = p + R.d(b)
    ep = ep + 2 * R.U32 * p.abs()
    assert ((pre.double() - p).abs() <= ep).all()
    a = R.act(act, p)
    ea = (1.2 * ep + 16 * R.U32 * p.abs()) * 0.5 + 4 * R.U32 * (a.abs() + res.double().abs())
    want = res.double() - 0.5 * a
    tol = ea + torch.finfo(out.dtype).eps / 2 * (want.abs() + ea)
    assert ((out.double() - want).abs() <= tol).all()
    again = torch.empty_like(out)
    rvq.moe_linear(x, w, n, rows, cols, again, ws, bias=b, act=rvq.MOE_ACTS[act], alpha=-0.5,
                   residual=res)
    assert torch.equal(again, out)


@pytest.mark.parametrize("n,rows,cols", [(757, 2000, 336), (300, 1000, 1000), (2999, 256, 264),
                                         (512, 2048, 2048), (161, 520, 1040)])
def test_linear_gradients_split_tiles(n, rows, cols):
    linear_train(n, rows, cols, BF if n % 2 else HF, "silu", True, alpha=0.5, extra=8, seed=n)


@pytest.mark.parametrize("n,rows,cols", [(662, 472, 1344), (400, 800, 3000), (256, 1024, 2048),
                                         (1688, 320, 512), (200, 264, 7168)])
def test_gated_gradients_split_tiles(n, rows, cols):
    test_gated_gradients(n, rows, cols)


def act_error(name, v):
    """Relative error of an activation's evaluation in fp32, in its own terms: the
    hardware exponential is good to 2 + 1.2 |a| units of the last place (2^-23) of
    exp(a), a's own rounding moves it by up to 3 |a| half steps, a division takes two
    units, and a polynomial and the remaining products a few."""
    a = {"silu": v.abs(), "gelu": v * v / 2,
         "gelu_tanh": 1.5957691216057308 * (v + 0.044715 * v ** 3).abs()}[name]
    return (16 + 3 * a) * 2.0 ** -23


def sweep(lo=-9.0, hi=9.0, count=4096):
    """Values as the sum of two bf16 ones, which the products with 1 add up again."""
    v = torch.linspace(lo, hi, count, device=DEV)
    a = v.to(BF)
    b = (v - a.float()).to(BF)
    return a, b


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("tokens_are", ["few", "many"])
def test_activations_are_accurate_in_the_tails(act, tokens_are):
    """Outputs in fp32 are within the evaluation's own relative error of the formula,
    for every pre-activation from -9 to 9."""
    a, b = sweep()
    ones = torch.zeros((8, 8), dtype=BF, device=DEV)
    ones[:, :2] = 1
    wide = torch.zeros((a.numel(), 8), dtype=BF, device=DEV)
    wide[:, 0], wide[:, 1] = a, b
    x, w = (ones[:1].clone(), wide) if tokens_are == "few" else (wide, ones)
    n, rows = x.shape[0], w.shape[0]
    ws = workspace(n, rows, 8)
    out, pre = (torch.empty((n, rows), device=DEV) for _ in range(2))
    rvq.moe_linear(x, w, n, rows, 8, out, ws, act=rvq.MOE_ACTS[act], pre=pre)
    v = (a.double() + b.double()) if tokens_are == "few" else (a.double() + b.double())[:, None]
    assert ((pre.double() - v).abs() <= 2.0 ** -22 * v.abs()).all()
    want = R.act(act, pre.double())
    if act == "gelu_tanh":     # 1 + tanh loses its last digits at -1 in any precision
        want = pre.double() * torch.sigmoid(
            1.5957691216057308 * (pre.double() + 0.044715 * pre.double() ** 3))
    err = (out.double() - want).abs()
    over = err - (act_error(act, pre.double()) * want.abs() + R.tiny(F32))
    i = over.argmax()
    assert (over <= 0).all(), (pre.reshape(-1)[i].item(), out.reshape(-1)[i].item(),
                               want.reshape(-1)[i].item())


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_slopes_are_accurate_in_the_tails(act):
    """dp = dout act'(pre) in bf16, for pre from -9 to 9: half a step, and the
    evaluation's error of the slope's two terms."""
    a, b = sweep()
    n = a.numel()
    pre = (a.float() + b.float())[:, None].expand(n, 8).contiguous()
    eye = torch.eye(8, dtype=BF, device=DEV)
    dx = torch.empty((n, 8), dtype=BF, device=DEV)
    ws = workspace(n, 8, 8)
    rvq.moe_linear_backward(torch.ones((n, 8), dtype=BF, device=DEV), None, eye, n, 8, 8, ws,
                            dx=dx, pre=pre, act=rvq.MOE_ACTS[act])
    v = pre.double()
    arg = {"silu": v, "gelu": None,
           "gelu_tanh": 1.5957691216057308 * (v + 0.044715 * v ** 3)}[act]
    if act == "gelu":
        one, two = 0.5 * torch.special.erfc(-v / 2 ** 0.5), \
            v * torch.exp(-0.5 * v * v) / (2 * torch.pi) ** 0.5
    else:
        da = 1.0 if act == "silu" else 1.5957691216057308 * (1 + 3 * 0.044715 * v * v)
        one = torch.sigmoid(arg)
        two = v * one * torch.sigmoid(-arg) * da
    want = one + two
    # 1 - s of a sigmoid near 1 is good to a half step of 1 only
    err = 2 * act_error(act, v) * (one.abs() + two.abs()) + 4 * R.U32 * (v * v).clamp(min=1) * one
    assert ((dx.double() - want).abs() <= R.half_step(BF) * (want.abs() + err) + err).all()


def test_one_workspace_for_every_batch():
    """A workspace made for the largest batch serves the smaller ones, which are cut
    otherwise, with the same results as one of their own."""
    rows, cols, most = 1000, 4096, 2048
    g = gen(1)
    x, dout = normal(g, (most, cols), BF), normal(g, (most, rows), BF)
    wg, wu = (normal(g, (rows, cols), BF, cols ** -0.5) for _ in range(2))
    big = workspace(most, rows, cols, True)
    for n in (most, 700, 400, 200, 30, 1):
        got = []
        for ws in (big, workspace(n, rows, cols, True)):
            out = torch.empty((n, rows), dtype=BF, device=DEV)
            pre = torch.empty((2, n, rows), dtype=F32, device=DEV)
            dx, dwg, dwu = (torch.empty(s, dtype=BF, device=DEV)
                            for s in ((n, cols), (rows, cols), (rows, cols)))
            rvq.moe_gated_linear(x[:n], wg, wu, n, rows, cols, out, ws, pre=pre)
            rvq.moe_gated_linear_backward(dout[:n], x[:n], wg, wu, pre, n, rows, cols, ws, dx=dx,
                                          dwg=dwg, dwu=dwu)
            assert rvq.rvq_ws_status(ws) == (0, 0)
            got.append((out, pre, dx, dwg, dwu))
        assert all(torch.equal(a, b) for a, b in zip(*got)), n


@pytest.mark.parametrize("n", [3, 300])
def test_columns_of_one_wider_matrix(n):
    """Input, output and residual beside each other in one matrix, and both weight
    gradients in one."""
    rows, cols = 72, 136
    g = gen(n)
    x, res = normal(g, (n, cols), BF), normal(g, (n, rows), BF)
    wide = torch.full((n, cols + 2 * rows), float("nan"), dtype=BF, device=DEV)
    xs, out, rs = wide[:, :cols], wide[:, cols:cols + rows], wide[:, cols + rows:]
    xs.copy_(x)
    rs.copy_(res)
    wg, wu = (normal(g, (rows, cols), BF, cols ** -0.5) for _ in range(2))
    ws = workspace(n, rows, cols, True)
    rvq.moe_linear(xs, wg, n, rows, cols, out, ws, residual=rs)
    R.check(out, R.linear(x, wg, None, "none", 1.0, res, BF)[0], "out")
    assert torch.equal(xs, x) and torch.equal(rs, res)
    pre = torch.empty((2, n, rows), dtype=F32, device=DEV)
    rvq.moe_gated_linear(xs, wg, wu, n, rows, cols, out, ws, pre=pre)
    dw = torch.empty((rows, 2 * cols), dtype=BF, device=DEV)
    apart = [torch.empty((rows, cols), dtype=BF, device=DEV) for _ in range(2)]
    for a, b in ((dw[:, :cols], dw[:, cols:]), apart):
        rvq.moe_gated_linear_backward(res, xs, wg, wu, pre, n, rows, cols, ws, dwg=a, dwu=b)
    assert torch.equal(dw, torch.cat(apart, 1))


# Every way of computing a product, and every pairing of ways of dx and dw that is not
# rare, at sizes that are not near another way: (n, rows, cols), whether dx and dw share
# a launch, and each product's way with the CTA pairs that split a tile.
FORWARD_WAYS = [
    (False, (7, 256, 512), "stream", 0), (False, (256, 512, 256), "tiles", 0),
    (False, (66, 8, 3968), "parts", 0), (False, (5300, 8, 872), "split", 2),
    (False, (50, 8, 864), "split", 4), (False, (250, 472, 1240), "split", 4),
    (True, (7, 256, 512), "stream", 0), (True, (256, 512, 256), "tiles", 0),
    (True, (71, 8, 2056), "parts", 0), (True, (257, 520, 4096), "parts", 0),
    (True, (69, 8, 752), "split", 2), (True, (113, 512, 1024), "split", 2)]
GRADIENT_WAYS = [
    (False, (31, 72, 1000), False, ("stream", 0), ("tiles", 0)),
    (False, (129, 264, 136), True, ("tiles", 0), ("tiles", 0)),
    (False, (709, 200, 8), True, ("split", 2), ("split", 2)),
    (False, (487, 928, 256), True, ("split", 4), ("split", 4)),
    (False, (3864, 3720, 312), False, ("parts", 0), ("parts", 0)),
    (False, (829, 5536, 8), False, ("parts", 0), ("split", 2)),
    (False, (70, 3112, 8), False, ("parts", 0), ("tiles", 0)),
    (False, (67, 1968, 8), False, ("split", 4), ("tiles", 0)),
    (False, (3062, 8, 8), False, ("tiles", 0), ("parts", 0)),
    (False, (1865, 8, 8), False, ("tiles", 0), ("split", 4)),
    (True, (31, 72, 1000), False, ("stream", 0), ("tiles", 0)),
    (True, (129, 264, 136), True, ("tiles", 0), ("tiles", 0)),
    (True, (256, 512, 256), True, ("split", 2), ("split", 2)),
    (True, (709, 200, 8), True, ("split", 4), ("split", 4)),
    (True, (3506, 2848, 8), False, ("parts", 0), ("parts", 0)),
    (True, (707, 2864, 8), False, ("parts", 0), ("split", 2)),
    (True, (71, 1616, 8), False, ("parts", 0), ("tiles", 0)),
    (True, (65, 904, 8), False, ("split", 4), ("tiles", 0)),
    (True, (3711, 360, 688), False, ("tiles", 0), ("parts", 0)),
    (True, (1865, 8, 8), False, ("tiles", 0), ("split", 4))]


def pairs_of(way):
    return way[0], way[1] if way[0] == "split" else 0


@pytest.mark.parametrize("gated,size,way,pairs", FORWARD_WAYS)
def test_forward_ways(gated, size, way, pairs):
    """The way is the one that the size is here for, and its results are right."""
    _, (w,) = rvq.rvq_selftest_dense_plan(gated, False, *size)
    assert pairs_of(w) == (way, pairs)
    test_every_way_of_a_product(*size)


@pytest.mark.parametrize("gated,size,joint,dx,dw", GRADIENT_WAYS)
def test_gradient_ways(gated, size, joint, dx, dw):
    together, ways = rvq.rvq_selftest_dense_plan(gated, True, *size)
    assert together == joint and [pairs_of(w) for w in ways] == [dx, dw]
    if gated:
        test_gated_gradients(*size)
    else:
        linear_train(*size, BF if size[0] % 2 else HF, "silu", True, alpha=0.5, extra=8,
                     seed=size[0])


def test_two_streams_at_once():
    """Calls of several ways on two streams with a workspace each, in flight together."""
    sizes = [(1, 2048, 2048), (40, 1000, 1736), (300, 520, 2048), (900, 1000, 1096)]
    g = gen(11)
    jobs = []
    for n, rows, cols in sizes:
        x, dout = normal(g, (n, cols), BF), normal(g, (n, rows), BF)
        wg, wu = (normal(g, (rows, cols), BF, cols ** -0.5) for _ in range(2))
        jobs.append((n, rows, cols, x, wg, wu, dout, [workspace(n, rows, cols, True)
                                                     for _ in range(2)]))

    def outputs(n, rows, cols):
        return [torch.zeros(s, dtype=t, device=DEV) for s, t in
                (((n, rows), BF), ((2, n, rows), F32), ((n, cols), BF), ((rows, cols), BF),
                 ((rows, cols), BF))]

    def step(job, i, o, stream=None):
        n, rows, cols, x, wg, wu, dout, ws = job
        rvq.moe_gated_linear(x, wg, wu, n, rows, cols, o[0], ws[i], pre=o[1], stream=stream)
        rvq.moe_gated_linear_backward(dout, x, wg, wu, o[1], n, rows, cols, ws[i], dx=o[2],
                                      dwg=o[3], dwu=o[4], stream=stream)

    want = [outputs(*j[:3]) for j in jobs]
    for j, o in zip(jobs, want):
        step(j, 0, o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[outputs(*j[:3]) for j in jobs] for _ in streams]
    torch.cuda.synchronize()
    for _ in range(4):
        for k in range(len(jobs)):
            for i, s in enumerate(streams):
                m = (k + i) % len(jobs)     # different calls at the same time
                step(jobs[m], i, got[i][m], s)
    torch.cuda.synchronize()
    for i in range(2):
        for j, a, b in zip(jobs, got[i], want):
            assert all(torch.equal(p, q) for p, q in zip(a, b)), (i, j[:3])
            assert rvq.rvq_ws_status(j[7][i]) == (0, 0)

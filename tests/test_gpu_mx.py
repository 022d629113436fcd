"""GPU parity of the microscaled operators against their float64 definitions:
quantisation bit for bit, the join with a microscaled output."""
import pytest
import torch

from tests import dense_ref as R
from tests import mx_ref as X

pytestmark = pytest.mark.gpu
rvq = pytest.importorskip("moe_expert_ffn_router_gb300")
DEV = "cuda"
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
F8, F4 = X.F8, X.F4
EPS = 1e-6
U = R.U32


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def new_mx(rows, cols, fmt, fill=0xEE):
    return (torch.full((rvq.moe_mx_code_bytes(fmt, rows, cols),), fill, dtype=torch.uint8,
                       device=DEV),
            torch.full((rvq.moe_mx_scale_bytes(rows, cols),), fill, dtype=torch.uint8, device=DEV))


def exactly_quantized(x, codes, scales, fmt, fill=0xEE):
    """Codes, scales and padding bit for bit; bytes of rows behind the last untouched.
    A code of zero may have either sign."""
    rows, cols = x.shape
    q, byte = X.quantize(x, fmt)
    got = X.unpack(codes, rows, cols, fmt)
    assert torch.equal(X.values(fmt, DEV)[got], q)
    pad = X.unpack(codes, rows, cols, fmt)[:, cols:]
    assert (pad == 0).all()
    assert torch.equal(X.from_tiles(scales, rows, cols), byte)
    behind = X.from_tiles(scales, X.up(rows, 128), cols)[rows:]
    assert (behind == fill).all()


SIZES = [(1, 8), (1, 7168), (3, 40), (33, 136), (127, 128), (129, 264), (257, 2040), (64, 512)]


@pytest.mark.parametrize("fmt", [F8, F4])
@pytest.mark.parametrize("dt", [BF, HF, F32])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_quantize(rows, cols, dt, fmt):
    g = gen(rows * 10007 + cols)
    x = torch.randn((rows, cols), device=DEV, generator=g)
    x *= torch.exp2(torch.randint(-12, 6, (rows, 1), device=DEV, generator=g).float())
    x = x.to(dt)
    codes, scales = new_mx(rows, cols, fmt)
    rvq.moe_mx_quantize(x, rows, cols, codes, scales, fmt)
    exactly_quantized(x, codes, scales, fmt)
    for ot in (BF, HF, F32):
        out = torch.full((rows, cols), 7.0, dtype=ot, device=DEV)
        rvq.moe_mx_dequantize(codes, scales, rows, cols, out, fmt)
        assert torch.equal(out, X.dequantize(codes, scales, rows, cols, fmt).to(F32).to(ot))


@pytest.mark.parametrize("fmt", [F8, F4])
def test_quantize_ties_and_ends(fmt):
    """Every midpoint between codes (ties to even), values at and over the largest, at
    several scales, signs and places in a block."""
    v = X.values(fmt, DEV)
    v = v[torch.isfinite(v) & (v >= 0)].unique()
    mid = (v[1:] + v[:-1]) / 2
    top = 2.0 ** X.LEAD[fmt]
    probe = torch.cat([v, mid, torch.tensor([1.99 * top, 1.8 * top], device=DEV).double()])
    probe = torch.cat([probe, -probe])
    rows = torch.zeros((len(probe), 32), device=DEV, dtype=F32)
    rows[:, 5] = top
    rows[:, 17] = probe.float()
    x = torch.cat([rows * 2.0 ** s for s in (-100, -3, 0, 40)], 1).contiguous()
    codes, scales = new_mx(*x.shape, fmt)
    rvq.moe_mx_quantize(x, *x.shape, codes, scales, fmt)
    exactly_quantized(x, codes, scales, fmt)


@pytest.mark.parametrize("fmt", [F8, F4])
def test_quantize_extremes(fmt):
    """Zeros, subnormal numbers, the largest, and blocks that are not finite."""
    x = torch.zeros((40, 64), device=DEV, dtype=F32)
    tiny = 2.0 ** -149
    for i, m in enumerate((tiny, 3 * tiny, 2.0 ** -127, 2.0 ** -126, 2.0 ** -119, 2.0 ** -118,
                           1.5 * 2.0 ** -124, 2.0 ** -117, 3.4e38, 2.0 ** 127, -3.4e38)):
        x[i, 3], x[i, 4], x[i, 40] = m, m / 3, -m
    for i, bad in enumerate((float("inf"), -float("inf"), float("nan"))):
        x[20 + i] = 1.0
        x[20 + i, 31 * i // 2] = bad
    x[23, 40], x[23, 41] = float("nan"), float("inf")
    x[24, 63] = -0.0
    codes, scales = new_mx(40, 64, fmt)
    rvq.moe_mx_quantize(x, 40, 64, codes, scales, fmt)
    exactly_quantized(x, codes, scales, fmt)
    out = torch.empty((40, 64), dtype=F32, device=DEV)
    rvq.moe_mx_dequantize(codes, scales, 40, 64, out, fmt)
    assert torch.isnan(out[20:23, :32]).all() and torch.isnan(out[23, 32:]).all()
    assert torch.isfinite(out[23, :32]).all() and torch.isfinite(out[:20]).all()


def test_every_code_read_back():
    """dequantize over every code and scale byte."""
    for fmt in (F8, F4):
        n = 256 if fmt == F8 else 16
        cols = 256
        q = torch.arange(cols, device=DEV) % n
        row = (q if fmt == F8 else q[0::2] + 16 * q[1::2]).to(torch.uint8)
        codes = row.expand(256, -1).contiguous().view(-1)
        byte = torch.arange(256, device=DEV).unsqueeze(1).expand(256, cols // 32)
        scales = X.to_tiles(byte)
        out = torch.empty((256, cols), dtype=F32, device=DEV)
        rvq.moe_mx_dequantize(codes, scales, 256, cols, out, fmt)
        want = X.dequantize(codes, scales, 256, cols, fmt).float()
        assert torch.equal(out.nan_to_num(1e30), want.nan_to_num(1e30))
        assert torch.equal(out.isnan(), want.isnan())


def test_quantize_strides_and_streams():
    """Columns of a wider matrix, and a side stream."""
    wide = torch.randn((70, 512), device=DEV, generator=gen(3)).to(BF)
    x = wide[:, 64:64 + 200]
    codes, scales = new_mx(70, 200, F8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        rvq.moe_mx_quantize(x, 70, 200, codes, scales)
    rvq.moe_mx_quantize(x, 70, 200, codes, scales, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    exactly_quantized(x, codes, scales, F8)
    out = torch.zeros((70, 512), device=DEV)
    rvq.moe_mx_dequantize(codes, scales, 70, 200, out[:, 8:208])
    assert torch.equal(out[:, 8:208].double(), X.dequantize(codes, scales, 70, 200, F8))
    assert (out[:, :8] == 0).all() and (out[:, 208:] == 0).all()


# ------------------------------------------------------------------ the join

def make(n, d, hdt, ydt, wdt, gate, post, seed=0, with_h=True, gains=True):
    g = gen(seed)

    def rnd(shape, dtype, std=1.0, mean=0.0):
        return (torch.randn(shape, device=DEV, generator=g) * std + mean).to(dtype)

    shape = {"none": None, "scalar": (1,), "token": (n, 1), "channel": (1, d), "full": (n, d)}[gate]
    return dict(h=rnd((n, d), hdt, 2.0) if with_h else None, y=rnd((n, d), ydt, 0.5),
                gate=None if shape is None else rnd(shape, hdt, 0.5, 0.3),
                w_post=rnd((d,), wdt, 0.1, 1.0) if gains and post else None,
                w_pre=rnd((d,), wdt, 0.1, 1.0) if gains else None)


def check_join(s, n, d, alpha, post, hdt, xdt, fmt, outs=("h_out", "xn", "rstd")):
    """h_out and xn in their types, the microscaled rows within half a step of the
    format.  A row's sum of squares is a tree of fp32 additions over at most 64 levels,
    each off by half a step; the rest are a few multiplications."""
    ho = torch.empty((n, d), dtype=hdt, device=DEV) if "h_out" in outs else None
    xn = torch.empty((n, d), dtype=xdt, device=DEV) if "xn" in outs else None
    rstd = torch.empty((2, n), dtype=F32, device=DEV) if "rstd" in outs else None
    codes, scales = new_mx(n, d, fmt)
    rvq.moe_norm_join_mx(s["y"], n, d, ho, codes, scales, fmt=fmt, xn=xn, h=s["h"], alpha=alpha,
                         gate=s["gate"], post_norm=post, w_post=s["w_post"], w_pre=s["w_pre"],
                         eps=EPS, rstd=rstd)
    wh, wx, r1, r2, z, gz = R.join(s["h"], s["y"], alpha, s["gate"], post, s["w_post"],
                                   s["w_pre"], EPS)
    ah = 0 if s["h"] is None else (alpha * s["h"].double()).abs()
    eh = 72 * U * gz.abs() + 4 * U * (ah + gz.abs())
    er2 = 64 * U * r2 + r2 ** 3 * (wh.abs() * eh).mean(1, keepdim=True)
    w = 1.0 if s["w_pre"] is None else s["w_pre"].double().abs()
    ex = (eh * r2 + wh.abs() * er2) * w + 4 * U * wx.abs()
    if ho is not None:
        R.check(ho, (wh, eh + R.half_step(hdt) * wh.abs() * 1.001 + R.tiny(hdt)), "h_out")
    if xn is not None:
        R.check(xn, (wx, ex + R.half_step(xdt) * wx.abs() * 1.001 + R.tiny(xdt)), "xn")
    if rstd is not None:
        R.check(rstd[0], (r1[:, 0], 66 * U * r1[:, 0]), "r1")
        R.check(rstd[1], (r2[:, 0], (er2 + U * r2)[:, 0]), "r2")
    X.check_quantized(codes, scales, n, d, fmt, wx, ex.expand_as(wx), "codes")
    behind = X.from_tiles(scales, X.up(n, 128), d)[n:]
    assert (behind == 0xEE).all()
    return codes, scales, xn


JOINS = [(1, 8, F32, BF), (1, 7168, F32, F32), (5, 40, BF, BF), (200, 136, F32, BF),
         (130, 2040, BF, BF), (3, 8200, F32, F32), (2, 16384, BF, HF), (333, 1000, HF, F32),
         (350, 1096, BF, F32), (610, 2056, BF, BF), (4100, 72, F32, BF), (400, 7168, F32, BF),
         (161, 8192, BF, BF)]


@pytest.mark.parametrize("fmt", [F8, F4])
@pytest.mark.parametrize("gate,post,alpha", [("none", False, 1.0), ("channel", True, 0.5),
                                             ("token", True, 1.0), ("full", False, 0.8125),
                                             ("scalar", True, 1.0)])
@pytest.mark.parametrize("n,d,hdt,ydt", JOINS)
def test_join(n, d, hdt, ydt, gate, post, alpha, fmt):
    s = make(n, d, hdt, ydt, F32 if n % 2 else BF, gate, post, seed=n + d)
    check_join(s, n, d, alpha, post, hdt, BF, fmt)


def test_join_parts():
    """Without h, without gains, without h_out, xn or rstd."""
    for outs in ((), ("xn",), ("h_out",), ("rstd",)):
        s = make(19, 264, BF, F32, F32, "none", True, with_h="h_out" in outs, gains=False)
        check_join(s, 19, 264, 1.0, True, BF, HF, F8, outs)


def test_join_agrees_with_quantize():
    """The microscaled rows are those of the fp32 xn beside them."""
    s = make(77, 712, F32, F32, F32, "channel", True, seed=5)
    for fmt in (F8, F4):
        codes, scales, xn = check_join(s, 77, 712, 1.0, True, F32, F32, fmt)
        c2, s2 = new_mx(77, 712, fmt)
        rvq.moe_mx_quantize(xn, 77, 712, c2, s2, fmt)
        assert torch.equal(codes, c2) and torch.equal(scales, s2)


@pytest.mark.parametrize("n,d", [(300, 520), (700, 1032)])
def test_join_in_place_and_zero_rows(n, d):
    """h_out over h, xn over y; a row of zeros (eps > 0) is a row of zeros."""
    s = make(n, d, F32, F32, F32, "none", False, seed=9)
    s["h"][7], s["y"][7] = 0, 0
    want = {k: None if v is None else v.clone() for k, v in s.items()}
    codes, scales = new_mx(n, d, F8)
    rvq.moe_norm_join_mx(s["y"], n, d, s["h"], codes, scales, xn=s["y"], h=s["h"], post_norm=False,
                         w_pre=s["w_pre"], eps=EPS)
    c2, s2, xn = check_join(want, n, d, 1.0, False, F32, F32, F8)
    assert torch.equal(codes, c2) and torch.equal(scales, s2) and torch.equal(s["y"], xn)
    assert (X.unpack(codes, n, d, F8)[7] == 0).all()
    assert (X.from_tiles(scales, n, d)[7] == 0).all()


@pytest.mark.parametrize("n,d", [(4, 264), (500, 1096)])
def test_join_non_finite_row(n, d):
    """A NaN makes its own row NaN and no other, and no padding."""
    s = make(n, d, F32, F32, F32, "none", False, seed=2)
    s["y"][2, 100] = float("nan")
    codes, scales = new_mx(n, d, F8)
    rvq.moe_norm_join_mx(s["y"], n, d, None, codes, scales, h=s["h"], post_norm=False, eps=EPS)
    byte, blocks = X.from_tiles(scales, n, d), -(-d // 32)
    assert (byte[2, :blocks] == 255).all() and (byte[:, blocks:] == 0).all()
    byte[2] = 0
    assert (byte < 255).all()
    assert (X.unpack(codes, n, d, F8)[2] == 0).all()


def test_join_gradient_straight_through():
    """rstd of the microscaled call feeds moe_norm_join_backward: the same gradients as
    after moe_norm_join."""
    n, d = 37, 648
    s = make(n, d, F32, BF, F32, "channel", True, seed=4)
    dxn = torch.randn((n, d), device=DEV, generator=gen(5)).to(BF)
    ws = torch.zeros(rvq.moe_norm_join_workspace_bytes(n, d), dtype=torch.uint8, device=DEV)
    got = []
    for mx in (True, False):
        rstd = torch.empty((2, n), device=DEV)
        if mx:
            rvq.moe_norm_join_mx(s["y"], n, d, None, *new_mx(n, d, F8), h=s["h"], gate=s["gate"],
                                 w_post=s["w_post"], w_pre=s["w_pre"], eps=EPS, rstd=rstd)
        else:
            xn = torch.empty((n, d), dtype=BF, device=DEV)
            rvq.moe_norm_join(s["y"], n, d, None, xn, h=s["h"], gate=s["gate"], w_post=s["w_post"],
                              w_pre=s["w_pre"], eps=EPS, rstd=rstd)
        dh, dy = torch.empty((n, d), device=DEV), torch.empty((n, d), dtype=BF, device=DEV)
        rvq.moe_norm_join_backward(None, dxn, s["y"], n, d, rstd, ws, h=s["h"], gate=s["gate"],
                                   w_post=s["w_post"], w_pre=s["w_pre"], dh=dh, dy=dy)
        got.append((rstd, dh, dy))
    # two orders of the sum of squares: 1/rms within 130 half steps of each other
    for a, b in zip(*got):
        rel = (a.double() - b.double()).norm() / b.double().norm()
        assert rel <= 260 * U + (R.half_step(BF) if a.dtype is BF else 0), rel


@pytest.mark.parametrize("n", [3, 400])
def test_join_streams_and_graph(n):
    """Two calls at once on two streams, and a captured call replayed on new rows, few
    and walked: the bits of a call alone."""
    d = 1032
    ins = [make(n, d, F32, BF, F32, "channel", True, seed=40 + i) for i in range(3)]

    def call(s, q, **kw):
        rvq.moe_norm_join_mx(s["y"], n, d, None, *q, h=s["h"], gate=s["gate"], w_post=s["w_post"],
                             w_pre=s["w_pre"], eps=EPS, **kw)

    alone = [new_mx(n, d, F8) for _ in ins]
    for s, q in zip(ins, alone):
        call(s, q)
    together = [new_mx(n, d, F8) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, q, st in zip(ins, together, streams):
            call(s, q, stream=st)
    torch.cuda.synchronize()
    for a, b in zip(alone, together):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    s, q = {k: None if v is None else v.clone() for k, v in ins[2].items()}, new_mx(n, d, F8)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(s, q)
    for i in range(3):
        for k, v in ins[i].items():
            s[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(q[0], alone[i][0]) and torch.equal(q[1], alone[i][1])


def test_past_two_gigabytes():
    """Matrices of more than 2^31 values: offsets of the last rows, of a tile boundary past
    2^31 and of the first, in every call."""
    n, d = 270000, 8192
    x = torch.empty((n, d), dtype=BF, device=DEV).normal_(generator=gen(1))
    codes, scales = new_mx(n, d, F8)
    rvq.moe_mx_quantize(x, n, d, codes, scales)
    places = (0, 262144 - 64, n - 100)

    def part(c, s, r):
        return (c.view(n, -1)[r:r + 100].reshape(-1),
                X.to_tiles(X.from_tiles(s, n, d)[r:r + 100]))

    for r in places:
        q, byte = X.quantize(x[r:r + 100], F8)
        c, s = part(codes, scales, r)
        assert torch.equal(X.values(F8, DEV)[X.unpack(c, 100, d, F8)], q)
        assert torch.equal(X.from_tiles(s, 100, d), byte)
    w, ws_, vw = X.random_mx(136, d, F4, gen(2), std=d ** -0.5)
    out = torch.zeros((n, 136), dtype=BF, device=DEV)
    ws = torch.zeros(rvq.moe_mx_linear_workspace_bytes(n, 136, d), dtype=torch.uint8, device=DEV)
    rvq.moe_mx_linear(codes, scales, w, ws_, n, 136, d, out, ws)
    assert rvq.rvq_ws_status(ws) == (0, 0)
    for r in places:
        v = X.dequantize(*part(codes, scales, r), 100, d, F8)
        y, e = R.product(v, vw)
        R.check(out[r:r + 100], (y, e + R.half_step(BF) * 1.001 * y.abs() + R.tiny(BF)), f"row {r}")
    rvq.moe_mx_dequantize(codes, scales, n, d, x)
    for r in places:
        assert torch.equal(x[r:r + 100].double(), X.dequantize(*part(codes, scales, r), 100, d, F8))
    h = torch.zeros((n, d), dtype=BF, device=DEV)
    rvq.moe_norm_join_mx(x, n, d, h, codes, scales, post_norm=False, eps=EPS)
    for r in places:
        y = x[r:r + 100].double()
        xn = y / torch.sqrt(y.square().mean(1, keepdim=True) + EPS)
        X.check_quantized(*part(codes, scales, r), 100, d, F8, xn, 72 * U * xn.abs(), f"row {r}")
        assert torch.equal(h[r:r + 100], x[r:r + 100])

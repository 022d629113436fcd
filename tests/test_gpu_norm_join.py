"""GPU parity of moe_norm_join and its gradients against the float64
definition: types, gates, odd row counts, aliases, zero rows."""
import itertools

import pytest
import torch

from tests import dense_ref as R

pytestmark = pytest.mark.gpu
rvq = pytest.importorskip("moe_expert_ffn_router_gb300")
DEV = "cuda"
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-6
U = R.U32


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def make(n, d, hdt, ydt, wdt, gate, post, gains=True, seed=0, with_h=True):
    g = gen(seed)

    def rnd(shape, dtype, std=1.0, mean=0.0):
        return (torch.randn(shape, device=DEV, generator=g) * std + mean).to(dtype)

    shape = {"none": None, "scalar": (1,), "token": (n, 1), "channel": (1, d), "full": (n, d)}[gate]
    return dict(h=rnd((n, d), hdt, 2.0) if with_h else None, y=rnd((n, d), ydt, 0.5),
                gate=None if shape is None else rnd(shape, hdt, 0.5, 0.3),
                w_post=rnd((d,), wdt, 0.1, 1.0) if gains and post else None,
                w_pre=rnd((d,), wdt, 0.1, 1.0) if gains else None)


def bounds_forward(s, alpha, post, hdt, xdt, rdt=F32):
    """Values and bounds.  A row's sum of squares is a tree of fp32 additions
    over at most 64 levels (a thread's columns, the warp, the warps), each off
    by half a step, so 1/rms is good to 64 half steps; the rest are a few
    multiplications."""
    ho, xn, r1, r2, z, gz = R.join(s["h"], s["y"], alpha, s["gate"], post, s["w_post"],
                                   s["w_pre"], EPS)
    ah = 0 if s["h"] is None else (alpha * s["h"].double()).abs()
    eho = 72 * U * gz.abs() + 4 * U * (ah + gz.abs())
    # r2's own error: 64 half steps, and what h_out's error puts into its mean square
    er2 = 64 * U * r2 + r2 ** 3 * (ho.abs() * eho).mean(1, keepdim=True)
    w = 1.0 if s["w_pre"] is None else s["w_pre"].double()
    exn = ((eho * r2 + ho.abs() * er2) * abs(w) + 4 * U * xn.abs()) if s["w_pre"] is None else \
        (eho * r2 + ho.abs() * er2) * w.abs() + 4 * U * xn.abs()
    return ((ho, eho + R.half_step(hdt) * ho.abs() * 1.001 + R.tiny(hdt)),
            (xn, exn + R.half_step(xdt) * xn.abs() * 1.001 + R.tiny(xdt)),
            r1, (r2, er2 + U * r2), z, gz, eho)


def forward(s, n, d, alpha, post, hdt, xdt):
    ho = torch.empty((n, d), dtype=hdt, device=DEV)
    xn = torch.empty((n, d), dtype=xdt, device=DEV)
    rstd = torch.empty((2, n), dtype=F32, device=DEV)
    rvq.moe_norm_join(s["y"], n, d, ho, xn, h=s["h"], alpha=alpha, gate=s["gate"], post_norm=post,
                      w_post=s["w_post"], w_pre=s["w_pre"], eps=EPS, rstd=rstd)
    return ho, xn, rstd


def check_forward(s, n, d, alpha, post, hdt, xdt):
    ho, xn, rstd = forward(s, n, d, alpha, post, hdt, xdt)
    who, wxn, r1, wr2, *_ = bounds_forward(s, alpha, post, hdt, xdt)
    R.check(ho, who, "h_out")
    R.check(xn, wxn, "xn")
    R.check(rstd[0], (r1[:, 0], 66 * U * r1[:, 0]), "r1")
    R.check(rstd[1], (wr2[0][:, 0], wr2[1][:, 0]), "r2")
    return rstd


def check_backward(s, n, d, alpha, post, hdt, ydt, xdt, wdt, rstd, seed=1, which="both"):
    g = gen(seed)
    dho = (torch.randn((n, d), device=DEV, generator=g)).to(hdt) if which != "dxn" else None
    dxn = (torch.randn((n, d), device=DEV, generator=g)).to(xdt) if which != "dho" else None
    (ho, _), _, r1, (r2, er2), z, gz, eho = bounds_forward(s, alpha, post, hdt, xdt)
    one = torch.ones((), dtype=torch.float64, device=DEV)
    wpost = one if s["w_post"] is None else s["w_post"].double()
    wpre = one if s["w_pre"] is None else s["w_pre"].double()
    gate = one if s["gate"] is None else s["gate"].double()
    y = s["y"].double()
    dh_ = torch.zeros_like(y) if dho is None else dho.double()
    dx_ = torch.zeros_like(y) if dxn is None else dxn.double()
    q = dx_ * wpre
    e = dh_ + r2 * q - ho * r2 ** 3 * (q * ho).mean(1, keepdim=True)
    dz = gate * e
    outs = dict(dh=None if s["h"] is None else torch.empty((n, d), dtype=hdt, device=DEV),
                dy=torch.empty((n, d), dtype=ydt, device=DEV),
                dgate=None if s["gate"] is None else torch.empty_like(s["gate"]),
                dw_post=torch.empty(d, dtype=wdt, device=DEV) if post else None,
                dw_pre=torch.empty(d, dtype=wdt, device=DEV) if dxn is not None else None)
    ws = torch.empty(rvq.moe_norm_join_workspace_bytes(n, d), dtype=torch.uint8, device=DEV)
    rvq.moe_norm_join_backward(dho, dxn, s["y"], n, d, rstd, ws, h=s["h"], alpha=alpha,
                               gate=s["gate"], post_norm=post, w_post=s["w_post"],
                               w_pre=s["w_pre"], **outs)

    def rounded(v, err, dtype):
        return v, err + R.half_step(dtype) * 1.001 * v.abs() + R.tiny(dtype)

    # magnitudes: every term's absolute value in place of the term, times the
    # relative errors met on the way (statistics 64 half steps, a row's sums
    # another 64, a few operations); `eho` enters through h_out.
    mag_ho = eho / U / 72 + ho.abs()
    k = 72 * U
    mS = (q.abs() * mag_ho).mean(1, keepdim=True)
    me = dh_.abs() + r2 * q.abs() + mag_ho * r2 ** 3 * mS
    ee = 4 * k * me
    if outs["dh"] is not None:
        R.check(outs["dh"], rounded(alpha * e, abs(alpha) * ee, hdt), "dh")
    if post:
        mean = (dz * wpost * y).mean(1, keepdim=True)
        dy = r1 * dz * wpost - y * r1 ** 3 * mean
        mmean = ((gate * wpost * y).abs() * me).mean(1, keepdim=True)
        mdy = r1 * (gate * wpost).abs() * me + y.abs() * r1 ** 3 * mmean
        R.check(outs["dy"], rounded(dy, 6 * k * mdy, ydt), "dy")
        # sums over n tokens: a chain of at most n fp32 additions in the worst
        # case (half a step each) on top of the terms' own errors
        nsum = (6 * k + n * U)
        R.check(outs["dw_post"], rounded((dz * y * r1).sum(0), nsum * ((gate * y).abs() * me * r1)
                                         .sum(0), wdt), "dw_post")
    else:
        R.check(outs["dy"], rounded(dz, gate.abs() * ee, ydt), "dy")
        nsum = (6 * k + n * U)
    if outs["dw_pre"] is not None:
        R.check(outs["dw_pre"], rounded((dx_ * ho * r2).sum(0), nsum * (dx_.abs() * mag_ho * r2)
                                        .sum(0), wdt), "dw_pre")
    if s["gate"] is not None:
        ez, mez = e * z, me * z.abs()
        dims = {tuple([n, d]): None, (n, 1): 1, (1, d): 0}
        shape = tuple(s["gate"].shape)
        if s["gate"].numel() == 1:
            want, mag = ez.sum().reshape(1), mez.sum().reshape(1)
        elif dims[shape] is None:
            want, mag = ez, mez
        else:
            want, mag = ez.sum(dims[shape], keepdim=True), mez.sum(dims[shape], keepdim=True)
        R.check(outs["dgate"].reshape(want.shape), rounded(want, nsum * mag, s["gate"].dtype),
                "dgate")
    return outs


SIZES = [(1, 8), (3, 64), (2, 2048), (5, 2056), (7, 7168), (33, 1000), (400, 264), (3, 8200),
         (2, 16384), (700, 4104)]
GATES = ["none", "scalar", "token", "channel", "full"]


@pytest.mark.parametrize("n,d", SIZES)
@pytest.mark.parametrize("gate", GATES)
def test_join_sizes_and_gates(n, d, gate):
    i = SIZES.index((n, d)) + GATES.index(gate)
    post = i % 3 != 0
    hdt, ydt, xdt, wdt = [(F32, F32, BF, BF), (BF, BF, BF, BF), (F32, BF, HF, F32),
                          (HF, F32, F32, HF)][i % 4]
    s = make(n, d, hdt, ydt, wdt, gate, post, gains=i % 5 != 0, seed=i)
    alpha = [1.0, 0.75][i % 2]
    rstd = check_forward(s, n, d, alpha, post, hdt, xdt)
    wdt2 = wdt if (s["w_post"] is not None or s["w_pre"] is not None) else F32
    check_backward(s, n, d, alpha, post, hdt, ydt, xdt, wdt2, rstd)


@pytest.mark.parametrize("which", ["dho", "dxn"])
@pytest.mark.parametrize("with_h", [True, False])
def test_join_one_gradient_arrives(which, with_h):
    s = make(21, 520, F32, BF, F32, "token", True, seed=4, with_h=with_h)
    rstd = check_forward(s, 21, 520, 1.0, True, F32, BF)
    check_backward(s, 21, 520, 1.0, True, F32, BF, BF, F32, rstd, which=which)


def test_join_every_type_mix():
    for hdt, ydt, xdt, wdt in itertools.product((F32, BF, HF), repeat=4):
        s = make(4, 136, hdt, ydt, wdt, "channel", True, seed=8)
        rstd = check_forward(s, 4, 136, 0.5, True, hdt, xdt)
        check_backward(s, 4, 136, 0.5, True, hdt, ydt, xdt, wdt, rstd)


# many rows (blocks that walk over them), at the limit of the block-per-row
# kernel, and the layouts of a walking block: two rows in shared memory, one (fp32
# with a full gate), none (long rows), types that no instance has
WALKS = [(304, 520, F32, BF, BF, BF, "token"), (305, 520, BF, BF, BF, BF, "channel"),
         (900, 8, BF, BF, BF, BF, "full"), (613, 136, HF, F32, HF, HF, "scalar"),
         (500, 7168, F32, F32, BF, F32, "full"), (333, 8192, F32, F32, F32, F32, "full"),
         (400, 8192, F32, F32, HF, HF, "channel"), (310, 8200, F32, F32, F32, F32, "channel"),
         (306, 16384, F32, F32, F32, F32, "full"), (306, 16384, BF, BF, BF, BF, "token"),
         (700, 264, BF, HF, F32, HF, "full"), (350, 2048, HF, BF, BF, F32, "none")]


@pytest.mark.parametrize("n,d,hdt,ydt,xdt,wdt,gate", WALKS)
def test_join_many_rows(n, d, hdt, ydt, xdt, wdt, gate):
    for post in (True, False):
        s = make(n, d, hdt, ydt, wdt, gate, post, seed=n)
        rstd = check_forward(s, n, d, 0.5, post, hdt, xdt)
        check_backward(s, n, d, 0.5, post, hdt, ydt, xdt, wdt, rstd)


def test_join_many_rows_full_gate_of_another_type():
    n, d = 320, 264
    s = make(n, d, F32, BF, F32, "full", True, seed=5)
    s["gate"] = s["gate"].to(BF)
    rstd = check_forward(s, n, d, 1.0, True, F32, BF)
    check_backward(s, n, d, 1.0, True, F32, BF, BF, F32, rstd)


def test_join_many_rows_without_some_tensors():
    n, d = 777, 1000
    for which, with_h in (("dho", True), ("dxn", False), ("both", False)):
        s = make(n, d, BF, BF, BF, "token", True, gains=which == "dxn", seed=4, with_h=with_h)
        rstd = check_forward(s, n, d, 1.0, True, BF, BF)
        wdt = BF if s["w_pre"] is not None else F32
        check_backward(s, n, d, 1.0, True, BF, BF, BF, wdt, rstd, which=which)
    # outputs over inputs, as for few rows
    s = make(n, d, BF, BF, BF, "channel", True, seed=2)
    ho, xn, rstd = forward(s, n, d, 1.0, True, BF, BF)
    for over in ("h", "y"):
        t = {k: None if v is None else v.clone() for k, v in s.items()}
        xn2 = torch.empty_like(xn)
        rvq.moe_norm_join(t["y"], n, d, t[over], xn2, h=t["h"], gate=t["gate"],
                          w_post=t["w_post"], w_pre=t["w_pre"], eps=EPS)
        assert torch.equal(t[over], ho) and torch.equal(xn2, xn)
    g = gen(3)
    dho, dxn = ((torch.randn((n, d), device=DEV, generator=g)).to(BF) for _ in range(2))
    ws = torch.empty(rvq.moe_norm_join_workspace_bytes(n, d), dtype=torch.uint8, device=DEV)
    kw = dict(h=s["h"], gate=s["gate"], w_post=s["w_post"], w_pre=s["w_pre"])
    dh, dy = torch.empty_like(dho), torch.empty_like(dho)
    rvq.moe_norm_join_backward(dho, dxn, s["y"], n, d, rstd, ws, dh=dh, dy=dy, **kw)
    a, b = dho.clone(), dxn.clone()
    rvq.moe_norm_join_backward(a, b, s["y"], n, d, rstd, ws, dh=a, dy=b, **kw)
    assert torch.equal(a, dh) and torch.equal(b, dy)


def test_join_aliases_and_partial_outputs():
    n, d = 6, 7168
    s = make(n, d, F32, F32, BF, "token", True, seed=2)
    ho, xn, rstd = forward(s, n, d, 1.0, True, F32, BF)
    for over in ("h", "y"):                       # h_out over h, or over y
        t = {k: None if v is None else v.clone() for k, v in s.items()}
        xn2 = torch.empty_like(xn)
        rvq.moe_norm_join(t["y"], n, d, t[over], xn2, h=t["h"], gate=t["gate"],
                          w_post=t["w_post"], w_pre=t["w_pre"], eps=EPS)
        assert torch.equal(t[over], ho) and torch.equal(xn2, xn)
    only = torch.empty_like(xn)
    rvq.moe_norm_join(s["y"], n, d, None, only, h=s["h"], gate=s["gate"], w_post=s["w_post"],
                      w_pre=s["w_pre"], eps=EPS)
    assert torch.equal(only, xn)
    only = torch.empty_like(ho)
    rvq.moe_norm_join(s["y"], n, d, only, None, h=s["h"], gate=s["gate"], w_post=s["w_post"],
                      eps=EPS)
    assert torch.equal(only, ho)
    # gradients over their own inputs
    g = gen(3)
    dho, dxn = torch.randn((n, d), device=DEV, generator=g), torch.randn((n, d), device=DEV,
                                                                          generator=g)
    ws = torch.empty(rvq.moe_norm_join_workspace_bytes(n, d), dtype=torch.uint8, device=DEV)
    kw = dict(h=s["h"], gate=s["gate"], w_post=s["w_post"], w_pre=s["w_pre"])
    dh, dy = torch.empty_like(dho), torch.empty_like(dho)
    rvq.moe_norm_join_backward(dho, dxn, s["y"], n, d, rstd, ws, dh=dh, dy=dy, **kw)
    a, b = dho.clone(), dxn.clone()
    rvq.moe_norm_join_backward(a, b, s["y"], n, d, rstd, ws, dh=a, dy=b, **kw)
    assert torch.equal(a, dh) and torch.equal(b, dy)


def test_join_zero_rows_and_non_finite():
    """A zero row norms to zero (eps > 0); a row with an infinity or NaN spoils
    only itself; a row whose gate is 0 passes the stream on."""
    n, d = 5, 256
    s = make(n, d, F32, F32, F32, "token", True, seed=6)
    s["y"][0] = 0
    s["h"][0] = 0
    s["y"][1, 7] = float("nan")
    s["h"][2, 9] = float("inf")
    s["gate"][3] = 0
    ho, xn, _ = forward(s, n, d, 1.0, True, F32, F32)
    assert (ho[0] == 0).all() and (xn[0] == 0).all()
    assert torch.isnan(ho[1]).all() and torch.isnan(xn[1]).all()
    assert torch.isinf(ho[2, 9]) and torch.isfinite(ho[2]).sum() == d - 1
    assert torch.equal(ho[3], s["h"][3])
    who, wxn, *_ = bounds_forward(s, 1.0, True, F32, F32)
    for r in (3, 4):
        R.check(ho[r], (who[0][r], who[1][r]), "h_out")
        R.check(xn[r], (wxn[0][r], wxn[1][r]), "xn")


def test_join_plain_norm_is_moe_rms_norm():
    """Without post norm, gate, residual and gains, xn is moe_rms_norm's value
    (both round 1/sqrt(mean + eps) of fp32 sums; the sums' order differs)."""
    n, d = 9, 7168
    x = torch.randn((n, d), device=DEV, generator=gen(1))
    a, b = torch.empty_like(x), torch.empty_like(x)
    rvq.moe_norm_join(x, n, d, None, a, post_norm=False, eps=EPS)
    rvq.moe_rms_norm(x, n, d, b, eps=EPS)
    assert ((a - b).abs() <= 130 * U * b.abs()).all()


def test_join_gradients_against_differences():
    n, d, alpha = 4, 64, 0.8
    s = make(n, d, F32, F32, F32, "channel", True, seed=12)
    _, _, rstd = forward(s, n, d, alpha, True, F32, F32)
    g = gen(13)
    dho, dxn = (torch.randn((n, d), device=DEV, generator=g) for _ in range(2))
    names = ["h", "y", "gate", "w_post", "w_pre"]
    outs = {"d" + k: torch.empty_like(s[k]) for k in names}
    ws = torch.empty(rvq.moe_norm_join_workspace_bytes(n, d), dtype=torch.uint8, device=DEV)
    rvq.moe_norm_join_backward(dho, dxn, s["y"], n, d, rstd, ws, h=s["h"], alpha=alpha,
                               gate=s["gate"], w_post=s["w_post"], w_pre=s["w_pre"], **outs)

    def loss(p):
        ho, xn, *_ = R.join(p["h"], p["y"], alpha, p["gate"], True, p["w_post"], p["w_pre"], EPS)
        return (dho.double() * ho + dxn.double() * xn).sum().item()

    base = {k: s[k].double() for k in names}
    for k in names:
        v = torch.randn(base[k].shape, device=DEV, generator=g, dtype=torch.float64)
        e = 1e-5
        diff = (loss({**base, k: base[k] + e * v}) - loss({**base, k: base[k] - e * v})) / (2 * e)
        got = (outs["d" + k].double() * v).sum().item()
        # fp32 gradients (a few hundred half steps) against differences whose
        # own error is of order e^2 times third derivatives (1e-10 x O(10))
        scale = (outs["d" + k].double().abs() * v.abs()).sum().item()
        assert abs(got - diff) <= 300 * U * scale + 1e-7 * abs(diff) + 1e-8, (k, got, diff)


def test_join_repeats_streams_and_graphs():
    n, d = 613, 2048
    s = make(n, d, BF, BF, BF, "scalar", True, seed=3)
    g = gen(14)
    dho, dxn = ((torch.randn((n, d), device=DEV, generator=g)).to(BF) for _ in range(2))
    ws = torch.empty(rvq.moe_norm_join_workspace_bytes(n, d), dtype=torch.uint8, device=DEV)

    def bufs():
        return dict(ho=torch.zeros((n, d), dtype=BF, device=DEV),
                    xn=torch.zeros((n, d), dtype=BF, device=DEV),
                    rstd=torch.zeros((2, n), device=DEV),
                    dh=torch.zeros((n, d), dtype=BF, device=DEV),
                    dy=torch.zeros((n, d), dtype=BF, device=DEV),
                    dgate=torch.zeros_like(s["gate"]), dw_post=torch.zeros_like(s["w_post"]),
                    dw_pre=torch.zeros_like(s["w_pre"]))

    def step(b, stream=None):
        rvq.moe_norm_join(s["y"], n, d, b["ho"], b["xn"], h=s["h"], gate=s["gate"],
                          w_post=s["w_post"], w_pre=s["w_pre"], rstd=b["rstd"], stream=stream)
        rvq.moe_norm_join_backward(dho, dxn, s["y"], n, d, b["rstd"], ws, h=s["h"], gate=s["gate"],
                                   w_post=s["w_post"], w_pre=s["w_pre"], dh=b["dh"], dy=b["dy"],
                                   dgate=b["dgate"], dw_post=b["dw_post"], dw_pre=b["dw_pre"],
                                   stream=stream)

    a, b, c = bufs(), bufs(), bufs()
    step(a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(b, side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(c)
    graph.replay()
    torch.cuda.synchronize()
    for k in a:
        assert torch.equal(a[k], b[k]) and torch.equal(a[k], c[k]), k


@pytest.mark.parametrize("half", [BF, HF])
@pytest.mark.parametrize("gate", ["token", "channel", "full"])
def test_join_threads_with_four_groups_of_columns(half, gate):
    """The gradients where a thread takes four groups of columns instead of two: 16-bit
    h with more rows than SMs and more than 1024 columns, fp32 h past 4096 columns."""
    for k, (hdt, ydt, xdt, wdt) in enumerate(itertools.product((F32, half), repeat=4)):
        n, d = (3, 4104) if hdt == F32 else (160, 1032)
        s = make(n, d, hdt, ydt, wdt, gate, True, seed=k)
        rstd = check_forward(s, n, d, 0.5, True, hdt, xdt)
        check_backward(s, n, d, 0.5, True, hdt, ydt, xdt, wdt, rstd)


@pytest.mark.parametrize("n,d,dtype", [(152, 2048, BF), (153, 2048, BF), (300, 1024, BF),
                                       (300, 1032, BF), (300, 4096, F32), (300, 4104, F32)])
def test_join_at_the_limits_of_narrow_threads(n, d, dtype):
    s = make(n, d, dtype, dtype, dtype, "channel", True, seed=d)
    rstd = check_forward(s, n, d, 0.75, True, dtype, BF)
    check_backward(s, n, d, 0.75, True, dtype, dtype, BF, dtype, rstd)


@pytest.mark.parametrize("n,d", [(6, 264), (400, 264), (400, 7168), (306, 16384)])
@pytest.mark.parametrize("gate", ["token", "full"])
def test_join_outputs_in_the_place_of_inputs(n, d, gate):
    """Rows of the same type may be written over: h, y and a full gate by the
    outputs, and h, y and a gate per row by the gradients."""
    s = make(n, d, F32, F32, F32, gate, True, seed=n)
    ho, xn, rstd = forward(s, n, d, 1.0, True, F32, F32)
    full = gate == "full"
    for a, b in [("h", "y"), ("y", "h")] + ([("gate", "h"), ("y", "gate")] if full else []):
        t = {k: v.clone() for k, v in s.items()}
        rvq.moe_norm_join(t["y"], n, d, t[a], t[b], h=t["h"], gate=t["gate"], w_post=t["w_post"],
                          w_pre=t["w_pre"], eps=EPS)
        assert torch.equal(t[a], ho) and torch.equal(t[b], xn), (a, b)
    g = gen(3)
    dho, dxn = (torch.randn((n, d), device=DEV, generator=g) for _ in range(2))
    ws = torch.empty(rvq.moe_norm_join_workspace_bytes(n, d), dtype=torch.uint8, device=DEV)

    def back(t, dh, dy, dgate):
        rvq.moe_norm_join_backward(dho, dxn, t["y"], n, d, rstd, ws, h=t["h"], gate=t["gate"],
                                   w_post=t["w_post"], w_pre=t["w_pre"], dh=dh, dy=dy, dgate=dgate)

    want = torch.empty_like(ho), torch.empty_like(ho), torch.empty_like(s["gate"])
    back(s, *want)
    for order in [("h", "y", "gate"), ("y", "h", "gate")] + ([("gate", "h", "y")] if full else []):
        t = {k: v.clone() for k, v in s.items()}
        back(t, *(t[k] for k in order))
        for k, w in zip(order, want):
            assert torch.equal(t[k], w), (order, k)


@pytest.mark.parametrize("n,d", [(3, 264), (400, 264), (310, 8200)])
@pytest.mark.parametrize("scale", [1e-14, 1.0, 1e14])
def test_join_gradients_of_any_scale(n, d, scale):
    """Rows whose norm is far from 1 (eps 0): the gradient's third power of 1/rms is
    beyond fp32, the gradient itself is not."""
    g = gen(n)
    h, y = (torch.randn((n, d), device=DEV, generator=g) * scale for _ in range(2))
    w_pre = torch.randn((d,), device=DEV, generator=g) * 0.1 + 1
    dxn = torch.randn((n, d), device=DEV, generator=g)
    xn, rstd = torch.empty_like(h), torch.empty((2, n), device=DEV)
    rvq.moe_norm_join(y, n, d, None, xn, h=h, alpha=0.5, post_norm=False, w_pre=w_pre, eps=0.0,
                      rstd=rstd)
    ws = torch.empty(rvq.moe_norm_join_workspace_bytes(n, d), dtype=torch.uint8, device=DEV)
    dh, dy, dw = torch.empty_like(h), torch.empty_like(h), torch.empty_like(w_pre)
    rvq.moe_norm_join_backward(None, dxn, y, n, d, rstd, ws, h=h, alpha=0.5, post_norm=False,
                               w_pre=w_pre, dh=dh, dy=dy, dw_pre=dw)
    ho = 0.5 * h.double() + y.double()
    r = 1 / torch.sqrt((ho * ho).mean(1, keepdim=True))
    q = dxn.double() * w_pre.double()
    e = r * q - ho * r ** 3 * (q * ho).mean(1, keepdim=True)
    # magnitudes of the terms times the errors met on the way: 1/rms and the row's sum
    # are each good to 64 half steps, the rest are a dozen operations
    mag = r * q.abs() + ho.abs() * r ** 3 * (q * ho).abs().mean(1, keepdim=True)
    err = 4 * 80 * U * mag
    R.check(dh, (0.5 * e, 0.5 * err), "dh")
    R.check(dy, (e, err), "dy")
    t = dxn.double() * ho * r
    R.check(dw, (t.sum(0), (80 + n) * U * t.abs().sum(0)), "dw_pre")


@pytest.mark.parametrize("d,wdt", [(5632, F32), (6144, F32), (6152, F32), (7168, BF), (7176, BF)])
def test_join_where_the_ring_gets_shorter(d, wdt):
    """fp32 rows at the ends of two of them in shared memory for the gradients: 6144
    columns with fp32 gains and 16-bit xn, 7168 with 16-bit gains."""
    n = 320
    for xdt in (BF, F32):
        s = make(n, d, F32, F32, wdt, "token", True, seed=d)
        rstd = check_forward(s, n, d, 1.0, True, F32, xdt)
        check_backward(s, n, d, 1.0, True, F32, F32, xdt, wdt, rstd)

"""GPU parity of moe_route_scored and its gradient against the float64 definition:
scores, biases, groups, ties and near ties, both ways of grouping, the layer call."""
import numpy as np
import pytest
import torch

from tests import route_ref as S

pytestmark = pytest.mark.gpu
rvq = pytest.importorskip("moe_expert_ffn_router_gb300")
DEV = "cuda"
F32, I32 = torch.float32, torch.int32
U = 2.0 ** -24


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def buffers(n, E, k):
    ws = torch.zeros(rvq.moe_route_scored_workspace_bytes(n, E), dtype=torch.uint8, device=DEV)
    return dict(topk_idx=torch.full((n, k), -7, dtype=I32, device=DEV),
                topk_w=torch.full((n, k), -7.0, device=DEV),
                offsets=torch.full((E + 1,), -7, dtype=I32, device=DEV),
                pairs=torch.full((n * k,), -7, dtype=I32, device=DEV), ws=ws)


def check(l, k, score, bias, groups, top, renorm, scale, status=(0, 0)):
    """Choice, offsets and pairs equal; weights within their error: the arguments of at
    most two exponentials are within |l| 2^-24 of the exact ones each, and a dozen
    roundings of sums and quotients."""
    n, E = l.shape
    b = buffers(n, E, k)
    kw = dict(score=rvq.MOE_SCORES[score], renorm=renorm, scale=scale)
    rvq.moe_route_scored(l, n, E, k, **b, bias=bias, groups=groups, top_groups=top, **kw)
    assert rvq.rvq_ws_status(b["ws"]) == status
    idx = S.choice(l, k, score, bias, groups, top)
    assert torch.equal(b["topk_idx"].long(), idx)
    off, pairs = S.grouping(idx, E)
    assert torch.equal(b["offsets"].long(), off) and torch.equal(b["pairs"].long(), pairs)
    w = S.weights(l, idx, score, renorm, scale)
    spread = (l.amax(1) - l.amin(1)).clamp(min=l.abs().amax(1)).double().unsqueeze(1)
    rel = (4 * spread + 64) * U
    assert ((b["topk_w"].double() - w).abs() <= rel * w + 1e-37).all()
    dw = torch.randn((n, k), device=DEV, generator=gen(1))
    dl = torch.full((n, E), 99.0, device=DEV)
    rvq.moe_route_scored_backward(dw, l, b["topk_idx"], n, E, k, dl, **kw)
    want = S.gradient(l, idx, dw, score, renorm, scale)
    # terms of both signs: the error is relative to the sum of their magnitudes
    ws_ = w.abs() / abs(scale)
    mag = (dw.double().abs() + (dw.double().abs() * ws_).sum(1, keepdim=True)) * abs(scale)
    p = S.scores(l, score)
    full = torch.zeros((n, E), dtype=torch.float64, device=DEV)
    if renorm:
        full.scatter_(1, idx, mag * ws_)
    elif score == "sigmoid":
        full.scatter_(1, idx, mag * p.gather(1, idx))
    else:
        full.scatter_(1, idx, mag)
        full = p * (full + (dw.double().abs() * p.gather(1, idx)).sum(1, keepdim=True) * abs(scale))
    assert ((dl.double() - want).abs() <= 2 * rel * full + 1e-37).all()
    return b


SHAPES = [(1, 256, 16), (1, 1, 1), (3, 8, 2), (64, 64, 8), (65, 64, 8), (8, 256, 32),
          (9, 33, 5), (300, 100, 7), (1500, 256, 16), (1191, 40, 3)]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm,scale,biased", [(True, 2.5, True), (True, 1.0, False),
                                                 (False, 1.0, True), (False, 2.5, False)])
@pytest.mark.parametrize("n,E,k", SHAPES)
def test_plain(n, E, k, score, renorm, scale, biased):
    g = gen(n * 1009 + E * 31 + k)
    l = torch.randn((n, E), device=DEV, generator=g) * 1.5
    bias = torch.randn((E,), device=DEV, generator=g) * 0.05 if biased else None
    check(l, k, score, bias, 1, 1, renorm, scale)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("n,E,k,groups,top", [(1, 256, 16, 8, 4), (70, 256, 8, 8, 1),
                                              (33, 60, 5, 5, 2), (200, 64, 4, 32, 3),
                                              (17, 16, 3, 16, 4), (500, 96, 12, 3, 2),
                                              (40, 256, 32, 2, 1), (5, 32, 8, 32, 31),
                                              (30, 192, 8, 2, 1), (21, 256, 8, 4, 2),
                                              (25, 128, 6, 4, 1), (12, 64, 5, 2, 1)])
def test_groups(n, E, k, groups, top, score):
    g = gen(n + E + groups)
    l = torch.randn((n, E), device=DEV, generator=g) * 1.5
    bias = torch.randn((E,), device=DEV, generator=g) * 0.1
    check(l, k, score, bias, groups, top, True, 1.0)
    check(l, k, score, None, groups, top, False, 1.0)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups,top", [(1, 1), (8, 3)])
@pytest.mark.parametrize("n", [6, 20, 200])
def test_ties_and_near_ties(n, groups, top, score):
    """Logits from few values, all equal, and an ulp apart, with biases that cancel what
    32 bits tell apart: the choice is the 64-bit one."""
    g = gen(3)
    few = torch.randint(-2, 3, (n, 64), device=DEV, generator=g).float()
    check(few, 8, score, None, groups, top, True, 1.0)
    check(few, 8, score, torch.randint(0, 2, (64,), device=DEV, generator=g).float() / 8, groups,
          top, True, 1.0)
    check(torch.zeros((n, 64), device=DEV), 8, score, None, groups, top, True, 1.0)
    ulp = 1.0 + torch.randint(0, 4, (n, 64), device=DEV, generator=g).float() * 2.0 ** -23
    check(ulp, 8, score, None, groups, top, False, 1.0)
    # c of all experts within a few 2^-24 of one another
    l = torch.randn((n, 64), device=DEV, generator=g)
    p = S.scores(l[:1], score)[0]
    noise = torch.randn((64,), device=DEV, generator=g).double() * 2.0 ** -24
    bias = (1 - p + noise).float()
    check(l[:1].expand(n, -1).contiguous(), 8, score, bias, groups, top, True, 1.0)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_extreme_logits(score):
    """Very large and very negative logits: weights keep their ratios and stay finite."""
    g = gen(4)
    for shift in (-200.0, -88.0, 80.0, 300.0):
        l = torch.randn((12, 32), device=DEV, generator=g) * 3 + shift
        check(l, 4, score, None, 1, 1, True, 1.0)
    l = torch.randn((5, 32), device=DEV, generator=g) * 40
    check(l, 4, score, None, 1, 1, True, 1.0)
    check(l, 4, score, None, 1, 1, False, 1.0)


@pytest.mark.parametrize("biased", [False, True])
def test_saturated_scores(biased):
    """Logits whose sigmoids are 1 (or 0) in 64 bits, and nearly so, among groups: ties go
    to the lower group, and scores a 2^-53 apart keep their order."""
    g = gen(12)
    for scale, shift in ((3.0, 34.0), (1.0, 17.0), (0.5, 60.0), (4.0, -40.0), (20.0, 0.0)):
        l = torch.randn((90, 64), device=DEV, generator=g) * scale + shift
        bias = torch.randint(-2, 3, (64,), device=DEV, generator=g).float() * 2.0 ** -50 if biased \
            else None
        idx = S.choice(l, 6, "sigmoid", bias, 8, 3)
        b = buffers(90, 64, 6)
        rvq.moe_route_scored(l, 90, 64, 6, **b, bias=bias, groups=8, top_groups=3)
        assert torch.equal(b["topk_idx"].long(), idx), (scale, shift)
        assert torch.equal(b["pairs"].long(), S.grouping(idx, 64)[1])


@pytest.mark.parametrize("n", [5, 130])
def test_non_finite_is_reported(n):
    """A logit or bias that is not finite counts as 0, and everything stays in range."""
    g = gen(6)
    l = torch.randn((n, 64), device=DEV, generator=g)
    bias = torch.randn((64,), device=DEV, generator=g) * 0.1
    bad, bb = l.clone(), bias.clone()
    bad[2, 5], bad[3, 7], bad[4] = float("nan"), float("inf"), -float("inf")
    bb[9] = float("nan")
    fixed, fb = bad.nan_to_num(0, 0, 0), bb.nan_to_num(0)
    for groups, top in ((1, 1), (8, 2)):
        b = buffers(n, 64, 8)
        rvq.moe_route_scored(bad, n, 64, 8, **b, bias=bb, groups=groups, top_groups=top)
        assert rvq.rvq_ws_status(b["ws"]) == (5, 2)
        want = S.choice(fixed, 8, "sigmoid", fb, groups, top)
        assert torch.equal(b["topk_idx"].long(), want)
        assert torch.equal(b["pairs"].long(), S.grouping(want, 64)[1])
        assert torch.isfinite(b["topk_w"]).all()


@pytest.mark.parametrize("score,renorm", [("sigmoid", True), ("softmax", False)])
def test_gradient_in_place_and_stray_indices(score, renorm):
    """dlogits in the logits' place; indices outside the experts take no part; the same
    expert twice adds up."""
    n, E, k = 33, 40, 4
    l = torch.randn((n, E), device=DEV, generator=gen(8))
    idx = S.choice(l, k, score, None, 1, 1).int()
    dw = torch.randn((n, k), device=DEV, generator=gen(9))
    kw = dict(score=rvq.MOE_SCORES[score], renorm=renorm)
    want = torch.empty((n, E), device=DEV)
    rvq.moe_route_scored_backward(dw, l, idx, n, E, k, want, **kw)
    got = l.clone()
    rvq.moe_route_scored_backward(dw, got, idx, n, E, k, got, **kw)
    assert torch.equal(got, want)
    stray = torch.cat([idx, torch.full((n, 2), E, dtype=I32, device=DEV)], 1)
    stray[:, 5] = -1
    dw2 = torch.cat([dw, torch.full((n, 2), 1e6, device=DEV)], 1)
    rvq.moe_route_scored_backward(dw2, l, stray.contiguous(), n, E, k + 2, got, **kw)
    assert torch.equal(got, want)
    if not renorm:
        twice = torch.cat([idx, idx[:, :1]], 1).contiguous()
        dw3 = torch.cat([dw, dw[:, :1]], 1).contiguous()
        merged = dw.clone()
        merged[:, 0] *= 2
        rvq.moe_route_scored_backward(dw3, l, twice, n, E, k + 1, got, **kw)
        rvq.moe_route_scored_backward(merged, l, idx, n, E, k, want, **kw)
        assert torch.allclose(got, want, rtol=1e-5, atol=1e-7)


def test_many_tokens():
    check(torch.randn((20000, 64), device=DEV, generator=gen(10)), 6, "sigmoid", None, 1, 1, True,
          1.0)
    n = 262144
    l = torch.randn((n, 8), device=DEV, generator=gen(11))
    b = buffers(n, 8, 2)
    rvq.moe_route_scored(l, n, 8, 2, **b)
    idx = S.choice(l, 2, "sigmoid", None, 1, 1)
    assert torch.equal(b["topk_idx"].long(), idx)
    off, pairs = S.grouping(idx, 8)
    assert torch.equal(b["offsets"].long(), off) and torch.equal(b["pairs"].long(), pairs)


def test_streams_and_graph():
    """Two calls at once on two streams, and a captured call replayed on new logits."""
    for n in (7, 20, 500):
        ls = [torch.randn((n, 64), device=DEV, generator=gen(20 + i)) for i in range(3)]
        bs = [buffers(n, 64, 8) for _ in range(3)]
        streams = [torch.cuda.Stream() for _ in range(2)]
        torch.cuda.synchronize()
        for _ in range(8):
            for i, s in enumerate(streams):
                rvq.moe_route_scored(ls[i], n, 64, 8, **bs[i], stream=s)
        torch.cuda.synchronize()
        l = ls[2].clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            rvq.moe_route_scored(l, n, 64, 8, **bs[2])
        for i in range(3):
            l.copy_(ls[i])
            graph.replay()
            torch.cuda.synchronize()
            idx = S.choice(ls[i], 8, "sigmoid", None, 1, 1)
            for b in (bs[2],) + ((bs[i],) if i < 2 else ()):
                assert torch.equal(b["topk_idx"].long(), idx)
                assert torch.equal(b["pairs"].long(), S.grouping(idx, 64)[1])


@pytest.mark.parametrize("n,tc", [(1, 0), (3, 0), (70, 0), (70, 1), (200, 6)])
def test_layer(n, tc):
    """The layer call with a rule: the separate calls' routing, and the combine of the
    experts that it chose."""
    from moe_expert_ffn_router_gb300.layer import MoeLayer, MoeStack
    from synth import workloads as W
    shape = W.LayerShape(d=512, f=512, E=16, k=4)
    src = W.ExpertSource(5, 0, shape)
    L = MoeLayer(16, 512, 512, 4)
    for e in range(16):
        mats = [(src.codes(e, m), src.codebooks(e, m)) for m in range(3)]
        L.load_expert(e, mats[0][0], mats[1][0], mats[2][0], np.stack([c for _, c in mats]))
    L.set_router(W.router_weight(src.lseed, 16, 512))
    bias = torch.randn((16,), device=DEV, generator=gen(2)) * 0.1
    L.set_scoring(bias=bias, groups=4, top_groups=2, scale=2.0)
    x = torch.randn((n, 512), device=DEV, generator=gen(n)).to(torch.bfloat16)
    b = L.forward(x, tc_min_tokens=tc)
    torch.cuda.synchronize()
    assert L.status(n) == (0, 0)
    idx = S.choice(b["logits"], 4, "sigmoid", bias, 4, 2)
    assert torch.equal(b["idx"].long(), idx)
    assert torch.equal(b["pairs"].long(), S.grouping(idx, 16)[1])
    s = L.forward_steps(x)
    for key in ("idx", "w", "offsets", "pairs"):
        assert torch.equal(s[key], b[key]), key
    want = x.double() + (s["y_pair"].view(n, 4, -1).double() * s["w"].double().unsqueeze(2)).sum(1)
    assert torch.allclose(s["out"].double(), want, rtol=1e-5, atol=1e-5)
    err = (b["out"].double() - want).abs().max() / (want - x.double()).square().mean().sqrt()
    assert err <= (2e-2 if tc else 1e-4), err
    if tc == 0:
        h = MoeStack([L]).forward(x.float())[0]
        assert torch.equal(h["idx"].long(), S.choice(h["logits"], 4, "sigmoid", bias, 4, 2))


@pytest.mark.parametrize("n", [5, 130])
@pytest.mark.parametrize("score,renorm", [("sigmoid", True), ("sigmoid", False),
                                          ("softmax", True), ("softmax", False)])
def test_gradient_of_non_finite_logits(score, renorm, n):
    """NaN and infinities, chosen and not: the gradient of the weights that the forward
    call returned, which took such a logit as 0."""
    E, k = 64, 8
    l = torch.randn((n, E), device=DEV, generator=gen(31))
    dw = torch.randn((n, k), device=DEV, generator=gen(32))
    bad = l.clone()
    bad[0, 3], bad[1, 7], bad[2, 9] = float("nan"), float("inf"), -float("inf")
    bad[3, :40] = float("nan")
    bad[4] = float("inf")
    fixed = bad.nan_to_num(0, 0, 0)
    idx = S.choice(fixed, k, score, None, 1, 1)
    idx[0, k - 1], idx[1, k - 1], idx[2, k - 1] = 3, 7, 9       # chosen all the same
    # and choices that are not the largest
    idx[:, 0] = torch.where(torch.arange(n, device=DEV) % 2 == 0, idx[:, 0], idx[:, 1])
    idx[:, 1] = torch.where(idx[:, 0] == idx[:, 1], 63 - idx[:, 1], idx[:, 1])
    kw = dict(score=rvq.MOE_SCORES[score], renorm=renorm, scale=2.5)
    got = {}
    for name, rows in (("bad", bad), ("fixed", fixed)):
        got[name] = torch.full((n, E), 99.0, device=DEV)
        rvq.moe_route_scored_backward(dw, rows, idx.int(), n, E, k, got[name], **kw)
    assert torch.equal(got["bad"], got["fixed"])
    want = S.gradient(fixed, idx, dw, score, renorm, 2.5)
    # terms of at most the sum of the magnitudes of scale dw, each after two exponentials
    # (two units of the last place and |l| 2^-24, |l| < 8), sums of up to 64 terms and a
    # few products and quotients
    bound = 256 * U * 2.5 * dw.double().abs().sum(1, keepdim=True)
    assert ((got["bad"].double() - want).abs() <= bound).all()
    place = bad.clone()
    rvq.moe_route_scored_backward(dw, place, idx.int(), n, E, k, place, **kw)
    assert torch.equal(place, got["bad"])


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("big", [1.0, 40.0, 1000.0, 1e5])
@pytest.mark.parametrize("E,groups,top,k", [(64, 8, 3, 4), (256, 8, 4, 8), (60, 5, 2, 3)])
def test_groups_of_large_biases_of_both_signs(E, groups, top, k, big, score):
    """A group's two largest c are about +big and -big: their sum is the scores', which 32
    bits of c do not hold."""
    n = 3000
    g = gen(51)
    l = torch.randn((n, E), device=DEV, generator=g)
    bias = torch.full((groups, E // groups), -big, device=DEV)
    bias[:, 1] = big
    bias = bias.view(-1) + torch.randint(0, 2, (E,), device=DEV, generator=g) * (big / 1024)
    b = buffers(n, E, k)
    for biases in (bias, bias.view(groups, -1).roll(1, 0).reshape(-1).contiguous()):
        rvq.moe_route_scored(l, n, E, k, **b, score=rvq.MOE_SCORES[score], bias=biases,
                             groups=groups, top_groups=top)
        assert rvq.rvq_ws_status(b["ws"]) == (0, 0)
        idx = S.choice(l, k, score, biases, groups, top)
        assert torch.equal(b["topk_idx"].long(), idx)

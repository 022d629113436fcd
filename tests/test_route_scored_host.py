"""Host side of the scored router (no GPU): sizes and refusals before any launch; the
tests' definition against differences."""
import ctypes

import pytest
import torch

import moe_expert_ffn_router_gb300 as rvq
from tests import route_ref as S

lib = rvq._lib
A = 0x10000000       # fake, aligned "device" addresses far apart (never dereferenced)
B, C, D, E_, F = (A + i * 0x10000000 for i in range(1, 6))
OK, EINVAL, EALIGN, ENOMEM = 0, 1, 2, 3
F32 = 0


def rule(score=1, bias=None, groups=1, top=1, renorm=1, scale=1.0):
    return rvq.MoeRouteRule(score, bias, groups, top, renorm, scale)


def test_workspace():
    f = rvq.moe_route_scored_workspace_bytes
    assert f(1, 256) == 256 and f(8, 256) == 256
    last = 0
    for n in (9, 64, 100, 1000, 1184, 2048, 262144):
        assert f(n, 256) >= max(last, 256 + min(148, (n + 7) // 8) * 1024)
        last = f(n, 256)
    for n, e in ((0, 8), (-1, 8), (262145, 8), (1, 0), (1, 257)):
        assert f(n, e) == 0


ROUTE = dict(logits=A, n=70, E=64, k=8, rule=rule(), idx=B, w=C, off=D, pairs=E_, ws=F,
             wsb=1 << 20, st=None)


def test_refusals():
    def route(**kw):
        return lib.moe_route_scored(*{**ROUTE, **kw}.values())

    G = F + 0x10000000
    for bad in (dict(n=0), dict(n=262145), dict(E=0), dict(E=257), dict(k=0), dict(k=33),
                dict(k=65), dict(rule=None), dict(rule=rule(score=2)), dict(rule=rule(score=-1)),
                dict(rule=rule(groups=0)), dict(rule=rule(groups=3)), dict(rule=rule(groups=64)),
                dict(rule=rule(groups=8, top=0)), dict(rule=rule(groups=8, top=9)),
                dict(rule=rule(groups=16, top=1)), dict(rule=rule(scale=float("nan"))),
                dict(logits=None), dict(idx=None), dict(w=None), dict(off=None), dict(pairs=None),
                dict(idx=A), dict(w=B), dict(pairs=C), dict(off=A + 64), dict(ws=None),
                dict(ws=F + 16), dict(rule=rule(bias=D)), dict(rule=rule(bias=E_ + 4))):
        assert route(**bad) == EINVAL, bad
    for bad in (dict(logits=A + 2), dict(idx=B + 1), dict(w=C + 2), dict(off=D + 2),
                dict(pairs=E_ + 3), dict(rule=rule(bias=G + 2))):
        assert route(**bad) == EALIGN, bad
    assert route(wsb=rvq.moe_route_scored_workspace_bytes(70, 64) - 1) == ENOMEM


def test_backward_refusals():
    base = dict(dw=A, logits=B, idx=C, n=4, E=64, k=8, rule=rule(), dl=D, st=None)

    def back(**kw):
        return lib.moe_route_scored_backward(*{**base, **kw}.values())

    for bad in (dict(n=0), dict(k=40), dict(E=300), dict(rule=None), dict(rule=rule(score=7)),
                dict(dw=None), dict(logits=None), dict(idx=None), dict(dl=None), dict(dl=A),
                dict(dl=C), dict(dl=B + 4), dict(dl=B - 4)):
        assert back(**bad) == EINVAL, bad
    for bad in (dict(dw=A + 2), dict(logits=B + 2), dict(idx=C + 2), dict(dl=D + 2)):
        assert back(**bad) == EALIGN, bad


def test_binding_refusals():
    f, i = torch.zeros(4 * 8), torch.zeros(4 * 2, dtype=torch.int32)
    w, off, ws = torch.zeros(4 * 2), torch.zeros(9, dtype=torch.int32), torch.zeros(256)
    with pytest.raises(ValueError, match="logits"):
        rvq.moe_route_scored(f[:16], 4, 8, 2, i, w, off, i, ws)
    with pytest.raises(TypeError, match="topk_idx"):
        rvq.moe_route_scored(f, 4, 8, 2, i.long(), w, off, i, ws)
    with pytest.raises(TypeError, match="bias"):
        rvq.moe_route_scored(f, 4, 8, 2, i, w, off, i, ws, bias=torch.zeros(8).double())
    with pytest.raises(ValueError, match="dlogits"):
        rvq.moe_route_scored_backward(w, f, i, 4, 8, 2, f[:8])


def test_layer_refuses_calls_that_choose_by_logits():
    from moe_expert_ffn_router_gb300.layer import MoeLayer
    layer = MoeLayer.__new__(MoeLayer)
    layer.E, layer.device, layer.rule = 8, torch.device("cpu"), None
    layer._by_logits("graph")
    layer.set_scoring(groups=2, top_groups=1)
    for call in (lambda: layer.forward_host(None, None), lambda: layer.graph(None, None)):
        with pytest.raises(ValueError, match="scores its experts"):
            call()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_definition_gradient(score, renorm):
    """The formula's gradient against central differences of the weights."""
    g = torch.Generator().manual_seed(1)
    l = torch.randn((3, 12), generator=g).double()
    dw = torch.randn((3, 4), generator=g).double()
    idx = S.choice(l, 4, score, None, 3, 2)
    got = S.gradient(l, idx, dw, score, renorm, 2.5)
    h = 1e-5
    for t in range(3):
        for e in range(12):
            d = torch.zeros_like(l)
            d[t, e] = h
            up, dn = (S.weights(l + s * d, idx, score, renorm, 2.5) for s in (1, -1))
            diff = float(((up - dn) * dw).sum() / (2 * h))
            assert abs(diff - float(got[t, e])) <= 1e-7
    # the header's form
    p = S.scores(l, score)
    ps = p.gather(1, idx)
    dp = 2.5 * dw
    if renorm:
        P = ps.sum(1, keepdim=True)
        dp = 2.5 * (dw - (dw * ps).sum(1, keepdim=True) / P) / P
    full = torch.zeros_like(l).scatter_(1, idx, dp)
    want = full * p * (1 - p) if score == "sigmoid" else p * (full - (dp * ps).sum(1, keepdim=True))
    assert torch.allclose(got, want, rtol=1e-12, atol=1e-14)


def test_definition_choice():
    l = torch.tensor([[0., 1., 2., 3., 3., 2., 1., 0.]])
    assert S.choice(l, 4, "sigmoid", None, 1, 1).tolist() == [[3, 4, 2, 5]]
    assert S.choice(l, 2, "softmax", None, 4, 1).tolist() == [[3, 2]]
    b = torch.tensor([5., 0, 0, 0, 0, 0, 0, 0])
    assert S.choice(l, 2, "sigmoid", b, 4, 1).tolist() == [[0, 1]]
    off, pairs = S.grouping(torch.tensor([[1, 0], [1, 2]]), 4)
    assert off.tolist() == [0, 1, 3, 4, 4] and pairs.tolist() == [1, 0, 2, 3]


def test_layer_refuses_a_rule_of_other_experts():
    """A rule's bias is as long as the bank has experts and on the call's device: the
    layer call would read behind it, or where the GPU cannot."""
    class Fake:
        device_index, cuda_stream = 0, 0

    bank = rvq.RvqMoeBank()
    rb = rvq.moe_bank_record_bytes(512, 512)
    assert lib.moe_bank_init(ctypes.byref(bank), A, rb * 32, 32, 512, 512, 0) == OK
    x = torch.zeros((4, 512))
    i32, f32 = torch.zeros(128, dtype=torch.int32), torch.zeros((4, 32))
    ws = torch.zeros(1 << 20, dtype=torch.uint8)

    def forward(rule):
        rvq.moe_layer_forward(bank, x, None, x, 4, 4, f32, i32, f32, i32, i32, x, ws, rule=rule,
                              stream=Fake())

    for n in (16, 64):
        with pytest.raises(ValueError, match="bias"):
            forward(rvq.moe_route_rule(n, bias=torch.zeros(n)))
    with pytest.raises(ValueError, match="on cpu, the call on cuda:0"):
        forward(rvq.moe_route_rule(32, bias=torch.zeros(32)))


@pytest.mark.parametrize("E,most", [(256, 4224), (64, 17024)])
def test_layer_token_limit(E, most):
    """The layer call takes as many tokens as the layer calls by logits; more are refused
    before any launch, as the header says."""
    assert rvq.moe_route_max_tokens(E) == most
    bank = rvq.RvqMoeBank()
    rb = rvq.moe_bank_record_bytes(512, 512)
    assert lib.moe_bank_init(ctypes.byref(bank), A, rb * E, E, 512, 512, 0) == OK

    def layer(n, ws):
        return lib.moe_layer_forward_scored(ctypes.byref(bank), A, None, rule(), A, F32, n, 4, B, C,
                                            D, E_, E_ + 0x1000000, F, F + 0x8000000, ws, None, F32,
                                            0, None, None)

    assert layer(most + 1, 1 << 60) == EINVAL
    assert f"max {most}".encode() in lib.rvq_last_error()
    assert layer(most, 0) == ENOMEM

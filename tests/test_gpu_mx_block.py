"""Blocks whose shared expert is microscaled and whose experts are scored, through the
classes a program uses: every call of a pass against its definition, on what the call
was given."""
import numpy as np
import pytest
import torch

import oracle
from synth import workloads as W
from tests import dense_ref as R
from tests import mx_ref as X
from tests import route_ref as S

pytestmark = pytest.mark.gpu
rvq = pytest.importorskip("moe_expert_ffn_router_gb300")
DEV, BF = "cuda", torch.bfloat16
D, F, E, K = 1024, 512, 8, 2
F8, F4 = X.F8, X.F4


def normal(shape, g, std, mean=0.0, dtype=BF):
    return (torch.randn(shape, device=DEV, generator=g) * std + mean).to(dtype)


def build(formats):
    from moe_expert_ffn_router_gb300.layer import (MoeLayer, MxSharedExpert, SharedExpert,
                                                   SharedExpertStack)
    g = torch.Generator(device=DEV).manual_seed(3)
    shape = W.LayerShape(d=D, f=F, E=E, k=K)
    blocks, sources = [], []
    for i, fmt in enumerate(formats):
        src = W.ExpertSource(98, i, shape)
        L = MoeLayer(E, D, F, K, layer=i)
        experts = {}
        for e in range(E):
            mats = [(src.codes(e, m), src.codebooks(e, m)) for m in range(3)]
            experts[e] = tuple(mats)
            L.load_expert(e, mats[0][0], mats[1][0], mats[2][0], np.stack([c for _, c in mats]))
        wr = W.router_weight(src.lseed, E, D)
        L.set_router(wr)
        L.set_scoring(bias=torch.randn((E,), device=DEV, generator=g) * 0.1, groups=4,
                      top_groups=2, scale=1.5)
        ws = [normal((F, D), g, D ** -0.5), normal((F, D), g, D ** -0.5),
              normal((D, F), g, F ** -0.5)]
        shared = SharedExpert(*ws) if fmt is None else MxSharedExpert(*ws, xfmt=fmt[0], wfmt=fmt[1])
        p = dict(w_pre=normal((D,), g, 0.1, 1.0), w_post=normal((D,), g, 0.1, 1.0),
                 gate=[None, normal((1, D), g, 0.1, 0.5, torch.float32)][i % 2])
        blocks.append((L, shared, p))
        sources.append((experts, wr))
    return SharedExpertStack(blocks, alpha=0.9), sources


def values(q, rows, cols, fmt):
    return X.dequantize(q[0], q[1], rows, cols, fmt)


@pytest.mark.parametrize("n,tc", [(1, 0), (70, 0), (300, 1)])
def test_stack(n, tc):
    """A microscaled block, a dense one, and another microscaled one."""
    stack, sources = build([(F8, F4), None, (F4, F4)])
    x = torch.randn((n, D), device=DEV, generator=torch.Generator(device=DEV).manual_seed(n))
    bufs = stack.forward(x, tc_min_tokens=tc)
    torch.cuda.synchronize()
    h = x
    for i, (L, sh, p) in enumerate(stack.blocks):
        b = bufs[i]
        assert L.status(n) == (0, 0) and sh.status(n) == (0, 0)
        # the choice
        idx = S.choice(b["logits"], K, "sigmoid", L.rule.keep, 4, 2)
        assert torch.equal(b["idx"].long(), idx)
        w = S.weights(b["logits"], idx, "sigmoid", True, 1.5)
        assert ((b["w"].double() - w).abs() <= 256 * R.U32 * w).all()
        # the normed rows in both types
        _, xn, *_ = R.join(None, h, 1.0, None, False, None, p["w_pre"], stack.eps)
        en = 256 * R.U32 * xn.abs() + 80 * R.U32
        R.check(b["xn"], (xn, en + R.half_step(BF) * xn.abs()), f"xn {i}")
        # the shared expert of the rows that it was given
        if i != 1:
            sb = sh.buffers(n)
            X.check_quantized(*sb["x"], n, D, sh.xfmt, xn, en, f"x {i}")
            vx = values(sb["x"], n, D, sh.xfmt)
            wg, wu = (values(q, F, D, sh.wfmt) for q in (sh.wg, sh.wu))
            a, u = vx @ wg.t(), vx @ wu.t()
            ea, eu = (R.product(vx, q)[1] for q in (wg, wu))
            hid = R.act("silu", a) * u
            eh = 1.2 * (ea + 16 * R.U32 * a.abs()) * u.abs() + a.abs() * eu + 4 * R.U32 * hid.abs()
            X.check_quantized(*sb["hidden"], n, F, sh.xfmt, hid, eh, f"hidden {i}")
            vh = values(sb["hidden"], n, F, sh.xfmt)
            y, ey = R.product(vh, values(sh.wd, D, F, sh.wfmt))
            R.check(sb["out"], (y, ey + 4 * R.U32 * y.abs()), f"shared {i}")
            shared = sb["out"].double()
        else:
            shared = sh.buffers(n)["out"].double()
        # the routed experts of the choice
        experts, _ = sources[i]
        x64 = b["xn"].double().cpu().numpy()
        routed = torch.zeros((n, D), dtype=torch.float64, device=DEV)
        few = range(min(n, 4))
        for t in few:
            for s in range(K):
                one = oracle.moe_layer(lambda e: experts[int(idx[t, s])], np.zeros((1, D), np.float32),
                                       x64[t:t + 1], 1, D, F, route_logits=np.zeros((1, 1), np.float32))
                out = torch.from_numpy(one["out"]).to(DEV)[0] - b["xn"][t].double()
                routed[t] += out * b["w"][t, s].double()
        want = (shared + routed)[:len(few)]
        tol = (2e-2 if tc else 1e-4) * routed[:len(few)].square().mean().sqrt()
        assert ((b["out"].double()[:len(few)] - want).abs() <= tol + 4 * R.U32 * want.abs()).all()
        ho, *_ = R.join(h, b["out"], 0.9, p["gate"], True, p["w_post"], None, stack.eps)
        R.check(b["h"], (ho, 80 * R.U32 * (ho.abs() + 0.9 * h.double().abs())), f"h {i}")
        h = b["h"]


def test_shared_expert_alone():
    """forward() quantises its tokens; the residual joins in; batch sizes keep their own
    buffers; a pass in a graph is replayed on new tokens."""
    from moe_expert_ffn_router_gb300.layer import MxSharedExpert
    g = torch.Generator(device=DEV).manual_seed(5)
    sh = MxSharedExpert(normal((264, 520), g, 0.05), normal((264, 520), g, 0.05),
                        normal((520, 264), g, 0.05, dtype=torch.float32))
    for n in (1, 130, 7):
        x, res = normal((n, 520), g, 1.0), normal((n, 520), g, 1.0, dtype=torch.float32)
        b = sh.forward(x, res)
        q, byte = X.quantize(x, F8)
        assert torch.equal(X.values(F8, DEV)[X.unpack(b["x"][0], n, 520, F8)], q)
        assert torch.equal(X.from_tiles(b["x"][1], n, 520), byte)
        vh = values(b["hidden"], n, 264, F8)
        y, ey = R.product(vh, values(sh.wd, 520, 264, F4))
        y = y + res.double()
        R.check(b["out"], (y, ey + 4 * R.U32 * y.abs()), "out")
        assert sh.status(n) == (0, 0)
    x = normal((7, 520), g, 1.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sh.forward(x)
    for _ in range(2):
        x.copy_(normal((7, 520), g, 1.0))
        graph.replay()
        torch.cuda.synchronize()
        got = sh.buffers(7)["out"].clone()
        assert torch.equal(got, sh.forward(x)["out"])


def test_example_leaves_the_given_stack():
    """The example's microscaled stack scores its experts; the stack that it was made from
    still chooses by logits, and gives the same bits."""
    import importlib.util
    import os
    at = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                      "shared_expert.py")
    spec = importlib.util.spec_from_file_location("shared_expert_example", at)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    stack = example.build(torch, n_blocks=2, d=512, f=512, n_experts=8, k=2)
    x = torch.randn((5, 512), device=DEV, generator=torch.Generator(device=DEV).manual_seed(1))
    keys = ("logits", "idx", "w", "out", "h")
    before = [{k: b[k].clone() for k in keys} for b in stack.forward(x)]
    mx = example.microscaled(torch, stack)
    for b in mx.forward(x):
        assert torch.equal(b["idx"].long(), S.choice(b["logits"], 2, "sigmoid", None, 4, 2))
    for L, _, _ in stack.blocks:
        assert L.rule is None
    for b, want in zip(stack.forward(x), before):
        assert all(torch.equal(b[k], want[k]) for k in keys)


@pytest.mark.parametrize("n", [1, 9, 130])
def test_stack_in_a_graph_and_on_a_stream(n):
    """A whole pass captured and replayed on new tokens, and one on a side stream, between
    passes of another batch size: the bits of a pass alone."""
    stack, _ = build([(F8, F4), (F4, F4)])
    g = torch.Generator(device=DEV).manual_seed(n)
    xs = [torch.randn((n, D), device=DEV, generator=g) for _ in range(3)]
    keys = ("logits", "idx", "w", "offsets", "pairs", "out", "h")

    def outputs(bufs):
        torch.cuda.synchronize()
        return [{k: b[k].clone() for k in keys} for b in bufs]

    def same(a, b):
        return all(torch.equal(p[k], q[k]) for p, q in zip(a, b) for k in keys)

    alone = [outputs(stack.forward(x)) for x in xs]
    x = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bufs = stack.forward(x)
    other = torch.randn((5, D), device=DEV, generator=g)
    for i in (2, 0, 1):
        x.copy_(xs[i])
        stack.forward(other)
        graph.replay()
        assert same(outputs(bufs), alone[i]), i
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        bufs = stack.forward(xs[2])
    assert same(outputs(bufs), alone[2])
    for L, sh, _ in stack.blocks:
        assert L.status(n) == (0, 0) and sh.status(n) == (0, 0)

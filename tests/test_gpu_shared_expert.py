"""The shared expert and the stack of blocks around it, through the classes a
program uses: the block's sum against the oracle's routed experts and a float64
shared expert, the joins against their definition, gradients of the whole shared
expert, and the example."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle
import synth
from synth import workloads as W
from tests import dense_ref as R

pytestmark = pytest.mark.gpu
pytest.importorskip("moe_expert_ffn_router_gb300")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEV, BF = "cuda", torch.bfloat16
D, F, E, K = 1024, 512, 8, 2


def build(n_blocks=2):
    from moe_expert_ffn_router_gb300.layer import MoeLayer, SharedExpert, SharedExpertStack
    g = torch.Generator(device=DEV).manual_seed(3)

    def normal(shape, std, mean=0.0, dtype=BF):
        return (torch.randn(shape, device=DEV, generator=g) * std + mean).to(dtype)

    shape = W.LayerShape(d=D, f=F, E=E, k=K)
    blocks, sources = [], []
    for i in range(n_blocks):
        src = W.ExpertSource(98, i, shape)
        L = MoeLayer(E, D, F, K, layer=i)
        experts = {}
        for e in range(E):
            mats = [(src.codes(e, m), src.codebooks(e, m)) for m in range(3)]
            experts[e] = tuple(mats)
            L.load_expert(e, mats[0][0], mats[1][0], mats[2][0], np.stack([c for _, c in mats]))
        wr = W.router_weight(src.lseed, E, D)
        L.set_router(wr)
        S = SharedExpert(normal((F, D), D ** -0.5), normal((F, D), D ** -0.5),
                         normal((D, F), F ** -0.5))
        p = dict(w_pre=normal((D,), 0.1, 1.0), w_post=normal((D,), 0.1, 1.0),
                 gate=[None, normal((1, D), 0.1, 0.5, torch.float32)][i % 2])
        blocks.append((L, S, p))
        sources.append((experts, wr))
    return SharedExpertStack(blocks, alpha=0.9), sources


@pytest.mark.parametrize("n", [1, 3, 70])
def test_stack_against_oracle(n):
    stack, sources = build()
    x = torch.randn((n, D), device=DEV, generator=torch.Generator(device=DEV).manual_seed(n))
    bufs = stack.forward(x)
    torch.cuda.synchronize()
    h = x
    for i, (L, S, p) in enumerate(stack.blocks):
        b = bufs[i]
        assert L.status(n) == (0, 0) and S.status(n) == (0, 0)
        x64 = b["xn"].double()
        experts, wr = sources[i]
        r = oracle.moe_layer(lambda e: experts[e], wr, x64.cpu().numpy(), K, D, F,
                             route_logits=b["logits"].cpu().numpy())
        assert np.array_equal(b["idx"].cpu().numpy(), r["idx"])
        routed = torch.from_numpy(r["out"]).to(DEV) - x64
        (a, ea), _, _ = R.gated(b["xn"], S.wg, S.wu, None, None, "silu")
        y, ey = R.product(a, S.wd.double())
        ey = ey + ea @ S.wd.double().abs().t()           # the hidden values' rounding
        ey = ey + 1e-4 * routed.square().mean().sqrt()   # the routed experts' tolerance
        R.check(b["out"], (y + routed, ey + 4 * R.U32 * (y + routed).abs()), f"y {i}")
        ho, *_ = R.join(h, b["out"], 0.9, p["gate"], True, p["w_post"], None, stack.eps)
        mag = ho.abs() + 0.9 * h.double().abs()
        R.check(b["h"], (ho, 80 * R.U32 * mag), f"h {i}")
        if i + 1 < len(stack.blocks):
            nxt = stack.blocks[i + 1][2]["w_pre"]
            _, xn, *_ = R.join(None, b["h"], 1.0, None, False, None, nxt, stack.eps)
            R.check(bufs[i + 1]["xn"], (xn, (R.half_step(BF) + 256 * R.U32) * xn.abs()
                                        + 80 * R.U32), f"xn {i + 1}")
        h = b["h"]


@pytest.mark.parametrize("n", [5, 130])
def test_shared_expert_gradients(n):
    stack, _ = build(1)
    S = stack.blocks[0][1]
    g = torch.Generator(device=DEV).manual_seed(9)
    x = torch.randn((n, D), device=DEV, generator=g).to(BF)
    dout = torch.randn((n, D), device=DEV, generator=g).to(BF)
    b = S.forward(x, train=True)
    S.backward(x, dout)
    assert S.status(n, True) == (0, 0)
    leaf = [t.double().requires_grad_(True) for t in (x, S.wg, S.wu, S.wd)]
    out = (R.act("silu", leaf[0] @ leaf[1].t()) * (leaf[0] @ leaf[2].t())) @ leaf[3].t()
    want = torch.autograd.grad(out, leaf, dout.double())
    assert ((b["out"].double() - out).norm() / out.norm()).item() <= 2 * R.half_step(BF)
    # roundings of half a step each on the way: hidden (dwd), the hidden
    # gradient, dg and du, and the result; independent, so their squares add
    for k, w, steps in (("dx", want[0], 3), ("dwg", want[1], 3), ("dwu", want[2], 3),
                        ("dwd", want[3], 2)):
        rel = ((b[k].double() - w).norm() / w.norm()).item()
        assert rel <= steps ** 0.5 * R.half_step(BF), (k, rel)


def test_example_runs():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "shared_expert.py"),
                        "--tokens", "130", "--steps", "5"], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    line = [v for v in r.stdout.splitlines() if v.startswith("training loss:")][0]
    losses = [float(v) for v in line.split(":")[1].split()]
    assert len(losses) == 5 and losses[-1] < losses[0]


def test_blocks_share_a_workspace():
    """The routed layers run one after another: one workspace (24 GB for a K3-shaped
    layer at 2048 tokens) serves them all."""
    stack, _ = build(3)
    for n in (3, 70):
        bufs = stack.forward(torch.randn((n, D), device=DEV))
        assert len({b["ws"].data_ptr() for b in bufs}) == 1
        for L, S, _ in stack.blocks:
            assert L.status(n) == (0, 0) and S.status(n) == (0, 0)

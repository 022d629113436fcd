"""A two-block stack of routed RVQ experts with shared experts: a prefill chunk,
decode steps, a training step of one shared expert, and decode with the shared experts
in microscaled formats.

    python examples/shared_expert.py [--tokens 512] [--steps 8]

Weights and tokens are seeded and synthetic (d = 2048, f = 1024, 16 routed
experts, 4 per token)."""
import argparse
import copy
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


def build(torch, n_blocks=2, d=2048, f=1024, n_experts=16, k=4):
    import numpy as np

    from moe_expert_ffn_router_gb300.layer import MoeLayer, SharedExpert, SharedExpertStack
    from synth import workloads as W

    g = torch.Generator(device="cuda").manual_seed(7)

    def normal(shape, std, mean=0.0, dtype=torch.bfloat16):
        return (torch.randn(shape, device="cuda", generator=g) * std + mean).to(dtype)

    shape = W.LayerShape(d=d, f=f, E=n_experts, k=k)
    blocks = []
    for i in range(n_blocks):
        src = W.ExpertSource(1, i, shape)
        L = MoeLayer(n_experts, d, f, k, layer=i)
        for e in range(n_experts):
            mats = [(src.codes(e, m), src.codebooks(e, m)) for m in range(3)]
            L.load_expert(e, mats[0][0], mats[1][0], mats[2][0], np.stack([c for _, c in mats]))
        L.set_router(W.router_weight(src.lseed, n_experts, d))
        L.validate()
        S = SharedExpert(normal((f, d), d ** -0.5), normal((f, d), d ** -0.5),
                         normal((d, f), f ** -0.5))
        gains = dict(w_pre=normal((d,), 0.1, 1.0), w_post=normal((d,), 0.1, 1.0),
                     gate=normal((1, d), 0.05, 0.5, torch.float32))
        blocks.append((L, S, gains))
    return SharedExpertStack(blocks)


def microscaled(torch, stack):
    """The stack for serving: shared experts in 4-bit weights and 8-bit tokens, experts
    chosen by sigmoid scores with a balance bias from two of four groups.  Its layers are
    others on the same expert records and workspaces, so the given stack goes on choosing
    by logits."""
    from moe_expert_ffn_router_gb300.layer import MxSharedExpert, SharedExpertStack

    blocks = []
    for L, S, p in stack.blocks:
        L = copy.copy(L)
        L.set_scoring(bias=torch.zeros(L.E, device="cuda"), groups=4, top_groups=2)
        blocks.append((L, MxSharedExpert(S.wg, S.wu, S.wd), p))
    return SharedExpertStack(blocks)


def train_step(torch, shared, x, target, lr):
    """One SGD step of a shared expert towards target (mean squared error);
    returns the loss before the step."""
    out = shared.forward(x, train=True)["out"]
    diff = out - target
    grads = shared.backward(x, (diff * (2.0 / diff.numel())).to(x.dtype))
    for w, dw in ((shared.wg, "dwg"), (shared.wu, "dwu"), (shared.wd, "dwd")):
        w.sub_(grads[dw], alpha=lr)
    return float(diff.square().mean())


def main():
    ap = argparse.ArgumentParser(description=__doc__,
                                 formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--steps", type=int, default=8)
    a = ap.parse_args()
    import torch

    stack = build(torch)
    g = torch.Generator(device="cuda").manual_seed(1)

    def timed(name, x, reps, stack=stack, **kw):
        stack.forward(x, **kw)
        s, e = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        s.record()
        for _ in range(reps):
            bufs = stack.forward(x, **kw)
        e.record()
        torch.cuda.synchronize()
        h = bufs[-1]["h"]
        print(f"{name}: {x.shape[0]} tokens, {s.elapsed_time(e) / reps:.3f} ms per pass, "
              f"|h| rms {float(h.square().mean().sqrt()):.4f}")

    d = stack.blocks[0][0].d
    timed("prefill", torch.randn((a.tokens, d), device="cuda", generator=g), 5, tc_min_tokens=1)
    timed("decode", torch.randn((1, d), device="cuda", generator=g), 20)

    shared = stack.blocks[0][1]
    x = torch.randn((a.tokens, d), device="cuda", generator=g).to(torch.bfloat16)
    target = torch.randn((a.tokens, d), device="cuda", generator=g) * 0.1
    losses = [train_step(torch, shared, x, target, lr=1.0) for _ in range(a.steps)]
    print("training loss:", " ".join(f"{v:.5f}" for v in losses))
    mx = microscaled(torch, stack)
    timed("microscaled decode", torch.randn((1, d), device="cuda", generator=g), 20, stack=mx)
    for _, S, _ in mx.blocks:
        for n in S._bufs:
            assert S.status(n) == (0, 0)
    for L, S, _ in stack.blocks:
        for n, train in S._bufs:
            assert S.status(n, train) == (0, 0)
        for n in L._ws:
            assert L.status(n) == (0, 0)


if __name__ == "__main__":
    main()

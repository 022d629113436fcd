"""The dense operators beside the routed experts, as measured cases.

Three operators surround an MoE layer's routed experts in a block with a shared
(always active, unquantised) expert:

  gated   h = act(x Wg^T + bg) * (x Wu^T + bu), the shared expert's first half,
          and in training dx, dWg, dWu, dbg, dbu from dh;
  linear  out = residual + alpha * act(x W^T + b), its second half (or any dense
          projection), and in training dx, dW, db from dout;
  join    h' = alpha * h + gate * norm(y) * w_post and xn = norm(h') * w_pre, the
          norms after one block and before the next joined with the block's gate
          and the residual's scale, and in training the gradients of all inputs
          (norm is the root-mean-square norm over the hidden dimension).

`run` computes them in plain torch operations, or, where `own` is true, through
moe_expert_ffn_router_gb300.  Sizes are those of the repository's layers
(d=7168/f=2048 and d=2048/f=1024, batches 1 to 64, chunks of 2048 tokens, the
256 x 512 single matrix) and ragged ones between them.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one token through the shared expert's first half: decode at batch 1, K3-shaped layer
        dict(name="gated_decode_1", op="gated", train=False, n=1, d=7168, f=2048, dtype="bf16",
             act="silu", bias=False),
        # a decode batch of 64 sequences
        dict(name="gated_decode_64", op="gated", train=False, n=64, d=7168, f=2048, dtype="bf16",
             act="silu", bias=False),
        # a 2048-token prefill chunk
        dict(name="gated_prefill_2048", op="gated", train=False, n=2048, d=7168, f=2048,
             dtype="bf16", act="silu", bias=False),
        # a fine-tuning step of the shared expert on two chunks: forward and every gradient
        dict(name="gated_train_4096", op="gated", train=True, n=4096, d=7168, f=2048,
             dtype="bf16", act="silu", bias=False),
        # a ragged step of the smaller layer, GELU gate with biases, fp16
        dict(name="gated_train_ragged", op="gated", train=True, n=1333, d=2048, f=1000,
             dtype="fp16", act="gelu_tanh", bias=True),
        # the smallest call: the repository's single 256 x 512 matrix, a few tokens
        dict(name="linear_tiny", op="linear", train=False, n=7, d=512, f=256, dtype="bf16",
             act="none", bias=True, residual=False),
        # one token through the shared expert's second half, added to a stream
        dict(name="linear_decode_1", op="linear", train=False, n=1, d=2048, f=7168, dtype="bf16",
             act="none", bias=False, residual=True),
        # the same for a prefill chunk
        dict(name="linear_prefill_2048", op="linear", train=False, n=2048, d=2048, f=7168,
             dtype="bf16", act="none", bias=False, residual=True),
        # a training step of a ragged projection with everything in its epilogue
        dict(name="linear_train_ragged", op="linear", train=True, n=1777, d=1736, f=4104,
             dtype="bf16", act="gelu", bias=True, residual=True),
        # between two blocks at decode: one row of the fp32 stream, gate per token
        dict(name="join_decode_1", op="join", train=False, n=1, d=7168, stream="fp32",
             block="fp32", norm="bf16", gate="token", post=True, alpha=1.0),
        # between two blocks of a prefill chunk
        dict(name="join_prefill_2048", op="join", train=False, n=2048, d=7168, stream="fp32",
             block="fp32", norm="bf16", gate="token", post=True, alpha=1.0),
        # a training step: bf16 streams, odd row count, gate per channel, scaled residual
        dict(name="join_train_4099", op="join", train=True, n=4099, d=2048, stream="bf16",
             block="bf16", norm="bf16", gate="channel", post=True, alpha=0.75),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    """Tokens from 1 to 4096 (any number), features in multiples of 8."""
    op = rng.choice(["gated", "linear", "join"])
    train = rng.random() < 0.4
    n = _log_int(rng, 1, 4096)
    if op == "gated":
        return dict(op=op, train=train, n=n, d=_log_int(rng, 512, 7168, 8),
                    f=_log_int(rng, 256, 2048, 8), dtype=rng.choice(["bf16", "bf16", "fp16"]),
                    act=rng.choice(["silu", "silu", "gelu_tanh", "gelu", "relu"]),
                    bias=rng.random() < 0.3)
    if op == "linear":
        return dict(op=op, train=train, n=n, d=_log_int(rng, 256, 2048, 8),
                    f=_log_int(rng, 256, 7168, 8), dtype=rng.choice(["bf16", "bf16", "fp16"]),
                    act=rng.choice(["none", "none", "silu", "gelu", "relu"]),
                    bias=rng.random() < 0.5, residual=rng.random() < 0.5)
    stream = rng.choice(["fp32", "bf16"])
    return dict(op=op, train=train, n=n, d=_log_int(rng, 256, 7168, 8), stream=stream,
                block=rng.choice([stream, "bf16"]), norm="bf16",
                gate=rng.choice(["none", "token", "channel", "full"]),
                post=rng.random() < 0.7, alpha=rng.choice([1.0, 0.5, 0.8125]))


# ----------------------------------------------------------------- the inputs

def _inputs(case, seed):
    """The tensors of a case, from the seed alone (a CUDA generator): normalised
    tokens, weights of standard deviation 0.02, gains near 1, gates in (0, 1)."""
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(shape, dtype, std=1.0, mean=0.0):
        t = torch.randn(shape, device="cuda", dtype=torch.float32, generator=g)
        return t.mul_(std).add_(mean).to(dtype)

    n, d = case["n"], case["d"]
    s = {}
    if case["op"] == "join":
        st, bl = DTYPES[case["stream"]], DTYPES[case["block"]]
        s["h"] = normal((n, d), st, 2.0)
        s["y"] = normal((n, d), bl, 0.5)
        s["w_post"] = normal((d,), st, 0.1, 1.0) if case["post"] else None
        s["w_pre"] = normal((d,), st, 0.1, 1.0)
        shape = {"none": None, "token": (n, 1), "channel": (1, d), "full": (n, d)}[case["gate"]]
        s["gate"] = None if shape is None else torch.rand(shape, device="cuda",
                                                          generator=g).to(st)
        if case["train"]:
            s["dh_out"] = normal((n, d), st, 0.1)
            s["dxn"] = normal((n, d), DTYPES[case["norm"]], 0.1)
        return s
    f, dt = case["f"], DTYPES[case["dtype"]]
    s["x"] = normal((n, d), dt)
    if case["op"] == "gated":
        s["wg"], s["wu"] = normal((f, d), dt, 0.02), normal((f, d), dt, 0.02)
        s["bg"] = normal((f,), dt, 0.1) if case["bias"] else None
        s["bu"] = normal((f,), dt, 0.1) if case["bias"] else None
    else:
        s["w"] = normal((f, d), dt, 0.02)
        s["bias"] = normal((f,), dt, 0.1) if case["bias"] else None
        s["residual"] = normal((n, f), dt) if case["residual"] else None
    if case["train"]:
        s["dout"] = normal((n, f), dt, 0.1)
    return s


def prepare(case, seed):
    """The inputs, and where the framework runs them the output buffers and the
    workspace that a program allocates once per batch size and keeps."""
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        import moe_expert_ffn_router_gb300 as rvq

        def out(shape, dtype):
            return torch.empty(shape, dtype=dtype, device="cuda")

        n, d, train = case["n"], case["d"], case["train"]
        if case["op"] == "join":
            st = DTYPES[case["stream"]]
            s["h_out"], s["xn"] = out((n, d), st), out((n, d), DTYPES[case["norm"]])
            nbytes = rvq.moe_norm_join_workspace_bytes(n, d)
            if train:
                s["rstd"] = out((2, n), torch.float32)
                s["dh"], s["dy"] = torch.empty_like(s["h"]), torch.empty_like(s["y"])
                for k in ("w_post", "w_pre", "gate"):
                    s["d" + k] = None if s[k] is None else torch.empty_like(s[k])
        else:
            f, dt = case["f"], DTYPES[case["dtype"]]
            gated = case["op"] == "gated"
            s["out"] = out((n, f), dt)
            size = rvq.moe_gated_linear_workspace_bytes if gated else rvq.moe_linear_workspace_bytes
            nbytes = size(n, f, d, train)
            if train:
                s["pre"] = out((2, n, f) if gated else (n, f), torch.float32) \
                    if gated or case["act"] != "none" else None
                s["dx"] = torch.empty_like(s["x"])
                for k in (("wg", "wu", "bg", "bu") if gated else ("w", "bias")):
                    s["d" + k] = None if s[k] is None else torch.empty_like(s[k])
        s["ws"] = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        rvq.rvq_ws_clear(s["ws"])
    return s


# ------------------------------------------------- the plain forms, in 32 bits

def _act(name, v):
    if name == "none":
        return v
    if name == "relu":
        return v * (v > 0)
    if name == "silu":
        return v / (1 + torch.exp(-v))
    if name == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))


def _act_grad(name, v):
    if name == "none":
        return torch.ones_like(v)
    if name == "relu":
        return (v > 0).to(v.dtype)
    if name == "silu":
        sg = 1 / (1 + torch.exp(-v))
        return sg * (1 + v * (1 - sg))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(v * math.sqrt(0.5))) \
            + v * torch.exp(-0.5 * v * v) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (v + 0.044715 * v * v * v))
    return 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * c * (1 + 3 * 0.044715 * v * v)


def _plain_gated(s, case):
    dt = s["x"].dtype
    x, wg, wu = s["x"].float(), s["wg"].float(), s["wu"].float()
    g, u = x @ wg.t(), x @ wu.t()
    if case["bias"]:
        g, u = g + s["bg"].float(), u + s["bu"].float()
    a = _act(case["act"], g)
    out = {"out": (a * u).to(dt)}
    if case["train"]:
        dh = s["dout"].float()
        dg, du = dh * u * _act_grad(case["act"], g), dh * a
        out["dx"] = (dg @ wg + du @ wu).to(dt)
        out["dwg"], out["dwu"] = (dg.t() @ x).to(dt), (du.t() @ x).to(dt)
        if case["bias"]:
            out["dbg"], out["dbu"] = dg.sum(0).to(dt), du.sum(0).to(dt)
    return out


def _plain_linear(s, case):
    dt = s["x"].dtype
    x, w = s["x"].float(), s["w"].float()
    p = x @ w.t()
    if case["bias"]:
        p = p + s["bias"].float()
    y = _act(case["act"], p)
    if case["residual"]:
        y = y + s["residual"].float()
    out = {"out": y.to(dt)}
    if case["train"]:
        dp = s["dout"].float() * _act_grad(case["act"], p)
        out["dx"], out["dw"] = (dp @ w).to(dt), (dp.t() @ x).to(dt)
        if case["bias"]:
            out["dbias"] = dp.sum(0).to(dt)
    return out


def _norm_grad(v, r, gv):
    """Gradient of v * r, r = 1 / sqrt(mean(v^2) + eps), given that of its value."""
    return r * gv - v * r * r * r * (gv * v).mean(1, keepdim=True)


def _plain_join(s, case):
    st = s["h"].dtype
    h, y = s["h"].float(), s["y"].float()
    z, ry = y, None
    if case["post"]:
        ry = 1 / torch.sqrt((y * y).mean(1, keepdim=True) + EPS)
        z = y * ry * s["w_post"].float()
    gate = None if s["gate"] is None else s["gate"].float()
    ho = case["alpha"] * h + (z if gate is None else gate * z)
    rh = 1 / torch.sqrt((ho * ho).mean(1, keepdim=True) + EPS)
    w_pre = s["w_pre"].float()
    out = {"h_out": ho.to(st), "xn": (ho * rh * w_pre).to(DTYPES[case["norm"]])}
    if case["train"]:
        dxn = s["dxn"].float()
        dho = s["dh_out"].float() + _norm_grad(ho, rh, dxn * w_pre)
        out["dw_pre"] = (dxn * ho * rh).sum(0).to(st)
        out["dh"] = (case["alpha"] * dho).to(st)
        dz = dho if gate is None else dho * gate
        if gate is not None:
            dgate = dho * z
            if case["gate"] != "full":
                dgate = dgate.sum(1 if case["gate"] == "token" else 0, keepdim=True)
            out["dgate"] = dgate.to(st)
        if case["post"]:
            out["dw_post"] = (dz * y * ry).sum(0).to(st)
            dz = _norm_grad(y, ry, dz * s["w_post"].float())
        out["dy"] = dz.to(s["y"].dtype)
    return out


# ----------------------------------------------------- the framework's kernels

def _own_gated(rvq, s, case):
    n, d, f = case["n"], case["d"], case["f"]
    act = rvq.MOE_ACTS[case["act"]]
    rvq.moe_gated_linear(s["x"], s["wg"], s["wu"], n, f, d, s["out"], s["ws"], bg=s["bg"],
                         bu=s["bu"], act=act, pre=s.get("pre"))
    out = {"out": s["out"]}
    if case["train"]:
        rvq.moe_gated_linear_backward(s["dout"], s["x"], s["wg"], s["wu"], s["pre"], n, f, d,
                                      s["ws"], dx=s["dx"], dwg=s["dwg"], dwu=s["dwu"],
                                      dbg=s["dbg"], dbu=s["dbu"], act=act)
        out.update({k: s[k] for k in ("dx", "dwg", "dwu")})
        if case["bias"]:
            out.update(dbg=s["dbg"], dbu=s["dbu"])
    return out


def _own_linear(rvq, s, case):
    n, d, f = case["n"], case["d"], case["f"]
    act = rvq.MOE_ACTS[case["act"]]
    rvq.moe_linear(s["x"], s["w"], n, f, d, s["out"], s["ws"], bias=s["bias"], act=act,
                   residual=s["residual"], pre=s.get("pre"))
    out = {"out": s["out"]}
    if case["train"]:
        rvq.moe_linear_backward(s["dout"], s["x"], s["w"], n, f, d, s["ws"], dx=s["dx"],
                                dw=s["dw"], dbias=s["dbias"], pre=s["pre"], act=act)
        out.update(dx=s["dx"], dw=s["dw"])
        if case["bias"]:
            out["dbias"] = s["dbias"]
    return out


def _own_join(rvq, s, case):
    n, d = case["n"], case["d"]
    rvq.moe_norm_join(s["y"], n, d, s["h_out"], s["xn"], h=s["h"], alpha=case["alpha"],
                      gate=s["gate"], post_norm=case["post"], w_post=s["w_post"],
                      w_pre=s["w_pre"], eps=EPS, rstd=s.get("rstd"))
    out = {"h_out": s["h_out"], "xn": s["xn"]}
    if case["train"]:
        rvq.moe_norm_join_backward(s["dh_out"], s["dxn"], s["y"], n, d, s["rstd"], s["ws"],
                                   h=s["h"], alpha=case["alpha"], gate=s["gate"],
                                   post_norm=case["post"], w_post=s["w_post"], w_pre=s["w_pre"],
                                   dh=s["dh"], dy=s["dy"], dw_post=s["dw_post"],
                                   dw_pre=s["dw_pre"], dgate=s["dgate"])
        out.update({k: s[k] for k in ("dh", "dy", "dw_post", "dw_pre", "dgate")
                    if s[k] is not None})
    return out


def run(state):
    case = state["case"]
    if own:
        import moe_expert_ffn_router_gb300 as rvq
        fn = {"gated": _own_gated, "linear": _own_linear, "join": _own_join}[case["op"]]
        return fn(rvq, state, case)
    fn = {"gated": _plain_gated, "linear": _plain_linear, "join": _plain_join}[case["op"]]
    return fn(state, case)


# --------------------------------------------------------------- what it takes

def work(case):
    """Inputs once, outputs once; two operations per multiply-add of a product.
    A training step's gradients read the forward's inputs again in principle,
    but they are counted once, and nothing saved in between is counted."""
    n, d = case["n"], case["d"]
    size = {k: torch.empty((), dtype=v).element_size() for k, v in DTYPES.items()}
    if case["op"] == "join":
        st, bl, no = size[case["stream"]], size[case["block"]], size[case["norm"]]
        gate = {"none": 0, "token": n, "channel": d, "full": n * d}[case["gate"]] * st
        gains = (d + (d if case["post"] else 0)) * st
        nbytes = n * d * (st + bl) + gate + gains + n * d * (st + no)
        flops = 12 * n * d
        if case["train"]:
            nbytes += n * d * (st + no) + n * d * (st + bl) + gate + gains
            flops += 24 * n * d
        return {"bytes": nbytes, "flops": flops}
    f, b = case["f"], size[case["dtype"]]
    mats = 2 if case["op"] == "gated" else 1
    weights = mats * (f * d + (f if case["bias"] else 0)) * b
    nbytes = n * d * b + weights + n * f * b
    if case.get("residual"):
        nbytes += n * f * b
    flops = 2 * mats * n * d * f
    if case["train"]:
        nbytes += n * f * b + n * d * b + weights
        flops += 4 * mats * n * d * f
    return {"bytes": nbytes, "flops": flops}


# -------------------------------------------- the definition, in 64 bits, apart

def _sigma(v):
    return torch.special.expit(v)


def _phi(v):
    return torch.special.ndtr(v)


def _curve(name, v):
    """(value, slope) of an activation, in the type of v."""
    if name == "none":
        return v, torch.ones_like(v)
    if name == "relu":
        return torch.clamp(v, min=0), torch.where(v > 0, 1.0, 0.0).to(v.dtype)
    if name == "silu":
        return v * _sigma(v), _sigma(v) + v * _sigma(v) * _sigma(-v)
    if name == "gelu":
        return v * _phi(v), _phi(v) + v * torch.exp(-v.square() / 2) * (2 * math.pi) ** -0.5
    # 0.5 (1 + tanh(t)) = sigma(2 t)
    t2 = 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v.pow(3))
    slope2 = 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * v.square())
    return v * _sigma(t2), _sigma(t2) + v * _sigma(t2) * _sigma(-t2) * slope2


def exact(case, seed):
    """The same outputs from the definitions in float64."""
    s = {k: None if v is None else v.double() for k, v in _inputs(case, seed).items()}
    if case["op"] == "join":
        return _exact_join(s, case)
    eq = "tk,rk->tr"
    if case["op"] == "linear":
        p = torch.einsum(eq, s["x"], s["w"])
        if s["bias"] is not None:
            p += s["bias"]
        val, slope = _curve(case["act"], p)
        out = {"out": val if s["residual"] is None else val + s["residual"]}
        if case["train"]:
            dp = slope * s["dout"]
            out["dx"] = torch.einsum("tr,rk->tk", dp, s["w"])
            out["dw"] = torch.einsum("tr,tk->rk", dp, s["x"])
            if s["bias"] is not None:
                out["dbias"] = torch.einsum("tr->r", dp)
        return out
    g, u = torch.einsum(eq, s["x"], s["wg"]), torch.einsum(eq, s["x"], s["wu"])
    if case["bias"]:
        g += s["bg"]
        u += s["bu"]
    val, slope = _curve(case["act"], g)
    out = {"out": val * u}
    if case["train"]:
        dg, du = s["dout"] * slope * u, s["dout"] * val
        out["dx"] = torch.einsum("tr,rk->tk", dg, s["wg"]) + torch.einsum("tr,rk->tk", du, s["wu"])
        out["dwg"] = torch.einsum("tr,tk->rk", dg, s["x"])
        out["dwu"] = torch.einsum("tr,tk->rk", du, s["x"])
        if case["bias"]:
            out["dbg"], out["dbu"] = torch.einsum("tr->r", dg), torch.einsum("tr->r", du)
    return out


def _exact_join(s, case):
    """Forward from the definition; gradients by automatic differentiation of
    it in float64."""
    names = ["h", "y", "w_post", "w_pre", "gate"]
    leaf = {k: None if s[k] is None else s[k].clone().requires_grad_(case["train"])
            for k in names}

    def unit(v):
        return v * torch.rsqrt(v.square().sum(1, keepdim=True) / v.shape[1] + EPS)

    branch = unit(leaf["y"]) * leaf["w_post"] if case["post"] else leaf["y"]
    if leaf["gate"] is not None:
        branch = leaf["gate"] * branch
    ho = leaf["h"] * case["alpha"] + branch
    xn = unit(ho) * leaf["w_pre"]
    out = {"h_out": ho.detach(), "xn": xn.detach()}
    if case["train"]:
        used = [k for k in names if leaf[k] is not None]
        grads = torch.autograd.grad([ho, xn], [leaf[k] for k in used], [s["dh_out"], s["dxn"]])
        out.update({"d" + k: v for k, v in zip(used, grads)})
    return out

"""A block's microscaled path and its scored router, as measured cases.

Five operators serve an MoE block whose shared expert is held in microscaled
formats and whose router scores experts with a balance bias and groups:

  quant   a matrix into a microscaled format: blocks of 32 values along a row share
          a power-of-two scale (8 bits), the values are held in 8 bits (4-bit
          exponent, 3-bit mantissa) or 4 (2-bit exponent, 1-bit mantissa);
  norm    h' = alpha h + gate * norm(y) * w_post, and norm(h') * w_pre straight into
          a microscaled format: the residual's addition, the norms and the
          quantisation in one pass;
  gated   act(x Wg^T + bg) * (x Wu^T + bu) of microscaled tokens and weights, in 16
          bits or microscaled for the next product;
  linear  residual + alpha * act(x W^T + b) of microscaled weights, the tokens
          microscaled already or 16-bit ones quantised on the way;
  route   experts chosen by sigmoid or softmax scores plus a bias, from the best
          groups, weights from the scores alone, and the token -> expert grouping;
          in training also the gradient of the logits.

`run` computes them in plain torch operations, or, where `own` is true, through
moe_expert_ffn_router_gb300.  Sizes are those of the repository's layers (d=7168,
f=2048, 256 experts of which 16 are chosen; d=2048, f=1024, 64 and 8; batches 1 to
64, chunks of 2048 tokens) and ragged ones between them.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6
BLOCK = 32       # values that share a scale
TILE = 128       # rows of a tile of scales; columns are padded to it
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one token's attention output on its way into an 8-bit projection: decode
        dict(name="quant_decode_1", op="quant", fmt="f8", n=1, d=7168, dtype="bf16"),
        # a projection matrix put into 4 bits and read back, as when weights are loaded
        # and checked
        dict(name="quant_weights_2048", op="quant", fmt="f4", n=2048, d=7168, dtype="fp32"),
        # the norms between two blocks at decode, 64 sequences
        dict(name="norm_decode_64", op="norm", fmt="f8", n=64, d=7168, stream="fp32", block="bf16",
             gate="none", post=False, alpha=1.0),
        # the same for a 2048-token prefill chunk, with a post norm and a gate per channel
        dict(name="norm_prefill_2048", op="norm", fmt="f8", n=2048, d=7168, stream="fp32",
             block="fp32", gate="channel", post=True, alpha=1.0),
        # a ragged batch of prompts through a small block
        dict(name="norm_ragged_1531", op="norm", fmt="f8", n=1531, d=2040, stream="bf16",
             block="bf16", gate="token", post=True, alpha=0.8125),
        # one token through the shared expert's first half: 8-bit tokens, 4-bit weights
        dict(name="gated_decode_1", op="gated", n=1, d=7168, f=2048, xfmt="f8", wfmt="f4",
             act="silu", bias=False, out="f8"),
        # a prefill chunk, all in 4 bits
        dict(name="gated_prefill_2048", op="gated", n=2048, d=7168, f=2048, xfmt="f4", wfmt="f4",
             act="silu", bias=False, out="bf16"),
        # the second half for a decode batch of 64 sequences, on the stream's fp32 residual
        dict(name="linear_decode_64", op="linear", n=64, d=2048, f=7168, xfmt="f8", wfmt="f4",
             act="none", bias=False, residual=True, given=True, out="fp32"),
        # a ragged batch of 16-bit tokens, quantised on the way
        dict(name="linear_ragged_777", op="linear", n=777, d=1736, f=4104, xfmt="f8", wfmt="f4",
             act="gelu", bias=True, residual=False, given=False, out="bf16"),
        # decode: one token's 16 of 256 experts, from 4 of 8 groups
        dict(name="route_decode_1", op="route", train=False, n=1, E=256, k=16, score="sigmoid",
             bias=True, groups=8, top=4, renorm=True, scale=2.5),
        # a 2048-token prefill chunk, the same router
        dict(name="route_prefill_2048", op="route", train=False, n=2048, E=256, k=16,
             score="sigmoid", bias=True, groups=8, top=4, renorm=True, scale=2.5),
        # a training batch of a softmax router without renormalisation, with the gradient
        dict(name="route_train_4096", op="route", train=True, n=4096, E=64, k=8, score="softmax",
             bias=False, groups=1, top=1, renorm=False, scale=1.0),
    ]


def _log_int(rng, low, high, step=1):
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    return max(low, min(high, v // step * step))


def draw(rng):
    op = rng.choice(["quant", "norm", "gated", "linear", "route"])
    n = _log_int(rng, 1, 2048)
    if op == "quant":
        return dict(op=op, fmt=rng.choice(["f8", "f4"]), n=n, d=_log_int(rng, 64, 7168, 8),
                    dtype=rng.choice(["bf16", "fp16", "fp32"]))
    if op == "norm":
        stream = rng.choice(["fp32", "bf16"])
        return dict(op=op, fmt="f8", n=n, d=_log_int(rng, 64, 7168, 8), stream=stream,
                    block=rng.choice([stream, "bf16"]),
                    gate=rng.choice(["none", "token", "channel", "full"]),
                    post=rng.random() < 0.6, alpha=rng.choice([1.0, 0.5, 0.8125]))
    if op == "gated":
        return dict(op=op, n=n, d=_log_int(rng, 256, 7168, 8), f=_log_int(rng, 64, 2048, 8),
                    xfmt=rng.choice(["f8", "f4"]), wfmt=rng.choice(["f4", "f4", "f8"]),
                    act=rng.choice(["silu", "silu", "gelu_tanh", "gelu", "relu"]),
                    bias=rng.random() < 0.3, out=rng.choice(["bf16", "fp16", "f8"]))
    if op == "linear":
        return dict(op=op, n=n, d=_log_int(rng, 64, 2048, 8), f=_log_int(rng, 64, 7168, 8),
                    xfmt=rng.choice(["f8", "f4"]), wfmt=rng.choice(["f4", "f4", "f8"]),
                    act=rng.choice(["none", "none", "silu", "gelu", "relu"]),
                    bias=rng.random() < 0.4, residual=rng.random() < 0.5,
                    given=rng.random() < 0.5, out=rng.choice(["fp32", "bf16"]))
    groups = rng.choice([1, 1, 2, 4, 8])
    E = _log_int(rng, max(8, 2 * groups), 256, groups)
    top = rng.randint(max(1, groups // 2), groups)
    return dict(op=op, train=rng.random() < 0.4, n=_log_int(rng, 1, 4096), E=E,
                k=rng.randint(1, min(16, E // groups * top)),
                score=rng.choice(["sigmoid", "sigmoid", "softmax"]), bias=rng.random() < 0.6,
                groups=groups, top=top, renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]))


# ----------------------------------------- microscaled matrices, in plain torch
#
# Codes: a row after the other, columns padded with zeros to a multiple of 128; 8-bit
# codes a byte each, 4-bit ones two to a byte, the lower column in the lower half.
# Scales: 2^(byte - 127), in tiles of 128 rows x 4 blocks of 32 columns: byte
# [row / 128][block / 4][row % 32][row / 32 % 4][block % 4]; rows behind the last of
# the matrix hold no scale.

def _up(v, m):
    return (v + m - 1) // m * m


def _mx_code_shape(rows, cols, fmt):
    return (rows, _up(cols, TILE) // (1 if fmt == "f8" else 2))


def _mx_scale_shape(rows, cols):
    return (_up(rows, TILE) // TILE, _up(cols, TILE) // TILE, 32, 4, 4)


def _pad(x, rows, cols):
    out = torch.zeros((rows, cols), dtype=x.dtype, device=x.device)
    out[:x.shape[0], :x.shape[1]] = x
    return out


def _scales_in_tiles(b):
    """[rows][blocks] -> tiles, rows and blocks padded with zeros."""
    rows, blocks = _up(b.shape[0], TILE), _up(b.shape[1], 4)
    return _pad(b, rows, blocks).view(rows // TILE, 4, 32, blocks // 4, 4).permute(0, 3, 2, 1, 4) \
        .contiguous()


def _scales_in_rows(t, rows):
    return t.permute(0, 3, 2, 1, 4).reshape(t.shape[0] * TILE, t.shape[1] * 4)[:rows]


def _mx_quantize(v, fmt):
    """fp32 [rows][cols] -> (values before their scales [rows][padded], scale bytes
    [rows][blocks]): the scale is the power of two that takes the block's largest
    magnitude below twice the format's largest power of two; values round to even and
    end at the format's largest."""
    rows, cols = v.shape
    v = _pad(v, rows, _up(cols, TILE)).view(rows, -1, BLOCK)
    top = v.abs().amax(2)
    expo = torch.frexp(top)[1] - 1          # floor(log2)
    byte = (expo - (8 if fmt == "f8" else 2) + 127).clamp(0, 254) * (top > 0)
    q = torch.ldexp(v, (127 - byte).unsqueeze(2))
    if fmt == "f8":
        q = q.clamp(-448, 448).to(E4M3).float()
    else:
        a = q.abs()
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
        q = torch.copysign((torch.round(a / step) * step).clamp(max=6), q)
    return q.view(rows, -1), byte.to(torch.uint8)


def _f4_codes(q):
    """e2m1 values -> packed codes."""
    where = torch.tensor([0, 1, 2, 3, 4, 0, 5, 0, 6, 0, 0, 0, 7], device=q.device)
    c = where[(q.abs() * 2).long()] + 8 * (q < 0)
    return (c[:, 0::2] + 16 * c[:, 1::2]).to(torch.uint8)


def _mx_codes(q, fmt):
    return q.to(E4M3).view(torch.uint8) if fmt == "f8" else _f4_codes(q)


def _mx_values(codes, tiles, rows, cols, fmt):
    """A microscaled matrix in fp32."""
    if fmt == "f8":
        q = codes.view(E4M3).float()
    else:
        table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
        table = torch.cat([table, -table])
        q = torch.stack([table[(codes & 15).long()], table[(codes >> 4).long()]], 2).view(rows, -1)
    e = _scales_in_rows(tiles, rows).int() - 127
    return torch.ldexp(q.view(rows, -1, BLOCK), e.unsqueeze(2)).reshape(rows, -1)[:, :cols]


# ----------------------------------------------------------------- the inputs

def _inputs(case, seed):
    """The tensors of a case, from the seed alone (a CUDA generator): normalised
    tokens, weights of standard deviation 0.02, gains near 1, gates in (0, 1), router
    logits of standard deviation 1.5 and a balance bias of 0.05."""
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(shape, dtype, std=1.0, mean=0.0):
        t = torch.randn(shape, device="cuda", dtype=torch.float32, generator=g)
        return t.mul_(std).add_(mean).to(dtype)

    def micro(name, shape, fmt, std):
        q, b = _mx_quantize(normal(shape, torch.float32, std), fmt)
        s[name], s[name + "_scales"] = _mx_codes(q, fmt), _scales_in_tiles(b)

    n, op = case["n"], case["op"]
    s = {}
    if op == "quant":
        s["x"] = normal((n, case["d"]), DTYPES[case["dtype"]], 0.02 if n > 64 else 1.0)
    elif op == "norm":
        d = case["d"]
        st, bl = DTYPES[case["stream"]], DTYPES[case["block"]]
        s["h"], s["y"] = normal((n, d), st, 2.0), normal((n, d), bl, 0.5)
        s["w_post"] = normal((d,), st, 0.1, 1.0) if case["post"] else None
        s["w_pre"] = normal((d,), st, 0.1, 1.0)
        shape = {"none": None, "token": (n, 1), "channel": (1, d), "full": (n, d)}[case["gate"]]
        s["gate"] = None if shape is None else torch.rand(shape, device="cuda",
                                                          generator=g).to(st)
    elif op == "gated":
        micro("x", (n, case["d"]), case["xfmt"], 1.0)
        micro("wg", (case["f"], case["d"]), case["wfmt"], 0.02)
        micro("wu", (case["f"], case["d"]), case["wfmt"], 0.02)
        for k in ("bg", "bu"):
            s[k] = normal((case["f"],), torch.float32, 0.1) if case["bias"] else None
    elif op == "linear":
        if case["given"]:
            micro("x", (n, case["d"]), case["xfmt"], 1.0)
        else:
            s["x"] = normal((n, case["d"]), torch.bfloat16)
        micro("w", (case["f"], case["d"]), case["wfmt"], 0.02)
        s["bias"] = normal((case["f"],), torch.float32, 0.1) if case["bias"] else None
        s["residual"] = normal((n, case["f"]), DTYPES[case["out"]]) if case["residual"] else None
    else:
        s["logits"] = normal((n, case["E"]), torch.float32, 1.5)
        s["bias"] = normal((case["E"],), torch.float32, 0.05) if case["bias"] else None
        if case["train"]:
            s["dw"] = normal((n, case["k"]), torch.float32, 0.1)
    return s


def prepare(case, seed):
    """The inputs, the output buffers that a program allocates once per batch size and
    keeps, and the framework's workspace."""
    s = _inputs(case, seed)
    s["case"] = case
    n, op = case["n"], case["op"]

    def new(shape, dtype):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    def micro(name, rows, cols, fmt):
        s[name] = new(_mx_code_shape(rows, cols, fmt), torch.uint8)
        s[name + "_scales"] = new(_mx_scale_shape(rows, cols), torch.uint8)

    if op == "quant":
        micro("q", n, case["d"], case["fmt"])
        if case["fmt"] == "f4":
            s["out"] = new((n, case["d"]), torch.bfloat16)
    elif op == "norm":
        s["h_out"] = torch.zeros_like(s["h"])
        micro("q", n, case["d"], case["fmt"])
    elif op == "gated" and case["out"] == "f8":
        micro("out", n, case["f"], "f8")
    elif op in ("gated", "linear"):
        s["out"] = new((n, case["f"]), DTYPES[case["out"]])
        if op == "linear" and not case["given"]:
            micro("q", n, case["d"], case["xfmt"])
    else:
        E, k = case["E"], case["k"]
        s["idx"], s["w"] = new((n, k), torch.int32), new((n, k), torch.float32)
        s["offsets"], s["pairs"] = new((E + 1,), torch.int32), new((n * k,), torch.int32)
        s["dlogits"] = new((n, E), torch.float32) if case["train"] else None
    if own and op in ("gated", "linear", "route"):
        import moe_expert_ffn_router_gb300 as rvq
        if op == "route":
            nbytes = rvq.moe_route_scored_workspace_bytes(n, case["E"])
        elif op == "gated":
            nbytes = rvq.moe_mx_gated_linear_workspace_bytes(n, case["f"], case["d"])
        else:
            nbytes = rvq.moe_mx_linear_workspace_bytes(n, case["f"], case["d"])
        s["ws"] = new((nbytes,), torch.uint8)
        rvq.rvq_ws_clear(s["ws"])
    return s


# ------------------------------------------------- the plain forms, in 32 bits

def _held(codes, tiles, cols):
    """8-bit codes and scales as the numbers that they stand for."""
    return {"q": codes.view(E4M3)[:, :cols], "scales": tiles.view(E8M0)}


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


def _plain_quant(s, case):
    q, b = _mx_quantize(s["x"].float(), case["fmt"])
    tiles = _scales_in_tiles(b)
    if case["fmt"] == "f8":
        return _held(_mx_codes(q, "f8"), tiles, case["d"])
    return {"out": _mx_values(_mx_codes(q, "f4"), tiles, case["n"], case["d"], "f4")
            .to(torch.bfloat16)}


def _plain_norm(s, case):
    h, y = s["h"].float(), s["y"].float()
    if case["post"]:
        y = y / torch.sqrt((y * y).mean(1, keepdim=True) + EPS) * s["w_post"].float()
    if s["gate"] is not None:
        y = y * s["gate"].float()
    h = case["alpha"] * h + y
    xn = h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) * s["w_pre"].float()
    q, b = _mx_quantize(xn, case["fmt"])
    return {"h_out": h.to(s["h"].dtype),
            **_held(_mx_codes(q, case["fmt"]), _scales_in_tiles(b), case["d"])}


def _plain_gated(s, case):
    n, d, f = case["n"], case["d"], case["f"]
    x = _mx_values(s["x"], s["x_scales"], n, d, case["xfmt"])
    g, u = (x @ _mx_values(s[k], s[k + "_scales"], f, d, case["wfmt"]).t() for k in ("wg", "wu"))
    if case["bias"]:
        g, u = g + s["bg"], u + s["bu"]
    h = _act(case["act"], g) * u
    if case["out"] != "f8":
        return {"out": h.to(DTYPES[case["out"]])}
    q, b = _mx_quantize(h, "f8")
    return _held(_mx_codes(q, "f8"), _scales_in_tiles(b), f)


def _plain_linear(s, case):
    n, d, f = case["n"], case["d"], case["f"]
    if case["given"]:
        x = _mx_values(s["x"], s["x_scales"], n, d, case["xfmt"])
    else:
        q, b = _mx_quantize(s["x"].float(), case["xfmt"])
        x = torch.ldexp(q.view(n, -1, BLOCK), b.int().unsqueeze(2) - 127).view(n, -1)[:, :d]
    y = x @ _mx_values(s["w"], s["w_scales"], f, d, case["wfmt"]).t()
    if case["bias"]:
        y = y + s["bias"]
    y = _act(case["act"], y)
    if case["residual"]:
        y = y + s["residual"].float()
    return {"out": y.to(DTYPES[case["out"]])}


def _plain_route(s, case):
    """Scores and choice in 64 bits: values next to each other decide."""
    n, E, k, groups, scale = (case[x] for x in ("n", "E", "k", "groups", "scale"))
    l = s["logits"].double()
    if case["score"] == "sigmoid":
        p = 1 / (1 + torch.exp(-l))
    else:
        p = torch.exp(l - l.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    c = p if s["bias"] is None else p + s["bias"].double()
    if case["top"] < groups:
        best = c.view(n, groups, -1).sort(2, descending=True)[0][:, :, :2].sum(2)
        kept = best.sort(dim=1, descending=True, stable=True)[1][:, :case["top"]]
        keep = torch.zeros((n, groups), dtype=torch.bool, device=c.device).scatter_(1, kept, True)
        keep = keep.unsqueeze(2).expand(n, groups, E // groups).reshape(n, E)
        c = torch.where(keep, c, -math.inf)
    idx = c.sort(dim=1, descending=True, stable=True)[1][:, :k]
    ps = p.gather(1, idx)
    total = ps.sum(1, keepdim=True) if case["renorm"] else 1.0
    w = ps / total
    flat = idx.reshape(-1)
    pairs = flat.sort(stable=True)[1]
    ends = (flat.unsqueeze(1) == torch.arange(E, device=c.device)).sum(0).cumsum(0)
    out = {"idx": idx.int(), "w": (scale * w).float(), "pairs": pairs.int(),
           "offsets": torch.cat([ends.new_zeros(1), ends]).int()}
    if case["train"]:
        dw = scale * s["dw"].double()
        if case["renorm"]:
            dw = (dw - (dw * w).sum(1, keepdim=True)) / total
        dp = torch.zeros_like(p).scatter_(1, idx, dw)
        dp = p * ((dp - (dp * p).sum(1, keepdim=True)) if case["score"] == "softmax"
                  else dp * (1 - p))
        out["dlogits"] = dp.float()
    return out


# ----------------------------------------------------- the framework's kernels

def _own_quant(rvq, s, case):
    n, d, fmt = case["n"], case["d"], rvq.MOE_MX[case["fmt"]]
    rvq.moe_mx_quantize(s["x"], n, d, s["q"], s["q_scales"], fmt)
    if case["fmt"] == "f8":
        return _held(s["q"], s["q_scales"], d)
    rvq.moe_mx_dequantize(s["q"], s["q_scales"], n, d, s["out"], fmt)
    return {"out": s["out"]}


def _own_norm(rvq, s, case):
    n, d = case["n"], case["d"]
    rvq.moe_norm_join_mx(s["y"], n, d, s["h_out"], s["q"], s["q_scales"],
                         fmt=rvq.MOE_MX[case["fmt"]], h=s["h"], alpha=case["alpha"],
                         gate=s["gate"], post_norm=case["post"], w_post=s["w_post"],
                         w_pre=s["w_pre"], eps=EPS)
    return {"h_out": s["h_out"], **_held(s["q"], s["q_scales"], d)}


def _own_gated(rvq, s, case):
    n, d, f = case["n"], case["d"], case["f"]
    rvq.moe_mx_gated_linear(s["x"], s["x_scales"], s["wg"], s["wg_scales"], s["wu"],
                            s["wu_scales"], n, f, d, s["out"], s["ws"],
                            xfmt=rvq.MOE_MX[case["xfmt"]], wfmt=rvq.MOE_MX[case["wfmt"]],
                            bg=s["bg"], bu=s["bu"], act=rvq.MOE_ACTS[case["act"]],
                            out_scales=s.get("out_scales"), ofmt=rvq.MOE_MX["f8"])
    if case["out"] == "f8":
        return _held(s["out"], s["out_scales"], f)
    return {"out": s["out"]}


def _own_linear(rvq, s, case):
    n, d, f, xfmt = case["n"], case["d"], case["f"], rvq.MOE_MX[case["xfmt"]]
    x = "x"
    if not case["given"]:
        x = "q"
        rvq.moe_mx_quantize(s["x"], n, d, s["q"], s["q_scales"], xfmt)
    rvq.moe_mx_linear(s[x], s[x + "_scales"], s["w"], s["w_scales"], n, f, d, s["out"], s["ws"],
                      xfmt=xfmt, wfmt=rvq.MOE_MX[case["wfmt"]], bias=s["bias"],
                      act=rvq.MOE_ACTS[case["act"]], residual=s["residual"])
    return {"out": s["out"]}


def _own_route(rvq, s, case):
    n, E, k = case["n"], case["E"], case["k"]
    score = rvq.MOE_SCORES[case["score"]]
    rvq.moe_route_scored(s["logits"], n, E, k, s["idx"], s["w"], s["offsets"], s["pairs"],
                         s["ws"], score=score, bias=s["bias"], groups=case["groups"],
                         top_groups=case["top"], renorm=case["renorm"], scale=case["scale"])
    out = {x: s[x] for x in ("idx", "w", "pairs", "offsets")}
    if case["train"]:
        rvq.moe_route_scored_backward(s["dw"], s["logits"], s["idx"], n, E, k, s["dlogits"],
                                      score=score, renorm=case["renorm"], scale=case["scale"])
        out["dlogits"] = s["dlogits"]
    return out


def run(state):
    case = state["case"]
    if own:
        import moe_expert_ffn_router_gb300 as rvq
        fn = {"quant": _own_quant, "norm": _own_norm, "gated": _own_gated, "linear": _own_linear,
              "route": _own_route}[case["op"]]
        return fn(rvq, state, case)
    fn = {"quant": _plain_quant, "norm": _plain_norm, "gated": _plain_gated,
          "linear": _plain_linear, "route": _plain_route}[case["op"]]
    return fn(state, case)


# --------------------------------------------------------------- what it takes

def _mx_bytes(rows, cols, fmt):
    return rows * cols // (1 if fmt == "f8" else 2) + rows * ((cols + BLOCK - 1) // BLOCK)


def work(case):
    """Inputs once, outputs once; two operations per multiply-add of a product.  What
    lies between two calls of a pass (4-bit codes read back, quantised tokens) is not
    counted."""
    n, op = case["n"], case["op"]
    size = {k: torch.empty((), dtype=v).element_size() for k, v in DTYPES.items()}
    if op == "quant":
        d = case["d"]
        out = _mx_bytes(n, d, "f8") if case["fmt"] == "f8" else 2 * n * d
        return {"bytes": n * d * size[case["dtype"]] + out, "flops": 4 * n * d}
    if op == "norm":
        d, st, bl = case["d"], size[case["stream"]], size[case["block"]]
        gate = {"none": 0, "token": n, "channel": d, "full": n * d}[case["gate"]] * st
        gains = (d + (d if case["post"] else 0)) * st
        return {"bytes": n * d * (2 * st + bl) + gate + gains + _mx_bytes(n, d, case["fmt"]),
                "flops": 16 * n * d}
    if op == "gated":
        d, f = case["d"], case["f"]
        out = _mx_bytes(n, f, "f8") if case["out"] == "f8" else 2 * n * f
        return {"bytes": _mx_bytes(n, d, case["xfmt"]) + 2 * _mx_bytes(f, d, case["wfmt"]) + out
                + (8 * f if case["bias"] else 0), "flops": 4 * n * d * f}
    if op == "linear":
        d, f, o = case["d"], case["f"], size[case["out"]]
        x = _mx_bytes(n, d, case["xfmt"]) if case["given"] else 2 * n * d
        return {"bytes": x + _mx_bytes(f, d, case["wfmt"]) + n * f * o
                * (2 if case["residual"] else 1) + (4 * f if case["bias"] else 0),
                "flops": 2 * n * d * f}
    E, k = case["E"], case["k"]
    nbytes = 4 * (n * E + 3 * n * k + E + 1 + (E if case["bias"] else 0))
    if case["train"]:
        nbytes += 4 * n * (E + k)
    return {"bytes": nbytes, "flops": 8 * n * E}


# -------------------------------------------- the definition, in 64 bits, apart

def _grid(fmt, device):
    """The format's values >= 0, in order."""
    if fmt == "f4":
        m, e = 2, range(0, 3)
    else:
        m, e = 8, range(-6, 9)
    v = [i / m * 2.0 ** e[0] for i in range(m)] + [(1 + i / m) * 2.0 ** x for x in e
                                                    for i in range(m)]
    return torch.tensor(v[:127] if fmt == "f8" else v, dtype=torch.float64, device=device)


def _nearest(a, grid):
    """a >= 0 to the grid, ties to the value of even place."""
    hi = torch.searchsorted(grid, a.contiguous()).clamp(max=grid.numel() - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - a, a - grid[lo]
    pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return grid[pick]


def _exact_quant(x, fmt):
    """(values over their scales, scales [rows][blocks]) of float64 [rows][cols]."""
    rows, cols = x.shape
    x = torch.nn.functional.pad(x, (0, -cols % TILE)).unflatten(1, (-1, BLOCK))
    top = x.abs().max(2)[0]
    grid = _grid(fmt, x.device)
    lead = 256.0 if fmt == "f8" else 4.0
    powers = torch.pow(2.0, torch.arange(-127, 128, dtype=torch.float64, device=x.device))
    scale = powers[(torch.searchsorted(powers * lead, top, right=True) - 1).clamp(min=0)]
    v = x / scale.unsqueeze(2)
    return (v.sign() * _nearest(v.abs(), grid)).flatten(1), scale


def _exact_value(s, name, rows, cols, fmt):
    """A microscaled matrix of the state in float64, code by code."""
    codes, tiles = s[name], s[name + "_scales"]
    grid = _grid(fmt, codes.device)
    if fmt == "f8":
        c = codes.long()
        v = grid[(c & 127).clamp(max=126)] * (1 - 2 * (c >> 7)).double()
    else:
        c = torch.stack((codes.long() % 16, codes.long() // 16), -1).flatten(1)
        v = grid[c % 8] * torch.where(c >= 8, -1.0, 1.0).double()
    r = torch.arange(rows, device=codes.device).unsqueeze(1)
    b = (torch.arange(cols, device=codes.device) // BLOCK).unsqueeze(0)
    byte = tiles[r // TILE, b // 4, r % 32, r // 32 % 4, b % 4]
    return v[:, :cols] * torch.pow(2.0, byte.double() - 127)


def _curve(name, v):
    if name == "none":
        return v
    if name == "relu":
        return torch.clamp(v, min=0)
    if name == "silu":
        return v * torch.special.expit(v)
    if name == "gelu":
        return v * torch.special.ndtr(v)
    # 0.5 (1 + tanh(t)) = sigma(2 t)
    return v * torch.special.expit(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v.pow(3)))


def exact(case, seed):
    """The same outputs from the definitions in float64.  A value that is quantised
    after a computation in 32 bits has no such value: next to a rounding border either
    neighbour is right."""
    s = _inputs(case, seed)
    n, op = case["n"], case["op"]
    if op == "quant":
        q, scale = _exact_quant(s["x"].double(), case["fmt"])
        if case["fmt"] == "f4":
            return {"out": (q.unflatten(1, (-1, BLOCK)) * scale.unsqueeze(2)).flatten(1)
                    [:, :case["d"]]}
        rows = _up(n, TILE)
        tiles = torch.full((rows, scale.shape[1]), 2.0 ** -127, dtype=torch.float64,
                           device=scale.device)
        tiles[:n] = scale
        return {"q": q[:, :case["d"]],
                "scales": tiles.unflatten(1, (-1, 4)).unflatten(0, (-1, 4, 32))
                .permute(0, 3, 2, 1, 4)}
    if op == "norm":
        y = s["y"].double()
        if case["post"]:
            y = torch.einsum("tc,t,c->tc", y, (y.square().mean(1) + EPS).rsqrt(),
                             s["w_post"].double())
        if s["gate"] is not None:
            y = s["gate"].double() * y
        return {"h_out": y + case["alpha"] * s["h"].double(), "q": None, "scales": None}
    if op == "gated":
        if case["out"] == "f8":
            return None
        f, d = case["f"], case["d"]
        x = _exact_value(s, "x", n, d, case["xfmt"])
        g, u = (torch.einsum("tk,rk->tr", x, _exact_value(s, w, f, d, case["wfmt"]))
                for w in ("wg", "wu"))
        if case["bias"]:
            g += s["bg"]
            u += s["bu"]
        return {"out": u * _curve(case["act"], g)}
    if op == "linear":
        f, d = case["f"], case["d"]
        if case["given"]:
            x = _exact_value(s, "x", n, d, case["xfmt"])
        else:
            q, scale = _exact_quant(s["x"].double(), case["xfmt"])
            x = (q.unflatten(1, (-1, BLOCK)) * scale.unsqueeze(2)).flatten(1)[:, :d]
        y = torch.einsum("tk,rk->tr", x, _exact_value(s, "w", f, d, case["wfmt"]))
        if case["bias"]:
            y += s["bias"]
        y = _curve(case["act"], y)
        return {"out": y if s["residual"] is None else y + s["residual"]}
    return _exact_route(s, case)


def _exact_route(s, case):
    n, E, k, groups = (case[x] for x in ("n", "E", "k", "groups"))
    l = s["logits"].double()
    p = torch.special.expit(l) if case["score"] == "sigmoid" else torch.softmax(l, 1)
    c = p.clone() if s["bias"] is None else s["bias"] + p
    if case["top"] < groups:
        size = E // groups
        best = c.unflatten(1, (groups, size)).topk(min(2, size), 2)[0].sum(2)
        # a group's place: how many are better, or as good and earlier
        ahead = best.unsqueeze(1) > best.unsqueeze(2)
        same = (best.unsqueeze(1) == best.unsqueeze(2)).tril(-1)
        place = (ahead | same).sum(2)
        c[(place >= case["top"]).repeat_interleave(size, 1)] = -math.inf
    idx = torch.empty((n, k), dtype=torch.int64, device=l.device)
    for j in range(k):
        best = c == c.max(1, keepdim=True)[0]
        idx[:, j] = torch.where(best, torch.arange(E, device=l.device), E).min(1)[0]
        c[torch.arange(n), idx[:, j]] = -math.inf
    p = p.requires_grad_(False)
    leaf = l.clone().requires_grad_(case["train"])
    ps = torch.special.expit(leaf) if case["score"] == "sigmoid" else torch.softmax(leaf, 1)
    ps = ps.gather(1, idx)
    w = case["scale"] * (ps / ps.sum(1, keepdim=True) if case["renorm"] else ps)
    order = torch.argsort(idx.flatten() * (n * k) + torch.arange(n * k, device=l.device))
    offsets = torch.searchsorted(idx.flatten().sort()[0], torch.arange(E + 1, device=l.device))
    out = {"idx": idx.int(), "w": w.detach(), "pairs": order.int(), "offsets": offsets.int()}
    if case["train"]:
        out["dlogits"] = torch.autograd.grad(w, leaf, s["dw"].double())[0]
    return out

"""Float64 definitions of the dense operators (moe_linear, moe_gated_linear,
moe_norm_join) and of their gradients, with the error bounds the tests hold the
kernels to.  Plain torch on whatever device the tensors are on."""
from __future__ import annotations

import math

import torch

ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]
U32 = 2.0 ** -24      # half a step of fp32, relative


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def act(name, v):
    if name == "none":
        return v
    if name == "relu":
        return v.clamp(min=0)
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "gelu":
        return 0.5 * v * torch.special.erfc(-v / math.sqrt(2.0))
    return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))


def slope(name, v):
    if name == "none":
        return torch.ones_like(v)
    if name == "relu":
        return (v > 0).double()
    if name == "silu":
        s = torch.sigmoid(v)
        return s * (1 + v * (1 - s))
    if name == "gelu":
        return 0.5 * torch.special.erfc(-v / math.sqrt(2.0)) \
            + v * torch.exp(-0.5 * v * v) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (v + 0.044715 * v ** 3))
    return 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * c * (1 + 3 * 0.044715 * v * v)


def d(t):
    return None if t is None else t.double()


def product(a, b):
    """a b^T in float64 and the error bound of an fp32 tensor-core sum: the
    products are exact, and each of the K/16 (rounded up) accumulations, and of
    the few joins of split sums, is off by at most two units of the last place
    (2^-22) of the sum of magnitudes."""
    K = a.shape[1]
    s = a @ b.t()
    mag = a.abs() @ b.abs().t()
    return s, (K / 16 + 16) * 2.0 ** -22 * mag


def linear(x, w, bias, name, alpha, residual, out_dtype):
    """(value, bound) of moe_linear's output; (pre, bound) of its pre."""
    p, ep = product(d(x), d(w))
    if bias is not None:
        p = p + d(bias)
    ep = ep + 2 * U32 * p.abs()
    v = alpha * act(name, p)
    # every activation's slope is within [-0.2, 1.2]; its evaluation is good to
    # a few units of fp32 of max(|v|, |p|)
    ev = abs(alpha) * (1.2 * ep + 16 * U32 * p.abs()) + 4 * U32 * v.abs()
    if residual is not None:
        v = v + d(residual)
    return (v, ev + (half_step(out_dtype) + 2 * U32) * v.abs() + tiny(out_dtype)), (p, ep)


def tiny(dtype):
    """Half the distance between subnormal numbers of the type."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps


def gated(x, wg, wu, bg, bu, name):
    g, eg = product(d(x), d(wg))
    u, eu = product(d(x), d(wu))
    if bg is not None:
        g = g + d(bg)
    if bu is not None:
        u = u + d(bu)
    eg, eu = eg + 2 * U32 * g.abs(), eu + 2 * U32 * u.abs()
    a = act(name, g)
    ea = 1.2 * eg + 16 * U32 * g.abs()
    v = a * u
    bound = ea * u.abs() + a.abs() * eu + ea * eu
    return (v, bound + (half_step(x.dtype) + 2 * U32) * v.abs() + tiny(x.dtype)), (g, eg), (u, eu)


def slope_err(g, eg):
    """Error of an activation's slope: its own slope is within [-1.2, 1.2]
    (relu steps at 0: within its argument's error of 0 anything goes), and its
    evaluation is good to a few units of fp32 of 1 + |g|."""
    return 1.2 * eg + 16 * U32 * (1 + g.abs())


def near_step(name, g, eg):
    return (g.abs() <= eg).double() if name == "relu" else torch.zeros_like(g)


def grads(dps, eps_, x, ws, dtype, products_rounded=True):
    """dx, dw and bias gradients from the float64 dp of each matrix and its
    bound; dp is rounded to dtype once as an operand."""
    h = half_step(dtype)
    x64 = d(x)
    dx, edx, out = 0, 0, []
    for dp, e, w in zip(dps, eps_, ws):
        edp = e + ((h * dp.abs() + tiny(dtype)) if products_rounded else 0)
        s, es = product(dp, d(w).t())
        dx, edx = dx + s, edx + es + edp @ d(w).abs()
        sw, ew = product(dp.t(), x64.t())
        ew = ew + edp.t() @ x64.abs()
        sb = dp.sum(0)
        eb = e.sum(0) + 64 * U32 * dp.abs().sum(0)
        out.append(((sw, ew + (h + 2 * U32) * sw.abs() + tiny(dtype)),
                    (sb, eb + (h + 2 * U32) * sb.abs() + tiny(dtype))))
    return (dx, edx + (h + 2 * U32) * dx.abs() + tiny(dtype)), out


def check(got, want, what, rms_factor=None, dtype=None):
    """Element by element within the bound; with rms_factor the 2-norm of the
    error is also within that many half steps of the type (a rounding is off by
    half a step / sqrt(3) in the mean, so 1 covers one rounding, 1.2 two)."""
    ref, bound = want
    assert tuple(got.shape) == tuple(ref.shape), (what, got.shape, ref.shape)
    err = (got.double() - ref).abs()
    assert torch.isfinite(got.double()).all(), what
    worst = (err - bound).max().item()
    assert worst <= 0, f"{what}: {worst:.3e} over the bound (max err {err.max().item():.3e})"
    if rms_factor is not None and ref.numel() >= 64:
        rel = (err.norm() / ref.norm()).item()
        lim = rms_factor * half_step(dtype or got.dtype)
        assert rel <= lim, f"{what}: relative error {rel:.3e} > {lim:.3e}"


# ------------------------------------------------------------------ norm join

def join(h, y, alpha, gate, post, w_post, w_pre, eps):
    """Float64 h_out, xn, r1, r2 and the intermediate z."""
    h, y, gate, w_post, w_pre = d(h), d(y), d(gate), d(w_post), d(w_pre)
    one = torch.ones((), dtype=torch.float64, device=y.device)
    r1 = 1 / torch.sqrt((y * y).mean(1, keepdim=True) + eps) if post \
        else torch.ones((y.shape[0], 1), dtype=torch.float64, device=y.device)
    z = y * r1 * (one if w_post is None else w_post) if post else y
    gz = z if gate is None else gate * z
    ho = gz if h is None else alpha * h + gz
    r2 = 1 / torch.sqrt((ho * ho).mean(1, keepdim=True) + eps)
    xn = ho * r2 * (one if w_pre is None else w_pre)
    return ho, xn, r1, r2, z, gz

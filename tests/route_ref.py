"""Float64 definition of moe_route_scored and its gradient, a row and an expert at a
time where order matters.  Plain torch."""
from __future__ import annotations

import torch


def scores(l, score):
    l = l.double()
    if score == "sigmoid":
        return torch.sigmoid(l)
    return torch.softmax(l, 1)


def choice(l, k, score, bias, groups, top):
    """int64 [n][k]; ties to the lower group and the lower expert."""
    n, E = l.shape
    p = scores(l, score)
    c = p if bias is None else p + bias.double()
    order = l.double() if bias is None else c   # p grows with l
    if top < groups:
        v = c.view(n, groups, E // groups).sort(dim=2, descending=True)[0][:, :, :2].sum(2)
        kept = v.sort(dim=1, descending=True, stable=True)[1][:, :top]
        keep = torch.zeros((n, groups), dtype=torch.bool, device=l.device)
        keep[torch.arange(n, device=l.device).unsqueeze(1), kept] = True
        order = order.masked_fill(~keep.repeat_interleave(E // groups, 1), -float("inf"))
    return order.sort(dim=1, descending=True, stable=True)[1][:, :k]


def weights(l, idx, score, renorm, scale):
    if renorm and score == "sigmoid":
        # logs, so that very negative logits keep their ratios
        a = torch.nn.functional.logsigmoid(l.double().gather(1, idx))
        return scale * torch.softmax(a, 1)
    if renorm:
        return scale * torch.softmax(l.double().gather(1, idx), 1)
    return scale * scores(l, score).gather(1, idx)


def grouping(idx, E):
    n, k = idx.shape
    flat = idx.reshape(-1)
    pairs = flat.sort(stable=True)[1]
    counts = torch.bincount(flat, minlength=E)
    return torch.cat([counts.new_zeros(1), counts.cumsum(0)]), pairs


def gradient(l, idx, dw, score, renorm, scale):
    """The formula, in float64."""
    l64 = l.double().clone().requires_grad_(True)
    w = weights_graph(l64, idx, score, renorm, scale)
    return torch.autograd.grad(w, l64, dw.double())[0]


def weights_graph(l64, idx, score, renorm, scale):
    if renorm:
        a = torch.nn.functional.logsigmoid(l64) if score == "sigmoid" else l64
        return scale * torch.softmax(a.gather(1, idx), 1)
    p = torch.sigmoid(l64) if score == "sigmoid" else torch.softmax(l64, 1)
    return scale * p.gather(1, idx)

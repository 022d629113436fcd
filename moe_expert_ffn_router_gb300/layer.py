"""Owning wrapper around one MoE layer's device buffers (expert bank, router,
outputs, workspace).  Marshalling only: every step runs in librvqmoe."""
from __future__ import annotations

import numpy as np
import torch

from . import (MOE_ACT_SILU, MOE_MX_F4, MOE_MX_F8, MOE_SCORE_SIGMOID, RVQ_WS_STATUS_BYTES,
               moe_bank_init, moe_bank_record_bytes, moe_bank_validate, moe_bank_write_expert, moe_cache_bank, moe_cache_create,
               moe_cache_destroy, moe_cache_stats, moe_combine, moe_expert_ffn,
               moe_gated_linear, moe_gated_linear_backward, moe_gated_linear_workspace_bytes,
               moe_layer_forward, moe_layer_forward_host, moe_layer_forward_prenorm,
               moe_layer_forward_streamed, moe_layer_graph_create, moe_linear,
               moe_linear_backward, moe_linear_workspace_bytes, moe_mx_code_bytes,
               moe_mx_gated_linear, moe_mx_gated_linear_workspace_bytes, moe_mx_linear,
               moe_mx_linear_workspace_bytes, moe_mx_quantize, moe_mx_scale_bytes,
               moe_norm_join, moe_norm_join_mx, moe_rms_norm, moe_route, moe_route_rule,
               moe_route_scored, moe_router_logits, moe_workspace_bytes, rvq_ws_clear, rvq_ws_status)


def _dev(a, device, dtype=None):
    if isinstance(a, torch.Tensor):
        return a.to(device=device, dtype=dtype or a.dtype).contiguous()
    t = torch.from_numpy(np.ascontiguousarray(a))
    return t.to(device=device, dtype=dtype or t.dtype)


class MoeLayer:
    """Expert bank of `n_experts` RVQ experts (d hidden, f intermediate) plus a
    linear router; top-k routing."""

    def __init__(self, n_experts: int, d: int, f: int, k: int, layer: int = 0,
                 device: str | torch.device = "cuda"):
        self.E, self.d, self.f, self.k, self.layer = n_experts, d, f, k, layer
        self.device = torch.device(device)
        rb = moe_bank_record_bytes(d, f)
        if rb == 0:
            raise ValueError(f"d={d}, f={f} must be multiples of 512")
        self.record_bytes = rb
        self.buf = torch.empty(rb * n_experts, dtype=torch.uint8, device=self.device)
        assert self.buf.data_ptr() % 256 == 0
        self.bank = moe_bank_init(self.buf, n_experts, d, f, layer)
        self.wr = None
        self.bias = None
        self.rule = None
        self._ws = {}

    # ---------------------------------------------------------------- loading
    def load_expert(self, e: int, gate_codes, up_codes, down_codes, codebooks):
        """Canonical codes uint8 [f][d/8][3], [f][d/8][3], [d][f/8][3] and
        codebooks fp32 [3 matrices][3][256][8] (numpy or tensors)."""
        dev = self.device
        g = _dev(gate_codes, dev, torch.uint8)
        u = _dev(up_codes, dev, torch.uint8)
        dn = _dev(down_codes, dev, torch.uint8)
        cb = _dev(codebooks, dev, torch.float32)
        assert g.numel() == self.f * self.d * 3 // 8 and dn.numel() == self.d * self.f * 3 // 8
        assert cb.numel() == 3 * 3 * 256 * 8
        moe_bank_write_expert(self.bank, e, g, u, dn, cb)

    def set_router(self, wr, bias=None):
        self.wr = _dev(wr, self.device, torch.float32)
        assert self.wr.shape == (self.E, self.d)
        self.bias = None if bias is None else _dev(bias, self.device, torch.float32)

    def set_scoring(self, score: int = MOE_SCORE_SIGMOID, bias=None, groups: int = 1,
                    top_groups: int = 1, renorm: bool = True, scale: float = 1.0):
        """Experts chosen by scores plus a balance bias (fp32 [E]) from the best groups
        (moe_route_scored) in forward() and forward_steps()."""
        bias = None if bias is None else _dev(bias, self.device, torch.float32)
        self.rule = moe_route_rule(self.E, score, bias, groups, top_groups, renorm, scale)

    def _by_logits(self, what: str):
        if self.rule is not None:
            raise ValueError(f"{what}: the layer scores its experts (set_scoring), and this call "
                             "chooses by logits")

    def validate(self):
        moe_bank_validate(self.bank)

    def record(self, e: int) -> torch.Tensor:
        return self.buf[e * self.record_bytes:(e + 1) * self.record_bytes]

    # ----------------------------------------------------------------- buffers
    def workspace(self, n: int) -> torch.Tensor:
        ws = self._ws.get(n)
        if ws is None:
            nbytes = moe_workspace_bytes(self.bank, n, self.k)
            ws = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
            rvq_ws_clear(ws)
            self._ws[n] = ws
        return ws

    def buffers(self, n: int) -> dict:
        dev, E, k = self.device, self.E, self.k
        return dict(
            logits=torch.empty((n, E), dtype=torch.float32, device=dev),
            idx=torch.empty((n, k), dtype=torch.int32, device=dev),
            w=torch.empty((n, k), dtype=torch.float32, device=dev),
            offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
            pairs=torch.empty(n * k, dtype=torch.int32, device=dev),
            out=torch.empty((n, self.d), dtype=torch.float32, device=dev),
            ws=self.workspace(n))

    # ----------------------------------------------------------------- compute
    def forward(self, x: torch.Tensor, bufs: dict | None = None, events=None,
                tc_min_tokens: int = 0, residual: torch.Tensor | None = None) -> dict:
        """Whole layer: out = residual + sum_slot w * expert(x) (residual
        defaults to x).  Experts with at least tc_min_tokens tokens use the
        tensor-core path (0: none)."""
        n = x.shape[0]
        b = bufs or self.buffers(n)
        moe_layer_forward(self.bank, self.wr, self.bias, x, n, self.k, b["logits"], b["idx"],
                          b["w"], b["offsets"], b["pairs"], b["out"], b["ws"], events=events,
                          tc_min_tokens=tc_min_tokens, residual=residual, rule=self.rule)
        return b

    def forward_host(self, x_host: torch.Tensor, out_host: torch.Tensor, bufs: dict | None = None,
                     tc_min_tokens: int = 0) -> dict:
        """The layer with its input read from and its output written to host
        tensors (pinned for asynchronous copies), through the library's
        host-buffer call; asynchronous on the current stream."""
        self._by_logits("forward_host")
        n = x_host.shape[0]
        b = bufs or self.buffers(n)
        xd = b.get("x_dev")
        if xd is None or xd.dtype != x_host.dtype or xd.shape != (n, self.d):
            xd = b["x_dev"] = torch.empty((n, self.d), dtype=x_host.dtype, device=self.device)
        moe_layer_forward_host(self.bank, self.wr, self.bias, x_host, n, self.k, xd, b["logits"],
                               b["idx"], b["w"], b["offsets"], b["pairs"], b["out"], out_host,
                               b["ws"], tc_min_tokens=tc_min_tokens)
        return b

    def graph(self, x_dev: torch.Tensor, bufs: dict, x_host: torch.Tensor | None = None,
              out_host: torch.Tensor | None = None, tc_min_tokens: int = 0):
        """A CUDA graph of this layer on x_dev and bufs (optionally with the
        copy of x_host into x_dev before it and of the output to out_host
        after it), recorded on a side stream; launch() runs it on the current
        stream."""
        self._by_logits("graph")
        side = torch.cuda.Stream(device=self.device)
        side.wait_stream(torch.cuda.current_stream())
        g = moe_layer_graph_create(self.bank, self.wr, self.bias, x_dev.shape[0], self.k, x_dev,
                                   bufs["logits"], bufs["idx"], bufs["w"], bufs["offsets"],
                                   bufs["pairs"], bufs["out"], bufs["ws"],
                                   tc_min_tokens=tc_min_tokens, x_host=x_host, out_host=out_host,
                                   stream=side)
        torch.cuda.current_stream().wait_stream(side)
        return g

    def forward_steps(self, x: torch.Tensor) -> dict:
        """Same layer through the separate calls (router, route, FFN, combine)."""
        n = x.shape[0]
        b = self.buffers(n)
        moe_router_logits(self.wr, self.bias, x, n, self.E, self.d, b["logits"])
        if self.rule is None:
            moe_route(b["logits"], n, self.E, self.k, b["idx"], b["w"], b["offsets"], b["pairs"],
                      b["ws"])
        else:
            r = self.rule
            moe_route_scored(b["logits"], n, self.E, self.k, b["idx"], b["w"], b["offsets"],
                             b["pairs"], b["ws"], r.score, r.keep, r.groups, r.top_groups,
                             r.renorm, r.scale)
        y = torch.empty((n * self.k, self.d), dtype=torch.float32, device=self.device)
        moe_expert_ffn(self.bank, x, n, self.k, b["offsets"], b["pairs"], y, b["ws"])
        moe_combine(y, b["w"], n, self.k, self.d, x, b["out"])
        b["y_pair"] = y
        return b

    def status(self, n: int) -> tuple[int, int]:
        return rvq_ws_status(self.workspace(n))


def _share_workspace(layers: list[MoeLayer], n: int):
    """One workspace for layers that run one after another on one stream (24 GB for
    a K3-shaped layer at 2048 tokens)."""
    ws = layers[0].workspace(n)
    for L in layers[1:]:
        if moe_workspace_bytes(L.bank, n, L.k) <= ws.numel():
            L._ws[n] = ws


class MoeStack:
    """Layers applied in order to a residual stream h (the first layer's
    input, then each layer's fp32 output): layer i computes
    out = h + sum_slot w * expert(rms_norm(h)), the normalised stream in
    bf16.  Each layer keeps its own buffers (its "xn" holds the normalised
    input), so the stream is never copied."""

    def __init__(self, layers: list[MoeLayer], eps: float = 1e-6):
        assert layers and all(L.d == layers[0].d for L in layers)
        self.layers = layers
        self.eps = eps
        self._bufs = {}

    def buffers(self, n: int) -> list[dict]:
        b = self._bufs.get(n)
        if b is None:
            _share_workspace(self.layers, n)
            b = [L.buffers(n) for L in self.layers]
            for L, bl in zip(self.layers, b):
                bl["xn"] = torch.empty((n, L.d), dtype=torch.bfloat16, device=L.device)
            self._bufs[n] = b
        return b

    def forward(self, x: torch.Tensor, events=None, tc_min_tokens: int = 0) -> list[dict]:
        """Runs every layer; returns the per-layer buffers (the last one's
        "out" is the stack output).  `events`, if given, are layer 0's."""
        n = x.shape[0]
        bufs = self.buffers(n)
        h = x
        for i, L in enumerate(self.layers):
            b = bufs[i]
            if L.rule is not None or (events is not None and i == 0):
                # scored experts, or per-kernel timing marks: the norm and the layer as
                # separate calls
                moe_rms_norm(h, n, L.d, b["xn"], eps=self.eps)
                L.forward(b["xn"], b, events=events if i == 0 else None,
                          tc_min_tokens=tc_min_tokens, residual=h)
            else:
                moe_layer_forward_prenorm(L.bank, L.wr, L.bias, h, n, L.k, self.eps, b["xn"],
                                          b["logits"], b["idx"], b["w"], b["offsets"], b["pairs"],
                                          b["out"], b["ws"], tc_min_tokens=tc_min_tokens)
            h = b["out"]
        return bufs


class MoeStreamedStack:
    """The same stack with its expert records in pinned host memory and an HBM
    cache of `slots` records (moe_layer_forward_streamed per layer): the
    pages' streaming engine with host memory in place of NVMe.  The layers'
    device banks are copied into one host bank and released.  With
    lookahead > 0 each layer prefetches the next layer's predicted experts."""

    def __init__(self, layers: list[MoeLayer], slots: int, lookahead: int = 0,
                 eps: float = 1e-6):
        assert layers and all(L.d == layers[0].d and L.f == layers[0].f and L.E == layers[0].E
                              for L in layers)
        for L in layers:
            L._by_logits("MoeStreamedStack")
        L0 = layers[0]
        self.n_layers, self.E, self.d, self.f, self.k = len(layers), L0.E, L0.d, L0.f, L0.k
        self.device = L0.device
        self.eps, self.lookahead = eps, lookahead
        rb = L0.record_bytes
        self.host = torch.empty(self.n_layers * self.E * rb, dtype=torch.uint8, pin_memory=True)
        for i, L in enumerate(layers):
            self.host[i * self.E * rb:(i + 1) * self.E * rb].copy_(L.buf)
            L.buf = None  # the device bank is no longer needed
        torch.cuda.synchronize()
        self.wr = [L.wr for L in layers]
        self.bias = [L.bias for L in layers]
        self.slots = torch.empty(slots * rb, dtype=torch.uint8, device=self.device)
        self.slot_map = torch.full((self.n_layers, self.E), -1, dtype=torch.int32,
                                   device=self.device)
        self.cache = moe_cache_create(self.host, self.n_layers, self.E, self.d, self.f,
                                      self.slots, self.slot_map)
        self._bufs = {}

    def buffers(self, n: int) -> list[dict]:
        b = self._bufs.get(n)
        if b is None:
            dev, E, k = self.device, self.E, self.k
            ws = torch.empty(moe_workspace_bytes(moe_cache_bank(self.cache, 0), n, k),
                             dtype=torch.uint8, device=dev)
            rvq_ws_clear(ws)
            b = [dict(logits=torch.empty((n, E), dtype=torch.float32, device=dev),
                      idx=torch.empty((n, k), dtype=torch.int32, device=dev),
                      w=torch.empty((n, k), dtype=torch.float32, device=dev),
                      offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
                      pairs=torch.empty(n * k, dtype=torch.int32, device=dev),
                      out=torch.empty((n, self.d), dtype=torch.float32, device=dev),
                      xn=torch.empty((n, self.d), dtype=torch.bfloat16, device=dev),
                      next_logits=torch.empty((n, E), dtype=torch.float32, device=dev),
                      ws=ws) for _ in range(self.n_layers)]
            self._bufs[n] = b
        return b

    def forward(self, x: torch.Tensor, tc_min_tokens: int = 0) -> list[dict]:
        n = x.shape[0]
        bufs = self.buffers(n)
        h = x
        for i in range(self.n_layers):
            bi = bufs[i]
            moe_rms_norm(h, n, self.d, bi["xn"], eps=self.eps)
            nxt = i + 1 < self.n_layers and self.lookahead > 0
            moe_layer_forward_streamed(
                self.cache, i, self.wr[i], self.bias[i], bi["xn"], n, self.k, bi["logits"],
                bi["idx"], bi["w"], bi["offsets"], bi["pairs"], bi["out"], bi["ws"],
                residual=h, tc_min_tokens=tc_min_tokens,
                next_wr=self.wr[i + 1] if nxt else None,
                next_bias=self.bias[i + 1] if nxt else None,
                lookahead=self.lookahead if nxt else 0,
                next_logits=bi["next_logits"] if nxt else None)
            h = bi["out"]
        return bufs

    def stats(self) -> dict:
        return moe_cache_stats(self.cache)

    def status(self, n: int) -> tuple[int, int]:
        return rvq_ws_status(self.buffers(n)[0]["ws"])

    def close(self):
        if self.cache:
            torch.cuda.synchronize()
            moe_cache_destroy(self.cache)
            self.cache = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class SharedExpert:
    """A dense (unquantised) feed-forward block that every token passes, beside
    the routed experts: out = (act(x Wg^T) * (x Wu^T)) Wd^T, with gradients.
    Weights are bf16 or fp16: gate and up [f][d], down [d][f]."""

    def __init__(self, wg, wu, wd, act: int = MOE_ACT_SILU, device: str | torch.device = "cuda"):
        self.device = torch.device(device)
        self.wg, self.wu, self.wd = (_dev(w, self.device) for w in (wg, wu, wd))
        self.f, self.d = self.wg.shape
        assert self.wu.shape == (self.f, self.d) and self.wd.shape == (self.d, self.f)
        for name, w in (("wg", self.wg), ("wu", self.wu), ("wd", self.wd)):
            if w.dtype not in (torch.bfloat16, torch.float16) or w.dtype != self.wg.dtype:
                raise TypeError(f"{name}: {w.dtype} (bf16 or fp16, one type for all three)")
        self.act = act
        self._bufs = {}

    def buffers(self, n: int, train: bool = False) -> dict:
        """Outputs and workspace for n tokens, kept; train adds what the
        gradients need and receive."""
        b = self._bufs.get((n, train))
        if b is None:
            def new(*shape, dtype=self.wg.dtype):
                return torch.empty(shape, dtype=dtype, device=self.device)

            nbytes = max(moe_gated_linear_workspace_bytes(n, self.f, self.d, train),
                         moe_linear_workspace_bytes(n, self.d, self.f, train))
            b = dict(hidden=new(n, self.f), out=new(n, self.d, dtype=torch.float32),
                     ws=new(nbytes, dtype=torch.uint8))
            if train:
                b.update(pre=new(2, n, self.f, dtype=torch.float32), dhidden=new(n, self.f),
                         dx=new(n, self.d), dwg=torch.empty_like(self.wg),
                         dwu=torch.empty_like(self.wu), dwd=torch.empty_like(self.wd))
            rvq_ws_clear(b["ws"])
            self._bufs[n, train] = b
        return b

    def forward(self, x: torch.Tensor, residual: torch.Tensor | None = None,
                train: bool = False) -> dict:
        """out (fp32) = residual + the block of x; with train the gradients'
        inputs are kept for backward()."""
        n = x.shape[0]
        b = self.buffers(n, train)
        moe_gated_linear(x, self.wg, self.wu, n, self.f, self.d, b["hidden"], b["ws"],
                         act=self.act, pre=b.get("pre"))
        moe_linear(b["hidden"], self.wd, n, self.d, self.f, b["out"], b["ws"], residual=residual)
        return b

    def backward(self, x: torch.Tensor, dout: torch.Tensor) -> dict:
        """Gradients of a forward(x, train=True): dx, dwg, dwu, dwd from dout (the
        weights' type); the residual's gradient is dout."""
        n = x.shape[0]
        b = self.buffers(n, True)
        moe_linear_backward(dout, b["hidden"], self.wd, n, self.d, self.f, b["ws"],
                            dx=b["dhidden"], dw=b["dwd"])
        moe_gated_linear_backward(b["dhidden"], x, self.wg, self.wu, b["pre"], n, self.f, self.d,
                                  b["ws"], dx=b["dx"], dwg=b["dwg"], dwu=b["dwu"], act=self.act)
        return b

    def status(self, n: int, train: bool = False) -> tuple[int, int]:
        return rvq_ws_status(self.buffers(n, train)["ws"])


class MxSharedExpert:
    """A shared expert in microscaled formats, for serving: out = residual +
    (act(x Wg^T) * (x Wu^T)) Wd^T.  The weights (gate and up [f][d], down [d][f]; fp32,
    bf16 or fp16) are quantised once to wfmt; tokens and hidden values are xfmt."""

    def __init__(self, wg, wu, wd, act: int = MOE_ACT_SILU, wfmt: int = MOE_MX_F4,
                 xfmt: int = MOE_MX_F8, device: str | torch.device = "cuda"):
        self.device = torch.device(device)
        self.act, self.wfmt, self.xfmt = act, wfmt, xfmt
        self.f, self.d = wg.shape
        assert wu.shape == (self.f, self.d) and wd.shape == (self.d, self.f)
        self.wg, self.wu, self.wd = (self._quantized(w, wfmt) for w in (wg, wu, wd))
        self._bufs = {}

    def _empty(self, rows: int, cols: int, fmt: int):
        """Codes and scales of a matrix (bytes of rows behind the last hold no scale)."""
        return (torch.empty(moe_mx_code_bytes(fmt, rows, cols), dtype=torch.uint8,
                            device=self.device),
                torch.zeros(moe_mx_scale_bytes(rows, cols), dtype=torch.uint8, device=self.device))

    def _quantized(self, w, fmt: int):
        w = _dev(w, self.device)
        q = self._empty(*w.shape, fmt)
        moe_mx_quantize(w, *w.shape, *q, fmt)
        return q

    def buffers(self, n: int) -> dict:
        """Microscaled tokens and hidden values (codes and scales each), the output and
        the workspace for n tokens, kept."""
        b = self._bufs.get(n)
        if b is None:
            nbytes = max(moe_mx_gated_linear_workspace_bytes(n, self.f, self.d),
                         moe_mx_linear_workspace_bytes(n, self.d, self.f))
            b = dict(x=self._empty(n, self.d, self.xfmt), hidden=self._empty(n, self.f, self.xfmt),
                     out=torch.empty((n, self.d), dtype=torch.float32, device=self.device),
                     ws=torch.empty(nbytes, dtype=torch.uint8, device=self.device))
            rvq_ws_clear(b["ws"])
            self._bufs[n] = b
        return b

    def forward(self, x: torch.Tensor, residual: torch.Tensor | None = None) -> dict:
        """out (fp32) = residual + the block of x [n][d] (fp32, bf16 or fp16)."""
        n = x.shape[0]
        moe_mx_quantize(x, n, self.d, *self.buffers(n)["x"], self.xfmt)
        return self.forward_quantized(n, residual)

    def forward_quantized(self, n: int, residual: torch.Tensor | None = None) -> dict:
        """The block of the n tokens that buffers(n)["x"] holds (moe_norm_join_mx writes
        them there)."""
        b = self.buffers(n)
        moe_mx_gated_linear(*b["x"], *self.wg, *self.wu, n, self.f, self.d, b["hidden"][0],
                            b["ws"], xfmt=self.xfmt, wfmt=self.wfmt, act=self.act,
                            out_scales=b["hidden"][1], ofmt=self.xfmt)
        moe_mx_linear(*b["hidden"], *self.wd, n, self.d, self.f, b["out"], b["ws"],
                      xfmt=self.xfmt, wfmt=self.wfmt, residual=residual)
        return b

    def status(self, n: int) -> tuple[int, int]:
        return rvq_ws_status(self.buffers(n)["ws"])


class SharedExpertStack:
    """Blocks of routed experts with a shared expert, normed before and after:
        xn = norm(h) * w_pre;  y = shared(xn) + sum_slot w * expert(xn)
        h  = alpha * h + gate * norm(y) * w_post
    for each block (MoeLayer, SharedExpert or MxSharedExpert, dict of w_pre, w_post,
    gate: tensors or None).  The norm after a block, its gate, the residual's scale and the
    norm before the next block are one launch (moe_norm_join), and the shared
    expert's output enters the routed layer as its residual.  h is fp32, xn bf16 (the
    routed layers take no fp16), so dense shared experts are bf16 (TypeError).  For a
    microscaled one the join before its block writes the normed rows in its format too."""

    def __init__(self, blocks, alpha: float = 1.0, eps: float = 1e-6):
        assert blocks and all(L.d == S.d == blocks[0][0].d for L, S, _ in blocks)
        for i, (_, S, _) in enumerate(blocks):
            if not isinstance(S, MxSharedExpert) and S.wg.dtype != torch.bfloat16:
                raise TypeError(f"block {i}: shared expert of {S.wg.dtype}, and the normed stream "
                                "that the routed experts read too is bf16")
        self.blocks, self.alpha, self.eps = list(blocks), alpha, eps
        self._bufs = {}

    def buffers(self, n: int) -> list[dict]:
        b = self._bufs.get(n)
        if b is None:
            b = []
            _share_workspace([L for L, _, _ in self.blocks], n)
            for L, _, _ in self.blocks:
                bl = L.buffers(n)
                bl["xn"] = torch.empty((n, L.d), dtype=torch.bfloat16, device=L.device)
                bl["h"] = torch.empty((n, L.d), dtype=torch.float32, device=L.device)
                b.append(bl)
            self._bufs[n] = b
        return b

    def forward(self, x: torch.Tensor, tc_min_tokens: int = 0) -> list[dict]:
        """x [n][d] fp32; returns the blocks' buffers ("xn" the normed input,
        "out" y, "h" the stream after the block)."""
        n = x.shape[0]
        bufs = self.buffers(n)

        def join(y, h_out, i, **kw):
            """The norm after a block joined with the one before block i, whose shared
            expert's format the normed rows are written in too."""
            nxt = self.blocks[i] if i < len(self.blocks) else None
            xn = bufs[i]["xn"] if nxt else None
            kw.update(w_pre=nxt[2].get("w_pre") if nxt else None, eps=self.eps)
            if nxt and isinstance(nxt[1], MxSharedExpert):
                moe_norm_join_mx(y, n, nxt[1].d, h_out, *nxt[1].buffers(n)["x"], fmt=nxt[1].xfmt,
                                 xn=xn, **kw)
            else:
                moe_norm_join(y, n, self.blocks[0][0].d, h_out, xn, **kw)

        join(x, None, 0, post_norm=False)
        h = x
        for i, (L, S, p) in enumerate(self.blocks):
            b = bufs[i]
            shared = S.forward_quantized(n) if isinstance(S, MxSharedExpert) else S.forward(b["xn"])
            L.forward(b["xn"], b, tc_min_tokens=tc_min_tokens, residual=shared["out"])
            join(b["out"], b["h"], i + 1, h=h, alpha=self.alpha, gate=p.get("gate"),
                 w_post=p.get("w_post"))
            h = b["h"]
        return bufs


__all__ = ["MoeLayer", "MoeStack", "MoeStreamedStack", "MxSharedExpert", "SharedExpert",
           "SharedExpertStack", "RVQ_WS_STATUS_BYTES"]

"""Python binding of librvqmoe (RVQ MoE expert FFN for GB300, sm_103a).

Argument marshalling only: every step runs in the library's CUDA kernels.
Functions carry the C names of include/rvqmoe.h and take torch tensors (device
memory) plus the current CUDA stream.  Importing fails loudly when the
compiled library is missing; there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os
import re

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "librvqmoe.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "rvqmoe.h")

RVQ_F32, RVQ_BF16, RVQ_F16 = 0, 1, 2
RVQ_WS_STATUS_BYTES = 256
RVQ_CODEBOOK_BYTES = 24576
RVQ_BANK_MAGIC = 0x31515652
RVQ_HDR_FLAG_CRC32 = 0x1
MOE_LAYER_EVENTS = 8
RVQMOE_PREFILL_MIN_TOKENS = 6
MOE_ACT_NONE, MOE_ACT_RELU, MOE_ACT_SILU, MOE_ACT_GELU, MOE_ACT_GELU_TANH = range(5)
MOE_ACTS = {"none": MOE_ACT_NONE, "relu": MOE_ACT_RELU, "silu": MOE_ACT_SILU,
            "gelu": MOE_ACT_GELU, "gelu_tanh": MOE_ACT_GELU_TANH}
MOE_WAYS = ("stream", "tiles", "parts", "split")
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = range(2)
MOE_SCORES = {"softmax": MOE_SCORE_SOFTMAX, "sigmoid": MOE_SCORE_SIGMOID}
MOE_MX_F8, MOE_MX_F4 = range(2)
MOE_MX = {"f8": MOE_MX_F8, "f4": MOE_MX_F4}
(MOE_GATE_NONE, MOE_GATE_SCALAR, MOE_GATE_TOKEN, MOE_GATE_CHANNEL, MOE_GATE_FULL) = range(5)
DEV_ERR_INDEX, DEV_ERR_NONFINITE, DEV_ERR_CORRUPT, DEV_ERR_TIMEOUT = 1, 2, 4, 8
STATUS = {0: "RVQ_OK", 1: "RVQ_EINVAL", 2: "RVQ_EALIGN", 3: "RVQ_ENOMEM", 4: "RVQ_ECORRUPT",
          5: "RVQ_EDEVICE", 6: "RVQ_ETIMEOUT", 7: "RVQ_ECUDA", 8: "RVQ_ENOTIMPL"}


class RvqError(RuntimeError):
    def __init__(self, name, code, msg):
        super().__init__(f"{name}: {STATUS.get(code, code)}: {msg}")
        self.code = code
        self.status = STATUS.get(code, str(code))


class RvqMoeBank(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("record_bytes", ctypes.c_uint64),
                ("n_experts", ctypes.c_int32), ("d", ctypes.c_int32),
                ("f", ctypes.c_int32), ("layer", ctypes.c_int32)]


class MoeRouteRule(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("bias", ctypes.c_void_p),
                ("groups", ctypes.c_int32), ("top_groups", ctypes.c_int32),
                ("renorm", ctypes.c_int32), ("scale", ctypes.c_float)]
    keep = None  # the tensor that `bias` points into (moe_route_rule)


class RvqCacheStats(ctypes.Structure):
    _fields_ = [("hits", ctypes.c_uint64), ("misses", ctypes.c_uint64),
                ("prefetched", ctypes.c_uint64), ("prefetch_used", ctypes.c_uint64),
                ("bytes_copied", ctypes.c_uint64), ("slots", ctypes.c_int32),
                ("pad", ctypes.c_int32)]


if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built: run `python -c 'import __graft_entry__ as g; "
                      "g.build()'` (nvcc, sm_103a)")

_vp, _i32, _u32, _u64, _sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint32,
                              ctypes.c_uint64, ctypes.c_size_t)
_i64, _f32 = ctypes.c_int64, ctypes.c_float
_lib = ctypes.CDLL(LIB_PATH)
_BANKP = ctypes.POINTER(RvqMoeBank)
_RULEP = ctypes.POINTER(MoeRouteRule)
_SIGS = {
    "rvq_status_string": (ctypes.c_char_p, [_i32]),
    "rvq_last_error": (ctypes.c_char_p, []),
    "rvq_version": (_u32, []),
    "rvq_code_bytes": (_sz, [_i32, _i32]),
    "rvq_pack": (_i32, [_vp, _i32, _i32, _vp, _sz, _vp]),
    "rvq_unpack": (_i32, [_vp, _i32, _i32, _vp, _sz, _vp]),
    "rvq_pack_codebooks": (_i32, [_vp, _vp, _vp]),
    "rvq_lut_build": (_i32, [_vp, _vp, _i32, _i32, _i32, _vp, _vp]),
    "rvq_gemv_workspace_bytes": (_sz, [_i32, _i32, _i32]),
    "rvq_gemv": (_i32, [_vp, _vp, _i32, _i32, _vp, _i32, _i32, _vp, _vp, _sz, _vp]),
    "rvq_gemv_noalloc": (_i32, [_vp, _vp, _i32, _i32, _vp, _i32, _i32, _vp, _vp]),
    "rvq_gemv_noalloc_status": (_i32, [ctypes.POINTER(_u32), _vp]),
    "moe_bank_record_bytes": (_u64, [_i32, _i32]),
    "moe_bank_init": (_i32, [_BANKP, _vp, _u64, _i32, _i32, _i32, _i32]),
    "moe_bank_write_expert": (_i32, [_BANKP, _i32, _vp, _vp, _vp, _vp, _vp]),
    "moe_bank_validate": (_i32, [_BANKP, _vp]),
    "moe_bank_seal": (_i32, [_BANKP, _vp]),
    "rvq_encode_workspace_bytes": (_sz, [_i32, _i32]),
    "rvq_encode": (_i32, [_vp, _i32, _i32, _i32, _vp, _vp, _vp, _sz, _vp]),
    "moe_cache_create": (_i32, [ctypes.POINTER(_vp), _vp, _i32, _i32, _i32, _i32, _vp, _u64,
                                _vp]),
    "moe_cache_destroy": (_i32, [_vp]),
    "moe_cache_stats": (_i32, [_vp, ctypes.POINTER(RvqCacheStats)]),
    "moe_cache_bank": (_i32, [_vp, _i32, _BANKP]),
    "moe_layer_forward_streamed": (_i32, [_vp, _i32, _vp, _vp, _vp, _i32, _i32, _i32, _vp, _vp,
                                          _vp, _vp, _vp, _vp, _vp, _sz, _vp, _i32, _i32, _vp,
                                          _vp, _i32, _vp, _vp]),
    "moe_bank_verify": (_i32, [_BANKP, _vp, _vp, _sz, _vp]),
    "moe_router_logits": (_i32, [_vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _vp]),
    "moe_route_max_tokens": (_i32, [_i32]),
    "moe_route": (_i32, [_vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "moe_route_scored_workspace_bytes": (_sz, [_i32, _i32]),
    "moe_route_scored": (_i32, [_vp, _i32, _i32, _i32, _RULEP, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "moe_route_scored_backward": (_i32, [_vp, _vp, _vp, _i32, _i32, _i32, _RULEP, _vp, _vp]),
    "moe_workspace_bytes": (_sz, [_BANKP, _i32, _i32]),
    "moe_expert_ffn": (_i32, [_BANKP, _vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _sz, _vp]),
    "moe_expert_ffn_ex": (_i32, [_BANKP, _vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _sz, _i32,
                                 _vp]),
    "moe_combine": (_i32, [_vp, _vp, _i32, _i32, _i32, _vp, _i32, _vp, _vp]),
    "moe_layer_forward": (_i32, [_BANKP, _vp, _vp, _vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp,
                                 _vp, _vp, _vp, _sz, _vp, _vp]),
    "moe_layer_forward_ex": (_i32, [_BANKP, _vp, _vp, _vp, _i32, _i32, _i32, _vp, _vp, _vp,
                                    _vp, _vp, _vp, _vp, _sz, _vp, _i32, _i32, _vp, _vp]),
    "moe_layer_forward_scored": (_i32, [_BANKP, _vp, _vp, _RULEP, _vp, _i32, _i32, _i32, _vp, _vp,
                                        _vp, _vp, _vp, _vp, _vp, _sz, _vp, _i32, _i32, _vp, _vp]),
    "moe_layer_forward_host": (_i32, [_BANKP, _vp, _vp, _vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp,
                                      _vp, _vp, _vp, _vp, _vp, _sz, _i32, _vp]),
    "moe_layer_graph_create": (_i32, [_BANKP, _vp, _vp, _vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp,
                                      _vp, _vp, _vp, _vp, _vp, _sz, _i32, _vp,
                                      ctypes.POINTER(ctypes.c_void_p)]),
    "moe_layer_graph_launch": (_i32, [_vp, _vp]),
    "moe_layer_graph_destroy": (_i32, [_vp]),
    "moe_layer_forward_prenorm": (_i32, [_BANKP, _vp, _vp, _vp, _i32, _i32, _i32, ctypes.c_float,
                                         _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _i32, _vp]),
    "moe_rms_norm": (_i32, [_vp, _i32, _i32, _i32, ctypes.c_float, _vp, _i32, _vp]),
    "moe_linear_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32]),
    "moe_linear": (_i32, [_vp, _i64, _vp, _i64, _vp, _i32, _i32, _i32, _i32, _i32, _f32, _vp, _i32,
                          _i64, _vp, _i32, _i64, _vp, _vp, _sz, _vp]),
    "moe_linear_backward": (_i32, [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _i32, _i32, _i32, _i32,
                                   _i32, _f32, _vp, _i64, _vp, _i64, _vp, _vp, _sz, _vp]),
    "moe_gated_linear_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32]),
    "moe_gated_linear": (_i32, [_vp, _i64, _vp, _vp, _i64, _vp, _vp, _i32, _i32, _i32, _i32, _i32,
                                _vp, _i64, _vp, _vp, _sz, _vp]),
    "moe_gated_linear_backward": (_i32, [_vp, _i64, _vp, _i64, _vp, _vp, _i64, _vp, _i32, _i32,
                                         _i32, _i32, _i32, _vp, _i64, _vp, _vp, _i64, _vp, _vp,
                                         _vp, _sz, _vp]),
    "moe_norm_join": (_i32, [_vp, _i32, _vp, _i32, _i32, _i32, _f32, _vp, _i32, _i32, _i32, _vp,
                             _vp, _i32, _f32, _vp, _vp, _i32, _vp, _vp]),
    "moe_norm_join_workspace_bytes": (_sz, [_i32, _i32]),
    "moe_norm_join_backward": (_i32, [_vp, _vp, _i32, _vp, _i32, _vp, _i32, _i32, _i32, _f32, _vp,
                                      _i32, _i32, _i32, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp,
                                      _vp, _vp, _sz, _vp]),
    "moe_mx_code_bytes": (_sz, [_i32, _i32, _i32]),
    "moe_mx_scale_bytes": (_sz, [_i32, _i32]),
    "moe_mx_quantize": (_i32, [_vp, _i64, _i32, _i32, _i32, _i32, _vp, _vp, _vp]),
    "moe_mx_dequantize": (_i32, [_vp, _vp, _i32, _i32, _i32, _vp, _i32, _i64, _vp]),
    "moe_mx_linear_workspace_bytes": (_sz, [_i32, _i32, _i32]),
    "moe_mx_gated_linear_workspace_bytes": (_sz, [_i32, _i32, _i32]),
    "moe_mx_linear": (_i32, [_vp, _vp, _i32, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _f32,
                             _vp, _i32, _i64, _vp, _i32, _i64, _vp, _sz, _vp]),
    "moe_mx_gated_linear": (_i32, [_vp, _vp, _i32, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _i32, _i32,
                                   _i32, _i32, _vp, _i32, _i64, _vp, _vp, _i32, _vp, _sz, _vp]),
    "moe_norm_join_mx": (_i32, [_vp, _i32, _vp, _i32, _i32, _i32, _f32, _vp, _i32, _i32, _i32, _vp,
                                _vp, _i32, _f32, _vp, _vp, _i32, _i32, _vp, _vp, _vp, _vp]),
    "rvq_selftest_dense_plan": (_i32, [_i32, _i32, _i32, _i32, _i32, ctypes.POINTER(_i32)]),
    "rvq_selftest_mx_plan": (_i32, [_i32, _i32, _i32, _i32, _i32, _i32, ctypes.POINTER(_i32)]),
    "rvq_selftest_prefill_timeout": (_i32, [_BANKP, _vp, _sz, _vp]),
    "rvq_ws_clear": (_i32, [_vp, _vp]),
    "rvq_ws_status": (_i32, [_vp, ctypes.POINTER(_u32), _vp]),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


def header_functions() -> list[str]:
    """Names of every function declared in include/rvqmoe.h."""
    txt = open(HEADER).read()
    txt = re.sub(r"/\*.*?\*/", "", txt, flags=re.S)
    return sorted(set(re.findall(r"\b(\w+)\s*\([^;{]*\)\s*;", txt)) - {"if", "while"})


def lib_has(name: str) -> bool:
    return hasattr(_lib, name)


# ------------------------------------------------------------------ helpers

def _p(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _nbytes(t) -> int:
    return t.numel() * t.element_size()


def _stream(stream=None):
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _dt(t) -> int:
    if t.dtype == torch.bfloat16:
        return RVQ_BF16
    if t.dtype == torch.float32:
        return RVQ_F32
    raise TypeError(f"unsupported dtype {t.dtype} (bf16 or fp32)")


def _check(name, rc):
    if rc != 0:
        raise RvqError(name, rc, last_error())


def status_string(code: int) -> str:
    return _lib.rvq_status_string(code).decode()


def last_error() -> str:
    return _lib.rvq_last_error().decode()


def rvq_version() -> int:
    return int(_lib.rvq_version())


# ------------------------------------------------------------------ RVQ calls

def rvq_code_bytes(rows: int, cols: int) -> int:
    return int(_lib.rvq_code_bytes(rows, cols))


def rvq_pack(codes, rows, cols, packed, stream=None):
    _check("rvq_pack", _lib.rvq_pack(_p(codes), rows, cols, _p(packed), _nbytes(packed),
                                     _stream(stream)))


def rvq_unpack(packed, rows, cols, codes, stream=None):
    _check("rvq_unpack", _lib.rvq_unpack(_p(packed), rows, cols, _p(codes), _nbytes(codes),
                                         _stream(stream)))


def rvq_pack_codebooks(cb, cb_packed, stream=None):
    _check("rvq_pack_codebooks", _lib.rvq_pack_codebooks(_p(cb), _p(cb_packed), _stream(stream)))


def rvq_lut_build(codebooks, x, n, cols, lut, stream=None):
    _check("rvq_lut_build", _lib.rvq_lut_build(_p(codebooks), _p(x), _dt(x), n, cols, _p(lut),
                                               _stream(stream)))


def rvq_gemv_workspace_bytes(rows, cols, n) -> int:
    return int(_lib.rvq_gemv_workspace_bytes(rows, cols, n))


def rvq_gemv(packed_codes, packed_cb, rows, cols, x, n, y, ws, stream=None):
    _check("rvq_gemv", _lib.rvq_gemv(_p(packed_codes), _p(packed_cb), rows, cols, _p(x), _dt(x),
                                     n, _p(y), _p(ws), _nbytes(ws), _stream(stream)))


RVQ_NOALLOC_SCRATCH_BYTES = 4 << 20


def rvq_gemv_noalloc(packed_codes, packed_cb, rows, cols, x, n, y, stream=None):
    """rvq_gemv without a workspace, for callers that cannot allocate device
    memory: the scratch is a fixed 4 MiB array inside the library, shared by
    all calls (calls that overlap on the GPU race).  Make the first call on a
    device before any stream capture."""
    _check("rvq_gemv_noalloc",
           _lib.rvq_gemv_noalloc(_p(packed_codes), _p(packed_cb), rows, cols, _p(x), _dt(x), n,
                                 _p(y), _stream(stream)))


def rvq_gemv_noalloc_status(stream=None) -> tuple[int, int]:
    """Device status of the no-allocation GEMV's fixed array: (status code,
    raw bits) after the stream's work; clears the bits."""
    bits = _u32(0)
    rc = _lib.rvq_gemv_noalloc_status(ctypes.byref(bits), _stream(stream))
    return int(rc), int(bits.value)


# ------------------------------------------------------------------ bank

def moe_bank_record_bytes(d: int, f: int) -> int:
    return int(_lib.moe_bank_record_bytes(d, f))


def moe_bank_init(buffer, n_experts, d, f, layer=0) -> RvqMoeBank:
    bank = RvqMoeBank()
    _check("moe_bank_init", _lib.moe_bank_init(ctypes.byref(bank), _p(buffer), _nbytes(buffer),
                                               n_experts, d, f, layer))
    return bank


def moe_bank_write_expert(bank, expert, gate_codes, up_codes, down_codes, codebooks, stream=None):
    _check("moe_bank_write_expert",
           _lib.moe_bank_write_expert(ctypes.byref(bank), expert, _p(gate_codes), _p(up_codes),
                                      _p(down_codes), _p(codebooks), _stream(stream)))


def moe_bank_validate(bank, stream=None):
    _check("moe_bank_validate", _lib.moe_bank_validate(ctypes.byref(bank), _stream(stream)))


def moe_bank_seal(bank, stream=None):
    _check("moe_bank_seal", _lib.moe_bank_seal(ctypes.byref(bank), _stream(stream)))


def rvq_encode_workspace_bytes(rows, cols) -> int:
    return int(_lib.rvq_encode_workspace_bytes(rows, cols))


def rvq_encode(w, rows, cols, iters, codes, codebooks, ws, stream=None):
    _check("rvq_encode", _lib.rvq_encode(_p(w), rows, cols, iters, _p(codes), _p(codebooks),
                                         _p(ws), _nbytes(ws), _stream(stream)))


def moe_cache_create(host_bank, n_layers, n_experts, d, f, slots, slot_map) -> int:
    """host_bank: pinned uint8 tensor of n_layers x n_experts records; slots:
    device uint8 tensor; slot_map: device int32 [n_layers][n_experts].
    Returns the cache handle (an address)."""
    h = _vp()
    _check("moe_cache_create",
           _lib.moe_cache_create(ctypes.byref(h), _p(host_bank), n_layers, n_experts, d, f,
                                 _p(slots), _nbytes(slots), _p(slot_map)))
    return h.value


def moe_cache_destroy(cache):
    _check("moe_cache_destroy", _lib.moe_cache_destroy(cache))


def moe_cache_stats(cache) -> dict:
    st = RvqCacheStats()
    _check("moe_cache_stats", _lib.moe_cache_stats(cache, ctypes.byref(st)))
    return {k: int(getattr(st, k)) for k, _ in RvqCacheStats._fields_ if k != "pad"}


def moe_cache_bank(cache, layer) -> RvqMoeBank:
    bank = RvqMoeBank()
    _check("moe_cache_bank", _lib.moe_cache_bank(cache, layer, ctypes.byref(bank)))
    return bank


def moe_layer_forward_streamed(cache, layer, wr, bias, x, n, k, logits, topk_idx, topk_w,
                               offsets, pairs, out, ws, residual=None, tc_min_tokens=0,
                               next_wr=None, next_bias=None, lookahead=0, next_logits=None,
                               stream=None):
    rdt = _dt(residual) if residual is not None else _dt(x)
    _check("moe_layer_forward_streamed",
           _lib.moe_layer_forward_streamed(
               cache, layer, _p(wr), _p(bias), _p(x), _dt(x), n, k, _p(logits), _p(topk_idx),
               _p(topk_w), _p(offsets), _p(pairs), _p(out), _p(ws), _nbytes(ws), _p(residual),
               rdt, tc_min_tokens, _p(next_wr), _p(next_bias), lookahead, _p(next_logits),
               _stream(stream)))


def moe_bank_verify(bank, crc, ws, stream=None):
    _check("moe_bank_verify", _lib.moe_bank_verify(ctypes.byref(bank), _p(crc), _p(ws),
                                                   _nbytes(ws), _stream(stream)))


# ------------------------------------------------------------------ MoE calls

def moe_router_logits(wr, bias, x, n, E, d, logits, stream=None):
    _check("moe_router_logits",
           _lib.moe_router_logits(_p(wr), _p(bias), _p(x), _dt(x), n, E, d, _p(logits),
                                  _stream(stream)))


def moe_route_max_tokens(E: int) -> int:
    return int(_lib.moe_route_max_tokens(E))


def moe_route(logits, n, E, k, topk_idx, topk_w, offsets, pairs, ws, stream=None):
    _check("moe_route", _lib.moe_route(_p(logits), n, E, k, _p(topk_idx), _p(topk_w),
                                       _p(offsets), _p(pairs), _p(ws), _nbytes(ws),
                                       _stream(stream)))


def moe_workspace_bytes(bank, n, k) -> int:
    return int(_lib.moe_workspace_bytes(ctypes.byref(bank), n, k))


def moe_expert_ffn(bank, x, n, k, offsets, pairs, y_pair, ws, stream=None):
    _check("moe_expert_ffn",
           _lib.moe_expert_ffn(ctypes.byref(bank), _p(x), _dt(x), n, k, _p(offsets), _p(pairs),
                               _p(y_pair), _p(ws), _nbytes(ws), _stream(stream)))


def moe_expert_ffn_ex(bank, x, n, k, offsets, pairs, y_pair, ws, tc_min_tokens, stream=None):
    _check("moe_expert_ffn_ex",
           _lib.moe_expert_ffn_ex(ctypes.byref(bank), _p(x), _dt(x), n, k, _p(offsets), _p(pairs),
                                  _p(y_pair), _p(ws), _nbytes(ws), int(tc_min_tokens),
                                  _stream(stream)))


def moe_combine(y_pair, topk_w, n, k, d, residual, out, stream=None):
    _check("moe_combine", _lib.moe_combine(_p(y_pair), _p(topk_w), n, k, d, _p(residual),
                                           _dt(residual), _p(out), _stream(stream)))


def moe_route_rule(E, score=MOE_SCORE_SIGMOID, bias=None, groups=1, top_groups=1, renorm=True,
                   scale=1.0) -> MoeRouteRule:
    """How moe_route_scored chooses among E experts; keeps a reference to the bias
    (fp32 [E])."""
    rule = MoeRouteRule(score, _vec(bias, E, "bias", torch.float32), groups, top_groups,
                        int(renorm), scale)
    rule.keep = bias
    return rule


def moe_route_scored_workspace_bytes(n, E) -> int:
    return int(_lib.moe_route_scored_workspace_bytes(n, E))


def moe_route_scored(logits, n, E, k, topk_idx, topk_w, offsets, pairs, ws,
                     score=MOE_SCORE_SIGMOID, bias=None, groups=1, top_groups=1, renorm=True,
                     scale=1.0, stream=None):
    """The k of E experts with the largest score plus bias in the top_groups best groups
    (a group's value: its two largest), weights from the scores, and the grouping of
    moe_route.  logits fp32 [n][E]."""
    rule = MoeRouteRule(score, _vec(bias, E, "bias", torch.float32), groups, top_groups,
                        int(renorm), scale)
    f32, i32 = torch.float32, torch.int32
    rc = _lib.moe_route_scored(_vec(logits, n * E, "logits", f32), n, E, k, rule,
                               _vec(topk_idx, n * k, "topk_idx", i32),
                               _vec(topk_w, n * k, "topk_w", f32),
                               _vec(offsets, E + 1, "offsets", i32),
                               _vec(pairs, n * k, "pairs", i32), ws.data_ptr(), ws.nbytes,
                               _stream_of(stream, logits, bias, topk_idx, topk_w, offsets, pairs,
                                          ws))
    if rc:
        _check("moe_route_scored", rc)


def moe_route_scored_backward(dtopk_w, logits, topk_idx, n, E, k, dlogits,
                              score=MOE_SCORE_SIGMOID, renorm=True, scale=1.0, stream=None):
    """dlogits (fp32 [n][E], may be logits itself) from the gradient of topk_w."""
    rule = MoeRouteRule(score, None, 1, 1, int(renorm), scale)
    f32 = torch.float32
    rc = _lib.moe_route_scored_backward(_vec(dtopk_w, n * k, "dtopk_w", f32),
                                        _vec(logits, n * E, "logits", f32),
                                        _vec(topk_idx, n * k, "topk_idx", torch.int32), n, E, k,
                                        rule, _vec(dlogits, n * E, "dlogits", f32),
                                        _stream_of(stream, dtopk_w, logits, topk_idx, dlogits))
    if rc:
        _check("moe_route_scored_backward", rc)


def moe_layer_forward(bank, wr, bias, x, n, k, logits, topk_idx, topk_w, offsets, pairs, out,
                      ws, events=None, stream=None, tc_min_tokens=0, residual=None, rule=None):
    """rule (moe_route_rule, for as many experts as the bank has): experts chosen by
    moe_route_scored instead of moe_route."""
    ev = None
    if events is not None:
        assert len(events) == MOE_LAYER_EVENTS
        ev = (ctypes.c_void_p * MOE_LAYER_EVENTS)(*[e.cuda_event for e in events])
    rdt = _dt(residual) if residual is not None else _dt(x)
    if rule is not None:
        _vec(rule.keep, bank.n_experts, "bias")
        raw = _stream_of(stream, rule.keep)
        _check("moe_layer_forward_scored",
               _lib.moe_layer_forward_scored(ctypes.byref(bank), _p(wr), _p(bias), rule, _p(x),
                                             _dt(x), n, k, _p(logits), _p(topk_idx), _p(topk_w),
                                             _p(offsets), _p(pairs), _p(out), _p(ws), _nbytes(ws),
                                             _p(residual), rdt, int(tc_min_tokens), ev, raw))
        return
    _check("moe_layer_forward",
           _lib.moe_layer_forward_ex(ctypes.byref(bank), _p(wr), _p(bias), _p(x), _dt(x), n, k,
                                     _p(logits), _p(topk_idx), _p(topk_w), _p(offsets),
                                     _p(pairs), _p(out), _p(ws), _nbytes(ws), _p(residual), rdt,
                                     int(tc_min_tokens), ev, _stream(stream)))


def moe_layer_forward_host(bank, wr, bias, x_host, n, k, x_dev, logits, topk_idx, topk_w,
                           offsets, pairs, out, out_host, ws, tc_min_tokens=0, stream=None):
    """The layer with x read from and out written to host tensors (pinned for
    asynchronous copies); x_dev is the device copy of x.  Asynchronous."""
    assert not x_host.is_cuda and not out_host.is_cuda and x_host.dtype == x_dev.dtype
    assert x_host.is_contiguous() and out_host.is_contiguous()
    assert out_host.dtype == torch.float32 and out_host.numel() >= n * out.shape[-1]
    _check("moe_layer_forward_host",
           _lib.moe_layer_forward_host(ctypes.byref(bank), _p(wr), _p(bias),
                                       ctypes.c_void_p(x_host.data_ptr()), _dt(x_dev), n, k,
                                       _p(x_dev), _p(logits), _p(topk_idx), _p(topk_w),
                                       _p(offsets), _p(pairs), _p(out),
                                       ctypes.c_void_p(out_host.data_ptr()), _p(ws), _nbytes(ws),
                                       int(tc_min_tokens), _stream(stream)))


class LayerGraph:
    """A CUDA graph of one layer call (moe_layer_graph_create): launch() runs
    the whole layer as one graph launch; close() frees it.  Holds references
    to the buffers it records, so they outlive it."""

    def __init__(self, handle, keep):
        self._h = handle
        self._keep = keep

    def launch(self, stream=None):
        _check("moe_layer_graph_launch", _lib.moe_layer_graph_launch(self._h, _stream(stream)))

    def close(self):
        if self._h is not None:
            _check("moe_layer_graph_destroy", _lib.moe_layer_graph_destroy(self._h))
            self._h = None
            self._keep = None

    def __del__(self):
        if getattr(self, "_h", None) is not None and _lib is not None:
            _lib.moe_layer_graph_destroy(self._h)


def moe_layer_graph_create(bank, wr, bias, n, k, x_dev, logits, topk_idx, topk_w, offsets, pairs,
                           out, ws, tc_min_tokens=0, x_host=None, out_host=None, stream=None):
    """Records one layer call (optionally with the copies of x_host in and of
    out back to out_host) as a CUDA graph; stream must be capturable (not the
    legacy default stream).  Returns a LayerGraph."""
    if (x_host is None) != (out_host is None):
        raise ValueError("x_host and out_host go together")
    if x_host is not None:
        assert not x_host.is_cuda and not out_host.is_cuda and x_host.dtype == x_dev.dtype
        assert x_host.is_contiguous() and out_host.is_contiguous()
        assert out_host.dtype == torch.float32 and out_host.numel() >= n * out.shape[-1]
    h = ctypes.c_void_p()
    _check("moe_layer_graph_create",
           _lib.moe_layer_graph_create(
               ctypes.byref(bank), _p(wr), _p(bias),
               None if x_host is None else ctypes.c_void_p(x_host.data_ptr()), _dt(x_dev), n, k,
               _p(x_dev), _p(logits), _p(topk_idx), _p(topk_w), _p(offsets), _p(pairs), _p(out),
               None if out_host is None else ctypes.c_void_p(out_host.data_ptr()), _p(ws),
               _nbytes(ws), int(tc_min_tokens), _stream(stream), ctypes.byref(h)))
    return LayerGraph(h, (bank, wr, bias, x_dev, logits, topk_idx, topk_w, offsets, pairs, out,
                          ws, x_host, out_host))


def moe_layer_forward_prenorm(bank, wr, bias, h, n, k, eps, xn, logits, topk_idx, topk_w, offsets,
                              pairs, out, ws, tc_min_tokens=0, stream=None):
    """out = h + MoE(bf16 rms_norm(h)); xn (bf16 [n][d]) receives the normalised rows."""
    _check("moe_layer_forward_prenorm",
           _lib.moe_layer_forward_prenorm(ctypes.byref(bank), _p(wr), _p(bias), _p(h), _dt(h), n, k,
                                          float(eps), _p(xn), _p(logits), _p(topk_idx),
                                          _p(topk_w), _p(offsets), _p(pairs), _p(out), _p(ws),
                                          _nbytes(ws), int(tc_min_tokens), _stream(stream)))


def rvq_selftest_prefill_timeout(bank, ws, stream=None):
    _check("rvq_selftest_prefill_timeout",
           _lib.rvq_selftest_prefill_timeout(ctypes.byref(bank), _p(ws), _nbytes(ws),
                                             _stream(stream)))


def moe_rms_norm(x, n, d, out, eps=1e-6, stream=None):
    _check("moe_rms_norm", _lib.moe_rms_norm(_p(x), _dt(x), n, d, float(eps), _p(out), _dt(out),
                                             _stream(stream)))


# ------------------------------------------------------------------ dense operators

_DTYPES = {torch.float32: RVQ_F32, torch.bfloat16: RVQ_BF16, torch.float16: RVQ_F16}


def _code(dtype) -> int:
    """dtype code of a dense operator's tensors."""
    try:
        return _DTYPES[dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {dtype} (bf16, fp16 or fp32)") from None


def _dt_any(t) -> int:
    """dtype code of a tensor (None: fp32, unused)."""
    return RVQ_F32 if t is None else _code(t.dtype)


# The dense calls take a few microseconds on the GPU at decode sizes, so their
# host side asks torch for as little as it can: raw stream handles, one look at
# each tensor's shape, strides and type, addresses taken along with the checks.
def _raw_stream(stream) -> int:
    """cudaStream_t of `stream`, or of the current device's current stream
    (the caller's CUDA tensors have initialised torch's CUDA state)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream


def _stream_of(stream, *tensors) -> int:
    """_raw_stream, once every tensor (or None) is on the stream's device."""
    device = torch._C._cuda_getDevice() if stream is None else stream.device_index
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError(f"a tensor is on {t.device}, the call on cuda:{device}")
    return torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream


def _mat(t, rows, cols, what, dtype=None):
    """(address, row pitch) of a [rows][cols] matrix with contiguous columns, or
    (None, 0)."""
    if t is None:
        return None, 0
    if t.shape != (rows, cols):
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected ({rows}, {cols})")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{what}: dtype {t.dtype}, expected {dtype}")
    pitch, step = t.stride()
    if step != 1:
        raise ValueError(f"{what}: columns are not contiguous (strides {t.stride()})")
    return t.data_ptr(), pitch if rows > 1 else max(cols, pitch // 8 * 8)


def _vec(t, numel, what, dtype=None):
    """Address of a contiguous tensor of numel elements, or None."""
    if t is None:
        return None
    if t.numel() != numel or not t.is_contiguous():
        raise ValueError(f"{what}: {tuple(t.shape)} with strides {t.stride()}, expected {numel} "
                         "contiguous elements")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{what}: dtype {t.dtype}, expected {dtype}")
    return t.data_ptr()


def _same_pitch(a, b, what):
    if a != b:
        raise ValueError(f"{what} have different row pitches")


def moe_linear_workspace_bytes(n, rows, cols, backward=False) -> int:
    return int(_lib.moe_linear_workspace_bytes(n, rows, cols, int(backward)))


def moe_linear(x, w, n, rows, cols, out, ws, bias=None, act=MOE_ACT_NONE, alpha=1.0, residual=None,
               pre=None, stream=None):
    """out = residual + alpha * act(x w^T + bias); x [n][cols], w [rows][cols]
    (bf16 or fp16, any row pitch), out and residual [n][rows].  pre (fp32
    [n][rows]) keeps x w^T + bias for moe_linear_backward."""
    dt = x.dtype
    px, ldx = _mat(x, n, cols, "x")
    pw, ldw = _mat(w, rows, cols, "w", dt)
    po, ldo = _mat(out, n, rows, "out")
    pr, ldr = _mat(residual, n, rows, "residual")
    rc = _lib.moe_linear(px, ldx, pw, ldw, _vec(bias, rows, "bias", dt), _dt_any(x), n, rows, cols,
                         act, alpha, pr, _dt_any(residual), ldr, po, _dt_any(out), ldo,
                         _vec(pre, n * rows, "pre", torch.float32), ws.data_ptr(), ws.nbytes,
                         _raw_stream(stream))
    if rc:
        _check("moe_linear", rc)


def moe_linear_backward(dout, x, w, n, rows, cols, ws, dx=None, dw=None, dbias=None, pre=None,
                        act=MOE_ACT_NONE, alpha=1.0, stream=None):
    """Gradients of moe_linear (those given a tensor): dx [n][cols], dw
    [rows][cols], dbias [rows]; the residual's gradient is dout itself."""
    dt = dout.dtype
    pd, ldd = _mat(dout, n, rows, "dout")
    px, ldx = _mat(x, n, cols, "x", dt)
    pw, ldw = _mat(w, rows, cols, "w", dt)
    pdx, lddx = _mat(dx, n, cols, "dx", dt)
    pdw, lddw = _mat(dw, rows, cols, "dw", dt)
    rc = _lib.moe_linear_backward(pd, ldd, px, ldx, pw, ldw,
                                  _vec(pre, n * rows, "pre", torch.float32), _dt_any(dout), n,
                                  rows, cols, act, alpha, pdx, lddx, pdw, lddw,
                                  _vec(dbias, rows, "dbias", dt), ws.data_ptr(), ws.nbytes,
                                  _raw_stream(stream))
    if rc:
        _check("moe_linear_backward", rc)


def moe_gated_linear_workspace_bytes(n, rows, cols, backward=False) -> int:
    return int(_lib.moe_gated_linear_workspace_bytes(n, rows, cols, int(backward)))


def moe_gated_linear(x, wg, wu, n, rows, cols, out, ws, bg=None, bu=None, act=MOE_ACT_SILU,
                     pre=None, stream=None):
    """out = act(x wg^T + bg) * (x wu^T + bu).  wg and wu share their row pitch
    (two halves of one tensor do).  pre (fp32 [2][n][rows]) keeps both projections
    for moe_gated_linear_backward."""
    dt = x.dtype
    px, ldx = _mat(x, n, cols, "x")
    pg, ldw = _mat(wg, rows, cols, "wg", dt)
    pu, ldu = _mat(wu, rows, cols, "wu", dt)
    _same_pitch(ldw, ldu, "wg and wu")
    po, ldo = _mat(out, n, rows, "out", dt)
    rc = _lib.moe_gated_linear(px, ldx, pg, pu, ldw, _vec(bg, rows, "bg", dt),
                               _vec(bu, rows, "bu", dt), _dt_any(x), n, rows, cols, act, po, ldo,
                               _vec(pre, 2 * n * rows, "pre", torch.float32), ws.data_ptr(),
                               ws.nbytes, _raw_stream(stream))
    if rc:
        _check("moe_gated_linear", rc)


def moe_gated_linear_backward(dout, x, wg, wu, pre, n, rows, cols, ws, dx=None, dwg=None, dwu=None,
                              dbg=None, dbu=None, act=MOE_ACT_SILU, stream=None):
    """Gradients of moe_gated_linear (those given a tensor) from the forward
    call's inputs and `pre`."""
    dt = dout.dtype
    pd, ldd = _mat(dout, n, rows, "dout")
    px, ldx = _mat(x, n, cols, "x", dt)
    pg, ldw = _mat(wg, rows, cols, "wg", dt)
    pu, ldu = _mat(wu, rows, cols, "wu", dt)
    _same_pitch(ldw, ldu, "wg and wu")
    pdx, lddx = _mat(dx, n, cols, "dx", dt)
    pdg, lddw = _mat(dwg, rows, cols, "dwg", dt)
    pdu, lddu = _mat(dwu, rows, cols, "dwu", dt)
    _same_pitch(lddw, lddu, "dwg and dwu")
    rc = _lib.moe_gated_linear_backward(pd, ldd, px, ldx, pg, pu, ldw,
                                        _vec(pre, 2 * n * rows, "pre", torch.float32),
                                        _dt_any(dout), n, rows, cols, act, pdx, lddx, pdg, pdu,
                                        lddw, _vec(dbg, rows, "dbg", dt),
                                        _vec(dbu, rows, "dbu", dt), ws.data_ptr(), ws.nbytes,
                                        _raw_stream(stream))
    if rc:
        _check("moe_gated_linear_backward", rc)


def rvq_selftest_dense_plan(gated, backward, n, rows, cols) -> tuple[bool, list[tuple[str, int, int]]]:
    """How the products of moe_linear or (gated) moe_gated_linear, or of their
    gradients, are computed: whether dx and dw share a launch, and for each product
    (the forward's; dx, dw) its way ("stream", "tiles", "parts" or "split"), the parts
    or CTA pairs a tile is cut into, and the tile's columns."""
    out = (_i32 * 7)()
    _check("rvq_selftest_dense_plan",
           _lib.rvq_selftest_dense_plan(int(gated), int(backward), n, rows, cols, out))
    ways = [(MOE_WAYS[out[i]], out[i + 1], out[i + 2]) for i in (1, 4)]
    return bool(out[0]), ways if backward else ways[:1]


def _gate_kind(gate, n, d) -> int:
    """MOE_GATE_* of a contiguous gate tensor: one element, [n][1], [1][d] or
    [d], or [n][d]."""
    if gate is None:
        return MOE_GATE_NONE
    if not gate.is_contiguous():
        raise ValueError(f"gate: not contiguous (strides {gate.stride()})")
    shape = gate.shape
    if shape == (n, 1):
        return MOE_GATE_TOKEN
    if shape == (n, d):
        return MOE_GATE_FULL
    if shape == (d,) or shape == (1, d):
        return MOE_GATE_CHANNEL
    if gate.numel() == 1:
        return MOE_GATE_SCALAR
    raise ValueError(f"gate: shape {tuple(shape)} does not broadcast over ({n}, {d})")


def moe_norm_join(y, n, d, h_out, xn, h=None, alpha=1.0, gate=None, post_norm=True, w_post=None,
                  w_pre=None, eps=1e-6, rstd=None, stream=None):
    """h_out = alpha * h + gate * norm(y) * w_post (post_norm; else y itself),
    xn = norm(h_out) * w_pre.  gate broadcasts over [n][d]; gains None are 1.
    h_out or xn may be None.  rstd (fp32 [2][n]) is kept for the gradients."""
    nd = n * d
    ho = h if h is not None else h_out
    wdt = w_post if w_post is not None else w_pre
    rc = _lib.moe_norm_join(
        _vec(h, nd, "h"), _dt_any(ho), _vec(y, nd, "y"), _dt_any(y), n, d, alpha,
        None if gate is None else gate.data_ptr(), _gate_kind(gate, n, d), _dt_any(gate),
        int(post_norm), _vec(w_post, d, "w_post"),
        _vec(w_pre, d, "w_pre", None if wdt is w_pre else wdt.dtype), _dt_any(wdt), eps,
        _vec(h_out, nd, "h_out", None if ho is h_out else ho.dtype), _vec(xn, nd, "xn"),
        _dt_any(xn), _vec(rstd, 2 * n, "rstd", torch.float32), _raw_stream(stream))
    if rc:
        _check("moe_norm_join", rc)


def moe_norm_join_workspace_bytes(n, d) -> int:
    return int(_lib.moe_norm_join_workspace_bytes(n, d))


def _first_dtype(*tensors):
    for t in tensors:
        if t is not None:
            return t.dtype
    return torch.float32


def moe_norm_join_backward(dh_out, dxn, y, n, d, rstd, ws, h=None, alpha=1.0, gate=None,
                           post_norm=True, w_post=None, w_pre=None, dh=None, dy=None, dgate=None,
                           dw_post=None, dw_pre=None, stream=None):
    """Gradients of moe_norm_join (those given a tensor) from its inputs and
    rstd.  dh_out or dxn may be None."""
    nd = n * d
    hdt = _first_dtype(h, dh_out, dh)
    wdt = _first_dtype(w_post, w_pre, dw_post, dw_pre)
    if gate is None:
        pg, pdg = None, None if dgate is None else dgate.data_ptr()
    else:
        pg, pdg = gate.data_ptr(), _vec(dgate, gate.numel(), "dgate", gate.dtype)
    rc = _lib.moe_norm_join_backward(
        _vec(dh_out, nd, "dh_out", hdt), _vec(dxn, nd, "dxn"), _dt_any(dxn), _vec(h, nd, "h", hdt),
        _code(hdt), _vec(y, nd, "y"), _dt_any(y), n, d, alpha, pg, _gate_kind(gate, n, d),
        _dt_any(gate), int(post_norm), _vec(w_post, d, "w_post", wdt),
        _vec(w_pre, d, "w_pre", wdt), _code(wdt), _vec(rstd, 2 * n, "rstd", torch.float32),
        _vec(dh, nd, "dh", hdt), _vec(dy, nd, "dy", y.dtype), pdg,
        _vec(dw_post, d, "dw_post", wdt), _vec(dw_pre, d, "dw_pre", wdt), ws.data_ptr(), ws.nbytes,
        _raw_stream(stream))
    if rc:
        _check("moe_norm_join_backward", rc)


# ------------------------------------------------------------------ microscaled operators

def moe_mx_code_bytes(fmt, rows, cols) -> int:
    return int(_lib.moe_mx_code_bytes(fmt, rows, cols))


def moe_mx_scale_bytes(rows, cols) -> int:
    return int(_lib.moe_mx_scale_bytes(rows, cols))


def _mx(codes, scales, rows, cols, fmt, what):
    """Addresses of a microscaled matrix's codes and scales (contiguous uint8 tensors
    of their sizes, any shape), or (None, None)."""
    if codes is None and scales is None:
        return None, None
    tiles = -(-cols // 128)
    n, m = rows * tiles * (64 if fmt == MOE_MX_F4 else 128), -(-rows // 128) * tiles * 512
    if codes is not None and scales is not None and codes.dtype is scales.dtype is torch.uint8 and \
            codes.numel() == n and scales.numel() == m and codes.is_contiguous() and \
            scales.is_contiguous():
        return codes.data_ptr(), scales.data_ptr()
    # one of them is refused, or left to the library (None)
    return _vec(codes, n, what, torch.uint8), _vec(scales, m, what + " scales", torch.uint8)


def moe_mx_quantize(x, rows, cols, codes, scales, fmt=MOE_MX_F8, stream=None):
    """codes, scales (uint8, moe_mx_code_bytes and moe_mx_scale_bytes long) = x [rows][cols]
    in a microscaled format."""
    px, ldx = _mat(x, rows, cols, "x")
    pc, ps = _mx(codes, scales, rows, cols, fmt, "codes")
    rc = _lib.moe_mx_quantize(px, ldx, _dt_any(x), rows, cols, fmt, pc, ps,
                              _stream_of(stream, x, codes, scales))
    if rc:
        _check("moe_mx_quantize", rc)


def moe_mx_dequantize(codes, scales, rows, cols, out, fmt=MOE_MX_F8, stream=None):
    """out [rows][cols] (bf16, fp16 or fp32) = the values of a microscaled matrix."""
    pc, ps = _mx(codes, scales, rows, cols, fmt, "codes")
    po, ldo = _mat(out, rows, cols, "out")
    rc = _lib.moe_mx_dequantize(pc, ps, fmt, rows, cols, po, _dt_any(out), ldo,
                                _stream_of(stream, codes, scales, out))
    if rc:
        _check("moe_mx_dequantize", rc)


def moe_mx_linear_workspace_bytes(n, rows, cols) -> int:
    return int(_lib.moe_mx_linear_workspace_bytes(n, rows, cols))


def moe_mx_gated_linear_workspace_bytes(n, rows, cols) -> int:
    return int(_lib.moe_mx_gated_linear_workspace_bytes(n, rows, cols))


def moe_mx_linear(x, x_scales, w, w_scales, n, rows, cols, out, ws, xfmt=MOE_MX_F8,
                  wfmt=MOE_MX_F4, bias=None, act=MOE_ACT_NONE, alpha=1.0, residual=None,
                  stream=None):
    """out = residual + alpha * act(x w^T + bias) of microscaled x [n][cols] and w
    [rows][cols] (codes and scales); bias fp32, out and residual [n][rows] in bf16, fp16
    or fp32."""
    px, pxs = _mx(x, x_scales, n, cols, xfmt, "x")
    pw, pws = _mx(w, w_scales, rows, cols, wfmt, "w")
    po, ldo = _mat(out, n, rows, "out")
    pr, ldr = _mat(residual, n, rows, "residual")
    rc = _lib.moe_mx_linear(px, pxs, xfmt, pw, pws, wfmt, _vec(bias, rows, "bias", torch.float32),
                            n, rows, cols, act, alpha, pr, _dt_any(residual), ldr, po,
                            _dt_any(out), ldo, ws.data_ptr(), ws.nbytes,
                            _stream_of(stream, x, x_scales, w, w_scales, bias, residual, out, ws))
    if rc:
        _check("moe_mx_linear", rc)


def moe_mx_gated_linear(x, x_scales, wg, wg_scales, wu, wu_scales, n, rows, cols, out, ws,
                        xfmt=MOE_MX_F8, wfmt=MOE_MX_F4, bg=None, bu=None, act=MOE_ACT_SILU,
                        out_scales=None, ofmt=MOE_MX_F8, stream=None):
    """act(x wg^T + bg) * (x wu^T + bu) of microscaled matrices: into out [n][rows] (bf16,
    fp16 or fp32), or, with out_scales, into out and out_scales as codes and scales."""
    px, pxs = _mx(x, x_scales, n, cols, xfmt, "x")
    pg, pgs = _mx(wg, wg_scales, rows, cols, wfmt, "wg")
    pu, pus = _mx(wu, wu_scales, rows, cols, wfmt, "wu")
    if out_scales is None:
        po, ldo = _mat(out, n, rows, "out")
        odt, pc, ps = _dt_any(out), None, None
    else:
        po, ldo, odt = None, 0, RVQ_F32
        pc, ps = _mx(out, out_scales, n, rows, ofmt, "out")
    rc = _lib.moe_mx_gated_linear(px, pxs, xfmt, pg, pgs, pu, pus, wfmt,
                                  _vec(bg, rows, "bg", torch.float32),
                                  _vec(bu, rows, "bu", torch.float32), n, rows, cols, act, po, odt,
                                  ldo, pc, ps, ofmt, ws.data_ptr(), ws.nbytes,
                                  _stream_of(stream, x, x_scales, wg, wg_scales, wu, wu_scales, bg,
                                             bu, out, out_scales, ws))
    if rc:
        _check("moe_mx_gated_linear", rc)


def rvq_selftest_mx_plan(gated, xfmt, wfmt, n, rows, cols) -> tuple[str, int]:
    """How moe_mx_linear or (gated) moe_mx_gated_linear computes its product: "stream" or
    "tiles", and the CTAs that the depth of a streamed one is split among."""
    out = (_i32 * 2)()
    _check("rvq_selftest_mx_plan",
           _lib.rvq_selftest_mx_plan(int(gated), xfmt, wfmt, n, rows, cols, out))
    return MOE_WAYS[out[0]], out[1]


def moe_norm_join_mx(y, n, d, h_out, codes, scales, fmt=MOE_MX_F8, xn=None, h=None, alpha=1.0,
                     gate=None, post_norm=True, w_post=None, w_pre=None, eps=1e-6, rstd=None,
                     stream=None):
    """moe_norm_join whose normed rows go into a microscaled matrix (codes, scales), and
    into xn too if it is given.  h_out may be None."""
    nd = n * d
    ho = h if h is not None else h_out
    wdt = w_post if w_post is not None else w_pre
    pc, ps = _mx(codes, scales, n, d, fmt, "codes")
    rc = _lib.moe_norm_join_mx(
        _vec(h, nd, "h"), _dt_any(ho), _vec(y, nd, "y"), _dt_any(y), n, d, alpha,
        None if gate is None else gate.data_ptr(), _gate_kind(gate, n, d), _dt_any(gate),
        int(post_norm), _vec(w_post, d, "w_post"),
        _vec(w_pre, d, "w_pre", None if wdt is w_pre else wdt.dtype), _dt_any(wdt), eps,
        _vec(h_out, nd, "h_out", None if ho is h_out else ho.dtype), _vec(xn, nd, "xn"),
        _dt_any(xn), fmt, pc, ps, _vec(rstd, 2 * n, "rstd", torch.float32),
        _stream_of(stream, y, h, gate, w_post, w_pre, h_out, codes, scales, xn, rstd))
    if rc:
        _check("moe_norm_join_mx", rc)


def rvq_ws_clear(ws, stream=None):
    _check("rvq_ws_clear", _lib.rvq_ws_clear(_p(ws), _stream(stream)))


def rvq_ws_status(ws, stream=None) -> tuple[int, int]:
    """Returns (status code, raw device bits); clears the bits."""
    bits = _u32(0)
    rc = _lib.rvq_ws_status(_p(ws), ctypes.byref(bits), _stream(stream))
    return int(rc), int(bits.value)

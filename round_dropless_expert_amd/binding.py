"""ctypes binding of libmoe_rounds.so (the C ABI in include/moe_rounds.h).

Argument marshalling only: every step of the layer runs in the library's HIP
kernels. Device buffers are torch tensors (or raw device addresses); torch
provides device memory and the current stream, nothing else. If the library
has not been built this module raises at load time: there is no fallback.
"""
from __future__ import annotations

import ctypes
import itertools
import math
import operator
import os

import numpy as np

import torch  # loads the HIP runtime the library must share

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "lib", "libmoe_rounds.so")

MOE_OK = 0
MOE_ERR_INVALID_ARGUMENT = 1
MOE_ERR_UNSUPPORTED = 2
MOE_ERR_WORKSPACE_TOO_SMALL = 3
MOE_ERR_HIP = 4

MOE_F32 = 0
MOE_BF16 = 1
MOE_F16 = 2  # ragged expert operators only

MOE_SCORE_SOFTMAX = 0
MOE_SCORE_SIGMOID = 1

MOE_WEIGHTS_ROW_MAJOR = 0
MOE_WEIGHTS_TILED = 1

EXPORTS = ("moe_status_string", "moe_last_error", "moe_hip_runtime_version",
           "moe_check_config", "moe_workspace_size", "moe_forward_workspace_size",
           "moe_workspace_layout",
           "moe_plan", "moe_launch_batches", "moe_dispatch", "moe_expert_ffn",
           "moe_expert_gate_up",
           "moe_expert_down", "moe_dispatch_gate_up", "moe_pack_weights", "moe_combine", "moe_forward",
           "moe_capacity_curve", "moe_capacity_for_rounds",
           "moe_backward_workspace_size", "moe_backward_layout",
           "moe_backward", "moe_forward_static",
           "moe_grouped_gemm", "moe_grouped_gemm_dx", "moe_grouped_gemm_dw",
           "moe_grouped_dw_workspace_size", "moe_swiglu", "moe_swiglu_backward",
           "moe_mxfp4_scale_stride", "moe_mxfp4_quantize", "moe_mxfp4_dequantize",
           "moe_mxfp4_grouped_gemm",
           "moe_route", "moe_route_backward", "moe_sort_workspace_size", "moe_sort",
           "moe_collect", "moe_collect_backward", "moe_int8_stride", "moe_int8_quantize",
           "moe_int8_dequantize", "moe_int8_grouped_gemm",
           "moe_orthogonalize_workspace_size", "moe_orthogonalize")


class MoeConfig(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("E", ctypes.c_int32),
                ("k", ctypes.c_int32), ("d_model", ctypes.c_int32),
                ("d_ff", ctypes.c_int32), ("C", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("weight_layout", ctypes.c_int32),
                ("group", ctypes.c_int32), ("round_buffers", ctypes.c_int32)]


LAYOUT_FIELDS = ("idx", "weight", "counts", "offsets", "n_rounds", "perm",
                 "pos", "round_of", "row_of", "rounds", "scratch", "xr", "h",
                 "z")


class MoeLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in LAYOUT_FIELDS] + \
        [("total", ctypes.c_size_t)]


BWD_LAYOUT_FIELDS = ("xr", "dyr", "gu", "hw", "dgu", "dz", "ones")


class MoeBackwardLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in BWD_LAYOUT_FIELDS] + \
        [("total", ctypes.c_size_t)]


class MoeGrouped(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("E", ctypes.c_int32),
                ("N", ctypes.c_int32), ("K", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("ld_x", ctypes.c_int64),
                ("ld_y", ctypes.c_int64)]


class MoeRouter(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("E", ctypes.c_int32), ("k", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("score", ctypes.c_int32),
                ("groups", ctypes.c_int32), ("top_groups", ctypes.c_int32),
                ("group_top", ctypes.c_int32), ("renormalize", ctypes.c_int32),
                ("scale", ctypes.c_float), ("ld", ctypes.c_int64)]


class MoeError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(msg)
        self.status = status


_lib = None


def load() -> ctypes.CDLL:
    """Load the HIP library (raises if it is missing: no fallback path)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with "
            "`python -c 'import __graft_entry__ as g; g.build()'` "
            "or `python round_dropless_expert_amd/csrc/build.py`")
    L = ctypes.CDLL(LIB_PATH)
    vp, sz, i32, i32p = (ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32,
                         ctypes.POINTER(ctypes.c_int32))
    cfgp = ctypes.POINTER(MoeConfig)
    L.moe_status_string.argtypes = [ctypes.c_int]
    L.moe_status_string.restype = ctypes.c_char_p
    L.moe_last_error.argtypes = []
    L.moe_last_error.restype = ctypes.c_char_p
    L.moe_hip_runtime_version.argtypes = []
    L.moe_hip_runtime_version.restype = ctypes.c_int32
    L.moe_check_config.argtypes = [cfgp]
    L.moe_workspace_size.argtypes = [cfgp, ctypes.POINTER(ctypes.c_size_t)]
    L.moe_forward_workspace_size.argtypes = [cfgp, ctypes.POINTER(ctypes.c_size_t)]
    L.moe_workspace_layout.argtypes = [cfgp, ctypes.POINTER(MoeLayout)]
    L.moe_plan.argtypes = [cfgp, vp, vp, sz, i32p, vp]
    L.moe_launch_batches.argtypes = [cfgp, i32p, i32, i32p, i32p, i32p]
    L.moe_dispatch.argtypes = [cfgp, i32, i32, vp, vp, sz, vp]
    L.moe_expert_ffn.argtypes = [cfgp, i32, i32, vp, vp, vp, i32p, vp, sz, vp]
    L.moe_expert_gate_up.argtypes = [cfgp, i32, i32, vp, vp, i32p, vp, sz, vp]
    L.moe_expert_down.argtypes = [cfgp, i32, i32, vp, i32p, vp, sz, vp]
    L.moe_dispatch_gate_up.argtypes = [cfgp, i32, i32, vp, vp, vp, i32p, vp, sz, vp]
    L.moe_pack_weights.argtypes = [cfgp, vp, vp, vp, vp, vp, vp, vp]
    L.moe_combine.argtypes = [cfgp, vp, sz, vp, vp]
    L.moe_forward.argtypes = [cfgp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.moe_forward_static.argtypes = [cfgp, vp, vp, vp, vp, vp, vp, vp]
    i64, i64p = ctypes.c_int64, ctypes.POINTER(ctypes.c_int64)
    L.moe_capacity_curve.argtypes = [cfgp, i32p, i64, i64p, i32, i32p,
                                     ctypes.POINTER(ctypes.c_size_t)]
    L.moe_capacity_for_rounds.argtypes = [cfgp, i32p, i64, i32, ctypes.c_double,
                                          i64p]
    L.moe_backward_workspace_size.argtypes = [cfgp, ctypes.POINTER(ctypes.c_size_t)]
    L.moe_backward_layout.argtypes = [cfgp, ctypes.POINTER(MoeBackwardLayout)]
    L.moe_backward.argtypes = [cfgp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                               vp, sz, vp, sz, vp]
    gp = ctypes.POINTER(MoeGrouped)
    L.moe_grouped_gemm.argtypes = [gp, vp, vp, vp, vp, vp]
    L.moe_grouped_gemm_dx.argtypes = [gp, vp, vp, vp, vp, vp]
    L.moe_grouped_dw_workspace_size.argtypes = [gp, ctypes.POINTER(ctypes.c_size_t)]
    L.moe_grouped_gemm_dw.argtypes = [gp, vp, vp, vp, vp, i32, vp, sz, vp]
    L.moe_swiglu.argtypes = [i32, i64, i64, vp, i64, vp, i64, vp, vp]
    L.moe_swiglu_backward.argtypes = [i32, i64, i64, vp, i64, vp, i64, vp, i64, vp, vp]
    L.moe_mxfp4_scale_stride.argtypes = [i64]
    L.moe_mxfp4_scale_stride.restype = i64
    L.moe_mxfp4_quantize.argtypes = [i32, i64, i64, vp, i64, i64, vp, i32, vp, vp, vp, vp]
    L.moe_mxfp4_dequantize.argtypes = [i32, i64, i64, vp, vp, vp, i64, vp, vp]
    L.moe_mxfp4_grouped_gemm.argtypes = [gp, vp, vp, vp, vp, vp, vp, vp]
    rp = ctypes.POINTER(MoeRouter)
    szp = ctypes.POINTER(ctypes.c_size_t)
    L.moe_route.argtypes = [rp, vp, vp, vp, vp, vp]
    L.moe_route_backward.argtypes = [rp, vp, vp, vp, vp, vp]
    L.moe_sort_workspace_size.argtypes = [i64, i32, szp]
    L.moe_sort.argtypes = [i64, i32, vp, vp, vp, vp, vp, sz, vp]
    L.moe_collect.argtypes = [i32, i64, i32, i64, i64, vp, i64, vp, vp, vp, i64, vp]
    L.moe_collect_backward.argtypes = [i32, i64, i32, i64, i64, vp, i64, vp, i64, vp, vp, vp,
                                       i64, vp, vp]
    L.moe_int8_stride.argtypes = [i64]
    L.moe_int8_stride.restype = i64
    L.moe_int8_quantize.argtypes = [i32, i64, i64, vp, i64, i64, vp, i32, vp, vp, vp, vp]
    L.moe_int8_dequantize.argtypes = [i32, i64, i64, vp, vp, vp, i64, vp, vp]
    L.moe_int8_grouped_gemm.argtypes = [gp, vp, vp, vp, vp, vp, vp, vp]
    L.moe_orthogonalize_workspace_size.argtypes = [i32, i32, i32, szp]
    L.moe_orthogonalize.argtypes = [i32, i32, i32, i32, vp, vp, i32, vp, ctypes.c_float, vp, sz,
                                    vp]
    for n in ("moe_route", "moe_route_backward", "moe_sort_workspace_size", "moe_sort",
              "moe_collect", "moe_collect_backward", "moe_int8_quantize",
              "moe_int8_dequantize", "moe_int8_grouped_gemm",
              "moe_orthogonalize_workspace_size", "moe_orthogonalize"):
        getattr(L, n).restype = ctypes.c_int
    for n in ("moe_grouped_gemm", "moe_grouped_gemm_dx", "moe_grouped_gemm_dw",
              "moe_grouped_dw_workspace_size", "moe_swiglu", "moe_swiglu_backward",
              "moe_mxfp4_quantize", "moe_mxfp4_dequantize", "moe_mxfp4_grouped_gemm",
              "moe_check_config", "moe_workspace_size", "moe_forward_workspace_size",
              "moe_workspace_layout",
              "moe_plan", "moe_launch_batches", "moe_dispatch", "moe_expert_ffn",
              "moe_expert_gate_up", "moe_expert_down", "moe_dispatch_gate_up",
              "moe_pack_weights",
              "moe_combine", "moe_forward", "moe_capacity_curve",
              "moe_capacity_for_rounds", "moe_backward_workspace_size",
              "moe_backward_layout", "moe_backward",
              "moe_forward_static"):
        getattr(L, n).restype = ctypes.c_int
    _lib = L
    return L


def check_runtime() -> None:
    """The library must run on the same HIP runtime instance as torch."""
    v = load().moe_hip_runtime_version()
    want = torch.version.hip
    if want is None:
        raise RuntimeError("torch was built without HIP")
    major, minor = (int(x) for x in want.split(".")[:2])
    if v < 0 or v // 10_000_000 != major or (v // 100_000) % 100 != minor:
        raise RuntimeError(f"libmoe_rounds sees HIP runtime {v}, torch uses {want}")


def _check(status: int) -> None:
    if status != MOE_OK:
        L = load()
        raise MoeError(status, f"{L.moe_status_string(status).decode()}: "
                               f"{L.moe_last_error().decode()}")


def config(T, E, k, d_model, d_ff, C, dtype,
           weight_layout=MOE_WEIGHTS_ROW_MAJOR, group=1,
           round_buffers=1) -> MoeConfig:
    """group: experts per capacity group (1 = strict per-expert capacity);
    round_buffers: 1, or 2 to overlap consecutive rounds in moe_forward."""
    if isinstance(dtype, str):
        dtype = {"f32": MOE_F32, "bf16": MOE_BF16}[dtype]
    elif isinstance(dtype, torch.dtype):
        dtype = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16}[dtype]
    if isinstance(weight_layout, str):
        weight_layout = {"row_major": MOE_WEIGHTS_ROW_MAJOR,
                         "tiled": MOE_WEIGHTS_TILED}[weight_layout]
    return MoeConfig(int(T), int(E), int(k), int(d_model), int(d_ff), int(C),
                     int(dtype), int(weight_layout), int(group),
                     int(round_buffers))


def buffer_geometry(cfg: MoeConfig) -> dict:
    """Round-buffer geometry: C' = min(C, T), P = C' rounded up to 64, the
    group size G, rows per group Q (P for G = 1, else G*(P+64)), the rows of
    one set of round buffers, the number of sets S (round r uses set r % S)
    and the rows M of each round table."""
    ce = min(cfg.C, cfg.T)
    pad = (ce + 63) // 64 * 64
    G = cfg.group if cfg.group > 0 else 1
    Q = pad if G == 1 else G * (pad + 64)
    S = cfg.round_buffers if cfg.round_buffers > 0 else 1
    return {"ce": ce, "pad": pad, "G": G, "Q": Q, "rows": (cfg.E // G) * Q,
            "S": S, "M": -(-cfg.T // ce)}


def check_config(cfg: MoeConfig) -> int:
    return load().moe_check_config(ctypes.byref(cfg))


def workspace_size(cfg: MoeConfig) -> int:
    n = ctypes.c_size_t(0)
    _check(load().moe_workspace_size(ctypes.byref(cfg), ctypes.byref(n)))
    return n.value


def forward_workspace_size(cfg: MoeConfig) -> int:
    """Bytes moe_forward and moe_backward need (the workspace up to xr when
    the forward gathers its rows from x)."""
    n = ctypes.c_size_t(0)
    _check(load().moe_forward_workspace_size(ctypes.byref(cfg), ctypes.byref(n)))
    return n.value


def workspace_layout(cfg: MoeConfig) -> dict:
    L = MoeLayout()
    _check(load().moe_workspace_layout(ctypes.byref(cfg), ctypes.byref(L)))
    return {n: getattr(L, n) for n in LAYOUT_FIELDS + ("total",)}


def _ptr(t) -> int:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _arg(t, name, dtype=None, numel=None):
    """Device address of a tensor argument, after checking what the C ABI
    cannot see from a pointer: a device (cuda) tensor, contiguous, of the
    element type and with at least the elements the config implies. A host
    tensor would otherwise reach a kernel as a host address. None and raw
    integer addresses pass unchanged."""
    if t is None or isinstance(t, int):
        return t
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor or an int address")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a device (cuda) tensor, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if numel is not None and t.numel() < numel:
        raise ValueError(f"{name}: {t.numel()} elements, the config needs {numel}")
    return t.data_ptr()


def _el(cfg) -> "torch.dtype":
    return torch.bfloat16 if cfg.dtype == MOE_BF16 else torch.float32


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _nbytes(ws) -> int:
    return ws.numel() * ws.element_size()


def moe_plan(cfg, logits, ws, read_rounds=True, stream=None,
             return_counts=False):
    """Route + plan. With read_rounds (waits for the stream) returns R, or
    (R, counts) with return_counts (counts: int32 numpy array of E, the
    counts_host argument of the expert calls)."""
    out = (ctypes.c_int32 * (cfg.E + 1))()
    _check(load().moe_plan(ctypes.byref(cfg),
                           _arg(logits, "logits", torch.float32, cfg.T * cfg.E),
                           _arg(ws, "ws"),
                           _nbytes(ws), out if read_rounds else None,
                           _stream(stream)))
    if not read_rounds:
        return None
    vals = np.frombuffer(out, dtype=np.int32).copy()
    return (int(vals[-1]), vals[:-1].copy()) if return_counts else int(vals[-1])


def _counts(counts_host):
    if counts_host is None:
        return None
    a = np.ascontiguousarray(counts_host, dtype=np.int32)
    return a.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), a


def launch_batches(cfg, counts_host):
    """The forward's launch batches for a step's counts: a list of
    (first_round, n_rounds)."""
    a = np.ascontiguousarray(counts_host, dtype=np.int32)
    n_max = max(1, -(-cfg.T // max(1, min(cfg.C, cfg.T))))
    first = np.zeros(n_max, dtype=np.int32)
    nr = np.zeros(n_max, dtype=np.int32)
    n = ctypes.c_int32(0)
    p32 = lambda v: v.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))
    _check(load().moe_launch_batches(ctypes.byref(cfg), p32(a), n_max, p32(first),
                                     p32(nr), ctypes.byref(n)))
    return [(int(first[i]), int(nr[i])) for i in range(n.value)]


def moe_dispatch(cfg, round_, x, ws, stream=None, n_rounds=1):
    _check(load().moe_dispatch(ctypes.byref(cfg), int(round_), int(n_rounds),
                               _arg(x, "x", _el(cfg), cfg.T * cfg.d_model),
                               _arg(ws, "ws"), _nbytes(ws), _stream(stream)))


def moe_expert_ffn(cfg, round_, w_gate, w_up, w_down, ws, stream=None,
                   counts_host=None, n_rounds=1):
    c = _counts(counts_host)
    nw = cfg.E * cfg.d_model * cfg.d_ff
    _check(load().moe_expert_ffn(ctypes.byref(cfg), int(round_), int(n_rounds),
                                 _arg(w_gate, "w_gate", _el(cfg), nw),
                                 _arg(w_up, "w_up", _el(cfg), nw),
                                 _arg(w_down, "w_down", _el(cfg), nw), c and c[0],
                                 _arg(ws, "ws"), _nbytes(ws), _stream(stream)))


def moe_expert_gate_up(cfg, round_, w_gate, w_up, ws, stream=None,
                       counts_host=None, n_rounds=1):
    c = _counts(counts_host)
    nw = cfg.E * cfg.d_model * cfg.d_ff
    _check(load().moe_expert_gate_up(ctypes.byref(cfg), int(round_), int(n_rounds),
                                     _arg(w_gate, "w_gate", _el(cfg), nw),
                                     _arg(w_up, "w_up", _el(cfg), nw), c and c[0],
                                     _arg(ws, "ws"), _nbytes(ws), _stream(stream)))


def moe_dispatch_gate_up(cfg, round_, x, w_gate, w_up, ws, stream=None,
                         counts_host=None, n_rounds=1):
    c = _counts(counts_host)
    nw = cfg.E * cfg.d_model * cfg.d_ff
    _check(load().moe_dispatch_gate_up(ctypes.byref(cfg), int(round_), int(n_rounds),
                                       _arg(x, "x", _el(cfg), cfg.T * cfg.d_model),
                                       _arg(w_gate, "w_gate", _el(cfg), nw),
                                       _arg(w_up, "w_up", _el(cfg), nw), c and c[0],
                                       _arg(ws, "ws"), _nbytes(ws), _stream(stream)))


def moe_expert_down(cfg, round_, w_down, ws, stream=None, counts_host=None,
                    n_rounds=1):
    c = _counts(counts_host)
    _check(load().moe_expert_down(ctypes.byref(cfg), int(round_), int(n_rounds),
                                  _arg(w_down, "w_down", _el(cfg),
                                       cfg.E * cfg.d_model * cfg.d_ff),
                                  c and c[0], _arg(ws, "ws"),
                                  _nbytes(ws), _stream(stream)))


def moe_pack_weights(cfg, w_gate, w_up, w_down, out_gate, out_up, out_down,
                     stream=None):
    """Row-major expert weights -> the tiled layout (MOE_WEIGHTS_TILED)."""
    nw, el = cfg.E * cfg.d_model * cfg.d_ff, _el(cfg)
    _check(load().moe_pack_weights(ctypes.byref(cfg), _arg(w_gate, "w_gate", el, nw),
                                   _arg(w_up, "w_up", el, nw),
                                   _arg(w_down, "w_down", el, nw),
                                   _arg(out_gate, "out_gate", el, nw),
                                   _arg(out_up, "out_up", el, nw),
                                   _arg(out_down, "out_down", el, nw), _stream(stream)))


def moe_combine(cfg, ws, y, stream=None):
    _check(load().moe_combine(ctypes.byref(cfg), _arg(ws, "ws"), _nbytes(ws),
                              _arg(y, "y", _el(cfg), cfg.T * cfg.d_model),
                              _stream(stream)))


def moe_forward(cfg, logits, x, w_gate, w_up, w_down, y, ws, stream=None):
    nw, el, nx = cfg.E * cfg.d_model * cfg.d_ff, _el(cfg), cfg.T * cfg.d_model
    _check(load().moe_forward(ctypes.byref(cfg),
                              _arg(logits, "logits", torch.float32, cfg.T * cfg.E),
                              _arg(x, "x", el, nx), _arg(w_gate, "w_gate", el, nw),
                              _arg(w_up, "w_up", el, nw), _arg(w_down, "w_down", el, nw),
                              _arg(y, "y", el, nx), _arg(ws, "ws"), _nbytes(ws),
                              _stream(stream)))


# bytes of the library's static workspace (MOE_STATIC_WORKSPACE_BYTES)
STATIC_WORKSPACE_BYTES = 64 << 20


def moe_forward_static(cfg, logits, x, w_gate, w_up, w_down, y, stream=None):
    """moe_forward on the library's static device workspace: the call
    allocates nothing (see moe_forward_static in the header)."""
    nw, el, nx = cfg.E * cfg.d_model * cfg.d_ff, _el(cfg), cfg.T * cfg.d_model
    _check(load().moe_forward_static(
        ctypes.byref(cfg), _arg(logits, "logits", torch.float32, cfg.T * cfg.E),
        _arg(x, "x", el, nx), _arg(w_gate, "w_gate", el, nw),
        _arg(w_up, "w_up", el, nw), _arg(w_down, "w_down", el, nw),
        _arg(y, "y", el, nx), _stream(stream)))


def backward_workspace_size(cfg: MoeConfig) -> int:
    n = ctypes.c_size_t(0)
    _check(load().moe_backward_workspace_size(ctypes.byref(cfg), ctypes.byref(n)))
    return n.value


def backward_layout(cfg: MoeConfig) -> dict:
    L = MoeBackwardLayout()
    _check(load().moe_backward_layout(ctypes.byref(cfg), ctypes.byref(L)))
    return {n: getattr(L, n) for n in BWD_LAYOUT_FIELDS + ("total",)}


def moe_backward(cfg, x, w_gate, w_up, w_down, dy, dx, dlogits,
                 dw_gate, dw_up, dw_down, ws, bws, stream=None):
    """The layer's backward after moe_forward (ws: its workspace; the
    weights as given to moe_forward)."""
    nw, el, nx = cfg.E * cfg.d_model * cfg.d_ff, _el(cfg), cfg.T * cfg.d_model
    f32 = torch.float32
    _check(load().moe_backward(
        ctypes.byref(cfg), _arg(x, "x", el, nx), _arg(w_gate, "w_gate", el, nw),
        _arg(w_up, "w_up", el, nw), _arg(w_down, "w_down", el, nw),
        _arg(dy, "dy", el, nx),
        _arg(dx, "dx", el, nx), _arg(dlogits, "dlogits", f32, cfg.T * cfg.E),
        _arg(dw_gate, "dw_gate", f32, nw), _arg(dw_up, "dw_up", f32, nw),
        _arg(dw_down, "dw_down", f32, nw), _arg(ws, "ws"), _nbytes(ws),
        _arg(bws, "bws"), _nbytes(bws), _stream(stream)))


def _counts_rows(cfg: MoeConfig, counts):
    """Observed counts as a C-contiguous int32 [n_steps, E] array."""
    import numpy as np
    a = np.ascontiguousarray(np.asarray(counts, dtype=np.int32))
    if a.ndim == 1:
        a = a.reshape(1, -1)
    if a.ndim != 2 or a.shape[1] != cfg.E:
        raise ValueError(f"counts must be [n_steps, {cfg.E}]")
    return a


def capacity_curve(cfg: MoeConfig, counts, capacities):
    """(rounds [n_C, n_steps], workspace bytes [n_C]) for each capacity C:
    the memory-against-rounds curve of the observed steps' counts."""
    import numpy as np
    a = _counts_rows(cfg, counts)
    caps = np.ascontiguousarray(np.asarray(capacities, dtype=np.int64))
    rounds = np.zeros((caps.size, a.shape[0]), dtype=np.int32)
    ws = (ctypes.c_size_t * caps.size)()
    _check(load().moe_capacity_curve(
        ctypes.byref(cfg), a.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
        a.shape[0], caps.ctypes.data_as(ctypes.POINTER(ctypes.c_int64)),
        caps.size, rounds.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), ws))
    return rounds, np.array(list(ws), dtype=np.int64)


def capacity_for_rounds(cfg: MoeConfig, counts, target_rounds=1,
                        quantile=1.0) -> int:
    """Smallest C with at most target_rounds rounds on a share `quantile` of
    the observed steps."""
    a = _counts_rows(cfg, counts)
    out = ctypes.c_int64(0)
    _check(load().moe_capacity_for_rounds(
        ctypes.byref(cfg), a.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
        a.shape[0], int(target_rounds), float(quantile), ctypes.byref(out)))
    return out.value


# ---------------------------------------------------------------------------
# Ragged expert operators (the header's section of that name): rows sorted by
# expert, expert e owning the rows offsets[e] .. offsets[e + 1] - 1.

_DTYPES = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16, torch.float16: MOE_F16}
_TORCH_DTYPES = {v: k for k, v in _DTYPES.items()}


def _int32(v, name):
    # ctypes keeps the low 32 bits of a larger int
    if not -2**31 <= int(v) < 2**31:
        raise ValueError(f"{name} = {v} does not fit 32 bits")
    return int(v)


def grouped(rows, E, N, K, dtype, ld_x=0, ld_y=0) -> MoeGrouped:
    """Shape of a grouped product: weights [E, N, K], buffers of `rows` rows
    with row strides ld_x and ld_y in elements (0: K and N)."""
    if isinstance(dtype, str):
        dtype = {"f32": MOE_F32, "bf16": MOE_BF16, "f16": MOE_F16}[dtype]
    elif isinstance(dtype, torch.dtype):
        dtype = _DTYPES[dtype]
    for v, name in ((E, "E"), (N, "N"), (K, "K")):
        _int32(v, name)
    return MoeGrouped(int(rows), int(E), int(N), int(K), int(dtype), int(ld_x),
                      int(ld_y))


def grouped_dw_workspace_size(g: MoeGrouped) -> int:
    n = ctypes.c_size_t(0)
    _check(load().moe_grouped_dw_workspace_size(ctypes.byref(g), ctypes.byref(n)))
    return n.value


def mxfp4_scale_stride(K: int) -> int:
    """Bytes of a row of MXFP4 scales."""
    if K < 32 or K % 32:
        raise ValueError(f"K = {K} must be a positive multiple of 32")
    return (K // 32 + 3) // 4 * 4


# The ragged calls are also made for single tokens, where the host's time per
# call counts: an argument that is what the call needs is passed by a few
# attribute reads, anything else goes through the functions that say what is
# wrong with it.
_get_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _call_stream(stream, dev):
    if stream is None and _get_raw_stream is not None:
        return _get_raw_stream(dev)
    if isinstance(stream, torch.cuda.Stream) and stream.device_index != dev:
        raise ValueError(f"stream: on {stream.device}, the current device is cuda:{dev}")
    return _stream(stream)


def _on_device(t, name, dev):
    if isinstance(t, torch.Tensor) and t.get_device() == dev:  # -1: the host's
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor or an int address")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a device (cuda) tensor, got {t.device}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: on {t.device}, the current device is cuda:{dev}")


def _dense(t, name, dtype, numel, dev):
    """Address of a contiguous tensor of at least numel elements on the
    current device."""
    if (isinstance(t, torch.Tensor) and t.get_device() == dev and t.dtype is dtype
            and t.is_contiguous() and t.numel() >= numel):
        return t.data_ptr()
    if t is None or isinstance(t, int):
        return t
    _on_device(t, name, dev)
    return _arg(t, name, dtype, numel)  # raises


def _matrices(t, name, dtype, shape, dev):
    """Address of a contiguous tensor of at least the elements of shape (...,
    height, width) whose trailing dimensions make rows of that width or whole
    matrices (a plain buffer has none): a transposed layout is refused."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.is_contiguous() and t.get_device() == dev):
        return t.data_ptr()
    if t is None or isinstance(t, int):
        return t
    _on_device(t, name, dev)
    address = _arg(t, name, dtype, math.prod(shape))
    groups = list(itertools.accumulate(reversed(t.shape[1:]), operator.mul))
    if shape[-1] not in groups and any(n < shape[-2] * shape[-1] for n in groups):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {shape}")
    return address


def _mat(t, name, dtype, rows, cols, ld, dev):
    """Address of a [rows, cols] matrix whose rows are ld elements apart."""
    if (isinstance(t, torch.Tensor) and t.get_device() == dev and t.dtype is dtype
            and t.shape == (rows, cols) and t.stride() == (ld, 1)):
        return t.data_ptr()
    if t is None or isinstance(t, int):
        return t
    _on_device(t, name, dev)
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.dim() != 2 or t.shape[0] != rows or t.shape[1] != cols:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected ({rows}, {cols})")
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: elements of a row must be adjacent")
    if rows > 1 and t.stride(0) != ld:
        raise ValueError(f"{name}: row stride {t.stride(0)}, expected {ld}")
    return t.data_ptr()


def _rows_of(t, name, dev):
    """(dtype, rows, width, row stride) of a matrix argument."""
    if isinstance(t, torch.Tensor) and t.get_device() == dev:
        shape, stride, dt = t.shape, t.stride(), t.dtype
        if (len(shape) == 2 and dt in _DTYPES and stride[1] == 1 and shape[0] > 1
                and stride[0] >= shape[1]):
            return dt, shape[0], shape[1], stride[0]
    _on_device(t, name, dev)
    if t.dim() != 2:
        raise ValueError(f"{name}: expected a matrix, got {t.dim()} dimensions")
    if t.dtype not in _DTYPES:
        raise ValueError(f"{name}: dtype {t.dtype} is not supported")
    r, c = t.shape
    ld, one = t.stride()
    if c > 1 and one != 1:
        raise ValueError(f"{name}: elements of a row must be adjacent")
    if r <= 1:
        ld = c
    if ld < c:
        raise ValueError(f"{name}: rows overlap (row stride {ld}, width {c})")
    return t.dtype, r, c, ld


def _pair_of(t, name, dtype, rows, cols, dev):
    """Address and row stride of a [rows, cols] matrix of any row stride."""
    if isinstance(t, torch.Tensor) and t.get_device() == dev:
        shape, stride = t.shape, t.stride()
        if (shape == (rows, cols) and t.dtype is dtype and rows > 1 and stride[1] == 1
                and stride[0] >= cols):
            return t.data_ptr(), stride[0]
    dt, r, c, ld = _rows_of(t, name, dev)
    if dt is not dtype:
        raise ValueError(f"{name}: dtype {dt}, expected {dtype}")
    if r != rows or c != cols:
        raise ValueError(f"{name}: shape ({r}, {c}), expected ({rows}, {cols})")
    return t.data_ptr(), ld


def _rows_like(t, name, dtype, cols, dev):
    """Address, row stride and rows of a matrix of any number of rows."""
    if isinstance(t, torch.Tensor) and t.get_device() == dev:
        shape, stride = t.shape, t.stride()
        if (len(shape) == 2 and shape[1] == cols and t.dtype is dtype and shape[0] > 1
                and stride[1] == 1 and stride[0] >= cols):
            return t.data_ptr(), stride[0], shape[0]
    _on_device(t, name, dev)
    rows = t.shape[0] if t.dim() else 0
    return (*_pair_of(t, name, dtype, rows, cols, dev), rows)


def _offsets(offsets, E, dev):
    return _dense(offsets, "offsets", torch.int32, E + 1, dev)


def _n_rows(n_rows, dev):
    # every number of rows is below 2^31, every device address far above
    if isinstance(n_rows, int) and n_rows < 2**32:
        raise TypeError(f"n_rows = {n_rows}: expected a one-element int32 device tensor")
    return None if n_rows is None else _dense(n_rows, "n_rows", torch.int32, 1, dev)


def _grouped_dims(g):
    if g.dtype not in _TORCH_DTYPES:
        raise ValueError(f"unknown dtype {g.dtype}")
    return _TORCH_DTYPES[g.dtype], g.ld_x or g.K, g.ld_y or g.N


def moe_grouped_gemm(g, offsets, x, w, y, stream=None):
    """y[i] = w[e] x[i] for the rows i of every expert e: x [rows, K], w
    [E, N, K], y [rows, N]; rows of no expert keep what they held."""
    el, ld_x, ld_y = _grouped_dims(g)
    rows, E, N, K, dev = g.rows, g.E, g.N, g.K, torch.cuda.current_device()
    _check(load().moe_grouped_gemm(
        g, _offsets(offsets, E, dev), _mat(x, "x", el, rows, K, ld_x, dev),
        _matrices(w, "w", el, (E, N, K), dev), _mat(y, "y", el, rows, N, ld_y, dev),
        _call_stream(stream, dev)))


def moe_grouped_gemm_dx(g, offsets, dy, w, dx, stream=None):
    """dx[i] = w[e]^T dy[i]."""
    el, ld_x, ld_y = _grouped_dims(g)
    rows, E, N, K, dev = g.rows, g.E, g.N, g.K, torch.cuda.current_device()
    _check(load().moe_grouped_gemm_dx(
        g, _offsets(offsets, E, dev), _mat(dy, "dy", el, rows, N, ld_y, dev),
        _matrices(w, "w", el, (E, N, K), dev), _mat(dx, "dx", el, rows, K, ld_x, dev),
        _call_stream(stream, dev)))


def moe_grouped_gemm_dw(g, offsets, x, dy, dw, ws=None, accumulate=False, stream=None):
    """dw[e] = sum over e's rows of dy[i] x[i]^T (fp32 [E, N, K]), added to dw
    with accumulate; ws: grouped_dw_workspace_size bytes (None if 0)."""
    el, ld_x, ld_y = _grouped_dims(g)
    rows, E, N, K, dev = g.rows, g.E, g.N, g.K, torch.cuda.current_device()
    w_ptr, w_bytes = _workspace(ws, dev)
    _check(load().moe_grouped_gemm_dw(
        g, _offsets(offsets, E, dev), _mat(x, "x", el, rows, K, ld_x, dev),
        _mat(dy, "dy", el, rows, N, ld_y, dev),
        _matrices(dw, "dw", torch.float32, (E, N, K), dev), 1 if accumulate else 0, w_ptr,
        w_bytes, _call_stream(stream, dev)))


def moe_swiglu(gu, h, n_rows=None, stream=None):
    """h = silu(g) u for rows gu = [g, u]: gu [rows, 2f], h [rows, f]. n_rows:
    a one-element int32 device tensor, rows from it on are left alone."""
    dev = torch.cuda.current_device()
    dt, rows, f, ld_h = _rows_of(h, "h", dev)
    gu_ptr, ld_gu = _pair_of(gu, "gu", dt, rows, 2 * f, dev)
    _check(load().moe_swiglu(_DTYPES[dt], rows, f, gu_ptr, ld_gu, h.data_ptr(), ld_h,
                             _n_rows(n_rows, dev), _call_stream(stream, dev)))


def moe_swiglu_backward(gu, dh, dgu, n_rows=None, stream=None):
    """dgu [rows, 2f] from gu [rows, 2f] and dh [rows, f]."""
    dev = torch.cuda.current_device()
    dt, rows, f, ld_dh = _rows_of(dh, "dh", dev)
    gu_ptr, ld_gu = _pair_of(gu, "gu", dt, rows, 2 * f, dev)
    dgu_ptr, ld_dgu = _pair_of(dgu, "dgu", dt, rows, 2 * f, dev)
    _check(load().moe_swiglu_backward(
        _DTYPES[dt], rows, f, gu_ptr, ld_gu, dh.data_ptr(), ld_dh, dgu_ptr, ld_dgu,
        _n_rows(n_rows, dev), _call_stream(stream, dev)))


def moe_mxfp4_quantize(x, codes, scales, index=None, index_div=1, n_rows=None,
                       stream=None):
    """Rows of x [src_rows, K] to MXFP4: codes uint8 [..., K / 2] and scales
    uint8 [..., mxfp4_scale_stride(K)], contiguous, of as many rows as index
    (int32) has entries, row i from x[index[i] // index_div] (zeros where that
    is no row); without index, of x's rows (a contiguous x may have more
    dimensions: weights [E, N, K])."""
    dev = torch.cuda.current_device()
    if isinstance(x, torch.Tensor) and x.dim() > 2 and x.is_contiguous():
        x = x.view(-1, x.shape[-1])
    dt, src, K, ld_x = _rows_of(x, "x", dev)
    rows, index_ptr = src, None
    if index is not None:
        rows = index.numel()
        index_ptr = _dense(index, "index", torch.int32, rows, dev)
    u8 = torch.uint8
    _check(load().moe_mxfp4_quantize(
        _DTYPES[dt], rows, K, x.data_ptr(), ld_x, src, index_ptr, _int32(index_div, "index_div"),
        _n_rows(n_rows, dev), _matrices(codes, "codes", u8, (rows, K // 2), dev),
        _matrices(scales, "scales", u8, (rows, mxfp4_scale_stride(K)), dev),
        _call_stream(stream, dev)))


def moe_mxfp4_dequantize(codes, scales, y, n_rows=None, stream=None):
    """The values of codes and scales, y [rows, K]."""
    dev = torch.cuda.current_device()
    dt, rows, K, ld_y = _rows_of(y, "y", dev)
    u8 = torch.uint8
    _check(load().moe_mxfp4_dequantize(
        _DTYPES[dt], rows, K, _matrices(codes, "codes", u8, (rows, K // 2), dev),
        _matrices(scales, "scales", u8, (rows, mxfp4_scale_stride(K)), dev),
        y.data_ptr(), ld_y, _n_rows(n_rows, dev), _call_stream(stream, dev)))


def moe_mxfp4_grouped_gemm(g, offsets, x_codes, x_scales, w_codes, w_scales, y,
                           stream=None):
    """moe_grouped_gemm on MXFP4 operands; y has g's dtype."""
    el, _, ld_y = _grouped_dims(g)
    rows, E, N, K, dev = g.rows, g.E, g.N, g.K, torch.cuda.current_device()
    S, u8 = mxfp4_scale_stride(K), torch.uint8
    _check(load().moe_mxfp4_grouped_gemm(
        g, _offsets(offsets, E, dev), _matrices(x_codes, "x_codes", u8, (rows, K // 2), dev),
        _matrices(x_scales, "x_scales", u8, (rows, S), dev),
        _matrices(w_codes, "w_codes", u8, (E, N, K // 2), dev),
        _matrices(w_scales, "w_scales", u8, (E, N, S), dev),
        _mat(y, "y", el, rows, N, ld_y, dev), _call_stream(stream, dev)))


# ---------------------------------------------------------------------------
# Around the experts' products (the header's section of that name): routing, the
# sort of its assignments, the sum of the outputs back to tokens, 8-bit integers
# and the orthogonalised update.

_SCORES = {"softmax": MOE_SCORE_SOFTMAX, "sigmoid": MOE_SCORE_SIGMOID}


def router(T, E, k, dtype="f32", score="softmax", groups=1, top_groups=0, group_top=0,
           renormalize=True, scale=1.0, ld=0) -> MoeRouter:
    """A router of T tokens to k of E experts. dtype and ld: of the logits
    (rows ld elements apart, 0: E). A token chooses from the top_groups best
    (0: all) of `groups` groups of neighbouring experts; a group's score is
    the sum of its group_top (1 or 2; 0: 2) best choice scores."""
    if isinstance(dtype, str):
        dtype = {"f32": MOE_F32, "bf16": MOE_BF16, "f16": MOE_F16}[dtype]
    elif isinstance(dtype, torch.dtype):
        dtype = _DTYPES[dtype]
    if isinstance(score, str):
        score = _SCORES[score]
    for v, name in ((E, "E"), (k, "k"), (groups, "groups"), (top_groups, "top_groups"),
                    (group_top, "group_top")):
        _int32(v, name)
    return MoeRouter(int(T), int(E), int(k), int(dtype), int(score), int(groups),
                     int(top_groups), int(group_top), 1 if renormalize else 0, float(scale),
                     int(ld))


def _router_dims(r):
    if r.dtype not in _TORCH_DTYPES:
        raise ValueError(f"unknown dtype {r.dtype}")
    return _TORCH_DTYPES[r.dtype], r.T, r.E, r.k, r.ld or r.E


def moe_route(r, logits, idx, weight, bias=None, stream=None):
    """logits [T, E] to idx int32 [T, k] and weight float32 [T, k]; bias
    float32 [E] steers the choice alone."""
    el, T, E, k, ld = _router_dims(r)
    dev = torch.cuda.current_device()
    _check(load().moe_route(
        r, _mat(logits, "logits", el, T, E, ld, dev),
        None if bias is None else _dense(bias, "bias", torch.float32, E, dev),
        _matrices(idx, "idx", torch.int32, (T, k), dev),
        _matrices(weight, "weight", torch.float32, (T, k), dev), _call_stream(stream, dev)))


def moe_route_backward(r, logits, idx, dweight, dlogits, stream=None):
    """dlogits [T, E] (rows r.ld apart, as the logits) from dweight [T, k]."""
    el, T, E, k, ld = _router_dims(r)
    dev = torch.cuda.current_device()
    _check(load().moe_route_backward(
        r, _mat(logits, "logits", el, T, E, ld, dev),
        _matrices(idx, "idx", torch.int32, (T, k), dev),
        _matrices(dweight, "dweight", torch.float32, (T, k), dev),
        _mat(dlogits, "dlogits", el, T, E, ld, dev), _call_stream(stream, dev)))


def sort_workspace_size(n: int, E: int) -> int:
    """Workspace of moe_sort for n assignments."""
    b = ctypes.c_size_t(0)
    _check(load().moe_sort_workspace_size(int(n), _int32(E, "E"), ctypes.byref(b)))
    return b.value


def _workspace(ws, dev):
    """(address, bytes) of a workspace tensor, or of none."""
    if ws is None:
        return None, 0
    _on_device(ws, "ws", dev)
    if not ws.is_contiguous():
        raise ValueError("ws: must be contiguous")
    size = _nbytes(ws)
    return (ws.data_ptr() if size else None), size  # an empty tensor has no address


def moe_sort(idx, E, perm, pos, offsets, ws=None, stream=None):
    """Assignments idx (int32, all its elements) by expert: perm and pos int32
    of as many elements, offsets int32 [E + 1]; ws: sort_workspace_size bytes
    (None if 0)."""
    dev = torch.cuda.current_device()
    i32 = torch.int32
    _on_device(idx, "idx", dev)
    n = idx.numel()
    w_ptr, w_bytes = _workspace(ws, dev)
    _check(load().moe_sort(n, _int32(E, "E"), _dense(idx, "idx", i32, n, dev),
                           _dense(perm, "perm", i32, n, dev), _dense(pos, "pos", i32, n, dev),
                           _offsets(offsets, E, dev), w_ptr, w_bytes, _call_stream(stream, dev)))


def _positions(pos, T, dev):
    """k and the address of pos [T, k]."""
    if isinstance(pos, torch.Tensor) and pos.get_device() == dev:
        shape = pos.shape
        if (len(shape) == 2 and shape[0] == T and pos.dtype is torch.int32
                and pos.is_contiguous()):
            return shape[1], pos.data_ptr()
    _on_device(pos, "pos", dev)
    if pos.dim() != 2 or pos.shape[0] != T:
        raise ValueError(f"pos: shape {tuple(pos.shape)}, expected ({T}, k)")
    return pos.shape[1], _dense(pos, "pos", torch.int32, pos.numel(), dev)


def moe_collect(z, pos, y, weight=None, stream=None):
    """y[t] = sum over j of weight[t, j] z[pos[t, j]]: z [rows, d], pos int32
    [T, k], y [T, d], weight float32 [T, k] (None: all 1)."""
    dev = torch.cuda.current_device()
    dt, T, d, ld_y = _rows_of(y, "y", dev)
    z_ptr, ld_z, rows = _rows_like(z, "z", dt, d, dev)
    k, pos_ptr = _positions(pos, T, dev)
    w_ptr = None if weight is None else _matrices(weight, "weight", torch.float32, (T, k), dev)
    _check(load().moe_collect(_DTYPES[dt], T, k, rows, d, z_ptr, ld_z, pos_ptr, w_ptr,
                              y.data_ptr(), ld_y, _call_stream(stream, dev)))


def moe_collect_backward(dy, pos, dz=None, weight=None, z=None, dweight=None, stream=None):
    """dz[pos[t, j]] = weight[t, j] dy[t] and, where dweight [T, k] is given,
    dweight[t, j] = <z[pos[t, j]], dy[t]>: dy [T, d], dz and z [rows, d]. With
    weight None, dz is a gather of dy's rows."""
    dev = torch.cuda.current_device()
    dt, T, d, ld_dy = _rows_of(dy, "dy", dev)
    k, pos_ptr = _positions(pos, T, dev)
    w_ptr = dw_ptr = z_ptr = dz_ptr = None
    ld_z = ld_dz = rows = 0
    if dz is not None:
        dz_ptr, ld_dz, rows = _rows_like(dz, "dz", dt, d, dev)
    elif dweight is None:
        raise ValueError("neither dz nor dweight is given")
    if dweight is not None:
        if z is None:
            raise ValueError("dweight needs z")
        dw_ptr = _matrices(dweight, "dweight", torch.float32, (T, k), dev)
    if z is not None:
        if dz is None:
            z_ptr, ld_z, rows = _rows_like(z, "z", dt, d, dev)
        else:
            z_ptr, ld_z = _pair_of(z, "z", dt, rows, d, dev)
    if weight is not None:
        w_ptr = _matrices(weight, "weight", torch.float32, (T, k), dev)
    _check(load().moe_collect_backward(
        _DTYPES[dt], T, k, rows, d, dy.data_ptr(), ld_dy, z_ptr, ld_z, pos_ptr, w_ptr, dz_ptr,
        ld_dz, dw_ptr, _call_stream(stream, dev)))


def int8_stride(K: int) -> int:
    """Codes of a row of 8-bit integers."""
    if not 1 <= K <= 2**20:
        raise ValueError(f"K = {K} must lie in [1, 2^20]")
    return (K + 15) // 16 * 16


def moe_int8_quantize(x, codes, scales, index=None, index_div=1, n_rows=None, stream=None):
    """Rows of x [src_rows, K] to 8-bit integers: codes int8 [...,
    int8_stride(K)] and scales float32 [...], contiguous; rows, index and
    index_div as for moe_mxfp4_quantize."""
    dev = torch.cuda.current_device()
    if isinstance(x, torch.Tensor) and x.dim() > 2 and x.is_contiguous():
        x = x.view(-1, x.shape[-1])
    dt, src, K, ld_x = _rows_of(x, "x", dev)
    rows, index_ptr = src, None
    if index is not None:
        rows = index.numel()
        index_ptr = _dense(index, "index", torch.int32, rows, dev)
    index_div = index_div if index_div == 1 else _int32(index_div, "index_div")
    _check(load().moe_int8_quantize(
        _DTYPES[dt], rows, K, x.data_ptr(), ld_x, src, index_ptr, index_div,
        _n_rows(n_rows, dev), _matrices(codes, "codes", torch.int8, (rows, int8_stride(K)), dev),
        _dense(scales, "scales", torch.float32, rows, dev), _call_stream(stream, dev)))


def moe_int8_dequantize(codes, scales, y, n_rows=None, stream=None):
    """The values of codes and scales, y [rows, K]."""
    dev = torch.cuda.current_device()
    dt, rows, K, ld_y = _rows_of(y, "y", dev)
    _check(load().moe_int8_dequantize(
        _DTYPES[dt], rows, K, _matrices(codes, "codes", torch.int8, (rows, int8_stride(K)), dev),
        _dense(scales, "scales", torch.float32, rows, dev), y.data_ptr(), ld_y,
        _n_rows(n_rows, dev), _call_stream(stream, dev)))


def moe_int8_grouped_gemm(g, offsets, x_codes, x_scales, w_codes, w_scales, y, stream=None):
    """moe_grouped_gemm on 8-bit rows: x_codes [rows, S], x_scales [rows],
    w_codes [E, N, S], w_scales [E, N] with S = int8_stride(K); y has g's dtype."""
    el, _, ld_y = _grouped_dims(g)
    rows, E, N, K, dev = g.rows, g.E, g.N, g.K, torch.cuda.current_device()
    S, i8, f32 = int8_stride(K), torch.int8, torch.float32
    _check(load().moe_int8_grouped_gemm(
        g, _offsets(offsets, E, dev), _matrices(x_codes, "x_codes", i8, (rows, S), dev),
        _dense(x_scales, "x_scales", f32, rows, dev),
        _matrices(w_codes, "w_codes", i8, (E, N, S), dev),
        _matrices(w_scales, "w_scales", f32, (E, N), dev),
        _mat(y, "y", el, rows, N, ld_y, dev), _call_stream(stream, dev)))


def orthogonalize_workspace_size(E: int, N: int, K: int) -> int:
    """Workspace of moe_orthogonalize for E matrices [N, K]."""
    b = ctypes.c_size_t(0)
    _check(load().moe_orthogonalize_workspace_size(_int32(E, "E"), _int32(N, "N"),
                                                   _int32(K, "K"), ctypes.byref(b)))
    return b.value


def moe_orthogonalize(g, y, ws, steps=5, coefficients=None, scale=1.0, stream=None):
    """The orthogonalised update of the matrices g [E, N, K] (or one [N, K]):
    y bfloat16 of the same shape. coefficients: `steps` triples (a, b, c), or
    None for the usual ones."""
    dev = torch.cuda.current_device()
    _on_device(g, "g", dev)
    if g.dim() not in (2, 3) or g.dtype not in _DTYPES:
        raise ValueError(f"g: shape {tuple(g.shape)}, dtype {g.dtype}: expected float matrices")
    if not g.is_contiguous():
        raise ValueError("g: must be contiguous")
    E, N, K = (1, *g.shape) if g.dim() == 2 else g.shape
    _on_device(y, "y", dev)
    if y.shape != g.shape or y.dtype is not torch.bfloat16 or not y.is_contiguous():
        raise ValueError(f"y: expected contiguous bfloat16 of shape {tuple(g.shape)}")
    c = None
    if coefficients is not None:
        flat = [float(v) for triple in coefficients for v in triple]
        if len(flat) != 3 * steps:
            raise ValueError(f"coefficients: expected {steps} triples")
        c = (ctypes.c_float * len(flat))(*flat)
    w_ptr, w_bytes = _workspace(ws, dev)
    _check(load().moe_orthogonalize(_DTYPES[g.dtype], E, N, K, g.data_ptr(), y.data_ptr(),
                                    _int32(steps, "steps"), c, float(scale), w_ptr, w_bytes,
                                    _call_stream(stream, dev)))


def workspace_views(cfg: MoeConfig, ws: torch.Tensor) -> dict:
    """torch views of the internal buffers of a uint8 workspace tensor.
    xr and h are returned as raw bytes of all sets of the round buffer (rows
    of d (f) elements in the tiled layout, see buffer_geometry); rounds is
    [9, M, E]: per (round, expert) rows, first index, rows of the group's
    lower experts, the same padded to 64, and the buffer row brow; then the
    pair tables indexed [b, v] (expert, rows, buffer row, first z row);
    round_pairs is [2, M]: rbeg and rend of every round."""
    L = workspace_layout(cfg)
    T, E, k = cfg.T, cfg.E, cfg.k
    geo = buffer_geometry(cfg)
    rows, M = geo["rows"] * geo["S"], geo["M"]
    el = torch.bfloat16 if cfg.dtype == MOE_BF16 else torch.float32
    es = 2 if cfg.dtype == MOE_BF16 else 4

    def view(name, n, dt, size):
        return ws[L[name]:L[name] + n * size].view(dt)

    i32 = torch.int32
    return {
        "idx": view("idx", T * k, i32, 4).view(T, k),
        "weight": view("weight", T * k, torch.float32, 4).view(T, k),
        "counts": view("counts", E, i32, 4),
        "offsets": view("offsets", E + 1, i32, 4),
        "n_rounds": view("n_rounds", 1, i32, 4),
        "perm": view("perm", T * k, i32, 4),
        "pos": view("pos", T * k, i32, 4),
        "round_of": view("round_of", T * k, i32, 4),
        "row_of": view("row_of", T * k, i32, 4),
        "rounds": view("rounds", 9 * M * E, i32, 4).view(9, M, E),
        "round_pairs": ws[L["rounds"] + 36 * M * E:L["rounds"] + 36 * M * E + 8 * M]
        .view(i32).view(2, M),
        "xr": view("xr", rows * cfg.d_model * es, torch.uint8, 1),
        "h": view("h", rows * cfg.d_ff * es, torch.uint8, 1),
        "z": view("z", T * k * cfg.d_model, el, es).view(T * k, cfg.d_model),
    }

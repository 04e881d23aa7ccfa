"""Thin Python binding of liblrm.so (include/lrm.h): argument marshalling only.

Every step of the path runs in the library's HIP kernels; PyTorch only supplies device memory
(tensors passed by data pointer) and the stream.  There is no fallback: if the library is not
built, loading raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("LRM_LIBRARY") or os.path.join(_PKG, "liblrm.so")

LRM_F32, LRM_BF16 = 0, 1
DEVERR = {1: "EXPERT_ID", 2: "L_CAP", 4: "K_CAP", 8: "QUOTA", 16: "NONFINITE", 32: "INDEX"}

EXPORTS = ("lrm_workspace_bytes", "lrm_plan_quotas", "lrm_admit_quotas", "lrm_score",
           "lrm_score_norms", "lrm_score_combine", "lrm_score_criterion",
           "lrm_select", "lrm_compact", "lrm_grouped_dw", "lrm_grouped_dx", "lrm_grouped_dw_dx",
           "lrm_swiglu_backward", "lrm_gather_tokens", "lrm_grouped_fc1_dw", "lrm_grouped_fc1_dx",
           "lrm_grouped_fc1_dw_dx", "lrm_scatter_tokens", "lrm_read_device_error",
           "lrm_status_string", "lrm_grouped_dw_dx_noalloc", "lrm_router_workspace_bytes",
           "lrm_route", "lrm_route_backward", "lrm_gate_dots", "lrm_forward_workspace_bytes",
           "lrm_grouped_fc1_swiglu", "lrm_grouped_fc2", "lrm_combine_tokens",
           "lrm_grad_workspace_bytes", "lrm_grad_norm", "lrm_clip_grads", "lrm_grouped_fc2_wide",
           "lrm_combine_tokens_wide")
_SIZES = ("lrm_workspace_bytes", "lrm_router_workspace_bytes", "lrm_forward_workspace_bytes",
          "lrm_grad_workspace_bytes")

QUOTA_KINDS = {"cap": 0, "proportional": 1, "waterfill": 2}
CRITERIA = {"lrm": 0, "grad_sq": 1, "grad_abs": 2, "random": 3}
GATES = {"topk": 0, "all": 1}


class Problem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("T", "k", "E", "e_lo", "E_loc", "h", "d", "dtype", "L_cap", "K_cap")]


class QuotaPolicy(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("full", "rho_num", "rho_den", "cap_abs", "kind")]


class Router(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "E", "k", "dtype", "gate")] + \
               [("balance_coef", ctypes.c_float)]


class Tensor(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("count", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


MAX_CANDIDATES = 16


class Admission(ctypes.Structure):
    _fields_ = [("n_cand", ctypes.c_int32), ("kind", ctypes.c_int32), ("cap_abs", ctypes.c_int32),
                ("full", ctypes.c_int32 * MAX_CANDIDATES),
                ("rho_num", ctypes.c_int32 * MAX_CANDIDATES),
                ("rho_den", ctypes.c_int32 * MAX_CANDIDATES),
                ("mem_budget", ctypes.c_int64), ("mem_base", ctypes.c_int64),
                ("mem_per_row", ctypes.c_int64), ("comm_budget", ctypes.c_int64),
                ("comm_per_row", ctypes.c_int64)]


def make_admission(candidates, mem_budget, mem_base=0, mem_per_row=0, comm_budget=-1,
                   comm_per_row=0, kind="cap", cap_abs=-1) -> Admission:
    """candidates: list of (full, rho_num, rho_den), tested in that order."""
    a = Admission()
    a.n_cand = len(candidates)
    a.kind = QUOTA_KINDS[kind] if isinstance(kind, str) else int(kind)
    a.cap_abs = cap_abs
    for i, (f, n, d) in enumerate(candidates):
        a.full[i], a.rho_num[i], a.rho_den[i] = int(f), int(n), int(d)
    a.mem_budget, a.mem_base, a.mem_per_row = mem_budget, mem_base, mem_per_row
    a.comm_budget, a.comm_per_row = comm_budget, comm_per_row
    return a


class LrmError(RuntimeError):
    pass


_LIB = None


def load_library(path: Optional[str] = None):
    """Load liblrm.so (raises if it has not been built)."""
    global _LIB
    if _LIB is not None and path is None:
        return _LIB
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise LrmError(f"{p} is missing: build the HIP library first "
                       "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(p)
    vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32
    PP, QP = ctypes.POINTER(Problem), ctypes.POINTER(QuotaPolicy)
    lib.lrm_workspace_bytes.argtypes = [PP]
    lib.lrm_plan_quotas.argtypes = [PP, QP] + [vp] * 7 + [sz, vp]
    lib.lrm_admit_quotas.argtypes = [PP, ctypes.POINTER(Admission)] + [vp] * 5 + [sz, vp]
    lib.lrm_score.argtypes = [PP] + [vp] * 7 + [sz, vp]
    lib.lrm_score_norms.argtypes = [PP] + [vp] * 3 + [sz, vp]
    lib.lrm_score_combine.argtypes = [PP] + [vp] * 5 + [sz, vp]
    lib.lrm_score_criterion.argtypes = [PP, i32] + [vp] * 8 + [sz, vp]
    lib.lrm_select.argtypes = [PP] + [vp] * 6 + [sz, vp]
    lib.lrm_compact.argtypes = [PP] + [vp] * 10 + [sz, vp]
    lib.lrm_grouped_dw.argtypes = [PP] + [vp] * 5 + [sz, vp]
    lib.lrm_grouped_dx.argtypes = [PP] + [vp] * 5 + [sz, vp]
    lib.lrm_grouped_dw_dx.argtypes = [PP] + [vp] * 7 + [sz, vp]
    lib.lrm_grouped_dw_dx_noalloc.argtypes = [PP] + [vp] * 6 + [vp]
    lib.lrm_swiglu_backward.argtypes = [PP] + [vp] * 6 + [sz, vp]
    lib.lrm_gather_tokens.argtypes = [PP] + [vp] * 5 + [sz, vp]
    lib.lrm_grouped_fc1_dw.argtypes = [PP] + [vp] * 5 + [sz, vp]
    lib.lrm_grouped_fc1_dx.argtypes = [PP] + [vp] * 5 + [sz, vp]
    lib.lrm_grouped_fc1_dw_dx.argtypes = [PP] + [vp] * 7 + [sz, vp]
    lib.lrm_scatter_tokens.argtypes = [PP] + [vp] * 5 + [sz, vp]
    lib.lrm_read_device_error.argtypes = [vp, ctypes.POINTER(i32), i32, vp]
    RP, TP = ctypes.POINTER(Router), ctypes.POINTER(Tensor)
    lib.lrm_router_workspace_bytes.argtypes = [RP]
    lib.lrm_route.argtypes = [RP] + [vp] * 9 + [sz, vp]
    lib.lrm_route_backward.argtypes = [RP] + [vp] * 7
    lib.lrm_gate_dots.argtypes = [PP] + [vp] * 6 + [sz, vp]
    lib.lrm_forward_workspace_bytes.argtypes = [PP]
    lib.lrm_grouped_fc1_swiglu.argtypes = [PP] + [vp] * 7 + [sz, vp]
    lib.lrm_grouped_fc2.argtypes = lib.lrm_grouped_fc2_wide.argtypes = [PP] + [vp] * 5 + [sz, vp]
    lib.lrm_combine_tokens.argtypes = [PP] + [vp] * 7 + [sz, vp]
    lib.lrm_combine_tokens_wide.argtypes = [PP] + [vp] * 7 + [sz, vp]
    lib.lrm_grad_workspace_bytes.argtypes = [TP, i32]
    lib.lrm_grad_norm.argtypes = [TP, i32, vp, vp, sz, vp]
    lib.lrm_clip_grads.argtypes = [TP, i32, ctypes.c_float, vp, vp, sz, vp]
    for f in EXPORTS:
        if f in _SIZES:
            getattr(lib, f).restype = sz
        elif f != "lrm_status_string":
            getattr(lib, f).restype = ctypes.c_int
    lib.lrm_status_string.argtypes = [ctypes.c_int]
    lib.lrm_status_string.restype = ctypes.c_char_p
    if path is None:
        _LIB = lib
    return lib


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(lib, status: int, what: str):
    if status != 0:
        raise LrmError(f"{what}: {lib.lrm_status_string(status).decode()} (status {status})")


def make_problem(T, k, E, e_lo, E_loc, h, d, dtype, L_cap, K_cap) -> Problem:
    dt = {"f32": LRM_F32, "bf16": LRM_BF16}.get(dtype, dtype)
    return Problem(T, k, E, e_lo, E_loc, h, d, dt, L_cap, K_cap)


def make_policy(full=0, rho_num=1, rho_den=1, cap_abs=-1, kind="cap") -> QuotaPolicy:
    kd = QUOTA_KINDS[kind] if isinstance(kind, str) else int(kind)
    return QuotaPolicy(int(full), int(rho_num), int(rho_den), int(cap_abs), kd)


def lrm_workspace_bytes(problem: Problem) -> int:
    return int(load_library().lrm_workspace_bytes(ctypes.byref(problem)))


def lrm_plan_quotas(problem, policy, topk_idx, counts, fwd_off, row_pair, quota, cmp_off, ws,
                    stream=None):
    lib = load_library()
    _check(lib, lib.lrm_plan_quotas(ctypes.byref(problem), ctypes.byref(policy), _ptr(topk_idx),
                                    _ptr(counts), _ptr(fwd_off), _ptr(row_pair), _ptr(quota),
                                    _ptr(cmp_off), _ptr(ws), ws.numel() * ws.element_size(),
                                    _stream(stream)), "lrm_plan_quotas")


def lrm_score(problem, topk_w, g, phi, row_pair, fwd_off, score, ws, stream=None):
    lib = load_library()
    _check(lib, lib.lrm_score(ctypes.byref(problem), _ptr(topk_w), _ptr(g), _ptr(phi),
                              _ptr(row_pair), _ptr(fwd_off), _ptr(score), _ptr(ws),
                              ws.numel() * ws.element_size(), _stream(stream)), "lrm_score")


def lrm_score_norms(problem, g, phi, ws, stream=None):
    lib = load_library()
    _check(lib, lib.lrm_score_norms(ctypes.byref(problem), _ptr(g), _ptr(phi), _ptr(ws),
                                    ws.numel() * ws.element_size(), _stream(stream)),
           "lrm_score_norms")


def lrm_score_combine(problem, topk_w, row_pair, fwd_off, score, ws, stream=None):
    lib = load_library()
    _check(lib, lib.lrm_score_combine(ctypes.byref(problem), _ptr(topk_w), _ptr(row_pair),
                                      _ptr(fwd_off), _ptr(score), _ptr(ws),
                                      ws.numel() * ws.element_size(), _stream(stream)),
           "lrm_score_combine")


def lrm_score_criterion(problem, criterion, topk_w, g, phi, keys, row_pair, fwd_off, score, ws,
                        stream=None):
    lib = load_library()
    crit = CRITERIA[criterion] if isinstance(criterion, str) else int(criterion)
    _check(lib, lib.lrm_score_criterion(ctypes.byref(problem), crit, _ptr(topk_w), _ptr(g),
                                        _ptr(phi), _ptr(keys), _ptr(row_pair), _ptr(fwd_off),
                                        _ptr(score), _ptr(ws), ws.numel() * ws.element_size(),
                                        _stream(stream)), "lrm_score_criterion")


def lrm_select(problem, score, fwd_off, quota, cmp_off, sel_row, ws, stream=None):
    lib = load_library()
    _check(lib, lib.lrm_select(ctypes.byref(problem), _ptr(score), _ptr(fwd_off), _ptr(quota),
                               _ptr(cmp_off), _ptr(sel_row), _ptr(ws),
                               ws.numel() * ws.element_size(), _stream(stream)), "lrm_select")


def lrm_compact(problem, sel_row, row_pair, cmp_off, topk_w, g, phi, Gc, Phic, sel_pair, ws,
                stream=None):
    lib = load_library()
    _check(lib, lib.lrm_compact(ctypes.byref(problem), _ptr(sel_row), _ptr(row_pair),
                                _ptr(cmp_off), _ptr(topk_w), _ptr(g), _ptr(phi), _ptr(Gc),
                                _ptr(Phic), _ptr(sel_pair), _ptr(ws),
                                ws.numel() * ws.element_size(), _stream(stream)), "lrm_compact")


def lrm_grouped_dw(problem, Gc, Phic, cmp_off, dW, ws, stream=None):
    lib = load_library()
    _check(lib, lib.lrm_grouped_dw(ctypes.byref(problem), _ptr(Gc), _ptr(Phic), _ptr(cmp_off),
                                   _ptr(dW), _ptr(ws), ws.numel() * ws.element_size(),
                                   _stream(stream)), "lrm_grouped_dw")


def lrm_grouped_dx(problem, Gc, W, cmp_off, dphi, ws, stream=None):
    lib = load_library()
    _check(lib, lib.lrm_grouped_dx(ctypes.byref(problem), _ptr(Gc), _ptr(W), _ptr(cmp_off),
                                   _ptr(dphi), _ptr(ws), ws.numel() * ws.element_size(),
                                   _stream(stream)), "lrm_grouped_dx")


def lrm_grouped_dw_dx(problem, Gc, Phic, W, cmp_off, dW, dphi, ws, stream=None):
    lib = load_library()
    _check(lib, lib.lrm_grouped_dw_dx(ctypes.byref(problem), _ptr(Gc), _ptr(Phic), _ptr(W),
                                      _ptr(cmp_off), _ptr(dW), _ptr(dphi), _ptr(ws),
                                      ws.numel() * ws.element_size(), _stream(stream)),
           "lrm_grouped_dw_dx")


def lrm_grouped_dw_dx_noalloc(problem, Gc, Phic, W, cmp_off, dW, dphi, stream=None):
    lib = load_library()
    _check(lib, lib.lrm_grouped_dw_dx_noalloc(ctypes.byref(problem), _ptr(Gc), _ptr(Phic), _ptr(W),
                                              _ptr(cmp_off), _ptr(dW), _ptr(dphi),
                                              _stream(stream)),
           "lrm_grouped_dw_dx_noalloc")


def lrm_admit_quotas(problem, admission, fwd_off, quota, cmp_off, admitted, ws, stream=None):
    lib = load_library()
    _check(lib, lib.lrm_admit_quotas(ctypes.byref(problem), ctypes.byref(admission), _ptr(fwd_off),
                                     _ptr(quota), _ptr(cmp_off), _ptr(admitted),
                                     _ptr(ws),
                                     ws.numel() * ws.element_size(), _stream(stream)),
           "lrm_admit_quotas")


def _ws(ws):
    return _ptr(ws), ws.numel() * ws.element_size()


def lrm_swiglu_backward(problem, sel_row, cmp_off, dphi, ac, dH, ws, stream=None):
    lib = load_library()
    _check(lib, lib.lrm_swiglu_backward(ctypes.byref(problem), _ptr(sel_row), _ptr(cmp_off),
                                        _ptr(dphi), _ptr(ac), _ptr(dH), *_ws(ws),
                                        _stream(stream)), "lrm_swiglu_backward")


def lrm_gather_tokens(problem, sel_pair, cmp_off, x, Xc, ws, stream=None):
    lib = load_library()
    _check(lib, lib.lrm_gather_tokens(ctypes.byref(problem), _ptr(sel_pair), _ptr(cmp_off),
                                      _ptr(x), _ptr(Xc), *_ws(ws), _stream(stream)),
           "lrm_gather_tokens")


def lrm_grouped_fc1_dw(problem, dH, Xc, cmp_off, dW1, ws, stream=None):
    lib = load_library()
    _check(lib, lib.lrm_grouped_fc1_dw(ctypes.byref(problem), _ptr(dH), _ptr(Xc), _ptr(cmp_off),
                                       _ptr(dW1), *_ws(ws), _stream(stream)), "lrm_grouped_fc1_dw")


def lrm_grouped_fc1_dx(problem, dH, W1, cmp_off, dX, ws, stream=None):
    lib = load_library()
    _check(lib, lib.lrm_grouped_fc1_dx(ctypes.byref(problem), _ptr(dH), _ptr(W1), _ptr(cmp_off),
                                       _ptr(dX), *_ws(ws), _stream(stream)), "lrm_grouped_fc1_dx")


def lrm_grouped_fc1_dw_dx(problem, dH, Xc, W1, cmp_off, dW1, dX, ws, stream=None):
    lib = load_library()
    _check(lib, lib.lrm_grouped_fc1_dw_dx(ctypes.byref(problem), _ptr(dH), _ptr(Xc), _ptr(W1),
                                          _ptr(cmp_off), _ptr(dW1), _ptr(dX), *_ws(ws),
                                          _stream(stream)), "lrm_grouped_fc1_dw_dx")


def lrm_scatter_tokens(problem, sel_pair, cmp_off, dX, dx, ws, stream=None):
    lib = load_library()
    _check(lib, lib.lrm_scatter_tokens(ctypes.byref(problem), _ptr(sel_pair), _ptr(cmp_off),
                                       _ptr(dX), _ptr(dx), *_ws(ws), _stream(stream)),
           "lrm_scatter_tokens")


# ---------------------------------------------------------------------------------------------
# The router, the experts' forward and the clipping of gradients.  A torch tensor's element type,
# size, layout and device are known here, so these calls check them before they pass the pointer
# on; a plain address (int) is passed as it is.
# ---------------------------------------------------------------------------------------------

_ELEM = {LRM_F32: (torch.float32,), LRM_BF16: (torch.bfloat16, torch.int16)}
_F32, _I32, _U8 = (torch.float32,), (torch.int32,), (torch.uint8, torch.bool)


def _arg(t, name, types, count, device, exact=False):
    """The address of tensor ``t`` of at least (or exactly) ``count`` elements, after its checks."""
    if t is None or t.__class__ is int:
        return t
    n = t.numel()
    if (n == count or n > count and not exact) and t.dtype in types and t.is_contiguous() and \
            t.get_device() == device:
        return t.data_ptr()
    if t.dtype not in types:
        raise LrmError(f"{name}: element type {t.dtype}, expected {types[0]}")
    if n < count or (exact and n != count):
        raise LrmError(f"{name}: {n} elements, expected {'' if exact else 'at least '}{count}")
    if not t.is_contiguous():
        raise LrmError(f"{name}: not contiguous")
    raise LrmError(f"{name}: on {t.device}, the call runs on cuda:{device}")


# The handle of torch's current stream.  A call of a serving step is a few microseconds of host time;
# forming a Stream object for its handle would be three more.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _queue(stream, device):
    if stream is None and _raw_stream is not None:
        return _raw_stream(device)
    if isinstance(stream, torch.cuda.Stream) and stream.device_index != device:
        raise LrmError(f"stream: on cuda:{stream.device_index}, the call runs on cuda:{device}")
    return _stream(stream)


def _device() -> int:
    return torch.cuda.current_device()


def _elem(dtype):
    if dtype not in _ELEM:
        raise LrmError(f"unknown element type {dtype}")
    return _ELEM[dtype]


def _space(ws, device):
    if isinstance(ws, int):
        raise LrmError("ws: a tensor is needed, its size is part of the call")
    if ws.is_contiguous() and ws.get_device() == device:
        return ws.data_ptr(), ws.nbytes
    return _arg(ws, "ws", (ws.dtype,), 0, device), 0   # raises


def make_router(T, E, k, dtype="f32", gate="topk", balance_coef=0.0) -> Router:
    """A router over E experts: ``gate`` "topk" renormalises the k weights, "all" keeps the
    probabilities over all experts; ``dtype`` is the logits'."""
    dt = {"f32": LRM_F32, "bf16": LRM_BF16}.get(dtype, dtype)
    return Router(T, E, k, dt, GATES[gate] if isinstance(gate, str) else int(gate), balance_coef)


def lrm_router_workspace_bytes(router: Router) -> int:
    return int(load_library().lrm_router_workspace_bytes(ctypes.byref(router)))


def lrm_forward_workspace_bytes(problem: Problem) -> int:
    return int(load_library().lrm_forward_workspace_bytes(ctypes.byref(problem)))


def lrm_route(router, logits, mask, topk_idx, topk_w, lse, counts, prob, loss, ws, stream=None):
    lib = load_library()
    r, d = router, _device()
    _check(lib, lib.lrm_route(ctypes.byref(r), _arg(logits, "logits", _elem(r.dtype), r.T * r.E, d, True),
                              _arg(mask, "mask", _U8, r.T, d, True),
                              _arg(topk_idx, "topk_idx", _I32, r.T * r.k, d),
                              _arg(topk_w, "topk_w", _F32, r.T * r.k, d),
                              _arg(lse, "lse", _F32, r.T, d), _arg(counts, "counts", _I32, r.E, d),
                              _arg(prob, "prob", _F32, r.E, d), _arg(loss, "loss", _F32, 1, d),
                              *_space(ws, d), _queue(stream, d)), "lrm_route")


def lrm_route_backward(router, logits, topk_idx, topk_w, counts, adot, dlogits, stream=None):
    lib = load_library()
    r, d = router, _device()
    _check(lib, lib.lrm_route_backward(
        ctypes.byref(r), _arg(logits, "logits", _elem(r.dtype), r.T * r.E, d, True),
        _arg(topk_idx, "topk_idx", _I32, r.T * r.k, d), _arg(topk_w, "topk_w", _F32, r.T * r.k, d),
        _arg(counts, "counts", _I32, r.E, d),
        _arg(adot, "adot", _F32, r.T * r.k, d), _arg(dlogits, "dlogits", _F32, r.T * r.E, d),
        _queue(stream, d)), "lrm_route_backward")


def lrm_gate_dots(problem, sel_pair, cmp_off, dphi, Phic, adot, ws, stream=None):
    lib = load_library()
    p, d = problem, _device()
    _check(lib, lib.lrm_gate_dots(
        ctypes.byref(p), _arg(sel_pair, "sel_pair", _I32, p.K_cap, d),
        _arg(cmp_off, "cmp_off", _I32, p.E_loc + 1, d), _arg(dphi, "dphi", _F32, p.K_cap * p.d, d),
        _arg(Phic, "Phic", _elem(p.dtype), p.K_cap * p.d, d), _arg(adot, "adot", _F32, p.T * p.k, d),
        *_space(ws, d), _queue(stream, d)), "lrm_gate_dots")


def lrm_grouped_fc1_swiglu(problem, row_pair, fwd_off, x, W1, ac, phi, ws, stream=None):
    """``ac`` None: the saved FC1 output is not kept (serving)."""
    lib = load_library()
    p, d = problem, _device()
    el = _elem(p.dtype)
    _check(lib, lib.lrm_grouped_fc1_swiglu(
        ctypes.byref(p), _arg(row_pair, "row_pair", _I32, p.L_cap, d),
        _arg(fwd_off, "fwd_off", _I32, p.E_loc + 1, d), _arg(x, "x", el, p.T * p.h, d),
        _arg(W1, "W1", el, p.E_loc * 2 * p.d * p.h, d), _arg(ac, "ac", el, p.L_cap * 2 * p.d, d),
        _arg(phi, "phi", el, p.L_cap * p.d, d), *_space(ws, d), _queue(stream, d)),
        "lrm_grouped_fc1_swiglu")


def _rows_of_y(p, y):
    """y's element type and whether a bf16 layer keeps it in float32 (the calls ending in _wide)."""
    wide = p.dtype == LRM_BF16 and getattr(y, "dtype", None) == torch.float32
    return (_F32 if wide else _elem(p.dtype)), wide


def lrm_grouped_fc2(problem, fwd_off, phi, W, y, ws, stream=None):
    """``y`` in the layer's type or in float32 (lrm_grouped_fc2_wide)."""
    lib = load_library()
    p, d = problem, _device()
    el, (ty, wide) = _elem(p.dtype), _rows_of_y(p, y)
    _check(lib, (lib.lrm_grouped_fc2_wide if wide else lib.lrm_grouped_fc2)(
        ctypes.byref(p), _arg(fwd_off, "fwd_off", _I32, p.E_loc + 1, d),
        _arg(phi, "phi", el, p.L_cap * p.d, d), _arg(W, "W", el, p.E_loc * p.h * p.d, d),
        _arg(y, "y", ty, p.L_cap * p.h, d), *_space(ws, d), _queue(stream, d)), "lrm_grouped_fc2")


def lrm_combine_tokens(problem, row_pair, fwd_off, topk_w, y, residual, out, ws, stream=None):
    """``residual`` None: the experts' output alone; ``out`` may be ``residual``; ``y`` in the layer's
    type or in float32 (lrm_combine_tokens_wide)."""
    lib = load_library()
    p, d = problem, _device()
    el, (ty, wide) = _elem(p.dtype), _rows_of_y(p, y)
    _check(lib, (lib.lrm_combine_tokens_wide if wide else lib.lrm_combine_tokens)(
        ctypes.byref(p), _arg(row_pair, "row_pair", _I32, p.L_cap, d),
        _arg(fwd_off, "fwd_off", _I32, p.E_loc + 1, d), _arg(topk_w, "topk_w", _F32, p.T * p.k, d),
        _arg(y, "y", ty, p.L_cap * p.h, d), _arg(residual, "residual", el, p.T * p.h, d),
        _arg(out, "out", el, p.T * p.h, d), *_space(ws, d), _queue(stream, d)), "lrm_combine_tokens")


class TensorList:
    """The (src, dst) tensors of lrm_grad_norm / lrm_clip_grads as the library's host array, made
    once and used for every step; it keeps the tensors alive."""

    def __init__(self, src, dst):
        self.src = list(src)
        self.dst = list(self.src if dst is None else dst)
        if len(self.src) != len(self.dst):
            raise LrmError(f"{len(self.src)} sources, {len(self.dst)} destinations")
        self.n = len(self.src)
        self.device = None
        self.array = (Tensor * max(1, self.n))()
        kinds = {torch.float32: LRM_F32, torch.bfloat16: LRM_BF16}
        for i, (a, b) in enumerate(zip(self.src, self.dst)):
            if a.dtype not in kinds or b.dtype != a.dtype:
                raise LrmError(f"tensor {i}: element types {a.dtype}, {b.dtype}: float32 or bfloat16, "
                               "the same for both")
            if a.device.type != "cuda":
                raise LrmError(f"tensor {i}: on {a.device}")
            if self.device is None:
                self.device = a.device.index
            n = a.numel()
            self.array[i] = Tensor(_arg(a, f"tensor {i}", (a.dtype,), n, self.device),
                                   _arg(b, f"destination {i}", (a.dtype,), n, self.device, True), n,
                                   kinds[a.dtype], 0)


def make_tensor_list(src, dst=None) -> TensorList:
    """float32 or bfloat16 tensors (contiguous, on one device) and where their clipped values go;
    ``dst`` None: in place."""
    return TensorList(src, dst)


def lrm_grad_workspace_bytes(tensors: TensorList) -> int:
    return int(load_library().lrm_grad_workspace_bytes(tensors.array, tensors.n))


def _on_device(tensors):
    d = _device()
    if tensors.device is not None and tensors.device != d:
        raise LrmError(f"tensors: on cuda:{tensors.device}, the call runs on cuda:{d}")
    return d


def lrm_grad_norm(tensors, norm, ws, stream=None):
    lib = load_library()
    d = _on_device(tensors)
    _check(lib, lib.lrm_grad_norm(tensors.array, tensors.n, _arg(norm, "norm", _F32, 1, d),
                                  *_space(ws, d), _queue(stream, d)), "lrm_grad_norm")


def lrm_clip_grads(tensors, max_norm, norm, ws, stream=None):
    lib = load_library()
    d = _on_device(tensors)
    _check(lib, lib.lrm_clip_grads(tensors.array, tensors.n, max_norm, _arg(norm, "norm", _F32, 1, d),
                                   *_space(ws, d), _queue(stream, d)), "lrm_clip_grads")


def lrm_read_device_error(ws, clear: bool = False, stream=None) -> int:
    lib = load_library()
    code = ctypes.c_int32(0)
    _check(lib, lib.lrm_read_device_error(_ptr(ws), ctypes.byref(code), int(clear),
                                          _stream(stream)), "lrm_read_device_error")
    return int(code.value)


def deverr_names(code: int):
    return [name for bit, name in DEVERR.items() if code & bit]

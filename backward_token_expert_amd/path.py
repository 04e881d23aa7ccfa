"""Device buffers and the call sequences of the hot path (marshalling only).

``DeviceBuffers`` allocates, with PyTorch, every output and the workspace of one problem; ``run``
enqueues lrm_plan_quotas -> lrm_score (or lrm_score_criterion) -> lrm_select -> lrm_compact ->
lrm_grouped_dw_dx (or lrm_grouped_dw -> lrm_grouped_dx) on one stream, or, given a second
stream, runs lrm_score_norms there beside lrm_plan_quotas and lrm_score_combine after both.
``LayerBuffers`` and ``run_layer`` do the same for the rest of the expert backward over the
retained rows:
lrm_swiglu_backward -> lrm_gather_tokens -> lrm_grouped_fc1_dw_dx (or the two FC1 calls) ->
lrm_scatter_tokens.

The layer's forward and what follows its backward have the same form: ``route`` over
``RouterBuffers`` (lrm_route), ``run_forward`` over ``ForwardBuffers`` (lrm_plan_quotas ->
lrm_grouped_fc1_swiglu -> lrm_grouped_fc2 -> lrm_combine_tokens), ``run_router_backward``
(lrm_gate_dots -> lrm_route_backward) and ``GradientClip`` (lrm_clip_grads over a fixed list of
gradients).  No step of the path is computed here.
"""
from __future__ import annotations

import numpy as np
import torch

from . import lrm


def storage_dtype(dtype: str):
    return torch.int16 if dtype == "bf16" else torch.float32


def to_device(a: np.ndarray, device="cuda") -> torch.Tensor:
    """Upload a host array; bf16 bit patterns (uint16) travel as int16."""
    if a.dtype == np.uint16:
        a = a.view(np.int16)
    return torch.from_numpy(np.ascontiguousarray(a)).to(device)


def to_host(t: torch.Tensor, bf16: bool = False) -> np.ndarray:
    a = t.detach().cpu().numpy()
    return a.view(np.uint16) if bf16 else a


class DeviceBuffers:
    """Outputs and workspace of one problem, sized to its capacities."""

    def __init__(self, problem: lrm.Problem, device="cuda"):
        p = problem
        i32 = dict(dtype=torch.int32, device=device)
        st = storage_dtype("bf16" if p.dtype == lrm.LRM_BF16 else "f32")
        self.problem = p
        self.counts = torch.zeros(p.E, **i32)
        self.fwd_off = torch.zeros(p.E_loc + 1, **i32)
        self.row_pair = torch.zeros(p.L_cap, **i32)
        self.quota = torch.zeros(p.E_loc, **i32)
        self.cmp_off = torch.zeros(p.E_loc + 1, **i32)
        self.admitted = torch.full((1,), -2, **i32)
        self.score = torch.zeros(p.L_cap, dtype=torch.float32, device=device)
        self.sel_row = torch.zeros(p.K_cap, **i32)
        self.sel_pair = torch.zeros(p.K_cap, **i32)
        self.Gc = torch.zeros((p.K_cap, p.h), dtype=st, device=device)
        self.Phic = torch.zeros((p.K_cap, p.d), dtype=st, device=device)
        self.dW = torch.zeros((p.E_loc, p.h, p.d), dtype=torch.float32, device=device)
        self.dphi = torch.zeros((p.K_cap, p.d), dtype=torch.float32, device=device)
        nws = lrm.lrm_workspace_bytes(p)
        if nws == 0:
            raise lrm.LrmError("invalid problem")
        self.ws = torch.zeros(nws, dtype=torch.uint8, device=device)


def _torch_stream(stream):
    if stream is None:
        return torch.cuda.current_stream()
    if isinstance(stream, int):
        return torch.cuda.ExternalStream(stream)
    return stream


def run(problem, policy, topk_idx, topk_w, g, phi, W, bufs: DeviceBuffers, stream=None,
        criterion: str = "lrm", keys=None, fused: bool = True, admission=None, side_stream=None):
    """Enqueue the whole hot path on `stream` (default: torch's current stream).  `criterion`
    picks the selection score (lrm_score for "lrm", else lrm_score_criterion; "random" ranks by
    `keys`, one float32 per pair).  `fused` runs both GEMMs as lrm_grouped_dw_dx, else as
    lrm_grouped_dw then lrm_grouped_dx.  With an `admission` (lrm.make_admission), the quotas are
    those of the first feasible candidate (lrm_admit_quotas after lrm_plan_quotas) and
    bufs.admitted receives its index (-1: none, every quota zero).  With a `side_stream` (LRM
    criterion only) the score's norm pass (lrm_score_norms) runs on it, forked from and joined back
    to `stream` with events, while lrm_plan_quotas runs on `stream`; the results are bitwise
    those of the one-stream sequence."""
    b = bufs
    split = criterion == "lrm" and side_stream is not None
    if split:
        main, side = _torch_stream(stream), _torch_stream(side_stream)
        fork, join = torch.cuda.Event(), torch.cuda.Event()
        fork.record(main)
        side.wait_event(fork)
        lrm.lrm_score_norms(problem, g, phi, b.ws, side)
        join.record(side)
    lrm.lrm_plan_quotas(problem, policy, topk_idx, b.counts, b.fwd_off, b.row_pair, b.quota,
                        b.cmp_off, b.ws, stream)
    if admission is not None:
        lrm.lrm_admit_quotas(problem, admission, b.fwd_off, b.quota, b.cmp_off, b.admitted, b.ws,
                             stream)
    if split:
        main.wait_event(join)
        lrm.lrm_score_combine(problem, topk_w, b.row_pair, b.fwd_off, b.score, b.ws, stream)
    elif criterion == "lrm":
        lrm.lrm_score(problem, topk_w, g, phi, b.row_pair, b.fwd_off, b.score, b.ws, stream)
    else:
        lrm.lrm_score_criterion(problem, criterion, topk_w, g, phi, keys, b.row_pair, b.fwd_off,
                                b.score, b.ws, stream)
    lrm.lrm_select(problem, b.score, b.fwd_off, b.quota, b.cmp_off, b.sel_row, b.ws, stream)
    lrm.lrm_compact(problem, b.sel_row, b.row_pair, b.cmp_off, topk_w, g, phi, b.Gc, b.Phic,
                    b.sel_pair, b.ws, stream)
    if fused:
        lrm.lrm_grouped_dw_dx(problem, b.Gc, b.Phic, W, b.cmp_off, b.dW, b.dphi, b.ws, stream)
    else:
        lrm.lrm_grouped_dw(problem, b.Gc, b.Phic, b.cmp_off, b.dW, b.ws, stream)
        lrm.lrm_grouped_dx(problem, b.Gc, W, b.cmp_off, b.dphi, b.ws, stream)


class LayerBuffers:
    """Outputs of the rest of the expert backward, sized to the problem's capacities."""

    def __init__(self, problem: lrm.Problem, device="cuda"):
        p = problem
        st = storage_dtype("bf16" if p.dtype == lrm.LRM_BF16 else "f32")
        f32 = dict(dtype=torch.float32, device=device)
        self.dH = torch.zeros((p.K_cap, 2 * p.d), dtype=st, device=device)
        self.Xc = torch.zeros((p.K_cap, p.h), dtype=st, device=device)
        self.dW1 = torch.zeros((p.E_loc, 2 * p.d, p.h), **f32)
        self.dX = torch.zeros((p.K_cap, p.h), **f32)
        self.dx = torch.zeros((p.T, p.h), **f32)


def run_layer(problem, ac, x, W1, bufs: DeviceBuffers, lay: LayerBuffers, stream=None,
              fused: bool = True):
    """Enqueue the rest of the expert backward after ``run`` on the same buffers: the activation's
    backward from dphi, FC1's input rows, the FC1 gradients and the return to the tokens."""
    b = bufs
    lrm.lrm_swiglu_backward(problem, b.sel_row, b.cmp_off, b.dphi, ac, lay.dH, b.ws, stream)
    lrm.lrm_gather_tokens(problem, b.sel_pair, b.cmp_off, x, lay.Xc, b.ws, stream)
    if fused:
        lrm.lrm_grouped_fc1_dw_dx(problem, lay.dH, lay.Xc, W1, b.cmp_off, lay.dW1, lay.dX, b.ws,
                                  stream)
    else:
        lrm.lrm_grouped_fc1_dw(problem, lay.dH, lay.Xc, b.cmp_off, lay.dW1, b.ws, stream)
        lrm.lrm_grouped_fc1_dx(problem, lay.dH, W1, b.cmp_off, lay.dX, b.ws, stream)
    lrm.lrm_scatter_tokens(problem, b.sel_pair, b.cmp_off, lay.dX, lay.dx, b.ws, stream)


class RouterBuffers:
    """Outputs and workspace of one router."""

    def __init__(self, router: lrm.Router, device="cuda"):
        r = router
        nws = lrm.lrm_router_workspace_bytes(r)
        if nws == 0:
            raise lrm.LrmError("invalid router")
        i32, f32 = dict(dtype=torch.int32, device=device), dict(dtype=torch.float32, device=device)
        self.topk_idx = torch.zeros(r.T * r.k, **i32)
        self.topk_w = torch.zeros(r.T * r.k, **f32)
        self.lse = torch.zeros(r.T, **f32)
        self.counts = torch.zeros(r.E, **i32)
        self.prob = torch.zeros(r.E, **f32)
        self.loss = torch.zeros(1, **f32)
        self.adot = torch.zeros(r.T * r.k, **f32)
        self.dlogits = torch.zeros((r.T, r.E), **f32)
        self.ws = torch.zeros(nws, dtype=torch.uint8, device=device)


def route(router, logits, rb: RouterBuffers, mask=None, stream=None):
    """Enqueue the routing of every token: choices, weights, counts and the balance loss."""
    lrm.lrm_route(router, logits, mask, rb.topk_idx, rb.topk_w, rb.lse, rb.counts, rb.prob, rb.loss,
                  rb.ws, stream)


class ForwardBuffers:
    """Outputs of the experts' forward, sized to the problem's capacities.  ``keep_ac`` False (serving):
    FC1's output is not kept for a backward.  ``wide_y``: a bf16 layer's expert outputs are kept in
    float32 on their way to the tokens, so that out is rounded once (see lrm_combine_tokens_wide)."""

    def __init__(self, problem: lrm.Problem, device="cuda", keep_ac: bool = True, wide_y: bool = False):
        p = problem
        st = storage_dtype("bf16" if p.dtype == lrm.LRM_BF16 else "f32")
        self.ac = torch.zeros((p.L_cap, 2 * p.d), dtype=st, device=device) if keep_ac else None
        self.phi = torch.zeros((p.L_cap, p.d), dtype=st, device=device)
        self.y = torch.zeros((p.L_cap, p.h), dtype=torch.float32 if wide_y else st, device=device)
        self.out = torch.zeros((p.T, p.h), dtype=st, device=device)


def run_forward(problem, policy, topk_idx, topk_w, x, W1, W, bufs: DeviceBuffers,
                fwd: ForwardBuffers, residual=None, stream=None):
    """Enqueue the experts' forward: the plan (counts, layout and the retention quotas that the
    backward over the same buffers keeps), FC1 with the activation, FC2, and the weighted sum back
    to the tokens.  ``fwd.phi`` and ``fwd.ac`` are then what ``run`` and ``run_layer`` take."""
    b = bufs
    lrm.lrm_plan_quotas(problem, policy, topk_idx, b.counts, b.fwd_off, b.row_pair, b.quota,
                        b.cmp_off, b.ws, stream)
    lrm.lrm_grouped_fc1_swiglu(problem, b.row_pair, b.fwd_off, x, W1, fwd.ac, fwd.phi, b.ws, stream)
    lrm.lrm_grouped_fc2(problem, b.fwd_off, fwd.phi, W, fwd.y, b.ws, stream)
    lrm.lrm_combine_tokens(problem, b.row_pair, b.fwd_off, topk_w, fwd.y, residual, fwd.out, b.ws,
                           stream)


def run_router_backward(problem, router, logits, bufs: DeviceBuffers, rb: RouterBuffers,
                        stream=None, balance: bool = True):
    """Enqueue the router's gradient after ``run`` on the same buffers: rb.dlogits holds that of the
    balance loss and of the retained pairs' gate weights.  Where a layer's experts are shared out and
    the shares' dlogits are summed, ``balance`` is True on one share alone: each holds the gate terms
    of its own pairs, but the balance loss of the whole layer."""
    lrm.lrm_gate_dots(problem, bufs.sel_pair, bufs.cmp_off, bufs.dphi, bufs.Phic, rb.adot, bufs.ws,
                      stream)
    if not balance:
        router = lrm.make_router(router.T, router.E, router.k, router.dtype, router.gate, 0.0)
    lrm.lrm_route_backward(router, logits, rb.topk_idx, rb.topk_w, rb.counts, rb.adot,
                           rb.dlogits, stream)


class GradientClip:
    """Clipping of a fixed list of gradients by their global norm, in place unless ``dst`` is given;
    the list, the norm and the workspace are kept between the steps."""

    def __init__(self, grads, dst=None):
        self.list = lrm.make_tensor_list(grads, dst)
        device = self.list.src[0].device if self.list.n else "cuda"
        nws = lrm.lrm_grad_workspace_bytes(self.list)
        if nws == 0:
            raise lrm.LrmError("invalid tensor list")
        self.norm = torch.zeros(1, dtype=torch.float32, device=device)
        self.ws = torch.zeros(nws, dtype=torch.uint8, device=device)

    def __call__(self, max_norm: float, stream=None) -> torch.Tensor:
        """Enqueue the clipping; the norm before it, a device tensor of one element."""
        lrm.lrm_clip_grads(self.list, max_norm, self.norm, self.ws, stream)
        return self.norm

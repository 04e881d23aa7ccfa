"""Refusals of the forward, router and clipping calls on the host (no GPU): every call below is
turned down before any launch, so its placeholder addresses are never used."""
import ctypes

import pytest
import torch

import backward_token_expert_amd as bte
from backward_token_expert_amd import lrm

FAKE = 0x100000


def _problem(**over):
    a = dict(T=4096, k=8, E=128, e_lo=0, E_loc=16, h=2048, d=768, dtype="bf16", L_cap=32768, K_cap=32768)
    a.update(over)
    return bte.make_problem(**a)


def test_struct_layouts():
    assert ctypes.sizeof(lrm.Router) == 24 and lrm.Router.balance_coef.offset == 20
    assert ctypes.sizeof(lrm.Tensor) == 32 and lrm.Tensor.dtype.offset == 24


def test_workspace_sizes():
    r = bte.make_router(4096, 128, 8)
    assert bte.lrm_router_workspace_bytes(r) >= 256 * 128 * 8
    p = _problem()
    n = bte.lrm_forward_workspace_bytes(p)
    assert 4096 * 8 * 4 + 256 <= n <= bte.lrm_workspace_bytes(p)
    assert bte.lrm_forward_workspace_bytes(_problem(h=60)) == 0
    for bad in (bte.make_router(0, 8, 2), bte.make_router(4, 8, 9), bte.make_router(4, 8, 0),
                bte.make_router(4, 5000, 2), bte.make_router(4, 8, 2, 7), bte.make_router(4, 8, 2, gate=2),
                bte.make_router(4, 8, 2, balance_coef=-1.0), bte.make_router(1 << 30, 8, 4),
                bte.make_router(4, 8, 2, balance_coef=float("nan")),
                bte.make_router(4, 8, 2, balance_coef=float("inf"))):
        assert bte.lrm_router_workspace_bytes(bad) == 0


def test_route_refusals():
    lib = bte.load_library()
    r = bte.make_router(64, 128, 8)
    R, n = ctypes.byref(r), bte.lrm_router_workspace_bytes(r)
    good = [FAKE] * 9
    for i in (0, 2, 3, 4, 5, 6, 7, 8):            # every pointer but the mask
        a = list(good)
        a[i] = None
        assert lib.lrm_route(R, *a, n, None) == 1, i
    assert lib.lrm_route(R, FAKE + 4, *good[1:], n, None) == 2
    assert lib.lrm_route(R, *good, n - 1, None) == 3
    assert lib.lrm_route(None, *good, n, None) == 1
    b = [FAKE] * 6
    for i in (0, 1, 2, 3, 5):                     # every pointer but adot
        a = list(b)
        a[i] = None
        assert lib.lrm_route_backward(R, *a, None) == 1, i
    assert lib.lrm_route_backward(R, *b[:5], FAKE + 4, None) == 2


def test_forward_refusals():
    lib = bte.load_library()
    p = _problem()
    P, n = ctypes.byref(p), bte.lrm_forward_workspace_bytes(p)
    for i in (0, 1, 2, 3, 5):                     # ac (4) may be NULL
        a = [FAKE] * 7
        a[i] = None
        assert lib.lrm_grouped_fc1_swiglu(P, *a, n, None) == 1, i
    for i in (2, 3, 4, 5):
        a = [FAKE] * 7
        a[i] += 8
        assert lib.lrm_grouped_fc1_swiglu(P, *a, n, None) == 2, i
    assert lib.lrm_grouped_fc1_swiglu(P, *[FAKE] * 7, n - 1, None) == 3
    assert lib.lrm_grouped_fc1_swiglu(P, *[FAKE] * 6, None, n, None) == 1
    # operands that 32-bit byte offsets do not reach: x of 2^31 + 2^16 bytes, one expert of 2^31 + ...
    big = _problem(T=2 ** 15 + 1, h=2 ** 15, k=1)
    assert lib.lrm_grouped_fc1_swiglu(ctypes.byref(big), *[FAKE] * 7, 1 << 40, None) == 2
    wide = _problem(T=16, h=2 ** 15, d=2 ** 15 + 8)
    assert lib.lrm_grouped_fc1_swiglu(ctypes.byref(wide), *[FAKE] * 7, 1 << 40, None) == 2
    assert lib.lrm_grouped_fc2(ctypes.byref(wide), *[FAKE] * 5, 1 << 40, None) == 2
    long_rows = _problem(T=16, h=8, d=2 ** 22 + 8)
    assert lib.lrm_grouped_fc2(ctypes.byref(long_rows), *[FAKE] * 5, 1 << 40, None) == 2
    for i in range(4):
        a = [FAKE] * 5
        a[i] = None
        assert lib.lrm_grouped_fc2(P, *a, n, None) == 1, i
    assert lib.lrm_grouped_fc2(P, FAKE, FAKE, FAKE, FAKE + 2, FAKE, n, None) == 2
    for i in (0, 1, 2, 3, 5):                     # residual (4) may be NULL
        a = [FAKE] * 7
        a[i] = None
        assert lib.lrm_combine_tokens(P, *a, n, None) == 1, i
    assert lib.lrm_combine_tokens(P, *[FAKE] * 4, FAKE + 4, FAKE, FAKE, n, None) == 2
    assert lib.lrm_combine_tokens(P, *[FAKE] * 7, 256, None) == 3
    for i in range(5):
        a = [FAKE] * 6
        a[i] = None
        assert lib.lrm_gate_dots(P, *a, n, None) == 1, i
    assert lib.lrm_gate_dots(P, FAKE, FAKE, FAKE + 4, FAKE, FAKE, FAKE, n, None) == 2


def _list(*entries):
    a = (lrm.Tensor * max(1, len(entries)))()
    for i, (src, dst, count, dtype) in enumerate(entries):
        a[i] = lrm.Tensor(src, dst, count, dtype, 0)
    return a, len(entries)


def _clip(entries, max_norm=1.0, ws=FAKE, n=1 << 30, norm=FAKE):
    a, m = _list(*entries)
    return bte.load_library().lrm_clip_grads(a, m, max_norm, norm, ws, n, None)


def test_clip_refusals():
    lib = bte.load_library()
    one = (0x200000, 0x300000, 16, 0)
    assert _clip([one], max_norm=0.0) == 1 and _clip([one], max_norm=-1.0) == 1
    assert _clip([one], max_norm=float("nan")) == 1 and _clip([one], max_norm=float("inf")) == 1
    assert _clip([one], norm=None) == 1 and _clip([one], ws=None) == 1
    assert _clip([one], ws=FAKE + 4) == 2 and _clip([one], n=256) == 3
    assert _clip([(None, 0x300000, 16, 0)]) == 1 and _clip([(0x200000, None, 16, 0)]) == 1
    assert _clip([(0x200000, 0x300000, -1, 0)]) == 1
    assert _clip([(0x200000, 0x300000, 16, 5)]) == 2
    assert _clip([(0x200002, 0x300000, 16, 0)]) == 2      # not aligned to its float32 elements
    assert _clip([(0x200001, 0x300000, 16, 1)]) == 2
    assert _clip([(0x200000, 0x300000, 1 << 46, 0)]) == 2
    # the same tensor twice; one entry's dst inside another's src; dst shifted against its own src
    assert _clip([(0x200000, 0x200000, 16, 0)] * 2) == 1
    assert _clip([one, (0x300020, 0x400000, 16, 0)]) == 1
    assert _clip([(0x200000, 0x200010, 16, 0)]) == 1
    assert _clip([one, (0x400000, 0x30003c, 16, 0)]) == 1  # the last element of the first dst
    # a long source that holds a later dst, behind another source
    assert _clip([(0x200000, 0x800000, 4096, 0), (0x200100, 0x900000, 4, 0), (0xA00000, 0x201000, 4, 0)]) == 1
    a, m = _list(one)
    assert lib.lrm_grad_norm(a, -1, FAKE, FAKE, 1 << 30, None) == 1
    assert lib.lrm_grad_norm(None, 1, FAKE, FAKE, 1 << 30, None) == 1
    assert lib.lrm_grad_norm(a, m, None, FAKE, 1 << 30, None) == 1
    assert lib.lrm_grad_norm(a, m, FAKE, FAKE, 256, None) == 3
    # two entries that only read one tensor pass the check of the list
    both, m = _list((0x200000, None, 16, 0), (0x200000, None, 16, 0))
    assert lib.lrm_grad_workspace_bytes(both, m) > 0
    a[0].reserved = 1
    assert lib.lrm_grad_workspace_bytes(a, 1) == 0


def test_binding_refuses_tensors_the_library_would_misread():
    r = bte.make_router(4, 8, 2)
    # host tensors: never passed on as device addresses
    for t, what in ((torch.zeros(4, 8, dtype=torch.float64), "element type"),
                    (torch.zeros(4, 7), "elements"), (torch.zeros(8, 4).t(), "contiguous"),
                    (torch.zeros(4, 8), "cpu")):
        with pytest.raises(lrm.LrmError, match=what):
            lrm._arg(t, "logits", (torch.float32,), 32, 0, True)
    with pytest.raises(lrm.LrmError, match="float32 or bfloat16"):
        bte.make_tensor_list([torch.zeros(4, dtype=torch.float16)])
    with pytest.raises(lrm.LrmError, match="destinations"):
        bte.make_tensor_list([torch.zeros(4)], [])
    with pytest.raises(lrm.LrmError, match="on cpu"):
        bte.make_tensor_list([torch.zeros(4)])
    assert r.gate == 0 and bte.make_router(4, 8, 2, gate="all").gate == 1

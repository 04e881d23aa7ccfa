"""Shares of a layer without any row: the forward calls and lrm_gate_dots with capacities of zero, whose
arrays of rows are empty (a torch tensor without elements has no address)."""
import ctypes

import pytest

import backward_token_expert_amd as bte
from backward_token_expert_amd import lrm

FAKE = 0x100000   # never used: every host call below is turned down before a launch


def _problem(L_cap, K_cap, dtype="bf16", T=64, k=2, E=8, E_loc=4, h=64, d=40):
    return bte.make_problem(T, k, E, 0, E_loc, h, d, dtype, L_cap, K_cap)


def test_capacities_of_zero_are_valid_and_need_no_rows():
    lib = bte.load_library()
    for caps in ((0, 0), (0, 5), (5, 0)):
        assert bte.lrm_forward_workspace_bytes(_problem(*caps)) > 0
    for caps in ((-1, 0), (0, -1)):
        assert bte.lrm_forward_workspace_bytes(_problem(*caps)) == 0
    none = ctypes.byref(_problem(0, 0))
    some = ctypes.byref(_problem(5, 5))
    # 3: everything before the workspace's size is accepted; 1: a pointer is missing
    calls = {
        "lrm_gate_dots": ([None, FAKE, None, None, FAKE], (0, 2, 3)),
        "lrm_grouped_fc1_swiglu": ([None, FAKE, FAKE, FAKE, None, None], (0, 5)),
        "lrm_grouped_fc2": ([FAKE, None, FAKE, None], (1, 3)),
        "lrm_combine_tokens": ([None, FAKE, FAKE, None, None, FAKE], (0, 3)),
    }
    for name, (args, rows) in calls.items():
        call = getattr(lib, name)
        assert call(none, *args, FAKE, 256, None) == 3, name
        given = [FAKE if a is None and i in rows else a for i, a in enumerate(args)]
        for i in rows:                            # with a capacity each is needed
            a = list(given)
            a[i] = None
            assert call(some, *a, FAKE, 256, None) == 1, (name, i)
        for i, a in enumerate(args):              # and the others always
            if a is not None:
                b = list(args)
                b[i] = None
                assert call(none, *b, FAKE, 256, None) == 1, (name, i)
    # the calls of the backward still need capacities
    assert bte.lrm_workspace_bytes(_problem(0, 0)) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,k", [(1, 2), (64, 2), (300, 70)])
def test_a_share_without_rows(T, k, dtype):
    import torch
    P = _problem(0, 0, dtype, T=T, k=k, E=max(8, k))
    t = torch.float32 if dtype == "f32" else torch.bfloat16

    def rows(n, *w, dt=t):
        return torch.full((n, *w), 3.0, dtype=dt, device="cuda")
    ws = torch.randint(0, 255, (lrm.lrm_forward_workspace_bytes(P),), dtype=torch.uint8, device="cuda")
    ws[:4] = 0
    off = torch.zeros(5, dtype=torch.int32, device="cuda")
    off[4] = 7                                    # more than the capacity: clamped
    pairs = torch.zeros(0, dtype=torch.int32, device="cuda")
    adot = rows(T * k, dt=torch.float32)
    lrm.lrm_gate_dots(P, pairs, off, rows(0, 40, dt=torch.float32), rows(0, 40), adot, ws)
    assert not adot.any()
    phi, y, out = rows(0, 40), rows(0, 64), rows(T, 64)
    lrm.lrm_grouped_fc1_swiglu(P, pairs, off, rows(T, 64), rows(4, 80, 64), rows(0, 80), phi, ws)
    lrm.lrm_grouped_fc1_swiglu(P, pairs, off, rows(T, 64), rows(4, 80, 64), None, phi, ws)
    lrm.lrm_grouped_fc2(P, off, phi, rows(4, 64, 40), y, ws)
    w = rows(T * k, dt=torch.float32)
    lrm.lrm_combine_tokens(P, pairs, off, w, y, None, out, ws)
    assert not out.any()
    residual = torch.randn(T, 64, device="cuda").to(t)
    lrm.lrm_combine_tokens(P, pairs, off, w, y, residual, out, ws)
    assert torch.equal(out, residual)
    assert lrm.lrm_read_device_error(ws) == 0

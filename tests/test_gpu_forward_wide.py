"""Expert outputs of a bf16 layer kept in float32 on their way to the tokens (lrm_grouped_fc2_wide,
lrm_combine_tokens_wide), against the float64 oracle.

With u = 2^-8, half a step of bf16 relative to the value, and S the sum of a product's absolute terms:
  y     d 2^-24 S (float32 accumulation; nothing is rounded to bf16)
  out   u |out| + sum |alpha| (error of y) + (k + 2) 2^-24 sum |terms|
The second bound does not hold a rounding of y to bf16, which adds u sum |alpha y|.
"""
import ctypes

import numpy as np
import pytest

import backward_token_expert_amd as bte
from oracle import forward_oracle as F
from tests.test_gpu_forward import CASES, IDS, Case, U32, _dev, _store

U = 2.0 ** -8


def bounds(c, phi64, residual):
    """The exact outputs and their bounds."""
    wy, size = F.fc2(phi64[:c.L], c.W64, c.off)
    ytol = c.d * U32 * size + 1e-37
    wout, terms = F.combine(wy, c.row_pair, c.w, c.T, c.k, c.res64 if residual else None)
    carried, _ = F.combine(ytol, c.row_pair, c.w, c.T, c.k)
    return wy, ytol, wout, U * np.abs(wout) + (carried + (c.k + 2) * U32 * (terms + carried)) * (1 + U) + 1e-37


def check(c, residual, wide=True, inplace=False):
    import torch
    from backward_token_expert_amd import lrm
    rng = np.random.default_rng(c.d)
    phi64, phi = _store(rng.normal(size=(c.L_cap, c.d)), c.dtype)
    phi[c.L:] = float("nan")
    rp, off = c.device_rows()
    y = torch.full((c.L_cap, c.h), 5.0, dtype=torch.float32 if wide else torch.bfloat16, device="cuda")
    lrm.lrm_grouped_fc2(c.P, off, phi, c.W, y, c.ws)
    res = c.res.clone() if residual else None
    out = res if inplace else c.rows(c.T, c.h, float("nan"))
    lrm.lrm_combine_tokens(c.P, rp, off, _dev(c.w), y, res, out, c.ws)
    torch.cuda.synchronize()
    assert lrm.lrm_read_device_error(c.ws) == 0
    wy, ytol, wout, tol = bounds(c, phi64, residual)
    g = y.double().cpu().numpy()
    assert np.all(g[c.L:] == 5.0)
    return np.all(np.abs(g[:c.L] - wy) <= ytol), np.all(np.abs(out.double().cpu().numpy() - wout) <= tol)


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_float32_rows_leave_out_its_own_rounding(case):
    print(f"[case] wide fc2 {case}", flush=True)
    c = Case(dtype="bf16", **case)
    assert check(c, residual=False) == (True, True)
    assert check(c, residual=True) == (True, True)
    assert check(c, residual=True, inplace=True) == (True, True)


@pytest.mark.gpu
def test_the_bound_tells_the_two_apart():
    """Rows in bf16 do not keep it, and float32 rows of a float32 layer are the plain call's."""
    import torch
    from backward_token_expert_amd import lrm
    c = Case(T=700, k=8, E=16, e_lo=0, E_loc=16, h=264, d=136, dtype="bf16")
    assert check(c, residual=False, wide=False) == (False, False)
    f = Case(T=90, k=2, E=4, e_lo=0, E_loc=4, h=64, d=40, dtype="f32")
    rp, off = f.device_rows()
    lib, P = bte.load_library(), ctypes.byref(f.P)
    phi, w = torch.randn(f.L_cap, f.d, device="cuda"), _dev(f.w)
    y, yw = f.rows(f.L_cap, f.h, 5.0), f.rows(f.L_cap, f.h, 5.0)
    out, ow = f.rows(f.T, f.h, 5.0), f.rows(f.T, f.h, 6.0)
    n, s = f.ws.numel(), torch.cuda.current_stream().cuda_stream
    lrm.lrm_grouped_fc2(f.P, off, phi, f.W, y, f.ws)
    lrm.lrm_combine_tokens(f.P, rp, off, w, y, f.res, out, f.ws)
    assert lib.lrm_grouped_fc2_wide(P, off.data_ptr(), phi.data_ptr(), f.W.data_ptr(), yw.data_ptr(),
                                    f.ws.data_ptr(), n, s) == 0
    assert lib.lrm_combine_tokens_wide(P, rp.data_ptr(), off.data_ptr(), w.data_ptr(), yw.data_ptr(),
                                       f.res.data_ptr(), ow.data_ptr(), f.ws.data_ptr(), n, s) == 0
    assert torch.equal(y, yw) and torch.equal(out, ow)


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,E", [(3000, 3, 8), (40, 70, 70)])
def test_wide_sequence_in_a_graph(T, k, E):
    """path.run_forward with float32 rows, captured and replayed on other inputs: the eager results, and
    those within the bound; with a plan that leaves room behind the last row."""
    import torch
    from backward_token_expert_amd import lrm, path
    c = Case(T=T, k=k, E=E, e_lo=0, E_loc=E, h=136, d=72, dtype="bf16", spare=0)
    c.P = lrm.make_problem(T, k, E, 0, E, 136, 72, "bf16", T * k + 9, T * k + 9)
    bufs, fwd, eager = path.DeviceBuffers(c.P), *[path.ForwardBuffers(c.P, wide_y=True) for _ in range(2)]
    assert fwd.y.dtype == torch.float32
    idx, w, x, full = _dev(c.idx), _dev(c.w), c.x.clone(), lrm.make_policy(1)
    path.run_forward(c.P, full, idx, w, x, c.W1, c.W, bufs, fwd, c.res)
    torch.cuda.synchronize()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        path.run_forward(c.P, full, idx, w, x, c.W1, c.W, bufs, fwd, c.res)
    for scale in (1.0, 0.5, 1.0):
        x.copy_(c.x * scale)
        graph.replay()
        torch.cuda.synchronize()
        other = path.DeviceBuffers(c.P)
        path.run_forward(c.P, full, idx, w, x, c.W1, c.W, other, eager, c.res)
        torch.cuda.synchronize()
        assert lrm.lrm_read_device_error(bufs.ws) == 0
        assert torch.equal(fwd.y[:c.L], eager.y[:c.L]) and torch.equal(fwd.out, eager.out)
        assert not fwd.y[c.L:].any()
        # the buffers hold bf16 as bit patterns
        phi64, out = [t.view(torch.bfloat16).double().cpu().numpy() for t in (fwd.phi, fwd.out)]
        _, _, wout, tol = bounds(c, phi64, True)
        assert np.all(np.abs(out - wout) <= tol)


def test_refusals():
    lib, fake = bte.load_library(), 0x100000      # turned down before any launch
    p = bte.make_problem(4096, 8, 128, 0, 16, 2048, 768, "bf16", 32768, 32768)
    P, n = ctypes.byref(p), bte.lrm_forward_workspace_bytes(p)
    for i in range(4):
        a = [fake] * 5
        a[i] = None
        assert lib.lrm_grouped_fc2_wide(P, *a, n, None) == 1, i
    assert lib.lrm_grouped_fc2_wide(P, fake, fake, fake, fake + 4, fake, n, None) == 2
    assert lib.lrm_grouped_fc2_wide(P, *[fake] * 5, n - 1, None) == 3
    for i in (0, 1, 2, 3, 5):                     # residual (4) may be NULL
        a = [fake] * 7
        a[i] = None
        assert lib.lrm_combine_tokens_wide(P, *a, n, None) == 1, i
    assert lib.lrm_combine_tokens_wide(P, *[fake] * 3, fake + 4, fake, fake, fake, n, None) == 2
    assert lib.lrm_combine_tokens_wide(P, *[fake] * 7, 256, None) == 3

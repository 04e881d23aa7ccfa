"""The router's gradient of a layer whose experts are shared out: the shares' dlogits, with the balance
loss in one of them, sum to the whole layer's."""
import numpy as np
import pytest

from tests.test_gpu_forward import Case, _dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gate", ["topk", "all"])
def test_shares_sum_to_the_layer(gate):
    """float32 rows: the shares' products are the layer's row by row, so the sums differ by roundings of
    the terms' float32 additions, at most 8 of 2^-24 of the terms' magnitudes (three terms a share)."""
    import torch
    from backward_token_expert_amd import lrm, path
    T, k, E, h, d, coef, shares = 200, 3, 12, 64, 48, 5.0, 3
    c = Case(T=T, k=k, E=E, e_lo=0, E_loc=E, h=h, d=d, dtype="f32", spare=0)
    rng = np.random.default_rng(4)
    logits = _dev(rng.normal(size=(T, E)).astype(np.float32))
    g = _dev(rng.normal(size=(T, h)).astype(np.float32))
    router, full = lrm.make_router(T, E, k, "f32", gate, coef), lrm.make_policy(1)

    def dlogits(e_lo, n, balance):
        P = lrm.make_problem(T, k, E, e_lo, n, h, d, "f32", T * k, T * k)
        rb, bufs, fwd = path.RouterBuffers(router), path.DeviceBuffers(P), path.ForwardBuffers(P)
        W1, W = c.W1[e_lo:e_lo + n].contiguous(), c.W[e_lo:e_lo + n].contiguous()
        path.route(router, logits, rb)
        path.run_forward(P, full, rb.topk_idx, rb.topk_w, c.x, W1, W, bufs, fwd)
        path.run(P, full, rb.topk_idx, rb.topk_w, g, fwd.phi, W, bufs)
        path.run_router_backward(P, router, logits, bufs, rb, balance=balance)
        torch.cuda.synchronize()
        assert lrm.lrm_read_device_error(bufs.ws) == 0
        return rb.dlogits.double(), rb.adot.double()
    whole, adot = dlogits(0, E, True)
    only_gate, _ = dlogits(0, E, False)
    n = E // shares
    parts = [dlogits(i * n, n, i == 1) for i in range(shares)]
    assert torch.equal(sum(a for _, a in parts), adot)          # every pair is in one share
    got = sum(p for p, _ in parts)
    scale = adot.reshape(T, k).abs().sum(1, keepdim=True) * 2 + (whole - only_gate).abs()
    assert bool(((got - whole).abs() <= 3 * 8 * 2.0 ** -24 * scale + 1e-37).all())
    # counted in every share, the balance loss would be there three times
    many = sum(dlogits(i * n, n, True)[0] for i in range(shares))
    assert bool(((many - whole - 2 * (whole - only_gate)).abs() <= 64 * 2.0 ** -24 * scale + 1e-37).all())
    assert float((many - whole).norm()) > float((got - whole).norm()) * 1e3

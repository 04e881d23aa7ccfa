"""The router on the GPU (lrm_route, lrm_route_backward, lrm_gate_dots) against the float64 oracle.

Whole numbers are exact.  Floating bounds, all from half a step of float32 (2^-24) per rounding:
  weights     an exponential of v - m carries |v - m| 2^-24 from its argument and a few steps of its
              own, a sum of positives its length's: |ln w| + 64 steps of 2^-23
  lse         (|m| + |lse| + 64) 2^-24
  prob, loss  sums of at most T non-negative float32: (T + 128) 2^-24 relative, worst case
  dlogits     the sum of its terms' magnitudes (the oracle gives it) times the relative error of a
              probability, (|ln p| + 128) 2^-23
  adot        float64 products and sums, one rounding: 2^-24 |adot| + 2^-45 sum |terms|
"""
import numpy as np
import pytest

import oracle as O
from oracle import forward_oracle as F

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def make_logits(T, E, seed, dtype, closed=0, ties=False):
    """float64 logits exact in `dtype`, and the device tensor."""
    import torch
    z = np.random.default_rng(seed).normal(size=(T, E)) * 2 - 1.2 * np.log(np.arange(1, E + 1))
    if ties:
        z = np.round(z * 2) / 2
    if closed:
        z[:, E - closed:] = -np.inf
    t = torch.from_numpy(z).to(torch.float32 if dtype == "f32" else torch.bfloat16)
    return t.double().numpy(), t.cuda()


def run_route(router, logits, mask=None):
    import torch
    from backward_token_expert_amd import lrm, path
    rb = path.RouterBuffers(router)
    rb.ws.random_()          # the workspace may hold anything
    path.route(router, logits, rb, None if mask is None else _dev(mask.astype(np.uint8)))
    torch.cuda.synchronize()
    return rb, lrm.lrm_read_device_error(rb.ws)


def check_route(rb, want, T):
    got = {n: getattr(rb, n).cpu().numpy() for n in ("topk_idx", "topk_w", "lse", "counts", "prob", "loss")}
    np.testing.assert_array_equal(got["topk_idx"], want["topk_idx"])
    np.testing.assert_array_equal(got["counts"], want["counts"])
    w = want["topk_w"]
    with np.errstate(divide="ignore"):
        tol = np.where(w > 1e-37, w * (np.abs(np.log(np.maximum(w, 1e-300))) + 64) * 2 * U, 1e-37)
    assert np.all(np.abs(got["topk_w"] - w) <= tol)
    m = np.abs(want["lse"])
    assert np.all(np.abs(got["lse"] - want["lse"]) <= (2 * m + 80) * U)
    assert np.all(np.abs(got["prob"] - want["prob"]) <= want["prob"] * (T + 256) * U + 1e-37)
    assert abs(got["loss"][0] - want["loss"]) <= want["loss"] * (T + 256) * U + 1e-37


# (T, E, k): one token, one expert, every expert chosen, odd sizes, more choices than a fast path
# may keep, the widest table, rows that are not 16-byte aligned, a large batch
SHAPES = [(1, 128, 8), (1, 1, 1), (3, 5, 5), (64, 8, 2), (65, 7, 3), (333, 60, 6), (1021, 128, 8),
          (100, 131, 9), (77, 160, 6), (50, 256, 16), (40, 300, 40), (33, 512, 8), (20, 1000, 22),
          (9, 2047, 4), (5, 4096, 12), (6, 4096, 40), (4096, 128, 8), (4097, 128, 2), (5000, 64, 4),
          (9001, 128, 16), (2100, 250, 8)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_route_and_backward(T, E, k, dtype):
    import torch
    from backward_token_expert_amd import lrm
    for gate, masked, closed in (("topk", False, 0), ("all", True, min(2, E // 4))):
        print(f"[case] route T={T} E={E} k={k} {dtype} {gate} masked={masked}", flush=True)
        z, logits = make_logits(T, E, T + E, dtype, closed, ties=dtype == "bf16")
        mask = np.random.default_rng(E).random(T) < 0.7 if masked else None
        coef = 0.37
        router = lrm.make_router(T, E, k, dtype, gate, coef)
        rb, err = run_route(router, logits, mask)
        assert err == 0
        want = F.route(z, k, gate, coef, mask)
        check_route(rb, want, T)
        adot = np.random.default_rng(k).normal(size=T * k).astype(np.float32)
        for a in (adot, None):
            out = torch.full((T, E), float("nan"), device="cuda")
            lrm.lrm_route_backward(router, logits, rb.topk_idx, rb.topk_w, rb.counts,
                                   None if a is None else _dev(a), out)
            d, size = F.route_backward(want, k, gate, coef, a)
            with np.errstate(divide="ignore"):
                lnp = np.where(want["p"] > 1e-37, np.abs(np.log(np.maximum(want["p"], 1e-300))), 0)
            got = out.cpu().numpy()
            assert np.all(np.abs(got - d) <= size * (lnp + 128 + 2 * k) * 2 * U + 1e-37), gate


def test_rows_that_leave_nothing():
    """Masked tokens, rows of -infinity, rows with fewer finite logits than choices, equal logits,
    both zeros, the type's lowest value; then no valid token at all."""
    from backward_token_expert_amd import lrm
    T, E, k = 12, 20, 4
    z = np.random.default_rng(5).normal(size=(T, E)).astype(np.float32)
    z[1] = -np.inf
    z[2, 2:] = -np.inf                                   # two finite logits, four choices
    z[3] = 0.25                                          # all equal: experts 0..3
    z[4] = 0.0
    z[4, ::2] = -0.0                                     # equal logits
    z[5] = np.finfo(np.float32).min
    z[6, :] = np.finfo(np.float32).min
    z[6, 7] = np.finfo(np.float32).max
    z[7] = 1e-42                                         # subnormal, equal
    z[7, 9] = 2e-42
    mask = np.ones(T, bool)
    mask[8] = False
    z[8] = np.nan                                        # masked: never looked at
    for gate in ("topk", "all"):
        router = lrm.make_router(T, E, k, "f32", gate, 1.0)
        rb, err = run_route(router, _dev(z), mask)
        assert err == 0
        zz = z.astype(np.float64)
        zz[8] = 0.0
        want = F.route(zz, k, gate, 1.0, mask)
        check_route(rb, want, T)
        idx = rb.topk_idx.cpu().numpy().reshape(T, k)
        assert list(idx[1]) == list(idx[8]) == [-1] * 4
        assert list(idx[3]) == list(idx[4]) == list(idx[5]) == [0, 1, 2, 3] and idx[7][0] == 9
        out = _dev(np.full((T, E), 7.0, np.float32))
        lrm.lrm_route_backward(router, _dev(z), rb.topk_idx, rb.topk_w, rb.counts, rb.topk_w, out)
        o = out.cpu().numpy()
        assert not o[1].any() and not o[8].any() and np.isfinite(o).all()
        none = np.zeros(T, bool)
        rb, err = run_route(router, _dev(z), none)
        assert err == 0 and rb.loss.item() == 0 and not rb.prob.any() and not rb.counts.any()
        assert (rb.topk_idx == -1).all() and not rb.topk_w.any()
        lrm.lrm_route_backward(router, _dev(z), rb.topk_idx, rb.topk_w, rb.counts, None, out)
        assert not out.any()


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_nonfinite_logits_are_reported_and_stay_in_their_row(value):
    from backward_token_expert_amd import lrm
    T, E, k = 40, 128, 8
    z, logits = make_logits(T, E, 3, "f32")
    logits[7, 5] = value
    rb, err = run_route(lrm.make_router(T, E, k), logits)
    assert err == 16
    idx = rb.topk_idx.cpu().numpy().reshape(T, k)
    assert np.all((idx >= 0) & (idx < E)) and all(len(set(r)) == k for r in idx)
    want = F.route(z, k)
    other = np.arange(T) != 7
    np.testing.assert_array_equal(idx[other], want["topk_idx"].reshape(T, k)[other])
    w = rb.topk_w.cpu().numpy().reshape(T, k)[other]
    assert np.allclose(w, want["topk_w"].reshape(T, k)[other], rtol=1e-5)
    rb, err = run_route(lrm.make_router(T, E, k), make_logits(T, E, 3, "f32")[1])
    assert err == 0                                       # the word is the call's own


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,k,K,d", [(1, 1, 1, 8), (5, 2, 7, 24), (300, 8, 700, 200), (64, 4, 0, 64),
                                     (1000, 8, 4001, 768), (17, 3, 51, 1032)])
def test_gate_dots(T, k, K, d, dtype):
    import torch
    from backward_token_expert_amd import lrm
    rng = np.random.default_rng(d)
    K_cap = K + 3
    P = lrm.make_problem(T, k, 8, 0, 8, 8, d, dtype, K_cap, K_cap)
    sel = rng.permutation(T * k)[:K].astype(np.int32)
    dphi = rng.normal(size=(K_cap, d)).astype(np.float32)
    phi = torch.from_numpy(rng.normal(size=(K_cap, d))).to(torch.float32 if dtype == "f32" else torch.bfloat16)
    dphi[K:] = np.nan                                     # the capacity's rows are not read
    off = np.zeros(9, np.int32)
    off[3:] = K
    ws = torch.randint(0, 255, (lrm.lrm_forward_workspace_bytes(P),), dtype=torch.uint8, device="cuda")
    ws[:4] = 0
    adot = torch.full((T * k,), 9.0, device="cuda")
    pad = np.concatenate([sel, np.full(3, -5, np.int32)])
    lrm.lrm_gate_dots(P, _dev(pad), _dev(off), _dev(dphi), phi.cuda(), adot, ws)
    assert lrm.lrm_read_device_error(ws) == 0
    want, size = F.gate_dots(dphi[:K].astype(np.float64), phi[:K].double().numpy(), sel, T * k)
    got = adot.cpu().numpy()
    assert np.all(np.abs(got - want) <= U * np.abs(want) + 2.0 ** -45 * size)
    if K >= 2:
        bad = pad.copy()
        bad[1] = bad[0]                                   # two rows name one pair
        lrm.lrm_gate_dots(P, _dev(bad), _dev(off), _dev(dphi), phi.cuda(), adot, ws)
        assert lrm.lrm_read_device_error(ws, clear=True) == 32
        bad[1] = T * k                                    # out of range
        lrm.lrm_gate_dots(P, _dev(bad), _dev(off), _dev(dphi), phi.cuda(), adot, ws)
        assert lrm.lrm_read_device_error(ws, clear=True) == 32


def test_route_repeats_bit_for_bit_and_in_a_graph():
    import torch
    from backward_token_expert_amd import lrm, path
    T, E, k = 3000, 128, 8
    _, logits = make_logits(T, E, 9, "f32")
    router = lrm.make_router(T, E, k, balance_coef=0.01)
    rb, _ = run_route(router, logits)
    first = [getattr(rb, n).clone() for n in ("topk_idx", "topk_w", "lse", "counts", "prob", "loss")]
    buf = path.RouterBuffers(router)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    static = logits.clone()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        path.route(router, static, buf)
        lrm.lrm_route_backward(router, static, buf.topk_idx, buf.topk_w, buf.counts, buf.topk_w,
                               buf.dlogits)
    for rep in range(3):
        static.copy_(logits if rep != 1 else logits.flip(0))
        g.replay()
        torch.cuda.synchronize()
        if rep != 1:
            for n, f in zip(("topk_idx", "topk_w", "lse", "counts", "prob", "loss"), first):
                assert torch.equal(getattr(buf, n), f), n
        eager, _ = run_route(router, static)
        assert torch.equal(eager.topk_w, buf.topk_w) and torch.equal(eager.loss, buf.loss)

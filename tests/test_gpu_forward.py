"""The experts' forward on the GPU (lrm_grouped_fc1_swiglu, lrm_grouped_fc2, lrm_combine_tokens)
against the float64 oracle, and one whole training and serving step of a layer.

With u = half a step of the output type (bf16 2^-8, float32 2^-24) and S the sum of a product's
absolute terms, a float32 accumulation of n terms is off by at most n 2^-24 S, so
  ac, y   u |v| + n 2^-24 S
  phi     u |phi| + 1.1 |c| da + |SiLU(a)| dc + 2^-20 |phi|   (|SiLU'| <= 1.1; da, dc the
          accumulations' parts above; the last term the exponential's and the division's steps)
  out     u |out| + sum |alpha| (error of y) + (k + 2) 2^-24 sum |terms|
"""
import numpy as np
import pytest

import oracle as O
from oracle import forward_oracle as F

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24


def _dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _half(dtype):
    return U32 if dtype == "f32" else 2.0 ** -8


def _store(v, dtype):
    """Rounded to the storage type: the exact float64 values, and the device tensor."""
    import torch
    t = torch.from_numpy(np.asarray(v)).to(torch.float32 if dtype == "f32" else torch.bfloat16)
    return t.double().numpy(), t.cuda()


class Case:
    """Inputs of one layer: idx [T, k] picks experts by `skew` (a share per global expert)."""

    def __init__(self, T, k, E, e_lo, E_loc, h, d, dtype, skew=None, seed=0, spare=5):
        from backward_token_expert_amd import lrm
        rng = np.random.default_rng(seed + T + h)
        self.T, self.k, self.E, self.e_lo, self.E_loc, self.h, self.d, self.dtype = T, k, E, e_lo, E_loc, h, d, dtype
        score = rng.gumbel(size=(T, E)) + (0 if skew is None else np.log(np.asarray(skew) + 1e-30))
        self.idx = np.argsort(-score, axis=1, kind="stable")[:, :k].astype(np.int32).reshape(-1)
        self.w = rng.uniform(0.05, 1.0, T * k).astype(np.float32)
        self.row_pair, self.off, self.L = self._layout()
        self.L_cap = self.L + spare
        self.x64, self.x = _store(rng.normal(size=(T, h)), dtype)
        local = np.zeros(T, bool)
        local[self.row_pair[:self.L] // k] = True
        if not local.all():                       # tokens of other ranks' experts are never read
            self.x[_dev(~local)] = float("nan")
        self.W164, self.W1 = _store(rng.normal(size=(E_loc, 2 * d, h)) / np.sqrt(h), dtype)
        self.W64, self.W = _store(rng.normal(size=(E_loc, h, d)) / np.sqrt(d), dtype)
        self.res64, self.res = _store(rng.normal(size=(T, h)), dtype)
        self.P = lrm.make_problem(T, k, E, e_lo, E_loc, h, d, dtype, self.L_cap, self.L_cap)
        import torch
        self.ws = torch.randint(0, 255, (lrm.lrm_forward_workspace_bytes(self.P),), dtype=torch.uint8, device="cuda")
        self.ws[:4] = 0

    def _layout(self):
        loc = self.idx - self.e_lo
        pairs = np.flatnonzero((loc >= 0) & (loc < self.E_loc))
        pairs = pairs[np.argsort(loc[pairs], kind="stable")]
        off = np.concatenate([[0], np.cumsum(np.bincount(loc[pairs], minlength=self.E_loc))])
        return pairs.astype(np.int32), off.astype(np.int32), len(pairs)

    def rows(self, n, width, fill):
        import torch
        return torch.full((n, width), fill, dtype=torch.float32 if self.dtype == "f32" else torch.bfloat16,
                          device="cuda")

    def device_rows(self):
        pad = np.full(self.L_cap, -7, np.int32)   # past the last row: never looked at
        pad[:self.L] = self.row_pair
        return _dev(pad), _dev(self.off)


def check_fc1(c, keep_ac=True):
    import torch
    from backward_token_expert_amd import lrm
    rp, off = c.device_rows()
    ac = c.rows(c.L_cap, 2 * c.d, 5.0) if keep_ac else None
    phi = c.rows(c.L_cap, c.d, 6.0)
    lrm.lrm_grouped_fc1_swiglu(c.P, rp, off, c.x, c.W1, ac, phi, c.ws)
    torch.cuda.synchronize()
    assert lrm.lrm_read_device_error(c.ws) == 0
    wac, wphi, size = F.fc1_swiglu(c.x64, c.W164, c.row_pair, c.off, c.k)
    u, acc = _half(c.dtype), c.h * U32 * size
    got = phi.double().cpu().numpy()
    a, b = wac[:, :c.d], wac[:, c.d:]
    silu = np.abs(a / (1 + np.exp(-a)))
    tol = u * np.abs(wphi) + 1.1 * np.abs(b) * acc[:, :c.d] + (silu + acc[:, :c.d]) * acc[:, c.d:] + \
        2.0 ** -20 * np.abs(wphi) + 1e-37
    assert np.all(np.abs(got[:c.L] - wphi) <= tol * (1 + u))
    assert np.all(got[c.L:] == 6.0)
    if keep_ac:
        g = ac.double().cpu().numpy()
        assert np.all(np.abs(g[:c.L] - wac) <= (u * np.abs(wac) + acc) * (1 + u) + 1e-37)
        assert np.all(g[c.L:] == 5.0)
    return phi, ac


def check_fc2(c, residual, inplace=False):
    import torch
    from backward_token_expert_amd import lrm
    rng = np.random.default_rng(c.d)
    phi64, phi = _store(rng.normal(size=(c.L_cap, c.d)), c.dtype)
    phi[c.L:] = float("nan")
    rp, off = c.device_rows()
    y = c.rows(c.L_cap, c.h, 5.0)
    lrm.lrm_grouped_fc2(c.P, off, phi, c.W, y, c.ws)
    res = c.res.clone() if residual else None
    out = res if inplace else c.rows(c.T, c.h, float("nan"))
    lrm.lrm_combine_tokens(c.P, rp, off, _dev(c.w), y, res, out, c.ws)
    torch.cuda.synchronize()
    assert lrm.lrm_read_device_error(c.ws) == 0
    wy, size = F.fc2(phi64[:c.L], c.W64, c.off)
    u = _half(c.dtype)
    ytol = (u * np.abs(wy) + c.d * U32 * size) * (1 + u) + 1e-37
    g = y.double().cpu().numpy()
    assert np.all(np.abs(g[:c.L] - wy) <= ytol)
    assert np.all(g[c.L:] == 5.0)
    wout, terms = F.combine(wy, c.row_pair, c.w, c.T, c.k, c.res64 if residual else None)
    carried, _ = F.combine(ytol, c.row_pair, c.w, c.T, c.k)
    tol = (u * np.abs(wout) + carried + (c.k + 2) * U32 * (terms + carried)) * (1 + u) + 1e-37
    assert np.all(np.abs(out.double().cpu().numpy() - wout) <= tol)


# one token and one expert; odd widths; local experts in the middle; empty experts; all rows on one
# expert; tiles that end inside an expert and inside a row of columns; more rows than one tile
CASES = [
    dict(T=1, k=1, E=1, e_lo=0, E_loc=1, h=8, d=8),
    dict(T=1, k=8, E=16, e_lo=0, E_loc=16, h=128, d=72),
    dict(T=3, k=2, E=6, e_lo=2, E_loc=3, h=40, d=24),
    dict(T=33, k=4, E=8, e_lo=0, E_loc=8, h=264, d=136),
    dict(T=65, k=1, E=4, e_lo=1, E_loc=2, h=72, d=520),
    dict(T=257, k=2, E=8, e_lo=0, E_loc=8, h=512, d=200, skew=[1, 0, 1, 0, 0, 1, 9, 1]),
    dict(T=700, k=3, E=12, e_lo=3, E_loc=7, h=136, d=264),
    dict(T=1000, k=1, E=3, e_lo=0, E_loc=3, h=256, d=128, skew=[0, 1, 0]),
    dict(T=2050, k=2, E=4, e_lo=0, E_loc=2, h=320, d=392),
    dict(T=40, k=2, E=140, e_lo=0, E_loc=140, h=64, d=64),
    dict(T=17, k=8, E=1024, e_lo=0, E_loc=1024, h=32, d=16),
    dict(T=5, k=2, E=64, e_lo=32, E_loc=4, h=1032, d=1048),
    # more units than workgroups, for every tile shape, with one, two and three steps of a unit (the
    # loads run ahead over one unit's end, or over several units), and FC2's mirror images
    dict(T=20000, k=1, E=2, e_lo=0, E_loc=2, h=8, d=1024),
    dict(T=20000, k=1, E=2, e_lo=0, E_loc=2, h=1024, d=8),
    dict(T=9000, k=2, E=70, e_lo=0, E_loc=70, h=136, d=512),
    dict(T=8000, k=2, E=100, e_lo=0, E_loc=100, h=8, d=1024),
    dict(T=8000, k=2, E=100, e_lo=0, E_loc=100, h=1024, d=72),
    dict(T=3000, k=2, E=300, e_lo=0, E_loc=300, h=72, d=1024),
    dict(T=3000, k=2, E=300, e_lo=0, E_loc=300, h=1032, d=16),
    dict(T=100, k=1, E=2, e_lo=0, E_loc=2, h=8, d=8),
]
IDS = ["T%dk%dE%d-%dh%dd%d" % (c["T"], c["k"], c["E"], c["E_loc"], c["h"], c["d"]) for c in CASES]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_fc1_swiglu(case, dtype):
    print(f"[case] fc1 {case} {dtype}", flush=True)
    c = Case(dtype=dtype, **case)
    phi, _ = check_fc1(c)
    phi2, _ = check_fc1(c, keep_ac=False)
    assert (phi[:c.L] == phi2[:c.L]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_fc2_and_combine(case, dtype):
    print(f"[case] fc2 {case} {dtype}", flush=True)
    c = Case(dtype=dtype, **case)
    check_fc2(c, residual=False)
    check_fc2(c, residual=True)
    check_fc2(c, residual=True, inplace=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_no_rows_at_all(dtype):
    """No token has a local expert: nothing but the residual is written."""
    import torch
    from backward_token_expert_amd import lrm
    c = Case(T=9, k=2, E=8, e_lo=6, E_loc=2, h=64, d=40, dtype=dtype, skew=[1, 1, 1, 1, 0, 0, 0, 0])
    assert c.L == 0
    check_fc1(c)
    check_fc2(c, residual=True)
    check_fc2(c, residual=False)


def test_rows_of_a_token_with_nan_stay_its_own():
    """NaN and infinity in one token's input reach that token's rows alone, also where rows share a
    tile and where the contracted width ends inside a step."""
    import torch
    from backward_token_expert_amd import lrm
    for dtype in ("f32", "bf16"):
        c = Case(T=70, k=2, E=2, e_lo=0, E_loc=2, h=40, d=24, dtype=dtype)
        rp, off = c.device_rows()
        good, ac = c.rows(c.L_cap, c.d, 0.0), c.rows(c.L_cap, 2 * c.d, 0.0)
        lrm.lrm_grouped_fc1_swiglu(c.P, rp, off, c.x, c.W1, ac, good, c.ws)
        x = c.x.clone()
        x[11] = float("nan")
        x[50, 39] = float("inf")
        phi = c.rows(c.L_cap, c.d, 0.0)
        lrm.lrm_grouped_fc1_swiglu(c.P, rp, off, x, c.W1, None, phi, c.ws)
        tok = c.row_pair // c.k
        clean = _dev(~np.isin(tok, (11, 50)))
        assert torch.equal(phi[:c.L][clean], good[:c.L][clean])
        assert not torch.isfinite(phi[:c.L][_dev(tok == 11)]).any()


def test_bad_rows_are_reported():
    import torch
    from backward_token_expert_amd import lrm
    c = Case(T=50, k=2, E=4, e_lo=0, E_loc=4, h=64, d=32, dtype="bf16")
    rp, off = c.device_rows()
    for value in (-1, 100, 2 ** 31 - 1):
        bad = rp.clone()
        bad[3] = value
        phi = c.rows(c.L_cap, c.d, 0.0)
        lrm.lrm_grouped_fc1_swiglu(c.P, bad, off, c.x, c.W1, None, phi, c.ws)
        assert lrm.lrm_read_device_error(c.ws, clear=True) == 32
        assert not phi[3].any()                   # that row reads x as zeros
        y, out = c.rows(c.L_cap, c.h, 1.0), c.rows(c.T, c.h, 0.0)
        lrm.lrm_combine_tokens(c.P, bad, off, _dev(c.w), y, None, out, c.ws)
        assert lrm.lrm_read_device_error(c.ws, clear=True) == 32
    bad = rp.clone()
    bad[3] = bad[60]                              # one pair twice
    lrm.lrm_combine_tokens(c.P, bad, off, _dev(c.w), y, None, out, c.ws)
    assert lrm.lrm_read_device_error(c.ws, clear=True) == 32
    # offsets beyond the capacity, or running backwards, are clamped: no access leaves the buffers
    wild = torch.tensor([0, 10 ** 6, -5, 40, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    phi = c.rows(c.L_cap, c.d, 0.0)
    lrm.lrm_grouped_fc1_swiglu(c.P, rp, wild, c.x, c.W1, None, phi, c.ws)
    torch.cuda.synchronize()
    lrm.lrm_read_device_error(c.ws, clear=True)


def test_padded_batch_through_the_sequences():
    """Masked tokens take no expert: their outputs are the residual, their gradients and adot zeros;
    the plan reports the pairs it left out and nothing else."""
    import torch
    from backward_token_expert_amd import lrm, path
    T, k, E, h, d = 90, 2, 8, 64, 48
    c = Case(T=T, k=k, E=E, e_lo=0, E_loc=E, h=h, d=d, dtype="f32", spare=0)
    c.P = lrm.make_problem(T, k, E, 0, E, h, d, "f32", T * k, T * k)
    router = lrm.make_router(T, E, k, "f32", "topk", 0.1)
    rb, bufs = path.RouterBuffers(router), path.DeviceBuffers(c.P)
    fwd, lay = path.ForwardBuffers(c.P), path.LayerBuffers(c.P)
    rng = np.random.default_rng(13)
    z, mask = rng.normal(size=(T, E)).astype(np.float32), rng.random(T) < 0.6
    g = _dev(rng.normal(size=(T, h)).astype(np.float32))
    full = lrm.make_policy(1)
    x = c.x.clone()
    x[_dev(~mask)] = float("nan")                  # padding may hold anything
    path.route(router, _dev(z), rb, _dev(mask.astype(np.uint8)))
    path.run_forward(c.P, full, rb.topk_idx, rb.topk_w, x, c.W1, c.W, bufs, fwd, c.res)
    path.run(c.P, full, rb.topk_idx, rb.topk_w, g, fwd.phi, c.W, bufs)
    path.run_layer(c.P, fwd.ac, x, c.W1, bufs, lay)
    path.run_router_backward(c.P, router, _dev(z), bufs, rb)
    assert lrm.lrm_read_device_error(bufs.ws) == 1   # EXPERT_ID
    off = _dev(~mask)
    assert int(bufs.cmp_off[-1]) == k * int(mask.sum()) == int(rb.counts.sum())
    assert torch.equal(fwd.out[off], c.res[off]) and not lay.dx[off].any() and not rb.dlogits[off].any()
    assert not rb.adot.reshape(T, k)[off].any()
    for t in (fwd.out, lay.dx, lay.dW1, bufs.dW, rb.dlogits):
        assert torch.isfinite(t).all()


def layer_step(c, router, logits, rb, bufs, fwd, lay, clip, inp, policy, stream=None):
    """One training step of the layer through the public sequences."""
    from backward_token_expert_amd import path
    path.route(router, logits, rb, stream=stream)
    path.run_forward(c.P, policy, rb.topk_idx, rb.topk_w, c.x, c.W1, c.W, bufs, fwd, c.res, stream)
    path.run(c.P, policy, rb.topk_idx, rb.topk_w, inp["g"], fwd.phi, c.W, bufs, stream)
    path.run_layer(c.P, fwd.ac, c.x, c.W1, bufs, lay, stream)
    path.run_router_backward(c.P, router, logits, bufs, rb, stream)
    clip(inp["max_norm"], stream)


@pytest.mark.parametrize("full", [True, False], ids=["full", "half"])
@pytest.mark.parametrize("gate", ["topk", "all"])
def test_training_step_against_autograd(gate, full):
    """The whole step in fp32 against torch float64 autograd of the layer: with every pair kept its
    gradients are the layer's; at half retention those of the layer whose dropped pairs' terms are
    constants.  The forward products' errors compound over four products of float32, so the
    gradients are held to 1e-4 of their norm."""
    import torch
    from backward_token_expert_amd import lrm, path
    T, k, E, h, d, coef = 192, 2, 8, 64, 48, 0.05
    rng = np.random.default_rng(11)
    z = rng.normal(size=(T, E)).astype(np.float32)
    c = Case(T=T, k=k, E=E, e_lo=0, E_loc=E, h=h, d=d, dtype="f32", spare=0, skew=None)
    L_cap = T * k
    c.P = lrm.make_problem(T, k, E, 0, E, h, d, "f32", L_cap, L_cap)
    router = lrm.make_router(T, E, k, "f32", gate, coef)
    rb, bufs = path.RouterBuffers(router), path.DeviceBuffers(c.P)
    fwd, lay = path.ForwardBuffers(c.P), path.LayerBuffers(c.P)
    g = rng.normal(size=(T, h)).astype(np.float32)
    clip = path.GradientClip([bufs.dW, lay.dW1, rb.dlogits],
                             [torch.zeros_like(t) for t in (bufs.dW, lay.dW1, rb.dlogits)])
    inp = dict(g=_dev(g), max_norm=1.0)
    policy = lrm.make_policy(int(full), 1, 2)
    layer_step(c, router, _dev(z), rb, bufs, fwd, lay, clip, inp, policy)
    torch.cuda.synchronize()
    assert lrm.lrm_read_device_error(bufs.ws) == 0 and lrm.lrm_read_device_error(rb.ws) == 0

    f64 = dict(dtype=torch.float64)
    zt, xt = torch.tensor(z, **f64).requires_grad_(), torch.tensor(c.x64).requires_grad_()
    W1, W = torch.tensor(c.W164).requires_grad_(), torch.tensor(c.W64).requires_grad_()
    p = torch.softmax(zt, 1)
    idx = torch.tensor(rb.topk_idx.cpu().numpy()).long().reshape(T, k)
    w = torch.gather(p, 1, idx)
    if gate == "topk":
        w = w / w.sum(1, keepdim=True)
    kept = torch.zeros(T * k, dtype=torch.bool)
    K = int(bufs.cmp_off[-1])
    kept[bufs.sel_pair[:K].cpu().long()] = True
    assert (K == T * k) == full
    out = torch.tensor(c.res64)
    for j in range(k):
        e = idx[:, j]
        hh = torch.einsum("tdh,th->td", W1[e], xt)
        yy = torch.einsum("thd,td->th", W[e], torch.nn.functional.silu(hh[:, :d]) * hh[:, d:])
        term = w[:, j:j + 1] * yy
        out = out + torch.where(kept.reshape(T, k)[:, j:j + 1], term, term.detach())
    f = torch.tensor(rb.counts.cpu().numpy() / (T * k))
    loss = coef * E * (f * p.mean(0)).sum()
    ((out * torch.tensor(g, **f64)).sum() + loss).backward()

    def near(a, b, tol=1e-4):
        a, b = a.detach().double().cpu(), b.detach()
        assert (a - b).norm() <= tol * b.norm(), ((a - b).norm() / b.norm()).item()
    near(fwd.out, out, 1e-5)
    near(rb.loss[0], loss, 1e-5)
    near(bufs.dW, W.grad)
    near(lay.dW1, W1.grad)
    near(lay.dx, xt.grad)
    near(rb.dlogits, zt.grad)
    total = sum(t.grad.square().sum() for t in (W, W1, zt)).sqrt()
    near(clip.norm[0], total)
    near(clip.list.dst[1], W1.grad / total)


def test_step_in_a_graph_and_serving_step():
    """The step captured once and replayed with other inputs equals the eager step bit for bit; a
    serving step without ac gives the same outputs."""
    import torch
    from backward_token_expert_amd import lrm, path
    T, k, E, h, d = 300, 4, 16, 256, 136
    c = Case(T=T, k=k, E=E, e_lo=0, E_loc=E, h=h, d=d, dtype="bf16", spare=0)
    c.P = lrm.make_problem(T, k, E, 0, E, h, d, "bf16", T * k, T * k)
    router = lrm.make_router(T, E, k, "f32", "topk", 0.01)
    policy = lrm.make_policy(0, 1, 2)
    rng = np.random.default_rng(12)
    zs = [_dev(rng.normal(size=(T, E)).astype(np.float32)) for _ in range(2)]
    _, g = _store(rng.normal(size=(T, h)), "bf16")

    def buffers():
        rb, bufs = path.RouterBuffers(router), path.DeviceBuffers(c.P)
        fwd, lay = path.ForwardBuffers(c.P), path.LayerBuffers(c.P)
        return rb, bufs, fwd, lay, path.GradientClip([bufs.dW, lay.dW1, rb.dlogits])

    def results(b):
        rb, bufs, fwd, lay, clip = b
        K, L = int(bufs.cmp_off[-1]), int(bufs.fwd_off[-1])
        return [rb.topk_idx, rb.topk_w, rb.loss, rb.dlogits, fwd.out, fwd.ac[:L], fwd.phi[:L], bufs.dW,
                bufs.dphi[:K], lay.dW1, lay.dx, clip.norm]
    inp = dict(g=g, max_norm=1.0)
    static = zs[0].clone()
    gb = buffers()
    s = torch.cuda.Stream()
    layer_step(c, router, static, *gb, inp, policy)       # look-ups of the first call
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        layer_step(c, router, static, *gb, inp, policy)
    for rep in (0, 1, 0):
        static.copy_(zs[rep])
        graph.replay()
        torch.cuda.synchronize()
        eb = buffers()
        layer_step(c, router, zs[rep], *eb, inp, policy)
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(results(gb), results(eb))):
            assert torch.equal(a, b), (rep, i)
    sv = path.ForwardBuffers(c.P, keep_ac=False)
    path.run_forward(c.P, lrm.make_policy(1), eb[0].topk_idx, eb[0].topk_w, c.x, c.W1, c.W, eb[1], sv, c.res)
    assert torch.equal(sv.out, eb[2].out)

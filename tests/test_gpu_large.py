"""Arrays past 2^31 elements, operands at the 2^31-byte limit, and calls on two streams at once.

Large results are compared row by row on samples that hold the last rows, in float64 on the GPU, with
the bounds of test_gpu_route, test_gpu_forward and test_gpu_clip."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U32, U16 = 2.0 ** -24, 2.0 ** -8


def _lrm():
    import torch
    from backward_token_expert_amd import lrm, path
    return torch, lrm, path


def _sample(torch, n):
    """Row ids: the first and last ones, those around 2^31 / 2048, and some between."""
    rng = np.random.default_rng(n)
    ids = [0, 1, n - 1, n - 2, n - 300] + [i for i in (2 ** 20 - 1, 2 ** 20, 2 ** 20 + 1) if i < n]
    return torch.from_numpy(np.unique(np.concatenate([ids, rng.integers(0, n, 200)]))).cuda()


def _layout(torch, idx, E_loc):
    flat = idx.reshape(-1).long()
    order = torch.argsort(flat, stable=True)
    n = torch.bincount(flat.clamp(max=E_loc), minlength=E_loc + 1)[:E_loc]
    off = torch.zeros(E_loc + 1, dtype=torch.int32, device="cuda")
    off[1:] = n.cumsum(0)
    return order[:int(off[-1])].to(torch.int32), off


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_expert_rows_past_32_bits(dtype):
    """ac, y and out of 2.25e9 elements."""
    torch, lrm, _ = _lrm()
    t = torch.float32 if dtype == "f32" else torch.bfloat16
    u = U32 if dtype == "f32" else U16
    T, E, h, d = 1_100_003, 3, 8, 1024
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    idx = torch.randint(0, E, (T, 1), generator=g, device="cuda")
    pairs, off = _layout(torch, idx, E)
    expert = idx.reshape(-1)[pairs.long()]
    rows = _sample(torch, T)
    x = torch.randn(T, h, generator=g, device="cuda").to(t)
    W1 = torch.randn(E, 2 * d, h, generator=g, device="cuda").to(t)
    P = lrm.make_problem(T, 1, E, 0, E, h, d, dtype, T, T)
    ws = torch.zeros(lrm.lrm_forward_workspace_bytes(P), dtype=torch.uint8, device="cuda")
    ac, phi = torch.zeros(T, 2 * d, dtype=t, device="cuda"), torch.zeros(T, d, dtype=t, device="cuda")
    lrm.lrm_grouped_fc1_swiglu(P, pairs, off, x, W1, ac, phi, ws)
    xs, Ws = x[pairs[rows].long()].double(), W1[expert[rows]].double()
    want, size = (Ws * xs[:, None, :]).sum(2), (Ws * xs[:, None, :]).abs().sum(2)
    acc = h * U32 * size
    assert bool(((ac[rows].double() - want).abs() <= (u * want.abs() + acc) * (1 + u) + 1e-37).all())
    a, b = want.chunk(2, 1)
    da, db = acc.chunk(2, 1)
    silu = a * torch.sigmoid(a)
    tol = (u + 2.0 ** -20) * (silu * b).abs() + 1.1 * b.abs() * da + (silu.abs() + da) * db + 1e-37
    assert bool(((phi[rows].double() - silu * b).abs() <= tol * (1 + u)).all())
    del ac, phi, W1, x
    # FC2 and the return to the tokens: the widths exchanged
    h, d = 2048, 8
    P = lrm.make_problem(T, 1, E, 0, E, h, d, dtype, T, T)
    phi = torch.randn(T, d, generator=g, device="cuda").to(t)
    W = torch.randn(E, h, d, generator=g, device="cuda").to(t)
    w = torch.rand(T, generator=g, device="cuda")
    out = torch.zeros(T, h, dtype=t, device="cuda")
    for y_type in ([t] if dtype == "f32" else [t, torch.float32]):
        y = torch.zeros(T, h, dtype=y_type, device="cuda")
        lrm.lrm_grouped_fc2(P, off, phi, W, y, ws)
        lrm.lrm_combine_tokens(P, pairs, off, w, y, None, out, ws)
        terms = W[expert[rows]].double() * phi[rows].double()[:, None, :]
        want = terms.sum(2)
        tol = (u if y_type == t else 0.0) * want.abs() + d * U32 * terms.abs().sum(2) + 1e-37
        assert bool(((y[rows].double() - want).abs() <= tol * (1 + u)).all())
        token = pairs[rows].long()
        full = w[token].double()[:, None] * y[rows].double()       # one row a token
        assert bool(((out[token].double() - full).abs() <= (u + 2 * U32) * full.abs() + 1e-37).all())
        del y
    assert lrm.lrm_read_device_error(ws) == 0


def test_input_of_two_gibibytes():
    """x at the limit of the 32-bit offsets: the last token's last columns, gathered."""
    torch, lrm, _ = _lrm()
    T, h, d, E = 2 ** 19, 2048, 64, 1024
    idx = torch.randint(1, E, (T, 1), device="cuda")
    local = _sample(torch, T)
    idx[local] = 0
    pairs, off = _layout(torch, idx, 1)
    x = torch.zeros(T, h, dtype=torch.bfloat16, device="cuda")
    x[local] = torch.randn(len(local), h, device="cuda").bfloat16()
    W1 = (torch.randn(1, 2 * d, h, device="cuda") / 45).bfloat16()
    P = lrm.make_problem(T, 1, E, 0, 1, h, d, "bf16", len(pairs), len(pairs))
    ws = torch.zeros(lrm.lrm_forward_workspace_bytes(P), dtype=torch.uint8, device="cuda")
    ac = torch.zeros(len(pairs), 2 * d, dtype=torch.bfloat16, device="cuda")
    phi = torch.zeros(len(pairs), d, dtype=torch.bfloat16, device="cuda")
    lrm.lrm_grouped_fc1_swiglu(P, pairs, off, x, W1, ac, phi, ws)
    rows = x[pairs.long()].double()
    want, size = rows @ W1[0].double().t(), rows.abs() @ W1[0].double().abs().t()
    assert bool(((ac.double() - want).abs() <= (U16 * want.abs() + h * U32 * size) * (1 + U16)).all())
    assert lrm.lrm_read_device_error(ws) == 0
    with pytest.raises(lrm.LrmError, match="status 2"):             # one token more
        Q = lrm.make_problem(T + 1, 1, E, 0, 1, h, d, "bf16", len(pairs), len(pairs))
        lrm.lrm_grouped_fc1_swiglu(Q, pairs, off, x.data_ptr(), W1, ac, phi,
                                   torch.zeros(lrm.lrm_forward_workspace_bytes(Q), dtype=torch.uint8, device="cuda"))


def test_router_past_32_bits():
    """2.2e9 logits and their gradient."""
    torch, lrm, path = _lrm()
    T, E, k = 2 ** 20 + 5, 2100, 2
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    logits = torch.randn(T, E, generator=g, device="cuda")
    router = lrm.make_router(T, E, k, "f32", "topk", 0.5)
    rb = path.RouterBuffers(router)
    path.route(router, logits, rb)
    adot = torch.randn(T * k, generator=g, device="cuda")
    lrm.lrm_route_backward(router, logits, rb.topk_idx, rb.topk_w, rb.counts, adot, rb.dlogits)
    assert lrm.lrm_read_device_error(rb.ws) == 0 and int(rb.counts.sum()) == T * k
    rows = _sample(torch, T)
    z = logits[rows].double()
    val, idx = torch.sort(z, dim=1, descending=True, stable=True)
    assert torch.equal(rb.topk_idx.reshape(T, k)[rows].long(), idx[:, :k])
    w = torch.softmax(val[:, :k], 1)
    assert bool(((rb.topk_w.reshape(T, k)[rows].double() - w).abs() <= w * (w.log().abs() + 64) * 2 * U32).all())
    p, f, c = torch.softmax(z, 1), rb.counts.double() / (T * k), 0.5 * E / T
    fp = (p * f).sum(1, keepdim=True)
    s = adot.reshape(T, k)[rows].double()
    S, mag = s.sum(1, keepdim=True), s.abs().sum(1, keepdim=True)
    d = (c * p * (f - fp)).scatter_add(1, idx[:, :k], s - w * S)
    size = (c * p * (f + fp)).scatter_add(1, idx[:, :k], s.abs() + w * mag)
    tol = size * (p.log().abs() + 128 + 2 * k) * 2 * U32 + 1e-37
    assert bool(((rb.dlogits[rows].double() - d).abs() <= tol).all())


def test_gate_dots_and_clipping_past_32_bits():
    torch, lrm, path = _lrm()
    K, d = 1_100_003, 2048
    P = lrm.make_problem(K, 1, 2, 0, 2, 8, d, "bf16", K, K)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    dphi = torch.randn(K, d, generator=g, device="cuda")
    phi = torch.empty(K, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    sel = torch.randperm(K, generator=g, device="cuda").to(torch.int32)
    off = torch.tensor([0, K // 3, K], dtype=torch.int32, device="cuda")
    ws = torch.zeros(lrm.lrm_forward_workspace_bytes(P), dtype=torch.uint8, device="cuda")
    adot = torch.zeros(K, device="cuda")
    lrm.lrm_gate_dots(P, sel, off, dphi, phi, adot, ws)
    assert lrm.lrm_read_device_error(ws) == 0
    rows = _sample(torch, K)
    terms = dphi[rows].double() * phi[rows].double()
    want = terms.sum(1)
    assert bool(((adot[sel[rows].long()].double() - want).abs() <=
                 U32 * want.abs() + 2.0 ** -45 * terms.abs().sum(1)).all())
    # the same arrays, 2.25e9 elements each, as gradients
    total = sum(float((t[i:i + 65536].double() ** 2).sum()) for t in (dphi, phi) for i in range(0, K, 65536)) ** 0.5
    keep = dphi[rows].clone(), phi[rows].clone()
    clip = path.GradientClip([dphi, phi])
    assert abs(clip(0.25 * total).item() - total) <= 2 * U32 * total
    for t, old, e in ((dphi, keep[0], 0.0), (phi, keep[1], U16)):
        want = old.double() * 0.25
        assert bool(((t[rows].double() - want).abs() <= (4 * U32 + e) * want.abs() + 1e-38).all())
    assert lrm.lrm_read_device_error(clip.ws) == 0


@pytest.mark.parametrize("T,dtype", [(1, "bf16"), (600, "bf16"), (600, "f32")])
def test_two_streams_at_once(T, dtype):
    """Two layers' steps of the router, the forward and the clipping on two streams, each with its own
    buffers, over and over: the results of the steps alone."""
    torch, lrm, path = _lrm()
    k, E, h, d = 4, 16, 520, 264
    t = torch.float32 if dtype == "f32" else torch.bfloat16

    class Layer:
        def __init__(self, seed):
            g = torch.Generator(device="cuda")
            g.manual_seed(seed)
            r = lambda *s: torch.randn(*s, generator=g, device="cuda")
            self.P = lrm.make_problem(T, k, E, 0, E, h, d, dtype, T * k, T * k)
            self.router = lrm.make_router(T, E, k, "f32", "topk", 0.1)
            self.z, self.x = r(T, E), r(T, h).to(t)
            self.W1, self.W = r(E, 2 * d, h).to(t), r(E, h, d).to(t)
            self.rb, self.bufs, self.fwd = path.RouterBuffers(self.router), path.DeviceBuffers(self.P), \
                path.ForwardBuffers(self.P)
            self.dst = [torch.zeros_like(self.z), torch.zeros_like(self.W1)]
            self.clip = path.GradientClip([self.z, self.W1], self.dst)

        def step(self, stream=None):
            path.route(self.router, self.z, self.rb, stream=stream)
            path.run_forward(self.P, lrm.make_policy(1), self.rb.topk_idx, self.rb.topk_w, self.x, self.W1,
                             self.W, self.bufs, self.fwd, self.x, stream)
            lrm.lrm_route_backward(self.router, self.z, self.rb.topk_idx, self.rb.topk_w, self.rb.counts,
                                   self.rb.topk_w, self.rb.dlogits, stream)
            self.clip(1.0, stream)

        def results(self):
            return [self.rb.topk_idx, self.rb.topk_w, self.rb.loss, self.rb.dlogits, self.fwd.phi, self.fwd.out,
                    self.clip.norm, *self.dst]
    layers = [Layer(1), Layer(2)]
    alone = []
    for layer in layers:
        layer.step()
        torch.cuda.synchronize()
        alone.append([r.clone() for r in layer.results()])
    streams = [torch.cuda.Stream() for _ in layers]
    for rep in range(5):
        for layer in layers:
            for r in layer.results():
                r.fill_(3)
        torch.cuda.synchronize()
        for layer, stream in zip(layers, streams):
            layer.step(stream)
        torch.cuda.synchronize()
        for layer, want in zip(layers, alone):
            assert lrm.lrm_read_device_error(layer.bufs.ws) == 0
            assert all(torch.equal(a, b) for a, b in zip(layer.results(), want)), rep

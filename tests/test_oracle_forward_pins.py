"""Pins of the forward oracle (CPU): autograd and differences of the definitions in float64, the
worked example of "Expert Parallel Math Deep", and closed forms."""
import json
import os

import numpy as np
import pytest
import torch

from oracle import forward_oracle as F

GOLDEN = os.path.join(os.path.dirname(os.path.abspath(__file__)), "golden")


def _logits(T, E, seed, closed=0):
    z = np.random.default_rng(seed).normal(size=(T, E))
    if closed:
        z[:, -closed:] = -np.inf
    return z


def test_balance_loss_of_the_worked_example():
    # the page: loads n of 8 experts, f_i = n_i / (T k), P_i = f_i gives E * sum f^2 = 1.204
    g = json.load(open(os.path.join(GOLDEN, "expert_parallel_math_worked_example.json")))
    n = np.array([30000, 24000, 20000, 16000, 14000, 12000, 8000, 7072])
    f = n / n.sum()
    assert abs(8 * float(f @ f) - 1.204) < 5e-4
    assert g  # the same example's golden file is the quota pins'
    # a router whose probabilities are the same for every token: P = p, the loss is E * sum f p
    z = np.log(f)[None, :].repeat(64, 0)
    r = F.route(z, 2, coef=1.0)
    assert np.allclose(r["prob"], f, atol=1e-15)
    want = 8 * (f[0] + f[1]) / 2          # every token chooses experts 0 and 1
    assert abs(r["loss"] - want) < 1e-12
    uniform = F.route(np.zeros((16, 8)), 2, coef=1.0)
    assert abs(uniform["loss"] - 1.0) < 1e-12 and list(uniform["topk_idx"][:2]) == [0, 1]


@pytest.mark.parametrize("gate", ["topk", "all"])
@pytest.mark.parametrize("masked", [False, True])
def test_router_gradient_is_autograd_and_differences(gate, masked):
    T, E, k, coef = 9, 12, 3, 0.7
    z = _logits(T, E, 1, closed=2)
    mask = np.arange(T) % 3 != 0 if masked else None
    r = F.route(z, k, gate, coef, mask)
    rng = np.random.default_rng(2)
    up = rng.normal(size=(T, k))                         # dL/dalpha
    adot = r["topk_w"] * up.reshape(-1)
    d, _ = F.route_backward(r, k, gate, coef, adot)

    def loss(zt):
        live = torch.tensor(r["live"])
        p = torch.softmax(zt, 1) * live[:, None]
        n = int(live.sum())
        idx = torch.tensor(np.maximum(r["topk_idx"].reshape(T, k), 0)).long()
        w = torch.gather(p, 1, idx)
        if gate == "topk":
            w = w / torch.where(live[:, None], w.sum(1, keepdim=True), torch.ones(T, 1, dtype=torch.float64))
        f = torch.tensor(r["counts"] / (n * k))
        return coef * E * (f * p.sum(0) / n).sum() + (w * live[:, None] * torch.tensor(up)).sum()

    zt = torch.tensor(z, requires_grad=True)
    loss(zt).backward()
    assert np.allclose(d, zt.grad.nan_to_num(0.0).numpy(), atol=1e-13)
    for t, e in ((1, 0), (4, 5), (7, int(r["topk_idx"][7 * k]))):
        h = 1e-6
        a, b = z.copy(), z.copy()
        a[t, e] += h
        b[t, e] -= h
        fd = (loss(torch.tensor(a)) - loss(torch.tensor(b))).item() / (2 * h)
        assert abs(fd - d[t, e]) < 1e-8


def test_forward_and_gate_dots_against_autograd_of_the_layer():
    # adot = alpha * d<g, out>/dalpha, through the experts, from dphi = W^T (alpha g)
    rng = np.random.default_rng(3)
    T, k, E, h, d = 5, 2, 3, 8, 16
    x, g = rng.normal(size=(T, h)), rng.normal(size=(T, h))
    W1, W = rng.normal(size=(E, 2 * d, h)), rng.normal(size=(E, h, d))
    idx = np.array([[0, 1], [2, 0], [1, 2], [0, 2], [1, 0]], np.int32).reshape(-1)
    w = rng.uniform(0.1, 0.9, T * k)
    row_pair = np.argsort(idx, kind="stable")
    off = np.concatenate([[0], np.cumsum(np.bincount(idx, minlength=E))])
    ac, phi, _ = F.fc1_swiglu(x, W1, row_pair, off, k)
    y, _ = F.fc2(phi, W, off)
    res = rng.normal(size=(T, h))
    out, _ = F.combine(y, row_pair, w, T, k, res)
    wt = torch.tensor(w, requires_grad=True)
    want = torch.tensor(res)
    for t in range(T):
        for j in range(k):
            e = int(idx[t * k + j])
            hh = torch.tensor(W1[e]) @ torch.tensor(x[t])
            want = want.index_add(0, torch.tensor([t]), (wt[t * k + j] * (
                torch.tensor(W[e]) @ (torch.nn.functional.silu(hh[:d]) * hh[d:])))[None])
    assert np.allclose(out, want.detach().numpy(), atol=1e-12)
    (want * torch.tensor(g)).sum().backward()
    dphi = np.stack([W[idx[p]].T @ (w[p] * g[p // k]) for p in row_pair])
    adot, _ = F.gate_dots(dphi, phi, row_pair, T * k)
    assert np.allclose(adot, w * wt.grad.numpy(), atol=1e-12)


def test_clip_keeps_the_direction_and_the_norm():
    rng = np.random.default_rng(4)
    gs = [rng.normal(size=n) for n in (1, 7, 100)]
    norm, out = F.clip(gs, 0.5)
    assert abs(np.sqrt(sum((o ** 2).sum() for o in out)) - 0.5) < 1e-12
    assert all(np.allclose(o * norm, 0.5 * g) for o, g in zip(out, gs))
    assert F.clip([np.zeros(3)], 1.0)[0] == 0.0 and F.clip(gs, 1e9)[1][2] is not None
    assert np.array_equal(F.clip(gs, 1e9)[1][1], gs[1])

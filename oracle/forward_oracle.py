"""Float64 oracle of the layer's forward, the router's gradient and gradient clipping.

TEST INFRASTRUCTURE ONLY.  Every function works on float64 values (widen storage types first) and
follows the definitions: "Expert Parallel Math Deep" for the routing and the auxiliary loss
coef * E * sum f_e P_e, LRMoE Appendix 7.1 Eq. (4) for the experts' output.
"""
from __future__ import annotations

import numpy as np


def live_tokens(logits, mask=None):
    """Tokens that route: not masked and with some logit above -infinity."""
    live = np.any(logits > -np.inf, axis=1)
    return live if mask is None else live & (np.asarray(mask) != 0)


def softmax(z):
    with np.errstate(invalid="ignore"):
        e = np.exp(z - z.max(axis=1, keepdims=True))
    return e / e.sum(axis=1, keepdims=True)


def route(logits, k: int, gate: str = "topk", coef: float = 0.0, mask=None) -> dict:
    z = np.asarray(logits, np.float64)
    T, E = z.shape
    live = live_tokens(z, mask)
    n = int(live.sum())
    p = np.zeros((T, E))
    p[live] = softmax(z[live])
    order = np.argsort(-z, axis=1, kind="stable")[:, :k]          # ties to the lower expert
    w = np.take_along_axis(p, order, 1)
    if gate == "topk":
        w[live] /= w[live].sum(axis=1, keepdims=True)
    lse = np.zeros(T)
    m = z[live].max(axis=1)
    lse[live] = m + np.log(np.exp(z[live] - m[:, None]).sum(axis=1))
    idx = np.where(live[:, None], order, -1).astype(np.int32)
    counts = np.bincount(idx[idx >= 0].reshape(-1), minlength=E).astype(np.int32)
    prob = p.sum(axis=0) / max(1, n)
    loss = coef * E * float(counts @ prob) / (max(1, n) * k)
    return dict(topk_idx=idx.reshape(-1), topk_w=w.reshape(-1), lse=lse, counts=counts, prob=prob,
                loss=loss, p=p, live=live)


def route_backward(r: dict, k: int, gate: str = "topk", coef: float = 0.0, adot=None):
    """dlogits from ``route``'s result; adot[p] = alpha_p dL/dalpha_p.  Also the sum of the terms'
    magnitudes, which a rounding error bound needs."""
    p, live = r["p"], r["live"]
    T, E = p.shape
    n = max(1, int(live.sum()))
    f = r["counts"] / (n * k)
    c = coef * E / n
    fp = p @ f
    d = c * p * (f[None, :] - fp[:, None])
    size = c * p * (f[None, :] + fp[:, None])
    if adot is not None:
        s = np.asarray(adot, np.float64).reshape(T, k)
        total, mag = s.sum(axis=1), np.abs(s).sum(axis=1)
        idx, w = r["topk_idx"].reshape(T, k), r["topk_w"].reshape(T, k)
        for t in np.flatnonzero(live):
            if gate == "topk":
                d[t, idx[t]] += s[t] - w[t] * total[t]
                size[t, idx[t]] += np.abs(s[t]) + w[t] * mag[t]
            else:
                d[t, idx[t]] += s[t]
                size[t, idx[t]] += np.abs(s[t])
                d[t] -= p[t] * total[t]
                size[t] += p[t] * mag[t]
    d[~live] = 0.0
    return d, size


def gate_dots(dphi, Phic, sel_pair, P: int):
    out, size = np.zeros(P), np.zeros(P)
    out[sel_pair] = (dphi * Phic).sum(axis=1)
    size[sel_pair] = np.abs(dphi * Phic).sum(axis=1)
    return out, size


def fc1_swiglu(x, W1, row_pair, fwd_off, k: int):
    """ac, phi and, for error bounds, sum |x||W1| of every ac element (float64)."""
    L, d2 = int(fwd_off[-1]), W1.shape[1]
    ac, size = np.zeros((L, d2)), np.zeros((L, d2))
    for e in range(W1.shape[0]):
        s = slice(int(fwd_off[e]), int(fwd_off[e + 1]))
        rows = x[row_pair[s] // k]
        ac[s] = rows @ W1[e].T
        size[s] = np.abs(rows) @ np.abs(W1[e]).T
    a, c = ac[:, :d2 // 2], ac[:, d2 // 2:]
    return ac, a / (1.0 + np.exp(-a)) * c, size


def fc2(phi, W, fwd_off):
    L = int(fwd_off[-1])
    y, size = np.zeros((L, W.shape[1])), np.zeros((L, W.shape[1]))
    for e in range(W.shape[0]):
        s = slice(int(fwd_off[e]), int(fwd_off[e + 1]))
        y[s] = phi[s] @ W[e].T
        size[s] = np.abs(phi[s]) @ np.abs(W[e]).T
    return y, size


def combine(y, row_pair, topk_w, T: int, k: int, residual=None):
    """The token outputs and the sum of their terms' magnitudes."""
    out = np.zeros((T, y.shape[1])) if residual is None else np.array(residual, np.float64)
    size = np.abs(out)
    for r, p in enumerate(row_pair[:y.shape[0]]):
        term = float(topk_w[p]) * y[r]
        out[p // k] += term
        size[p // k] += np.abs(term)
    return out, size


def clip(grads, max_norm: float):
    norm = float(np.sqrt(sum(float((g.astype(np.float64) ** 2).sum()) for g in grads)))
    coef = min(1.0, max_norm / norm) if norm > 0 else 1.0
    return norm, [g.astype(np.float64) * coef for g in grads]

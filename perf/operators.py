"""What the operators around the expert backward are measured on: the router with its balance loss
and gradient, the experts' forward products, and the clipping of the layer's gradients.

`run` computes each operator in elementary torch operations, or, with `own` set, through
backward_token_expert_amd's entry points; `exact` computes it again in 64 bits."""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------

def _route(name, T, E, k, dtype="f32", gate="topk", pad=False, closed=0):
    return {"name": name, "op": "route", "T": T, "E": E, "k": k, "dtype": dtype, "gate": gate,
            "pad": pad, "closed": closed}


def _grad(name, T, E, k, E_loc, d, keep, dtype="bf16", gate="topk", pad=False):
    return {"name": name, "op": "router_grad", "T": T, "E": E, "k": k, "E_loc": E_loc, "d": d,
            "keep": keep, "dtype": dtype, "gate": gate, "pad": pad}


def _fc(op, name, T, E, k, E_loc, h, d, dtype="bf16", residual=False):
    return {"name": name, "op": op, "T": T, "E": E, "k": k, "E_loc": E_loc, "h": h, "d": d,
            "dtype": dtype, "residual": residual}


def _clip(name, tensors, longest, shortest, dtype="f32"):
    return {"name": name, "op": "clip", "tensors": tensors, "longest": longest,
            "shortest": shortest, "dtype": dtype}


def listed():
    return [
        # one token of a serving loop: latency alone
        _route("route one token", 1, 128, 8),
        # a training batch of the 128-expert layers
        _route("route 32768x128", 32768, 128, 8),
        # a padded batch of a 160-expert router without renormalised weights, bf16 logits, and
        # experts that are never routed to
        _route("route padded 16384x160 bf16", 16384, 160, 6, "bf16", "all", True, 3),
        # the router's gradient of the Qwen3-30B-A3B-shaped share at half retention
        _grad("router grad qwen3 share", 32768, 128, 8, 16, 768, 0.5),
        # a small fp32 layer, padded batch, every expert local
        _grad("router grad small fp32", 1021, 8, 2, 8, 512, 0.6, "f32", "all", True),
        # FC1 and the activation of the GLM4.5-shaped share: the largest product
        _fc("fc1", "fc1 glm4.5 share", 32768, 128, 8, 16, 4096, 1408),
        # 32 sequences of a serving loop over a whole Qwen3-shaped layer: two rows an expert
        _fc("fc1", "fc1 decode 32", 32, 128, 8, 128, 2048, 768),
        # the small fp32 layer
        _fc("fc1", "fc1 small fp32", 4096, 8, 2, 8, 256, 512, "f32"),
        # FC2 and the return to the tokens of the Qwen3-shaped share
        _fc("fc2", "fc2 qwen3 share", 32768, 128, 8, 16, 2048, 768, "bf16", True),
        # one token of a serving loop over a whole layer
        _fc("fc2", "fc2 one token", 1, 128, 8, 128, 2048, 768, "bf16", True),
        # the GLM4.5-shaped share's expert gradients (FC2 and FC1 of 16 experts) and its router's
        _clip("clip glm4.5 share", 3, 16 * 2816 * 4096, 128 * 4096),
        # the many small, odd tensors of the rest of a model, bf16
        _clip("clip 40 odd bf16", 40, 300007, 5, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "router_grad", "fc1", "fc2", "clip"])
    dtype = rng.choice(["f32", "bf16"])
    if op == "clip":
        tensors = rng.randint(1, 48)
        longest = _log(rng, 1000, 20_000_000 if tensors > 8 else 100_000_000)
        return {"op": op, "tensors": tensors, "longest": longest,
                "shortest": rng.randint(1, 999), "dtype": dtype}
    E = rng.choice([8, 16, 60, 64, 96, 128, 160, 256])
    k = rng.randint(1, 8)
    gate = rng.choice(["topk", "all"])
    if op == "route":
        return {"op": op, "T": _log(rng, 1, 32768), "E": E, "k": k, "dtype": dtype, "gate": gate,
                "pad": rng.random() < 0.4, "closed": rng.choice([0, 0, 3])}
    E_loc = max(1, E // rng.choice([1, 4, 8]))
    if op == "router_grad":
        return {"op": op, "T": _log(rng, 16, 16384), "E": E, "k": k, "E_loc": E_loc,
                "d": 8 * rng.randint(8, 176), "keep": rng.choice([0.25, 0.5, 1.0]),
                "dtype": dtype, "gate": gate, "pad": rng.random() < 0.4}
    # a few experts' rows over short and long batches; fp32 layers are small ones
    h, d = (8 * rng.randint(8, 128), 8 * rng.randint(8, 96)) if dtype == "f32" else \
        (8 * rng.randint(16, 512), 8 * rng.randint(16, 176))
    return {"op": op, "T": _log(rng, 1, 4096 if dtype == "f32" else 8192), "E": E, "k": k,
            "E_loc": E_loc, "h": h, "d": d, "dtype": dtype, "residual": rng.random() < 0.5}


# ---------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------

def _logits(g, T, E, dtype, closed=0, device=DEV):
    """Random logits with a Zipf-shaped constant per expert, the first experts being the hottest;
    the last `closed` experts are never chosen."""
    out = torch.randn(T, E, generator=g, device=device)
    out -= 1.8 * torch.log(torch.arange(1, E + 1, device=device))
    if closed and E > 2 * closed + 8:
        out[:, E - closed:] = -math.inf
    return out.to(TYPES[dtype])


def _mask(g, T, pad):
    return (torch.rand(T, generator=g, device=DEV) < 0.8).to(torch.uint8) if pad else None


def _choose(logits, k, gate):
    """The k largest logits of each row, ties to the lower expert, and their weights, in 32 bits."""
    val, idx = torch.sort(logits.float(), dim=1, descending=True, stable=True)
    lse = torch.logsumexp(logits.float(), 1)
    val, idx = val[:, :k], idx[:, :k].to(torch.int32)
    w = torch.exp(val - (torch.logsumexp(val, 1) if gate == "topk" else lse)[:, None])
    return idx, w, lse


def _layout(idx, E_loc):
    """Pairs of the experts below E_loc, ordered by (expert, pair), and the experts' offsets."""
    flat = idx.reshape(-1).long()
    flat = torch.where(flat < 0, torch.full_like(flat, E_loc), flat)
    order = torch.argsort(flat, stable=True).to(torch.int32)
    n = torch.bincount(torch.clamp(flat, max=E_loc), minlength=E_loc + 1)[:E_loc]
    off = torch.zeros(E_loc + 1, dtype=torch.int32, device=DEV)
    off[1:] = torch.cumsum(n, 0).to(torch.int32)
    return order, off, n.tolist()


def _segments(n):
    """(expert, first row, end) of the experts that have rows."""
    out, at = [], 0
    for e, m in enumerate(n):
        if m:
            out.append((e, at, at + m))
        at += m
    return out, at


def _swiglu_rows(g, rows, d):
    a = torch.randn(rows, d, generator=g, device=DEV)
    return a / (1.0 + torch.exp(-a)) * torch.randn(rows, d, generator=g, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": case}
    op, t = case["op"], TYPES[case["dtype"]]
    if op == "clip":
        n, hi, lo = case["tensors"], case["longest"], case["shortest"]
        step = (hi / lo) ** (1.0 / max(1, n - 1))
        sizes = [max(1, min(hi, int(hi / step ** i))) for i in range(n)]
        s["grads"] = [(torch.randn(m, generator=g, device=DEV) * (0.1 + i)).to(t)
                      for i, m in enumerate(sizes)]
        # a norm that has to be cut, as in a run's first steps
        s["max_norm"] = 0.25 * math.sqrt(sum(m * (0.1 + i) ** 2 for i, m in enumerate(sizes)))
        return s
    T, E, k = case["T"], case["E"], case["k"]
    if op == "route":
        s["logits"] = _logits(g, T, E, case["dtype"], case["closed"])
        s["mask"] = _mask(g, T, case["pad"])
        return s
    E_loc, d = case["E_loc"], case["d"]
    if op == "router_grad":
        # the router works in 32 bits; the experts' rows have the layer's type
        s["logits"], s["mask"] = _logits(g, T, E, "f32"), _mask(g, T, case["pad"])
        idx, w, s["lse"] = _choose(s["logits"], k, case["gate"])
        if s["mask"] is not None:
            live = s["mask"].bool()
            idx = torch.where(live[:, None], idx, torch.full_like(idx, -1))
            w = torch.where(live[:, None], w, torch.zeros_like(w))
            s["lse"] = torch.where(live, s["lse"], torch.zeros_like(s["lse"]))
        s["topk_idx"], s["topk_w"] = idx.reshape(-1), w.reshape(-1)
        s["counts"] = torch.bincount(idx[idx >= 0].long(), minlength=E).to(torch.int32)
        order, off, n = _layout(idx, E_loc)
        cap = int(case["keep"] * sum(n) / E_loc) if case["keep"] < 1.0 else max(n)
        rows = [off[e].item() + torch.randperm(m, generator=g, device=DEV)[:min(m, cap)].sort()[0]
                for e, m in enumerate(n)]
        s["sel_pair"] = order[torch.cat(rows)]
        s["cmp_off"] = torch.tensor([0] + [len(r) for r in rows], device=DEV).cumsum(0).to(torch.int32)
        K = s["sel_pair"].numel()
        s["Phic"] = _swiglu_rows(g, K, d).to(t)
        s["dphi"] = torch.randn(K, d, generator=g, device=DEV) * s["topk_w"][s["sel_pair"].long()][:, None]
        return s
    h = case["h"]
    idx, w, _ = _choose(_logits(g, T, E, "f32"), k, "topk")
    order, s["fwd_off"], n = _layout(idx, E_loc)
    s["segments"], L = _segments(n)
    # rows past the last segment are the capacity's: no call reads or writes them
    s["row_pair"] = order[:T * min(k, E_loc)].contiguous()
    s["topk_w"] = w.reshape(-1)
    if op == "fc1":
        s["x"] = torch.randn(T, h, generator=g, device=DEV).to(t)
        s["W1"] = (torch.randn(E_loc, 2 * d, h, generator=g, device=DEV) / math.sqrt(h)).to(t)
    else:
        s["phi"] = _swiglu_rows(g, s["row_pair"].numel(), d).to(t)
        s["W"] = (torch.randn(E_loc, h, d, generator=g, device=DEV) / math.sqrt(d)).to(t)
        s["residual"] = torch.randn(T, h, generator=g, device=DEV).to(t) if case["residual"] else None
    s["rows"] = L
    return s


# ---------------------------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------------------------

COEF = 0.01  # of the balance loss


def _plain_route(s):
    c = s["case"]
    idx, w, lse = _choose(s["logits"], c["k"], c["gate"])
    p = torch.exp(s["logits"].float() - lse[:, None])
    n = float(c["T"])
    if s["mask"] is not None:
        live = s["mask"].bool()[:, None]
        idx = torch.where(live, idx, torch.full_like(idx, -1))
        w, p = w * live, p * live
        lse = lse * live[:, 0]
        n = live.sum().float().clamp(min=1.0)
    chosen = idx.reshape(-1).long()
    # masked pairs count for one more expert, which is left out
    counts = torch.bincount(torch.where(chosen < 0, torch.full_like(chosen, c["E"]), chosen),
                            minlength=c["E"] + 1)[:c["E"]]
    prob = p.sum(0) / n
    loss = COEF * c["E"] * (counts.float() / (n * c["k"]) * prob).sum()
    return {"topk_idx": idx.reshape(-1), "topk_w": w.reshape(-1), "lse": lse,
            "counts": counts.to(torch.int32), "prob": prob, "loss": loss.reshape(1)}


def _plain_router_grad(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    adot = torch.zeros(T * k, device=DEV)
    adot[s["sel_pair"].long()] = (s["dphi"] * s["Phic"].float()).sum(1)
    p = torch.exp(s["logits"] - s["lse"][:, None])
    n = (s["counts"].sum() / k).clamp(min=1.0)
    f = s["counts"].float() / (n * k)
    d = COEF * E / n * p * (f - (p * f).sum(1, keepdim=True))
    a = adot.reshape(T, k)
    at = s["topk_idx"].reshape(T, k).long().clamp(min=0)
    total = a.sum(1, keepdim=True)
    if c["gate"] == "topk":
        d = d.scatter_add(1, at, a - s["topk_w"].reshape(T, k) * total)
    else:
        d = d.scatter_add(1, at, a) - p * total
    if s["mask"] is not None:
        d = d * s["mask"][:, None]
    return {"adot": adot, "dlogits": d}


def _plain_fc1(s):
    t = s["x"].dtype
    rows = s["x"][s["row_pair"][:s["rows"]].long() // s["case"]["k"]].float()
    h = torch.zeros(s["row_pair"].numel(), s["W1"].shape[1], device=DEV)
    for e, i, j in s["segments"]:
        torch.matmul(rows[i:j], s["W1"][e].float().t(), out=h[i:j])
    a, c = h.chunk(2, 1)
    return {"ac": h.to(t), "phi": (a / (1.0 + torch.exp(-a)) * c).to(t)}


def _plain_fc2(s):
    c, t = s["case"], s["phi"].dtype
    y = torch.zeros(s["row_pair"].numel(), c["h"], device=DEV)
    for e, i, j in s["segments"]:
        torch.matmul(s["phi"][i:j].float(), s["W"][e].float().t(), out=y[i:j])
    out = s["residual"].float() if s["residual"] is not None else torch.zeros(c["T"], c["h"], device=DEV)
    pair = s["row_pair"][:s["rows"]].long()
    out = out.index_add(0, pair // c["k"], y[:s["rows"]] * s["topk_w"][pair][:, None])
    return {"y": y.to(t), "out": out.to(t)}


def _plain_clip(s):
    norm = torch.sqrt(sum(g.float().square().sum() for g in s["grads"]))
    coef = torch.clamp(s["max_norm"] / norm, max=1.0)
    return {"norm": norm.reshape(1), "grads": [(g.float() * coef).to(g.dtype) for g in s["grads"]]}


# ---------------------------------------------------------------------------------------------
# The framework's calls; a program keeps the buffers and the workspace between its steps
# ---------------------------------------------------------------------------------------------

def _problem(s):
    from backward_token_expert_amd import lrm
    c = s["case"]
    rows = s["sel_pair"].numel() if c["op"] == "router_grad" else s["row_pair"].numel()
    return lrm.make_problem(c["T"], c["k"], c["E"], 0, c["E_loc"], c.get("h", 8), c["d"],
                            c["dtype"], rows, rows)


def _own_route(s):
    from backward_token_expert_amd import lrm, path
    c = s["case"]
    if "bufs" not in s:
        s["router"] = lrm.make_router(c["T"], c["E"], c["k"], c["dtype"], c["gate"], COEF)
        s["bufs"] = path.RouterBuffers(s["router"])
    b = s["bufs"]
    lrm.lrm_route(s["router"], s["logits"], s["mask"], b.topk_idx, b.topk_w, b.lse, b.counts,
                  b.prob, b.loss, b.ws)
    return {"topk_idx": b.topk_idx, "topk_w": b.topk_w, "lse": b.lse, "counts": b.counts,
            "prob": b.prob, "loss": b.loss}


def _own_router_grad(s):
    from backward_token_expert_amd import lrm
    c = s["case"]
    if "ws" not in s:
        s["router"] = lrm.make_router(c["T"], c["E"], c["k"], "f32", c["gate"], COEF)
        s["problem"] = _problem(s)
        s["ws"] = torch.zeros(lrm.lrm_forward_workspace_bytes(s["problem"]), dtype=torch.uint8, device=DEV)
        s["adot"] = torch.empty(c["T"] * c["k"], device=DEV)
        s["dlogits"] = torch.empty(c["T"], c["E"], device=DEV)
    lrm.lrm_gate_dots(s["problem"], s["sel_pair"], s["cmp_off"], s["dphi"], s["Phic"], s["adot"], s["ws"])
    lrm.lrm_route_backward(s["router"], s["logits"], s["topk_idx"], s["topk_w"], s["counts"],
                           s["adot"], s["dlogits"])
    return {"adot": s["adot"], "dlogits": s["dlogits"]}


def _own_fc1(s):
    from backward_token_expert_amd import lrm
    if "ws" not in s:
        s["problem"] = _problem(s)
        s["ws"] = torch.zeros(lrm.lrm_forward_workspace_bytes(s["problem"]), dtype=torch.uint8, device=DEV)
        d = s["case"]["d"]
        s["ac"] = torch.zeros(s["row_pair"].numel(), 2 * d, dtype=s["x"].dtype, device=DEV)
        s["phi"] = torch.zeros(s["row_pair"].numel(), d, dtype=s["x"].dtype, device=DEV)
    lrm.lrm_grouped_fc1_swiglu(s["problem"], s["row_pair"], s["fwd_off"], s["x"], s["W1"], s["ac"],
                               s["phi"], s["ws"])
    return {"ac": s["ac"], "phi": s["phi"]}


def _own_fc2(s):
    from backward_token_expert_amd import lrm
    c = s["case"]
    if "ws" not in s:
        s["problem"] = _problem(s)
        s["ws"] = torch.zeros(lrm.lrm_forward_workspace_bytes(s["problem"]), dtype=torch.uint8, device=DEV)
        s["y"] = torch.zeros(s["row_pair"].numel(), c["h"], dtype=s["phi"].dtype, device=DEV)
        s["out"] = torch.empty(c["T"], c["h"], dtype=s["phi"].dtype, device=DEV)
    lrm.lrm_grouped_fc2(s["problem"], s["fwd_off"], s["phi"], s["W"], s["y"], s["ws"])
    lrm.lrm_combine_tokens(s["problem"], s["row_pair"], s["fwd_off"], s["topk_w"], s["y"],
                           s["residual"], s["out"], s["ws"])
    return {"y": s["y"], "out": s["out"]}


def _own_clip(s):
    from backward_token_expert_amd import lrm
    if "ws" not in s:
        s["dst"] = [torch.empty_like(g) for g in s["grads"]]
        s["list"] = lrm.make_tensor_list(s["grads"], s["dst"])
        s["norm"] = torch.empty(1, device=DEV)
        s["ws"] = torch.zeros(lrm.lrm_grad_workspace_bytes(s["list"]), dtype=torch.uint8, device=DEV)
    lrm.lrm_clip_grads(s["list"], s["max_norm"], s["norm"], s["ws"])
    return {"norm": s["norm"], "grads": s["dst"]}


PLAIN = {"route": _plain_route, "router_grad": _plain_router_grad, "fc1": _plain_fc1,
         "fc2": _plain_fc2, "clip": _plain_clip}
OWN = {"route": _own_route, "router_grad": _own_router_grad, "fc1": _own_fc1, "fc2": _own_fc2,
       "clip": _own_clip}


def run(state):
    op = state["case"]["op"]
    return OWN[op](state) if own else PLAIN[op](state)


# ---------------------------------------------------------------------------------------------
# Bytes and operations that a pass cannot do without
# ---------------------------------------------------------------------------------------------

def _routed(case):
    """Expected rows of every local expert, and tokens with a local row, from a sample of routings."""
    T, E, k, E_loc = case["T"], case["E"], case["k"], case["E_loc"]
    g = torch.Generator()
    g.manual_seed(0)
    pick = _logits(g, 2048, E, "f32", device="cpu").topk(k, 1)[1]
    share = torch.bincount(pick.reshape(-1), minlength=E)[:E_loc].double() / 2048
    return T * share, T * (pick < E_loc).any(1).double().mean().item()


def work(case):
    op, b = case["op"], 4 if case["dtype"] == "f32" else 2
    if op == "clip":
        n, hi, lo = case["tensors"], case["longest"], case["shortest"]
        step = (hi / lo) ** (1.0 / max(1, n - 1))
        total = sum(max(1, min(hi, int(hi / step ** i))) for i in range(n))
        return {"bytes": 2 * total * b, "flops": 3 * total}
    T, E, k = case["T"], case["E"], case["k"]
    if op == "route":
        return {"bytes": T * E * b + 8 * T * k + 4 * T + 8 * E, "flops": 4 * T * E}
    n, tokens = _routed(case)
    L, used = n.sum().item(), (1.0 - (1.0 - n / T) ** T).sum().item()
    d = case["d"]
    if op == "router_grad":
        K = n.clamp(max=case["keep"] * L / case["E_loc"]).sum().item() if case["keep"] < 1.0 else L
        return {"bytes": K * (d * (4 + b) + 4) + T * E * 8 + T * k * 12 + 4 * T,
                "flops": 2 * K * d + 8 * T * E}
    h = case["h"]
    if op == "fc1":
        return {"bytes": (tokens * h + used * 2 * d * h + 3 * L * d) * b, "flops": 4 * L * h * d}
    return {"bytes": (L * d + used * h * d + L * h + T * h * (2 if case["residual"] else 1)) * b,
            "flops": 2 * L * h * d + 2 * L * h}


# ---------------------------------------------------------------------------------------------
# The same results in 64 bits, from the definitions
# ---------------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        total = 0.0
        for g in s["grads"]:
            v = g.double()
            total = total + torch.dot(v, v).item()
        scale = min(1.0, s["max_norm"] / math.sqrt(total))
        return {"norm": torch.tensor([math.sqrt(total)], dtype=torch.float64),
                "grads": [g.double().mul_(scale) for g in s["grads"]]}
    k = case["k"]
    if op == "route":
        z = s["logits"].double()
        live = torch.ones(case["T"], dtype=torch.bool, device=DEV) if s["mask"] is None else s["mask"] != 0
        prob = torch.softmax(z, 1)
        pick = torch.sort(z, dim=1, descending=True, stable=True)[1][:, :k]
        w = torch.gather(prob, 1, pick)
        if case["gate"] == "topk":
            w = w / w.sum(1, keepdim=True)
        w[~live] = 0.0
        lse = torch.logsumexp(z, 1)
        lse[~live] = 0.0
        kept, n = pick[live], max(1, int(live.sum()))
        counts = torch.stack([(kept == e).sum() for e in range(case["E"])])
        mean = prob[live].sum(0) / n
        loss = COEF * case["E"] * torch.dot(counts.double() / (n * k), mean)
        return {"topk_idx": None, "topk_w": w.reshape(-1), "lse": lse, "counts": None,
                "prob": mean, "loss": loss.reshape(1)}
    if op == "router_grad":
        T, E = case["T"], case["E"]
        live = torch.ones(T, dtype=torch.bool, device=DEV) if s["mask"] is None else s["mask"] != 0
        dots = torch.zeros(T * k, dtype=torch.float64, device=DEV)
        for i in range(0, s["sel_pair"].numel(), 65536):
            j = slice(i, i + 65536)
            dots[s["sel_pair"][j].long()] = (s["dphi"][j].double() * s["Phic"][j].double()).sum(1)
        # the Jacobians of the two softmaxes, from 64-bit logits
        z = s["logits"].double()
        p = torch.softmax(z, 1)
        n = max(1, int(live.sum()))
        f = s["counts"].double() / (n * k)
        up = (COEF * E / n) * f[None, :].expand(T, E)   # dL/dp of the balance loss
        pick = torch.where(live[:, None], s["topk_idx"].reshape(T, k).long(), 0)
        each = torch.gather(p, 1, pick)
        if case["gate"] == "all":
            # dL/dp_idx = dots / p_idx, joined to the balance loss' in one softmax gradient
            out = p * (up - (p * up).sum(1, keepdim=True))
            mine = torch.zeros(T, E, dtype=torch.float64, device=DEV).scatter_add_(1, pick, dots.reshape(T, k))
            out = out + mine - p * mine.sum(1, keepdim=True)
        else:
            out = p * (up - (p * up).sum(1, keepdim=True))
            each = each / each.sum(1, keepdim=True)
            part = dots.reshape(T, k)
            out = out.scatter_add(1, pick, part - each * part.sum(1, keepdim=True))
        out[~live] = 0.0
        return {"adot": dots, "dlogits": out}
    token = torch.div(s["row_pair"][:s["rows"]].long(), k, rounding_mode="floor")
    if op == "fc1":
        ac = torch.zeros(s["row_pair"].numel(), 2 * case["d"], dtype=torch.float64, device=DEV)
        for e, i, j in s["segments"]:
            ac[i:j] = s["x"][token[i:j]].double() @ s["W1"][e].double().T
        gate, up = ac[:, :case["d"]], ac[:, case["d"]:]
        return {"ac": ac, "phi": gate * torch.sigmoid(gate) * up}
    y = torch.zeros(s["row_pair"].numel(), case["h"], dtype=torch.float64, device=DEV)
    for e, i, j in s["segments"]:
        y[i:j] = s["phi"][i:j].double() @ s["W"][e].double().T
    out = torch.zeros(case["T"], case["h"], dtype=torch.float64, device=DEV)
    w = s["topk_w"].double()[s["row_pair"][:s["rows"]].long()]
    for i in range(0, s["rows"], 65536):
        j = min(i + 65536, s["rows"])
        out.index_add_(0, token[i:j], y[i:j] * w[i:j, None])
    return {"y": y, "out": out if s["residual"] is None else out + s["residual"].double()}

"""lrm_grad_norm and lrm_clip_grads on the GPU against float64.

The squares and sums are float64, so norm is off by one float32 rounding (2^-24 relative; 2^-23 is
allowed, for the float64 sums' order).  coef = max_norm / norm adds one rounding of its own and the
product another: 4 steps of 2^-24 on a float32 value, and half a step of bf16 (2^-8) on top there."""
import numpy as np
import pytest

from oracle import forward_oracle as F

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _tensors(sizes, seed, dtype, offset=0):
    """Device tensors that start `offset` elements into their allocation (views of odd alignment)."""
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kinds = {"f32": [torch.float32], "bf16": [torch.bfloat16], "mixed": [torch.float32, torch.bfloat16]}[dtype]
    return [(torch.randn(n + offset, generator=g, device="cuda") * (1 + i % 5)).to(kinds[i % len(kinds)])[offset:]
            for i, n in enumerate(sizes)]


def check(grads, dst, norm, max_norm):
    want_norm, want = F.clip([t.double().cpu().numpy() for t in grads], max_norm)
    assert abs(norm - want_norm) <= 2 * U * want_norm
    for a, w in zip(dst, want):
        e = 4 * U + (2.0 ** -8 if a.element_size() == 2 else 0)
        # a value below the type's normal range rounds at the spacing of the subnormals instead
        assert np.all(np.abs(a.double().cpu().numpy() - w) <= e * np.abs(w) + 1e-38)


SIZES = [[1], [0], [], [7, 0, 1, 3], [8191, 8192, 8193, 16384], [5] * 64, [3] * 65 + [70001],
         [100003, 1, 4096 * 33], list(range(1, 200))]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "mixed"])
@pytest.mark.parametrize("sizes", SIZES, ids=[f"{len(s)}x{max(s, default=0)}" for s in SIZES])
@pytest.mark.parametrize("offset", [0, 1, 3])
def test_clip(sizes, dtype, offset):
    import torch
    from backward_token_expert_amd import lrm, path
    print(f"[case] clip {len(sizes)} tensors {dtype} offset {offset}", flush=True)
    src = _tensors(sizes, 7, dtype, offset)
    keep = [t.clone() for t in src]
    total = float(np.sqrt(sum(t.double().square().sum().item() for t in src)))
    for max_norm in ((0.3 * total, 2 * total) if total > 0 else (1.0,)):
        dst = [torch.full_like(t, 9.0) for t in src]
        c = path.GradientClip(src, dst)
        c.ws.random_()
        norm = c(max_norm).item()
        assert lrm.lrm_read_device_error(c.ws) == 0
        check(src, dst, norm, max_norm)
        assert all(torch.equal(a, b) for a, b in zip(src, keep))
        only = torch.zeros(1, device="cuda")
        lrm.lrm_grad_norm(c.list, only, c.ws)
        assert only.item() == norm
        inplace = [t.clone() for t in src]
        c2 = path.GradientClip(inplace)
        assert c2(max_norm).item() == norm
        assert all(torch.equal(a, b) for a, b in zip(inplace, dst))


def test_neighbours_of_a_view_stay_as_they_were():
    import torch
    from backward_token_expert_amd import path
    for dt in (torch.float32, torch.bfloat16):
        base = torch.randn(40000, device="cuda").to(dt)
        keep = base.clone()
        v = base[3:39990]
        path.GradientClip([v])(0.5)
        torch.cuda.synchronize()
        assert torch.equal(base[:3], keep[:3]) and torch.equal(base[39990:], keep[39990:])
        assert not torch.equal(v, keep[3:39990])


def test_norms_without_a_square_in_float32_and_nonfinite_norms():
    import torch
    from backward_token_expert_amd import lrm, path
    big = torch.full((1000,), 1e30, device="cuda")        # the squares exceed float32
    c = path.GradientClip([big])
    assert abs(c(1.0).item() - 1e30 * np.sqrt(1000)) <= 4 * U * 1e30 * np.sqrt(1000)
    assert torch.allclose(big, torch.full_like(big, float(1 / np.sqrt(1000))), rtol=1e-6)
    tiny = torch.full((10,), 1e-30, device="cuda")
    c = path.GradientClip([tiny])
    assert abs(c(1.0).item() - 1e-30 * np.sqrt(10)) <= 1e-36
    assert torch.equal(tiny, torch.full_like(tiny, 1e-30))
    for bad in (float("nan"), float("inf")):
        t = torch.ones(5000, device="cuda")
        t[4321] = bad
        u = torch.ones(77, device="cuda", dtype=torch.bfloat16)
        c = path.GradientClip([t, u])
        n = c(0.1).item()
        assert not np.isfinite(n) and lrm.lrm_read_device_error(c.ws) == 16
        assert t[0].item() == 1.0 and (u == 1).all()      # nothing is written
        t[4321] = 1.0
        assert abs(c(0.1).item() - np.sqrt(5077)) < 1e-4 and lrm.lrm_read_device_error(c.ws) == 0


def test_clip_repeats_bit_for_bit_on_another_stream_and_in_a_graph():
    import torch
    from backward_token_expert_amd import path
    src = _tensors([300007, 5, 70000], 3, "mixed")
    dst = [torch.zeros_like(t) for t in src]
    c = path.GradientClip(src, dst)
    n0 = c(1.0).clone()
    first = [t.clone() for t in dst]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c(1.0, stream=s)
    s.synchronize()
    assert torch.equal(c.norm, n0) and all(torch.equal(a, b) for a, b in zip(dst, first))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        c(1.0)
    for rep in range(3):
        for t in dst:
            t.fill_(3.0)
        if rep == 1:
            src[0].mul_(2.0)
        g.replay()
        torch.cuda.synchronize()
        check(src, dst, c.norm.item(), 1.0)
        if rep == 0:
            assert torch.equal(c.norm, n0) and all(torch.equal(a, b) for a, b in zip(dst, first))

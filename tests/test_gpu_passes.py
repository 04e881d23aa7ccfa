"""Sizes at which a workgroup goes on to further tokens, rows, chunks or units: what it carries from one to
the next (partial sums, LDS rows that have to be cleared, a ring that is already loading) and the odd
tail.  The bounds are those of test_gpu_route, test_gpu_forward and test_gpu_clip."""
import numpy as np
import pytest

from oracle import forward_oracle as F
from tests.test_gpu_forward import Case, check_fc1, check_fc2
from tests.test_gpu_route import U, _dev, check_route, make_logits, run_route

pytestmark = pytest.mark.gpu


# The router has 256 workgroups: second passes from 513 tokens (E > 512, and k > 16), 4097 (E > 256),
# 16385 (E > 128) and 32769.  Its gradient has 2048: from 4097, 32769 and 65537 tokens.
@pytest.mark.parametrize("T,E,k,dtype,gate", [
    (520, 1000, 4, "f32", "topk"), (1700, 4096, 3, "bf16", "all"), (700, 600, 20, "f32", "all"),
    (1300, 40, 18, "bf16", "topk"), (4200, 512, 8, "f32", "topk"), (16500, 160, 6, "bf16", "all"),
    (33100, 60, 2, "f32", "topk"), (33000, 128, 16, "bf16", "topk")])
def test_route(T, E, k, dtype, gate):
    print(f"[case] route T={T} E={E} k={k} {dtype} {gate}", flush=True)
    from backward_token_expert_amd import lrm
    z, logits = make_logits(T, E, T + E, dtype, ties=dtype == "bf16")
    mask = np.random.default_rng(E).random(T) < 0.8
    mask[-1] = True
    rb, err = run_route(lrm.make_router(T, E, k, dtype, gate, 0.37), logits, mask)
    assert err == 0
    check_route(rb, F.route(z, k, gate, 0.37, mask), T)


@pytest.mark.parametrize("T,E,k,gate", [(4101, 600, 8, "topk"), (4300, 1031, 5, "all"), (32801, 300, 4, "topk"),
                                        (65601, 8, 2, "topk"), (65601, 136, 3, "all")])
def test_router_gradient(T, E, k, gate):
    print(f"[case] router gradient T={T} E={E} k={k} {gate}", flush=True)
    import torch
    from backward_token_expert_amd import lrm
    z, logits = make_logits(T, E, T, "f32")
    mask = np.random.default_rng(k).random(T) < 0.8
    coef, router = 0.37, lrm.make_router(T, E, k, "f32", gate, 0.37)
    rb, err = run_route(router, logits, mask)
    assert err == 0
    want = F.route(z, k, gate, coef, mask)
    np.testing.assert_array_equal(rb.topk_idx.cpu().numpy(), want["topk_idx"])
    adot = np.random.default_rng(E).normal(size=T * k).astype(np.float32)
    out = torch.full((T, E), float("nan"), device="cuda")
    lrm.lrm_route_backward(router, logits, rb.topk_idx, rb.topk_w, rb.counts, _dev(adot), out)
    d, size = F.route_backward(want, k, gate, coef, adot)
    lnp = np.where(want["p"] > 1e-37, np.abs(np.log(np.maximum(want["p"], 1e-300))), 0)
    assert np.all(np.abs(out.cpu().numpy() - d) <= size * (lnp + 128 + 2 * k) * 2 * U + 1e-37)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gate_dots(dtype):
    """65536 rows and 524288 pairs to a pass."""
    import torch
    from backward_token_expert_amd import lrm
    T, k, K, d = 70001, 8, 530003, 16
    P = lrm.make_problem(T, k, 8, 0, 8, 8, d, dtype, K, K)
    rng = np.random.default_rng(1)
    sel = rng.permutation(T * k)[:K].astype(np.int32)
    dphi = rng.normal(size=(K, d)).astype(np.float32)
    phi = torch.from_numpy(rng.normal(size=(K, d))).to(torch.float32 if dtype == "f32" else torch.bfloat16)
    off = np.zeros(9, np.int32)
    off[1:] = K
    ws = torch.randint(0, 255, (lrm.lrm_forward_workspace_bytes(P),), dtype=torch.uint8, device="cuda")
    ws[:4] = 0
    adot = torch.full((T * k,), 9.0, device="cuda")
    lrm.lrm_gate_dots(P, _dev(sel), _dev(off), _dev(dphi), phi.cuda(), adot, ws)
    assert lrm.lrm_read_device_error(ws) == 0
    want, size = F.gate_dots(dphi.astype(np.float64), phi.double().numpy(), sel, T * k)
    assert np.all(np.abs(adot.cpu().numpy() - want) <= U * np.abs(want) + 2.0 ** -45 * size)


# rows an expert pick the tile: Low below 24, MidFew below 96, Mid below 256, Big.  Every case has more units
# than workgroups (256, of Low 512) in FC1 or FC2, of five to sixteen K steps, more than a ring holds;
# the last step is partial.
FC = [dict(T=1000, k=2, E=100, h=264, d=1024), dict(T=1000, k=2, E=100, h=1032, d=328),
      dict(T=1000, k=2, E=100, h=1032, d=328, skew=[60] + [1] * 99),
      dict(T=3000, k=2, E=100, h=264, d=1024), dict(T=3000, k=2, E=100, h=1032, d=264),
      dict(T=3000, k=2, E=100, h=264, d=1032, skew=[40, 0, 0] + [1] * 97),
      dict(T=8000, k=2, E=100, h=264, d=1024), dict(T=8000, k=2, E=100, h=1032, d=264),
      dict(T=20000, k=1, E=20, h=264, d=1032), dict(T=20000, k=1, E=20, h=1032, d=264)]
FC_IDS = ["T%dh%dd%d%s" % (c["T"], c["h"], c["d"], "skewed" if "skew" in c else "") for c in FC]


@pytest.mark.parametrize("case", FC, ids=FC_IDS)
def test_expert_products(case):
    print(f"[case] {case}", flush=True)
    c = Case(dtype="bf16", e_lo=0, E_loc=case["E"], **case)
    check_fc1(c)
    check_fc2(c, residual=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("E,E_loc", [(2, 2), (300, 2)])
def test_return_to_more_tokens_than_wavefronts(E, E_loc, dtype):
    """65536 wavefronts to a pass; few local rows are looked up without the map."""
    c = Case(T=70001, k=1, E=E, e_lo=0, E_loc=E_loc, h=8, d=16, dtype=dtype)
    assert (c.L_cap <= 1024) == (E == 300)
    check_fc2(c, residual=True)
    check_fc2(c, residual=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("sizes", [[9_000_001, 7], [3] * 64 + [9_000_001, 5], [1, 75_000_003, 30_000_011]],
                         ids=["chunks", "launches", "past the kept part"])
def test_clip(sizes, dtype):
    """1024 chunks of 32 KiB to a pass; 64 tensors to a launch; 192 MB of a launch's list stay in the
    memory-side cache, what lies before streams past it."""
    import torch
    from backward_token_expert_amd import lrm, path
    t = torch.float32 if dtype == "f32" else torch.bfloat16
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    src = [torch.randn(n, generator=g, device="cuda").to(t) for n in sizes]
    total = sum(float(torch.dot(a.double(), a.double())) for a in src) ** 0.5
    dst = [torch.full_like(a, 9.0) for a in src]
    clip = path.GradientClip(src, dst)
    clip.ws.random_()
    norm = clip(0.3 * total).item()
    assert lrm.lrm_read_device_error(clip.ws) == 0
    assert abs(norm - total) <= 2 * U * total
    e = 4 * U + (2.0 ** -8 if dtype == "bf16" else 0)
    for a, b in zip(src, dst):
        want = a.double() * 0.3
        assert bool(((b.double() - want).abs() <= e * want.abs() + 1e-38).all())
    only = torch.zeros(1, device="cuda")
    lrm.lrm_grad_norm(clip.list, only, clip.ws)
    assert only.item() == norm
    inplace = path.GradientClip(src)
    assert inplace(0.3 * total).item() == norm
    assert all(torch.equal(a, b) for a, b in zip(src, dst))


# the serving kernel, float32's of up to 128 tokens, float32's and bf16's of more
@pytest.mark.parametrize("T,dtype", [(1, "bf16"), (40, "f32"), (200, "f32"), (40, "bf16"), (3000, "bf16")])
def test_wild_offsets_stay_inside_the_buffers(T, dtype):
    """Offsets past the capacity, negative, or running backwards are clamped: rows of the capacity may be
    written, nothing beside it, and pairs that are none are reported."""
    import torch
    from backward_token_expert_amd import lrm
    c = Case(T=T, k=2, E=4, e_lo=0, E_loc=4, h=64, d=32, dtype=dtype)
    rp, _ = c.device_rows()                       # the spare rows' pair ids are none
    off = torch.tensor([0, 10 ** 6, -5, 2 * T // 3, 2 ** 31 - 1], dtype=torch.int32, device="cuda")

    def guarded(width):
        base = c.rows(c.L_cap + 600, width, 5.0)
        return base, base[300:300 + c.L_cap]

    def whole(base):
        return bool((base[:300] == 5.0).all()) and bool((base[300 + c.L_cap:] == 5.0).all())
    (ab, ac), (pb, phi), (yb, y) = guarded(2 * c.d), guarded(c.d), guarded(c.h)
    x = torch.nan_to_num(c.x)
    lrm.lrm_grouped_fc1_swiglu(c.P, rp, off, x, c.W1, ac, phi, c.ws)
    assert lrm.lrm_read_device_error(c.ws, clear=True) == 32
    assert whole(ab) and whole(pb)
    spare = phi[c.L:]                             # rows of no pair read x as zeros
    assert not spare.any()
    lrm.lrm_grouped_fc2(c.P, off, phi, c.W, y, c.ws)
    assert whole(yb) and whole(pb)
    ob = c.rows(c.T + 600, c.h, 5.0)
    lrm.lrm_combine_tokens(c.P, rp, off, _dev(c.w), y, None, ob[300:300 + c.T], c.ws)
    assert lrm.lrm_read_device_error(c.ws, clear=True) == 32
    assert bool((ob[:300] == 5.0).all()) and bool((ob[300 + c.T:] == 5.0).all())


@pytest.mark.parametrize("h,d", [(1032, 4104), (4104, 1032), (2048, 1024)])
def test_one_token_of_wide_and_narrow_products(h, d):
    """One token's products on either side of what the serving kernel takes (by its units of work)."""
    c = Case(T=1, k=8, E=8, e_lo=0, E_loc=8, h=h, d=d, dtype="bf16")
    check_fc1(c)
    check_fc1(c, keep_ac=False)
    check_fc2(c, residual=True)
    s = Case(T=1, k=8, E=32, e_lo=8, E_loc=8, h=h, d=d, dtype="bf16")     # a share: two of its experts
    check_fc1(s)
    check_fc2(s, residual=False)

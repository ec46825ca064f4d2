"""The router (rfp2_moe_route) against its formula in float64: ids equal as whole numbers; weights within 2^-20 of
themselves (expf 2 ulp on an argument that is rounded once, sums of up to 1024 terms in a tree, a quotient, a
factor: under 16 roundings of 2^-24)."""
import numpy as np
import pytest

import _feedforward as plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import gemm_rocmfp2_mul_gb300 as g
    g.build()
    g.lib()
    return g


def check(g, x, top_k, bias=None, **kw):
    """x: a tensor of logits on the GPU."""
    import torch
    ids, weights = g.rfp2_moe_route(x, top_k, bias=None if bias is None else torch.from_numpy(bias).cuda(), **kw)
    want, w = plain.route(x.double().cpu().numpy(), top_k, bias=bias, **kw)
    np.testing.assert_array_equal(ids.cpu().numpy(), want)
    got = weights.double().cpu().numpy()
    np.testing.assert_array_equal(np.isnan(got), np.isnan(w))
    ok = ~np.isnan(w)
    assert np.all(np.abs(got - w)[ok] <= np.abs(w)[ok] * 2.0 ** -20 + 2.0 ** -140)
    return ids, weights


def logits(T, E, dtype="float32", seed=0, masked=0.0):
    import torch
    r = torch.Generator(device="cuda").manual_seed(seed)
    x = 1.5 * torch.randn((T, E), generator=r, device="cuda") + 0.7 * torch.randn((1, E), generator=r, device="cuda")
    x[torch.rand((T, E), generator=r, device="cuda") < masked] = -float("inf")
    return x.to(getattr(torch, dtype))


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("E,top_k", [(1, 1), (2, 2), (8, 2), (31, 5), (32, 32), (33, 4), (60, 4), (64, 6), (100, 8), (160, 6),
                                     (256, 8), (384, 9), (512, 32), (777, 7), (1024, 10)])
def test_choice(g, E, top_k, scoring, biased):
    bias = 0.1 * np.random.default_rng(1).standard_normal(E).astype(np.float32) if biased else None
    for dtype, masked in (("float32", 0.0), ("bfloat16", 0.3), ("float16", 0.0)):
        check(g, logits(150, E, dtype, E, masked), top_k, bias, scoring=scoring, renormalise=dtype != "float16", scale=2.5)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("E,groups,keep,top_k", [(256, 8, 4, 8), (256, 8, 1, 8), (64, 8, 3, 6), (60, 4, 2, 4), (160, 5, 5, 3),
                                                 (32, 32, 7, 7), (512, 16, 4, 12), (96, 3, 2, 8), (256, 2, 1, 4), (256, 4, 3, 5), (512, 4, 2, 8),
                                                 (512, 8, 5, 8), (1024, 8, 3, 5), (768, 8, 2, 4)])
def test_groups(g, E, groups, keep, top_k, group_top, biased, scoring):
    bias = 0.1 * np.random.default_rng(2).standard_normal(E).astype(np.float32) if biased else None
    for dtype, masked in (("float32", 0.0), ("bfloat16", 0.6), ("float32", 0.97)):
        check(g, logits(120, E, dtype, E + keep, masked), top_k, bias, scoring=scoring, groups=groups, keep=keep,
              group_top=group_top)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_ties_go_to_the_lowest_index(g, scoring, groups):
    """Rows of one value, of few values, and 16-bit logits whose biases are zero: exact ties."""
    import torch
    kw = dict(scoring=scoring, groups=groups, keep=2 if groups > 1 else 1, group_top=2)
    for E in (32, 256):
        flat = torch.zeros((3, E), device="cuda")
        few = torch.randint(0, 3, (40, E), device="cuda", generator=torch.Generator(device="cuda").manual_seed(3)).float()
        for bias in (None, np.zeros(E, np.float32), np.full(E, 0.25, np.float32)):
            zeros = torch.where(few > 0, 0.0, -0.0)   # both zeros are one value
            for x in (flat, few, zeros, logits(60, E, "bfloat16", 4)):
                check(g, x, 8, bias, **kw)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [48, 256])
def test_values_too_near_for_fp32(g, scoring, E):
    """Biases that take every expert's value to 1 within half a step of fp32: 64 bits decide.  All of a row's,
    a few of them, and pairs."""
    x = logits(1, E, seed=5).cpu()
    v = x.double().numpy()[0]
    score = np.exp(v - v.max()) / np.exp(v - v.max()).sum() if scoring == "softmax" else 1 / (1 + np.exp(-v))
    near = (1.0 - score).astype(np.float32)
    rows = x.repeat(4, 1)
    for some in (slice(None), slice(3, 9), slice(0, None, 7)):
        bias = np.full(E, -0.5, np.float32)
        bias[some] = near[some]
        for groups in (1, 4):
            check(g, rows.cuda(), 6, bias, scoring=scoring, groups=groups, keep=2 if groups > 1 else 1, group_top=2)


def test_saturated_scores(g):
    """Sigmoids of 1 within a step of fp32, and of 0: without a bias the logits decide."""
    import torch
    r = np.random.default_rng(6)
    x = torch.from_numpy(np.concatenate([20 + r.random((20, 128)), -90 - 30 * r.random((20, 128))]).astype(np.float32)).cuda()
    check(g, x, 8, scoring="sigmoid")
    check(g, x, 8, scoring="sigmoid", groups=8, keep=3, group_top=1)
    check(g, x, 8, np.zeros(128, np.float32), scoring="sigmoid")
    check(g, 40 * x, 8, scoring="softmax", renormalise=False)


def test_masks_infinities_and_nan(g):
    """Rows that a mask leaves nothing or too little, masks of the type's lowest value, rows without an answer."""
    import torch
    inf, low = float("inf"), torch.finfo(torch.float32).min
    x = logits(8, 64, seed=7)
    x[0] = -inf
    x[1, 3:] = -inf
    x[2, 5:] = low
    x[3, 9] = float("nan")
    x[4, 11] = inf
    x[5] = low
    for scoring in ("softmax", "sigmoid"):
        for renormalise in (True, False):
            check(g, x, 6, scoring=scoring, renormalise=renormalise)
            check(g, x, 6, scoring=scoring, renormalise=renormalise, groups=8, keep=2)
            bias = np.zeros(64, np.float32)
            bias[:10] = -np.inf
            check(g, x, 6, bias, scoring=scoring, renormalise=renormalise)
            bias[0] = np.nan
            ids, w = check(g, x, 6, bias, scoring=scoring, renormalise=renormalise)
            assert bool((ids == -1).all()) and bool(w.isnan().all())


def test_strides_nothing_to_do_and_refusals(g):
    import torch
    wide = logits(50, 200, seed=8)
    x = wide[:, 3:131]
    a, b = g.rfp2_moe_route(x, 4), g.rfp2_moe_route(x.contiguous(), 4)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert g.rfp2_moe_route(x[:0], 4)[0].shape == (0, 4)
    one = torch.ones(128, device="cuda")
    for kw in (dict(top_k=33), dict(top_k=129), dict(top_k=0), dict(top_k=2, groups=3), dict(top_k=2, groups=4, keep=5),
               dict(top_k=2, groups=4, keep=0), dict(top_k=2, group_top=3), dict(top_k=2, scale=float("inf")),
               dict(top_k=2, groups=64)):
        with pytest.raises(g.RFP2Error):
            g.rfp2_moe_route(x, **kw)
    for call in (lambda: g.rfp2_moe_route(x, 4, bias=one[:5]), lambda: g.rfp2_moe_route(x[0], 4, ids=a[0], weights=a[1]),
                 lambda: g.rfp2_moe_route(x, 5, ids=a[0], weights=a[1]), lambda: g.rfp2_moe_route(x, 4, ids=a[0][:3], weights=a[1]),
                 lambda: g.rfp2_moe_route(x.T, 4)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        g.rfp2_moe_route(x.long(), 4)
    with pytest.raises(KeyError):
        g.rfp2_moe_route(x, 4, scoring="tanh")
    with pytest.raises(RuntimeError, match="gradient"):
        g.rfp2_moe_route(x.clone().requires_grad_(), 4)

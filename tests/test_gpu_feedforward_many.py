"""The feed-forward operators where their kernels go around more than once, on random data throughout: CTA pairs
that take several units of experts of uneven sizes, plans of many pairs, CTAs that walk over many tokens, rows of
several runs a thread.  Bounds as in the operators' own tests."""
import numpy as np
import pytest

import _feedforward as plain
import test_gpu_combine
import test_gpu_norm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import gemm_rocmfp2_mul_gb300 as g
    g.build()
    g.lib()
    return g


def blocks(E, M, K, seed, scales=(0, 28)):
    r = np.random.default_rng(seed)
    W = r.integers(0, 256, (E, M, K // 32, 10), dtype=np.uint8)
    W[..., 8:] = r.integers(*scales, W[..., 8:].shape)
    return W


def routed(T, E, k, seed, liked=1.5):
    r = np.random.default_rng(seed)
    score = r.standard_normal((T, E)) + liked * r.standard_normal((1, E))
    return np.argsort(-score, axis=1)[:, :k].astype(np.int32)


def check_products(g, W, ids, seed, bias=None, kind="none", each=False):
    """All rows of y against float64, the experts' one after another."""
    import torch
    E, M, K = W.shape[0], W.shape[1], W.shape[2] * 32
    T, k = ids.shape
    r = torch.Generator(device="cuda").manual_seed(seed)
    X = torch.randn((T, k, K) if each else (T, K), generator=r, device="cuda").bfloat16()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = g.rfp2_moe_gemm(torch.from_numpy(W).cuda(), E, M, K, torch.from_numpy(ids).cuda(), X,
                        None if bias is None else torch.from_numpy(bias).cuda(), kind, dev_status=status)
    assert int(status) == 0
    rows = (X if each else X[:, None].expand(T, k, K)).reshape(T * k, K).double()
    flat = y.flatten(0, 1).double()
    pairs = torch.from_numpy(ids).cuda().flatten()
    assert not flat[pairs < 0].any()
    step = K / 8 * 2.0 ** -23 + 2.0 ** -22    # of the sum of sizes, as in plain.experts
    for e in range(E):
        at = (pairs == e).nonzero()[:, 0]
        if not at.numel():
            continue
        w, x = torch.from_numpy(plain.weights_of(W[e])).cuda(), rows[at]
        z, size = x @ w.T, x.abs() @ w.abs().T
        if bias is not None:
            b = torch.from_numpy(bias[e]).cuda().double()
            z, size = z + b, size + b.abs()
        off = size * step
        if kind != "none":
            (a, u), (da, du) = z.chunk(2, 1), off.chunk(2, 1)
            v = a if kind == "silu" else 2.0 * (2.0 / np.pi) ** 0.5 * (a + 0.044715 * a ** 3)
            act = a * torch.sigmoid(v)
            # act changes by at most 1.13 of its argument's change; the fast exponential of v and the roundings of
            # v itself are off by 2^-21 (2 + |v|) of act, which is below 2^-19 |a|
            z, off = act * u, (1.13 * da + 2.0 ** -19 * a.abs()) * (u.abs() + du) + act.abs() * du
        bound = (off + z.abs() * 2.0 ** -8) * (1 + 2.0 ** -8) + 2.0 ** -133
        assert bool(((flat[at] - z).abs() <= bound).all()), e


@pytest.mark.parametrize("kind,biased,each", [("none", False, False), ("silu", True, False), ("gelu", False, True)])
@pytest.mark.parametrize("T,E,M,K,k", [(600, 128, 512, 256, 4),      # tiles of 64 tokens: 256 units and more
                                       (700, 64, 1024, 512, 5),      # of 128
                                       (2000, 16, 4096, 256, 3)])    # of 256
def test_pairs_that_take_many_units(g, T, E, M, K, k, kind, biased, each):
    bias = np.random.default_rng(4).standard_normal((E, M)).astype(np.float32) if biased else None
    check_products(g, blocks(E, M, K, 1), routed(T, E, k, 2), 3, bias, kind, each)


@pytest.mark.parametrize("kind", ["none", "silu"])
def test_plans_of_many_pairs(g, kind):
    """More pairs than a warp of the plan keeps in registers, some of them without an expert."""
    W, ids = blocks(200, 96, 256, 5), routed(1600, 200, 6, 6)
    ids[np.random.default_rng(7).random(ids.shape) < 0.1] = -1
    check_products(g, W, ids, 8, kind=kind)


def test_one_expert_of_thousands_among_narrow_tiles(g):
    W, ids = blocks(256, 256, 256, 9), routed(1000, 256, 8, 10)
    ids[:, 2:5] = 7
    check_products(g, W, ids, 11, kind="silu")


@pytest.mark.parametrize("kind", ["none", "gelu"])
def test_scales_of_every_size(g, kind):
    W = blocks(3, 256, 256, 12, (0, 127))
    W[0, :127, 0, 8] = np.arange(127)
    check_products(g, W, routed(150, 3, 2, 13), 14, kind=kind)


@pytest.mark.parametrize("dtype,otype", [("bfloat16", "bfloat16"), ("float16", "float32"), ("float32", "float32")])
@pytest.mark.parametrize("T,k,M", [(2500, 8, 2048), (2500, 9, 1001), (20000, 3, 96), (3000, 4, 333)])
def test_combinations_of_many_tokens(g, T, k, M, dtype, otype):
    import torch
    made = test_gpu_combine.made
    y, w, rest = made((T, k, M), dtype, 1), made((T, k), "float32", 2), made((T, M), otype, 3)
    ids = torch.randint(-1, 4, (T, k), device="cuda", generator=torch.Generator(device="cuda").manual_seed(4), dtype=torch.int32)
    out = g.rfp2_moe_combine(y, w, ids=ids, residual=rest)
    test_gpu_combine.check(out, y, w, ids, rest)
    test_gpu_combine.check(g.rfp2_moe_combine(y, w), y, w)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("T,K", [(701, 64), (701, 1000), (701, 2048), (400, 5120), (330, 16384), (701, 4097)])
def test_norms_of_many_rows(g, T, K, dtype):
    import torch
    made = test_gpu_norm.made
    x, rest = made(T, K, dtype, 1), made(T, K, dtype, 2, 3.0)
    weight = 1.0 + 0.3 * made(1, K, "float32", 3)[0]
    n = g.rfp2_rms_norm(x, weight, residual=rest)
    assert torch.equal(n.total, (x.float() + rest.float()).to(x.dtype))
    test_gpu_norm.check(n.total, weight, n)

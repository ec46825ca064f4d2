"""The routed experts' products (rfp2_moe_gemm) against the formula in float64 on the weights that the blocks stand
for: sums and activations in fp32 as tests/_feedforward.py bounds them, then one rounding to bf16."""
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


def blocks(E, M, K, seed):
    """Selectors at random, scales of every size that keeps a row's sums in range."""
    r = np.random.default_rng(seed)
    W = r.integers(0, 256, (E, M, K // 32, 10), dtype=np.uint8)
    W[..., 8:] = r.integers(0, 28, W[..., 8:].shape)
    return W


def routed(T, E, k, seed, liked=0.7):
    r = np.random.default_rng(seed)
    score = r.standard_normal((T, E)) + liked * r.standard_normal((1, E))
    return np.argsort(-score, axis=1)[:, :k].astype(np.int32)


def run(g, W, ids, X, bias=None, kind="none", **kw):
    import torch
    E, M, K = W.shape[0], W.shape[1], W.shape[2] * 32
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = g.rfp2_moe_gemm(torch.from_numpy(W).cuda(), E, M, K, torch.from_numpy(ids).cuda(), X,
                        None if bias is None else torch.from_numpy(bias).cuda(), kind, dev_status=status, **kw)
    return y, int(status)


def check(y, W, ids, X, bias=None, kind="none"):
    ref, off = plain.experts(W, ids, X.double().cpu().numpy(), bias, kind)
    got = y.double().cpu().numpy()
    assert np.all(np.abs(got - ref) <= (off + np.abs(ref) * 2.0 ** -8) * (1 + 2.0 ** -8) + 2.0 ** -133)


def tokens(shape, seed):
    import torch
    r = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=r, device="cuda").bfloat16()


@pytest.mark.parametrize("kind", ["none", "silu", "gelu"])
@pytest.mark.parametrize("T,E,M,K,k", [(1, 1, 32, 256, 1), (1, 4, 96, 512, 2), (5, 8, 256, 256, 8), (17, 3, 288, 768, 2),
                                       (40, 16, 544, 256, 4), (300, 2, 64, 256, 1), (700, 3, 320, 512, 2), (33, 60, 32, 256, 4)])
@pytest.mark.parametrize("biased,each", [(False, False), (True, True)])
def test_products(g, T, E, M, K, k, kind, biased, each):
    W, ids = blocks(E, M, K, 1), routed(T, E, k, 2)
    X = tokens((T, k, K) if each else (T, K), 3)
    bias = np.random.default_rng(4).standard_normal((E, M)).astype(np.float32) if biased else None
    y, status = run(g, W, ids, X, bias, kind)
    assert status == 0
    check(y, W, ids, X, bias, kind)


@pytest.mark.parametrize("M", [16, 48, 144, 272])
def test_rows_that_end_inside_a_tile(g, M):
    W, ids, X = blocks(3, M, 256, 5), routed(70, 3, 2, 6), tokens((70, 256), 7)
    y, _ = run(g, W, ids, X)
    check(y, W, ids, X)


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 127, 128, 129, 255, 256, 257, 513])
def test_lengths_of_an_experts_run(g, n):
    """One expert has n tokens, the next none, another three."""
    W, X = blocks(4, 64, 256, 8), tokens((n + 3, 256), 9)
    ids = np.full((n + 3, 1), 1, np.int32)
    ids[np.random.default_rng(10).permutation(n + 3)[:3]] = 3
    y, _ = run(g, W, ids, X, kind="silu")
    check(y, W, ids, X, kind="silu")


def test_all_slots_of_one_expert(g):
    """The same expert for every slot, and twice for one token."""
    W, X = blocks(5, 64, 256, 11), tokens((50, 256), 12)
    ids = np.full((50, 3), 2, np.int32)
    y, _ = run(g, W, ids, X)
    check(y, W, ids, X)
    assert bool((y[:, 0] == y[:, 1]).all())


def test_ids_without_an_expert(g):
    """-1: a row of zeros and no error; another id outside: NaN and RFP2_EBADID; neither touches its neighbours."""
    W, X, ids = blocks(6, 96, 256, 13), tokens((64, 256), 14), routed(64, 6, 3, 15)
    lost = np.random.default_rng(16).random(ids.shape) < 0.2
    ids[lost] = -1
    y, status = run(g, W, ids, X, kind="gelu")
    assert status == 0 and not y[lost].any()
    check(y, W, ids, X, kind="gelu")
    bad = ids.copy()
    bad[3, 1], bad[40, 0], bad[7, 2] = 6, -2, 2 ** 31 - 1
    z, status = run(g, W, bad, X, kind="gelu")
    assert status == 7
    changed = bad != ids
    assert bool(z[changed].isnan().all()) and bool((z[~changed] == y[~changed]).all())
    none, status = run(g, W, np.full((9, 2), -1, np.int32), X[:9])
    assert status == 0 and not none.any()


def test_outputs_and_workspace_of_the_caller(g):
    """A workspace may be larger than its call needs, hold anything, and be used again; bytes beside it stay."""
    import torch
    W, X, ids = blocks(8, 64, 256, 17), tokens((90, 256), 18), routed(90, 8, 2, 19)
    want, _ = run(g, W, ids, X)
    n = g.rfp2_moe_gemm_workspace_bytes(90, 2, 8)
    held = torch.randint(0, 256, (n + 512,), dtype=torch.uint8, device="cuda")
    copy = held.clone()
    Y = torch.full((90, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    for count in (90, 90, 11):
        y, _ = run(g, W, ids[:count], X[:count], Y=Y[:count], workspace=held[:n])
        assert torch.equal(y, want[:count])
    assert torch.equal(held[n:], copy[n:])
    with pytest.raises(g.RFP2Error):
        run(g, W, ids, X, workspace=held[: n - 1])
    with pytest.raises(g.RFP2Error):
        run(g, W, ids, X, workspace=held[1: n + 1])


def test_values_that_are_not_finite(g):
    """A token's infinities and NaN stay with its own rows."""
    import torch
    W, X, ids = blocks(4, 64, 256, 20), tokens((40, 256), 21), routed(40, 4, 2, 22)
    want, _ = run(g, W, ids, X)
    X = X.clone()
    X[5, 17], X[9, 200] = float("nan"), float("inf")
    y, _ = run(g, W, ids, X)
    assert bool(y[5].isnan().all()) and not bool(y[9].isfinite().any())
    rest = [t for t in range(40) if t not in (5, 9)]
    assert torch.equal(y[rest], want[rest])


def test_agrees_with_the_gemv(g):
    """What rfp2_moe_gemv computes for a few tokens, but for its 8-bit activations and the rounding to bf16: each
    activation is off by at most 1/254 of its block's largest, uniformly."""
    import torch
    W, ids, X = blocks(16, 128, 512, 23), routed(8, 16, 4, 24), tokens((8, 512), 25)
    y, _ = run(g, W, ids, X)
    v = g.rfp2_moe_gemv(torch.from_numpy(W).cuda(), 16, 128, 512, torch.from_numpy(ids).cuda(), X.float())
    assert float((y.float() - v).norm() / v.norm()) < 0.02


def test_refusals(g):
    import torch
    W, X, ids = torch.from_numpy(blocks(2, 64, 256, 26)).cuda(), tokens((4, 256), 27), torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    assert g.rfp2_moe_gemm(W, 2, 64, 256, ids[:0], X[:0]).shape == (0, 2, 64)
    with pytest.raises(g.RFP2Error):  # gated rows that are no whole number of 16
        g.rfp2_moe_gemm(torch.zeros((2, 48, 8, 10), dtype=torch.uint8, device="cuda"), 2, 48, 256, ids, X, activation="silu")
    with pytest.raises(g.RFP2Error):
        g.rfp2_moe_gemm(torch.zeros((2, 64, 1, 10), dtype=torch.uint8, device="cuda"), 2, 64, 32, ids, X[:, :32].contiguous())
    for call in (lambda: g.rfp2_moe_gemm(W, 2, 64, 512, ids, X), lambda: g.rfp2_moe_gemm(W, 2, 32, 256, ids, X),
                 lambda: g.rfp2_moe_gemm(W, 2, 64, 256, ids, X[:3]), lambda: g.rfp2_moe_gemm(W, 2, 64, 256, ids, X[:, None]),
                 lambda: g.rfp2_moe_gemm(W, 2, 64, 256, ids, X, bias=torch.zeros((2, 32), device="cuda")),
                 lambda: g.rfp2_moe_gemm(W, 2, 64, 256, ids[0], X, Y=torch.empty((4, 2, 64), device="cuda").bfloat16(), workspace=W.view(-1)),
                 lambda: g.rfp2_moe_gemm(W, 2, 64, 256, ids, X, activation="silu", Y=torch.empty((4, 2, 64), device="cuda").bfloat16())):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        g.rfp2_moe_gemm(W, 2, 64, 256, ids, X.float())
    with pytest.raises(KeyError):
        g.rfp2_moe_gemm(W, 2, 64, 256, ids, X, activation="relu")
    with pytest.raises(RuntimeError, match="gradient"):
        g.rfp2_moe_gemm(W, 2, 64, 256, ids, X.clone().requires_grad_())

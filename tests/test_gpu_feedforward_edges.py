"""The feed-forward operators at the ends of their ranges."""
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


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups", [(64, 4), (256, 8), (256, 4), (1024, 8), (60, 5)])
def test_biases_of_the_lowest_and_the_largest_value(g, E, groups, scoring):
    """A bias of the type's lowest value switches experts off, but it is a value: a group whose two largest sum
    past fp32 has experts all the same, and counts as the formula in 64 bits says.  So does one of the largest."""
    import torch
    r = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((12, E), generator=r, device="cuda")
    x[3, E // 2:] = -float("inf")
    low, size = np.float32(np.finfo(np.float32).min), E // groups
    off, some, far, ever = (np.zeros(E, np.float32) for _ in range(4))
    off[size:] = low                                       # all groups but the first
    some[:] = low
    some[: 2 * size: 3] = 0.25                             # a few experts of the first two
    far[:] = np.repeat(low * np.linspace(0.6, 1.0, groups)[::-1].astype(np.float32), size)   # sums 1.2 ... 2 times the lowest
    ever[size: 2 * size: 5] = np.inf
    for bias in (off, some, far, -far, ever, np.full(E, low), np.full(E, -low)):
        for keep in (1, 2, groups - 1, groups):
            ids, weights = g.rfp2_moe_route(x, 8, scoring=scoring, bias=torch.from_numpy(bias).cuda(), groups=groups, keep=keep, group_top=2)
            want, w = plain.route(x.double().cpu().numpy(), 8, scoring, bias, groups, keep, 2)
            np.testing.assert_array_equal(ids.cpu().numpy(), want)
            assert np.all(np.abs(weights.double().cpu().numpy() - w) <= w * 2.0 ** -20)


def products(g, gate, up, kind):
    """rfp2_moe_gemm of rows whose gate and up values are exactly these bf16 numbers: y [T]."""
    import torch
    W = np.zeros((1, 32, 8, 10), np.uint8)
    W[..., :8] = 0xAA                       # level 1 everywhere
    W[0, :16, 0, 8] = W[0, 16:, 0, 9] = 64  # gate rows see the first 16 columns, up rows the next, with scale 1
    X = torch.zeros((len(gate), 256), dtype=torch.bfloat16, device="cuda")
    X[:, 3], X[:, 20] = gate, up
    ids = torch.zeros((len(gate), 1), dtype=torch.int32, device="cuda")
    y = g.rfp2_moe_gemm(torch.from_numpy(W).cuda(), 1, 32, 256, ids, X, activation=kind)
    assert bool(((y == y[..., :1]) | y.isnan()).all())
    return y[:, 0, 0]


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_activations_of_very_negative_gates(g, kind):
    """act(gate) far below 1, times an up value that brings it back: where 1 + exp(-v) is near the end of fp32's
    range and past it.  v is off by five roundings of up to 2^-24 |v| and its exponential by (2 + 1.2 |v|) 2^-23:
    2^-13 of the result at |v| <= 170, beside its own rounding."""
    import torch
    gate = torch.linspace(-160, 2, 649, device="cuda") if kind == "silu" else torch.linspace(-12.5, 1, 649, device="cuda")
    gate = gate.bfloat16()
    for up in (1.0, -2.0 ** 100):
        y = products(g, gate, torch.full_like(gate, up), kind).double().cpu().numpy()
        a = gate.double().cpu().numpy()
        v = a if kind == "silu" else 2.0 * np.sqrt(2.0 / np.pi) * (a + 0.044715 * a ** 3)
        ref = a / (1.0 + np.exp(-v)) * up
        # (below 2^-126 a bf16 has steps of 2^-133)
        assert np.all(np.abs(y - ref) <= np.abs(ref) * (2.0 ** -8 + 2.0 ** -13) + 2.0 ** -133)


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_activations_at_the_ends(g, kind):
    """Gates of any size and NaN: 0 below, the gate above."""
    import torch
    gate = torch.tensor([-3e38, -1e20, -1e10, -300.0, 0.0, 300.0, 1e10, 1e20, 3e38, float("nan")], device="cuda").bfloat16()
    y = products(g, gate, torch.ones_like(gate), kind)
    assert not y[:5].any() and torch.equal(y[5:9], gate[5:9]) and bool(y[9].isnan())


@pytest.mark.parametrize("M,kind", [(16, "none"), (32, "silu"), (1040, "none"), (4128, "gelu")])
def test_rows_without_an_expert(g, M, kind):
    """Most rows lost, in stretches and here and there, of every length that a warp writes: zeros for -1, NaN for
    another id, the others as without them."""
    import torch
    r = np.random.default_rng(4)
    T, k, E = 900, 4, 6
    W = r.integers(0, 256, (E, M, 8, 10), dtype=np.uint8)
    W[..., 8:] %= 28
    W, X = torch.from_numpy(W).cuda(), torch.randn((T, 256), device="cuda").bfloat16()
    ids = r.integers(0, E, (T, k)).astype(np.int32)
    want = g.rfp2_moe_gemm(W, E, M, 256, torch.from_numpy(ids).cuda(), X, activation=kind)
    lost = r.random((T, k)) < 0.5
    lost[200:700] = True
    bad = lost & (r.random((T, k)) < 0.3)
    ids[lost] = -1
    ids[bad] = E + 3
    Y = torch.full_like(want, 5.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    g.rfp2_moe_gemm(W, E, M, 256, torch.from_numpy(ids).cuda(), X, activation=kind, Y=Y, dev_status=status)
    assert int(status) == 7
    assert bool(Y[bad].isnan().all()) and not Y[lost & ~bad].any() and torch.equal(Y[~lost], want[~lost])


def test_rows_without_an_expert_hold_nothing_up(g):
    """57344 of 65536 rows without an expert, 822 MB of zeros: written at a fair share of the rate of a plain fill
    (a tenth at least, beside the products of the others), where a value at a time took far longer than that
    and kept the tensor cores waiting, whose waits have a limit."""
    import torch
    T, k, M, K, E = 8192, 8, 7168, 256, 8
    W = torch.zeros((E, M, K // 32, 10), dtype=torch.uint8, device="cuda")
    X = torch.randn((T, K), device="cuda").bfloat16()
    ids = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    ids[:, 0] = torch.arange(T, device="cuda") % E
    Y, workspace = torch.empty((T, k, M), dtype=torch.bfloat16, device="cuda"), g.rfp2_moe_gemm_workspace(ids, E)

    def best(call):
        times = []
        for _ in range(6):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            call()
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        return min(times[1:])

    fill = best(Y.zero_)
    some = best(lambda: g.rfp2_moe_gemm(W, E, M, K, ids[:, :1].contiguous(), X, workspace=workspace))
    both = best(lambda: g.rfp2_moe_gemm(W, E, M, K, ids, X, Y=Y, workspace=workspace))
    print(f"fill {fill:.3f} ms, products {some:.3f} ms, together {both:.3f} ms")
    assert both - some < 10 * fill


@pytest.mark.parametrize("scoring,renormalise", [("softmax", True), ("softmax", False), ("sigmoid", True)])
def test_weights_of_experts_far_apart(g, scoring, renormalise):
    """Weights are within 2^-20 of themselves however far apart the logits are: what a difference of two loses
    (2^-18 where it is 64) is not lost to its exponential."""
    import torch
    r = np.random.default_rng(2)
    x = torch.from_numpy((-60.0 * r.random((200, 16)) ** 2 - (0.1 if scoring == "softmax" else 18.0)).astype(np.float32)).cuda()
    ids, weights = g.rfp2_moe_route(x, 16, scoring=scoring, renormalise=renormalise)
    want, w = plain.route(x.double().cpu().numpy(), 16, scoring, renormalise=renormalise)
    np.testing.assert_array_equal(ids.cpu().numpy(), want)
    assert np.all(np.abs(weights.double().cpu().numpy() - w) <= w * 2.0 ** -20)


@pytest.mark.parametrize("K", [1, 64, 1001])
def test_an_eps_near_the_largest_value(g, K):
    """Also where it leaves fp32's range together with a mean that does not."""
    import torch
    x = torch.randn((4, K), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").double()
    x[1:3] *= (torch.tensor([[2.0 ** 125.9], [2.0 ** 127.9]], device="cuda") / x[1:3].square().sum(-1, keepdim=True)).sqrt()
    x[3] *= 2.0 ** 100
    x = x.float()
    for eps in (1e38, 3.3e38, float(np.finfo(np.float32).max)):
        y = g.rfp2_rms_norm(x, torch.full((K,), 2.0 ** 40, device="cuda"), eps=eps).y.double().cpu().numpy()
        ref = plain.norm(x.double().cpu().numpy(), np.full(K, 2.0 ** 40), np.float64(np.float32(eps)))
        assert np.all(np.abs(y - ref) <= np.abs(ref) * 31 * plain.U)


def test_outputs_that_require_a_gradient_are_refused(g):
    """What autograd knows of such a tensor would no longer be true of its values."""
    import torch
    x, w = torch.randn((4, 64), device="cuda"), torch.ones(64, device="cuda")
    leaf = lambda *shape, dtype=torch.float32: torch.zeros(shape, dtype=dtype, device="cuda", requires_grad=True)
    grown = (leaf(4, 64) * 2.0)
    W, X = torch.zeros((2, 64, 8, 10), dtype=torch.uint8, device="cuda"), torch.zeros((4, 256), dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    calls = [lambda: g.rfp2_rms_norm(x, w, y=leaf(4, 64)), lambda: g.rfp2_rms_norm(x, w, y=grown),
             lambda: g.rfp2_rms_norm(x, w, residual=x, total=grown), lambda: g.rfp2_rms_norm(x, w, want="q8", d=leaf(4, 2)),
             lambda: g.rfp2_moe_route(x, 2, weights=leaf(4, 2)), lambda: g.rfp2_moe_combine(x.view(4, 2, 32), x[:, :2].contiguous(), out=grown[:, :32]),
             lambda: g.rfp2_moe_gemm(W, 2, 64, 256, ids, X, Y=leaf(4, 2, 64, dtype=torch.bfloat16))]
    for call in calls:
        with pytest.raises(RuntimeError, match="gradient"):
            call()
        with torch.no_grad():
            call()


def test_router_gemv_combination(g):
    """The path of a few tokens: router, rfp2_moe_gemv, combination.  A slot whose id is -1 has a row of NaN from the
    products, as that call answers any id outside, which the combination with ids does not read."""
    import torch
    r = np.random.default_rng(5)
    T, E, M, K, k = 6, 12, 64, 256, 4
    W = r.integers(0, 256, (E, M, K // 32, 10), dtype=np.uint8)
    W[..., 8:] %= 28
    logits = torch.from_numpy(r.standard_normal((T, E)).astype(np.float32)).cuda()
    logits[2, 2:] = logits[4] = -float("inf")
    x = torch.from_numpy(r.standard_normal((T, K)).astype(np.float32)).cuda()
    rest = torch.from_numpy(r.standard_normal((T, M)).astype(np.float32)).cuda()
    ids, weights = g.rfp2_moe_route(logits, k)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = g.rfp2_moe_gemv(torch.from_numpy(W).cuda(), E, M, K, ids, x, dev_status=status)
    assert int(status) == 7 and bool((y.isnan().all(-1) == (ids < 0)).all()) and int((ids < 0).sum()) == 2 + k
    out = g.rfp2_moe_combine(y, weights, ids=ids, residual=rest)
    # activations in 8 bits: off by half a step of 1/127 of their block's largest at most
    w, X = plain.weights_of(W), x.double().cpu().numpy()
    half = np.abs(X).reshape(T, -1, 32).max(-1).repeat(32, -1) / 254
    found, probs = ids.cpu().numpy(), weights.double().cpu().numpy()
    for t in range(T):
        ref, off = rest[t].double().cpu().numpy(), 2.0 ** -20
        for j in range(k):
            if found[t, j] >= 0:
                a = w[found[t, j]]
                ref, off = ref + probs[t, j] * (a @ X[t]), off + probs[t, j] * (np.abs(a) @ (half[t] + 2.0 ** -18 * np.abs(X[t])))
        assert np.all(np.abs(out[t].double().cpu().numpy() - ref) <= off)
    assert torch.equal(out[4], rest[4])


FIRST = """
import sys
import torch
import gemm_rocmfp2_mul_gb300 as g
x, w = torch.ones((4, 256), device="cuda"), torch.ones(256, device="cuda")
W = torch.full((2, 64, 8, 10), 0xAA, dtype=torch.uint8, device="cuda")
W[..., 8:] = 64
stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
stream.wait_stream(torch.cuda.current_stream())
with torch.cuda.stream(stream):
    with torch.cuda.graph(graph, stream=stream):
        n = g.rfp2_rms_norm(x, w, residual=x, dtype=torch.bfloat16)
        ids, weights = g.rfp2_moe_route(x[:, :2], 2)
        y = g.rfp2_moe_gemm(W, 2, 64, 256, ids, n.y)
        out = g.rfp2_moe_combine(y, weights, ids=ids)
    for _ in range(2):
        out.zero_()
        graph.replay()
stream.synchronize()
assert bool((out == 256).all()), out
"""


def test_first_calls_are_captured():
    """A process whose first calls are captured: what a call sets up once is set up there."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_calls_of_several_threads(g):
    """Host threads on streams of their own, the same weights, every operator."""
    import threading
    import torch
    r = np.random.default_rng(6)
    W = r.integers(0, 256, (8, 128, 8, 10), dtype=np.uint8)
    W[..., 8:] %= 28
    W, w = torch.from_numpy(W).cuda(), torch.ones(256, device="cuda")
    inputs = [torch.randn((70 + 40 * i, 256), device="cuda") for i in range(4)]

    def layer(x):
        n = g.rfp2_rms_norm(x, w, residual=x, dtype=torch.bfloat16)
        ids, weights = g.rfp2_moe_route(x[:, :8], 3, scoring="sigmoid")
        y = g.rfp2_moe_gemm(W, 8, 128, 256, ids, n.y, activation="silu")
        return g.rfp2_moe_combine(y, weights, ids=ids)

    want = [layer(x) for x in inputs]
    torch.cuda.synchronize()
    got, failed = [None] * 4, []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got[i] = layer(inputs[i])
                torch.cuda.current_stream().synchronize()
        except Exception as e:
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    assert all(torch.equal(a, b) for a, b in zip(got, want))

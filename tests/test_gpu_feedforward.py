"""The feed-forward operators together, as they are used: the layer of examples/expert_layer.py from a replayed
graph, calls on several streams and workspaces shared by graphs, tensors of another device."""
import importlib.util
import os

import numpy as np
import pytest

import _feedforward as plain

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def g():
    import gemm_rocmfp2_mul_gb300 as g
    g.build()
    g.lib()
    return g


@pytest.fixture(scope="module")
def example(g):
    spec = importlib.util.spec_from_file_location("expert_layer", os.path.join(ROOT, "examples", "expert_layer.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    return example


@pytest.mark.parametrize("tokens", [1, 8, 9, 100, 700])
def test_expert_layer(example, tokens):
    """The residual stream is exact but for the last sum.  A token's part of the experts: values enter the products
    as bf16, off by 2^-8 at most and 2^-8 / sqrt(3) in the mean, three times over (norm, hidden rows, the experts'
    rows), each through sums that keep a relative error as it is; the shared expert's Q8 blocks add 0.5 % (half a
    step of 1/127 of the largest of 32, uniform).  1.5 % covers their sum for every token."""
    layer, steps = example.run(tokens)
    for x, residual, out, logits, ids in steps:
        want, _ = plain.route(logits.double().cpu().numpy(), example.TOP_K, "sigmoid", layer.balance.cpu().numpy(),
                              example.GROUPS, example.KEEP, 2)
        np.testing.assert_array_equal(ids.cpu().numpy(), want)
        ref, total = example.reference(layer, x, residual, logits, ids)
        off = (out.double() - total - ref).norm(dim=-1) / ref.norm(dim=-1)
        assert float(off.max()) < 0.015, off.max()
    assert int(layer.status) == 0


def test_two_streams(g, example):
    """Calls that run at the same time, each with its own workspace, do not disturb one another."""
    import torch
    layers = [example.Layer(300, seed) for seed in (1, 2)]
    inputs = [torch.randn((2, 300, example.HIDDEN), device="cuda") for _ in layers]
    want = [layer(*x)[0].clone() for layer, x in zip(layers, inputs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    got = [None, None]
    for _ in range(10):
        for i, (layer, x, s) in enumerate(zip(layers, inputs, streams)):
            with torch.cuda.stream(s):
                got[i] = layer(*x)[0]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_two_graphs_share_a_workspace(g, example):
    """Graphs of calls of other sizes with one workspace, replayed in turn on one stream."""
    import torch
    layer = example.Layer(400, 3)
    x, residual = torch.randn((2, 400, example.HIDDEN), device="cuda")
    sizes = (400, 7, 130)
    want = [layer(x[:n], residual[:n])[0].clone() for n in sizes]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], []
    with torch.cuda.stream(stream):
        for n in sizes:
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=stream):
                outs.append(layer(x[:n], residual[:n])[0])
        for _ in range(3):
            for graph in graphs:
                graph.replay()
    stream.synchronize()
    for a, b in zip(outs, want):
        assert torch.equal(a, b)


def test_offsets_past_32_bits(g):
    """Arrays of more than 2^32 bytes, and of more than 2^31 values: their last rows, against the same rows alone."""
    import torch
    r = torch.Generator(device="cuda").manual_seed(4)
    K, T = 32768, 66000
    x = torch.zeros((T, K), dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn((3, K), generator=r, device="cuda").bfloat16()
    w = 1.0 + 0.1 * torch.randn(K, generator=r, device="cuda")
    far, near = g.rfp2_rms_norm(x, w, residual=x, want="both"), g.rfp2_rms_norm(x[-3:], w, residual=x[-3:], want="both")
    for a, b in zip(far, near):   # (few rows go by another variant: the last bit of a sum may differ)
        assert a[-3:].float().isfinite().all() and not a[:-3].any()
        assert float((a[-3:].float() - b.float()).abs().max()) <= 2.0 ** -7 * float(b.float().abs().max())
    y = x.view(T // 8, 8, K)
    weights = torch.ones((T // 8, 8), device="cuda")
    assert torch.equal(g.rfp2_moe_combine(y, weights)[-1:], g.rfp2_moe_combine(y[-1:], weights[-1:]))
    del far, near, y
    X = x[:, :16384].reshape(-1, 16384)[: 2 * T // 2].repeat(2, 1)   # 132000 rows of 32 KB
    ids = torch.zeros((X.shape[0], 1), dtype=torch.int32, device="cuda")
    W = torch.randint(0, 256, (1, 32, 512, 10), generator=r, device="cuda", dtype=torch.uint8)
    W[..., 8:] %= 24
    out = g.rfp2_moe_gemm(W, 1, 32, 16384, ids, X)
    alone = g.rfp2_moe_gemm(W, 1, 32, 16384, ids[-3:], X[-3:].contiguous())
    assert torch.equal(out[-3:], alone) and bool(alone.any()) and not out[T: -3].any()
    # the last expert's weights, 5 GB in
    E, M = 4, 262144
    W = torch.zeros((E, M, 512, 10), dtype=torch.uint8, device="cuda")
    W[-1, -64:] = torch.randint(0, 256, (64, 512, 10), generator=r, device="cuda", dtype=torch.uint8)
    W[-1, -64:, :, 8:] %= 24
    X, ids = X[-3:].contiguous(), torch.full((3, 1), E - 1, dtype=torch.int32, device="cuda")
    out = g.rfp2_moe_gemm(W, E, M, 16384, ids, X)
    alone = g.rfp2_moe_gemm(W[-1, -64:].contiguous()[None], 1, 64, 16384, torch.zeros_like(ids), X)
    assert torch.equal(out[..., -64:], alone) and not out[..., :-64].any()


def test_tensors_of_another_device_are_refused(g):
    """As with the other operators: without memory, so that no call below can come to a launch."""
    import torch

    class Elsewhere(torch.Tensor):
        @staticmethod
        def __new__(cls, *shape, dtype=torch.float32):
            strides = [1]
            for n in shape[:0:-1]:
                strides.insert(0, strides[0] * n)
            return torch.Tensor._make_wrapper_subclass(cls, shape, strides=strides, dtype=dtype,
                                                       device=f"cuda:{torch.cuda.current_device() + 1}")

        @classmethod
        def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
            raise AssertionError(f"{func} of a tensor without memory")

    x, w, y = Elsewhere(3, 256), Elsewhere(256), Elsewhere(3, 2, 64)
    ids, weights = Elsewhere(3, 2, dtype=torch.int32), Elsewhere(3, 2)
    W, X = Elsewhere(2, 64, 8, 10, dtype=torch.uint8), Elsewhere(3, 256, dtype=torch.bfloat16)
    Y, workspace = Elsewhere(3, 2, 64, dtype=torch.bfloat16), Elsewhere(1 << 20, dtype=torch.uint8)
    for call in (lambda: g.rfp2_rms_norm(x, w, y=x), lambda: g.rfp2_moe_route(x, 2, ids=ids, weights=weights),
                 lambda: g.rfp2_moe_combine(y, weights, out=Elsewhere(3, 64)),
                 lambda: g.rfp2_moe_gemm(W, 2, 64, 256, ids, X, Y=Y, workspace=workspace)):
        with pytest.raises(ValueError, match="current device"):
            call()

"""The sum of a token's experts (rfp2_moe_combine) against its formula in float64: top_k fused additions and the
residual's in fp32 are each off by 2^-24 of what is summed at most, and the result is rounded once."""
import numpy as np
import pytest

import _feedforward as plain

pytestmark = pytest.mark.gpu
TYPES = ["float32", "bfloat16", "float16"]


@pytest.fixture(scope="module")
def g():
    import gemm_rocmfp2_mul_gb300 as g
    g.build()
    g.lib()
    return g


def made(shape, dtype, seed):
    import torch
    r = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=r, device="cuda").to(getattr(torch, dtype))


def check(out, y, w, ids=None, residual=None):
    host = lambda t: None if t is None else t.double().cpu().numpy()
    ref, size = plain.combine(host(y), host(w), None if ids is None else ids.cpu().numpy(), host(residual))
    name = str(out.dtype).split(".")[1]
    bound = (y.shape[1] + 2) * plain.U * size + plain.HALF[name] * np.abs(ref) * (1 + 2.0 ** -20) + plain.TINY[name]
    assert np.all(np.abs(host(out) - ref) <= bound)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("otype", TYPES)
@pytest.mark.parametrize("T,k,M", [(1, 1, 1), (1, 8, 2048), (3, 2, 7), (5, 3, 1001), (40, 6, 256), (2, 9, 64), (1, 33, 24), (300, 4, 96)])
def test_sums(g, T, k, M, dtype, otype):
    import torch
    y, w, rest = made((T, k, M), dtype, 1), made((T, k), "float32", 2), made((T, M), otype, 3)
    ids = torch.randint(-1, 3, (T, k), device="cuda", generator=torch.Generator(device="cuda").manual_seed(4), dtype=torch.int32)
    y[ids < 0] = float("nan")   # rows that are not read
    check(g.rfp2_moe_combine(y, w, ids=ids, residual=rest), torch.where((ids < 0)[..., None], 0, y), w, ids, rest)
    y = torch.where((ids < 0)[..., None], 1, y).to(y.dtype)
    out = g.rfp2_moe_combine(y, w, dtype=getattr(torch, otype))
    assert out.dtype == getattr(torch, otype)
    check(out, y, w)
    rest2 = rest.clone()
    g.rfp2_moe_combine(y, w, ids=ids, residual=rest, out=rest2)
    check(rest2, y, w, ids, rest)


def test_in_place_and_strides(g):
    import torch
    y = made((30, 5, 4, 80), "bfloat16", 5)
    w, wide = made((30, 4), "float32", 6), made((30, 200), "bfloat16", 7)
    for part, rest in ((y[:, 2, :, 8:72], wide[:, 40:104]), (y[:, 1, :, 3:60], wide[:, 1:58])):
        want = g.rfp2_moe_combine(part.contiguous(), w, residual=rest.contiguous())
        check(want, part, w, None, rest)
        kept = wide.clone()
        at = rest.storage_offset()
        mine = kept[:, at: at + rest.shape[1]]
        assert g.rfp2_moe_combine(part, w, residual=mine, out=mine) is mine
        assert torch.equal(mine, want)
        kept[:, at: at + rest.shape[1]] = rest
        assert torch.equal(kept, wide)
        with pytest.raises(g.RFP2Error):
            g.rfp2_moe_combine(part[:29], w[:29], residual=mine[:29], out=mine[1:])


def test_weights_of_nothing_and_nan(g):
    """A slot without an expert adds its weight times 0: a row that has no answer (weights NaN) keeps saying so."""
    import torch
    y, w = made((3, 2, 64), "float32", 8), torch.tensor([[0.5, 0.5], [1.0, 0.0], [float("nan")] * 2], device="cuda")
    ids = torch.tensor([[-1, -1], [3, -1], [-1, -1]], device="cuda", dtype=torch.int32)
    y[0] = y[2] = float("inf")
    y[1, 1] = float("nan")
    out = g.rfp2_moe_combine(y, w, ids=ids)
    assert not out[0].any() and torch.equal(out[1], y[1, 0]) and bool(out[2].isnan().all())


def test_nothing_to_do_and_refusals(g):
    import torch
    y, w = made((4, 2, 64), "float32", 9), made((4, 2), "float32", 10)
    assert g.rfp2_moe_combine(y[:0], w[:0]).shape == (0, 64) and g.rfp2_moe_combine(y[..., :0], w).shape == (4, 0)
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    for call in (lambda: g.rfp2_moe_combine(y, w[:3]), lambda: g.rfp2_moe_combine(y, w, ids=ids[:, :1]),
                 lambda: g.rfp2_moe_combine(y, w, residual=y[:3, 0]), lambda: g.rfp2_moe_combine(y, w, out=y[:, 0, :32]),
                 lambda: g.rfp2_moe_combine(y[0], w), lambda: g.rfp2_moe_combine(y.transpose(1, 2), w),
                 lambda: g.rfp2_moe_combine(y, w, residual=y[:, 0].half(), out=torch.empty((4, 64), device="cuda"))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: g.rfp2_moe_combine(y, w.half()), lambda: g.rfp2_moe_combine(y, w, ids=ids.long()),
                 lambda: g.rfp2_moe_combine(y.int(), w)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(RuntimeError, match="gradient"):
        g.rfp2_moe_combine(y.clone().requires_grad_(), w)

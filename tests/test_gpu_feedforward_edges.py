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

"""The angle that the rotation turns by: position times frequency, exactly."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("how", ["rope", "kv_write"])
def test_the_angle_is_not_rounded(how):
    """cos and sin come back where (1, 0) is turned, each within a unit or two of its last place, so the angle that
    they stand for is off by rounding alone, 3e-8 rad, whichever the angle is.  Were the turn held in one float32,
    between -1/2 and 1/2, that float's rounding (up to 2^-26 turn, 4e-8 rad rms) would show in the result with a
    slope of 1.  The slope's own deviation over N angles is (3e-8 / 4e-8) / sqrt(N): 0.003 for 65536."""
    import torch
    import gemm_rocmfp2_mul_gb300 as g
    g.build()
    T, n = 2048, 32
    r = np.random.default_rng(0)
    f = r.uniform(0.01, 1.0, n).astype(np.float32)
    positions = r.integers(0, 50000, T).astype(np.int32)
    x = np.zeros((T, 1, 2 * n), np.float32)
    x[:, 0, :n] = 1.0
    if how == "kv_write":
        # one pair a block of 32, so that a block's code and scale give the larger of the two to 24 bits
        f = f[:1]
        x = np.zeros((T, 1, 32), np.float32)
        x[:, 0, 0] = 1.0
    args = torch.from_numpy(positions).cuda(), torch.from_numpy(f).cuda()
    if how == "rope":
        y = g.rfp2_rope(torch.from_numpy(x).cuda(), *args).double().cpu().numpy()[:, 0]
        c, s = y[:, :n], y[:, n:]
    turns = positions.astype(np.float64)[:, None] * f.astype(np.float64) / (2 * np.pi)
    turns -= np.round(turns)
    rounded = (turns * 2.0 ** 32).astype(np.float32).astype(np.float64) * 2.0 ** -32
    by_float = 2 * np.pi * (rounded - turns)
    theta = 2 * np.pi * turns
    if how == "rope":
        off = s * np.cos(theta) - c * np.sin(theta)
    else:
        cache = g.rfp2_kv_alloc(T // 16, 1, 16, 32)
        k = torch.from_numpy(x).cuda()
        g.rfp2_kv_write(cache, k, k, torch.arange(T, device="cuda"), *args)
        top = cache[1].double().cpu().numpy().reshape(T, 1) * 127.0     # the larger of |cos|, |sin|
        # its angle from the axis that it is next to, by the smaller's sine or the larger's cosine
        by_cosine = np.abs(np.cos(theta)) >= np.abs(np.sin(theta))
        exact = np.where(by_cosine, np.abs(np.cos(theta)), np.abs(np.sin(theta)))
        slope = np.where(by_cosine, -np.sin(theta) * np.sign(np.cos(theta)), np.cos(theta) * np.sign(np.sin(theta)))
        keep = np.abs(slope) > 0.3
        off, by_float = ((top - exact) / np.where(keep, slope, 1.0))[keep], by_float[keep]
    assert np.abs(off).max() < 1.3e-7 / (1.0 if how == "rope" else 0.3), np.abs(off).max()
    along = float((off * by_float).sum() / (by_float ** 2).sum())
    assert abs(along) < (0.05 if how == "rope" else 0.2), along

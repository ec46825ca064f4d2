"""Rotary positions (rfp2_rope, rfp2_rope_frequencies) against the formula in float64.

Tolerances.  theta is exact to 2^-32 turn and the float that goes into sincospi, in [-1, 1), to 2^-25:
1.0e-7 rad; sincospi adds about 1 ulp.  A rotated value a cos - b sin is then off by at most
(|a| + |b|)(1.0e-7 + 2 * 2^-24) plus three roundings of terms at most |a| + |b|: 5e-7 (|a| + |b|) covers
it.  16-bit outputs add half a unit of their last place (2^-9 relative for bf16, 2^-12 for f16 with a
floor of 2^-25)."""
import numpy as np
import pytest

import _attention as plain

pytestmark = pytest.mark.gpu
HALF_ULP = {"float32": 0.0, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}


@pytest.fixture(scope="module")
def g():
    import gemm_rocmfp2_mul_gb300 as g
    g.build()
    g.lib()
    return g


def _inputs(T, H, D, dtype, seed, top=100000):
    import torch
    r = np.random.default_rng(seed)
    x = torch.from_numpy(r.standard_normal((T, H, D)).astype(np.float32)).to(getattr(torch, dtype))
    positions = r.integers(-top // 8, top, T).astype(np.int32)
    return x, positions


def _check(y, x, positions, f, dtype, **kw):
    x64 = x.double().numpy()
    ref = plain.rope(x64, positions, f, **kw)
    n = len(f)
    pair = np.zeros_like(ref)
    i = np.arange(n)
    a, b = (2 * i, 2 * i + 1) if kw.get("interleaved") else (i, i + n)
    pair[..., a] = pair[..., b] = np.abs(x64[..., a]) + np.abs(x64[..., b])
    bound = 5e-7 * pair * abs(kw.get("factor", 1.0)) + HALF_ULP[dtype] * np.abs(ref) + (2.0 ** -25 if dtype == "float16" else 0)
    err = np.abs(y.double().cpu().numpy() - ref)
    assert np.all(err <= bound), (err - bound).max()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("T,H,D,R", [(1, 1, 128, 128), (5, 8, 64, 32), (33, 3, 96, 64), (7, 20, 192, 64),
                                     (2, 5, 34, 18), (130, 9, 256, 256), (3, 2, 128, 0), (1, 40, 2, 2)])
def test_rope_against_the_formula(g, T, H, D, R, dtype, interleaved):
    x, positions = _inputs(T, H, D, dtype, T + H + D)
    import torch
    f, _ = g.rfp2_rope_frequencies(max(R, 2), device="cpu")
    f = f[: R // 2]
    y = g.rfp2_rope(x.cuda(), torch.from_numpy(positions).cuda(), f.cuda(), interleaved=interleaved, factor=1.25)
    _check(y, x, positions, f.numpy(), dtype, interleaved=interleaved, factor=1.25)


def test_angles_of_long_contexts(g):
    """The largest positions an int32 holds, and frequencies that are no power of anything."""
    import torch
    r = np.random.default_rng(4)
    f = r.uniform(0.3, 1.0, 32).astype(np.float32)
    positions = np.array([0, 1, -1, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31, 12345678], np.int32)
    x = torch.from_numpy(r.standard_normal((7, 2, 64)).astype(np.float32))
    y = g.rfp2_rope(x.cuda(), torch.from_numpy(positions).cuda(), torch.from_numpy(f).cuda())
    # the fraction of a turn per position is exact to 2^-53 or so: 2^31 positions make 2^-22 turn = 1.5e-6 rad
    ref = plain.rope(x.numpy(), positions, f)
    tol = 5e-7 + np.abs(positions.astype(np.float64)) * 2.0 ** -53 * 2 * np.pi
    err = np.abs(y.double().cpu().numpy() - ref).max(axis=(1, 2))
    assert np.all(err <= 8 * tol), err / tol


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_strides_unaligned_rows_and_in_place(g, dtype, interleaved):
    """Heads inside wider rows, at an odd offset, written over themselves or to another layout."""
    import torch
    T, H, D, R = 6, 5, 64, 32
    r = np.random.default_rng(8)
    f, _ = g.rfp2_rope_frequencies(R, device="cpu")
    positions = r.integers(0, 5000, T).astype(np.int32)
    for lead in (0, 3, 8):
        whole = torch.from_numpy(r.standard_normal((T, lead + (H + 2) * D + 5)).astype(np.float32)).to(getattr(torch, dtype))
        x = whole[:, lead: lead + H * D].unflatten(1, (H, D))
        dev = whole.cuda()
        view = dev[:, lead: lead + H * D].unflatten(1, (H, D))
        out = torch.full((H, T, D), 7.0, dtype=x.dtype, device="cuda").transpose(0, 1)
        pos = torch.from_numpy(positions).cuda()
        g.rfp2_rope(view, pos, f.cuda(), out=out, interleaved=interleaved)
        _check(out, x, positions, f.numpy(), dtype, interleaved=interleaved)
        assert g.rfp2_rope(view, pos, f.cuda(), out=view, interleaved=interleaved).data_ptr() == view.data_ptr()
        _check(view, x, positions, f.numpy(), dtype, interleaved=interleaved)
        # nothing outside the heads moved
        mask = torch.ones(whole.shape[1], dtype=torch.bool)
        mask[lead: lead + H * D] = False
        assert torch.equal(dev.cpu()[:, mask], whole[:, mask])


def test_gradient_is_the_inverse(g):
    """Against the formula's transpose, and against differences of the forward call."""
    import torch
    T, H, D, R = 4, 2, 64, 64
    r = np.random.default_rng(3)
    f, _ = g.rfp2_rope_frequencies(R)
    pos = torch.from_numpy(r.integers(0, 9000, T).astype(np.int32)).cuda()
    x, gy, step = (torch.from_numpy(r.standard_normal((T, H, D)).astype(np.float32)).cuda() for _ in range(3))
    for interleaved in (False, True):
        run = lambda t, **kw: g.rfp2_rope(t, pos, f, interleaved=interleaved, factor=1.5, **kw).double()  # noqa: E731
        gx = run(gy, inverse=True)
        ref = plain.rope(gy.cpu().numpy(), pos.cpu().numpy(), f.cpu().numpy(), interleaved=interleaved, inverse=True, factor=1.5)
        assert np.abs(gx.cpu().numpy() - ref).max() <= 5e-7 * 1.5 * 2 * float(gy.abs().max())
        # the map is linear: a difference over any step is its derivative, up to rounding
        diff = ((run(x + step) - run(x - step)) * gy).sum() / 2
        dot = (gx * step).sum()
        size = float((gy.abs().double().sum()) * 4 * 1.5)
        assert abs(float(diff - dot)) <= 2e-6 * size
        # forward then inverse (without its factor): the factor times the identity
        back = g.rfp2_rope(run(x).float(), pos, f, interleaved=interleaved, inverse=True)
        assert float((back.double() - 1.5 * x.double()).abs().max()) <= 1.5 * 2e-6 * 2 * float(x.abs().max())


def test_stream_order(g):
    """The call reads what the current stream wrote just before, on a stream of its own."""
    import torch
    s = torch.cuda.Stream()
    f, _ = g.rfp2_rope_frequencies(128)
    pos = torch.zeros(512, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        x = torch.zeros((512, 32, 128), device="cuda")
        for k in range(20):
            x.fill_(float(k))
            y = g.rfp2_rope(x, pos, f)
            assert bool((y == float(k)).all())


def test_refusals(g):
    import torch
    f, _ = g.rfp2_rope_frequencies(64)
    x = torch.zeros((4, 2, 64), device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        g.rfp2_rope(x.double(), pos, f)
    with pytest.raises(TypeError):
        g.rfp2_rope(x, pos.long(), f)
    with pytest.raises(TypeError):
        g.rfp2_rope(x.cpu(), pos, f)
    with pytest.raises(ValueError):
        g.rfp2_rope(x, pos[:3], f)
    with pytest.raises(ValueError):
        g.rfp2_rope(x.transpose(1, 2), pos, f)
    with pytest.raises(ValueError):
        g.rfp2_rope(x, pos, f, out=torch.zeros((4, 2, 32), device="cuda"))
    with pytest.raises(g.RFP2Error) as e:   # more rotated values than the head has
        g.rfp2_rope(x, pos, torch.zeros(33, device="cuda"))
    assert e.value.status == 2
    assert g.rfp2_rope(x[:0], pos[:0], f).shape == (0, 2, 64)

"""The root-mean-square norm (rfp2_rms_norm) against its formula in float64.

Tolerances: a sum of K <= 32768 squares in fp32, at most 32 in a row and then in a tree of ten levels, is off by
43 roundings (2^-24 each) at most; mean, eps, root and reciprocal add 4; half of the first, then two products: r
and y are within 30 2^-24 of themselves, and a block's scale within 32 2^-24, beside their own last rounding.
Codes are exact: they are compared as whole numbers with those of extended precision."""
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


def made(T, K, dtype, seed=0, size=1.0):
    import torch
    r = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((T, K), generator=r, device="cuda") * torch.exp(0.5 * torch.randn((T, 1), generator=r, device="cuda"))
    return (x * size).to(getattr(torch, dtype))


def check(s, weight, n, eps=1e-6):
    """n: a Norm, of the sums s."""
    s64, w64 = s.double().cpu().numpy(), weight.double().cpu().numpy()
    ref = plain.norm(s64, w64, eps)
    if n.y is not None:
        name = str(n.y.dtype).split(".")[1]
        bound = np.abs(ref) * (30 * plain.U + plain.HALF[name]) + plain.TINY[name] + 2.0 ** -149
        assert np.all(np.abs(n.y.double().cpu().numpy() - ref) <= bound)
    if n.q is not None:
        want = plain.codes(s64, w64)
        d = np.abs(ref).reshape(len(ref), -1, 32).max(-1) / 127
        got = n.d.double().cpu().numpy()
        assert np.all(np.abs(got - d) <= d * 33 * plain.U + 2.0 ** -149)
        want[np.repeat(got == 0, 32, axis=-1)] = 0
        np.testing.assert_array_equal(n.q.cpu().numpy(), want)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,K", [(1, 1), (1, 32), (3, 31), (5, 96), (2, 1000), (7, 1001), (4, 4096), (33, 2048),
                                 (1, 32768), (2, 32767), (700, 64), (400, 5120), (1, 16384)])
def test_rows(g, T, K, dtype):
    import torch
    x, rest = made(T, K, dtype, 1), made(T, K, dtype, 2, 3.0)
    weight = 1.0 + 0.3 * made(1, K, "float32", 3)[0]
    want = "both" if K % 32 == 0 else "y"
    n = g.rfp2_rms_norm(x, weight, residual=rest, want=want)
    s = (x.float() + rest.float()).to(x.dtype)
    assert torch.equal(n.total, s)
    check(s, weight, n)
    check(x, weight, g.rfp2_rms_norm(x, weight, eps=1e-3, want=want), 1e-3)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("wtype", TYPES)
@pytest.mark.parametrize("ytype", TYPES)
def test_types(g, dtype, wtype, ytype):
    import torch
    x, rest = made(9, 416, dtype, 4), made(9, 416, dtype, 5)
    weight = (1.0 + 0.3 * made(1, 416, "float32", 6)[0]).to(getattr(torch, wtype))
    n = g.rfp2_rms_norm(x, weight, residual=rest, want="both", dtype=getattr(torch, ytype))
    assert n.y.dtype == getattr(torch, ytype)
    check(n.total, weight, n)
    q8 = g.rfp2_rms_norm(x, weight, residual=rest, want="q8")
    assert q8.y is None and torch.equal(q8.q, n.q) and torch.equal(q8.d, n.d)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K,shift", [(256, 0), (256, 1), (264, 0), (250, 2)])
def test_strides_and_alignment(g, dtype, K, shift):
    """Rows that are parts of wider ones, at any offset; outputs beside which nothing is written."""
    import torch
    T = 6
    wide = made(T, 2 * K + 19, dtype, 7)
    x, rest = wide[:, shift: shift + K], wide[:, K + shift + 5: 2 * K + shift + 5]
    weight = 1.0 + 0.3 * made(1, K + shift, "float32", 8)[0, shift:]
    y, total = (torch.full((T, K + 9), 7.0, device="cuda", dtype=x.dtype) for _ in range(2))
    n = g.rfp2_rms_norm(x, weight, residual=rest, y=y[:, shift: shift + K], total=total[:, shift: shift + K])
    s = (x.float() + rest.float()).to(x.dtype)
    assert torch.equal(n.total, s)
    check(s, weight, n)
    for t in (y, total):
        assert bool((t[:, :shift] == 7).all()) and bool((t[:, shift + K:] == 7).all())


@pytest.mark.parametrize("dtype", TYPES)
def test_in_place(g, dtype):
    import torch
    x, rest = made(50, 1024, dtype, 9), made(50, 1024, dtype, 10)
    weight = 1.0 + 0.3 * made(1, 1024, "float32", 11)[0]
    n = g.rfp2_rms_norm(x, weight, residual=rest)
    a, b = x.clone(), rest.clone()
    m = g.rfp2_rms_norm(a, weight, residual=b, total=b, y=a)
    assert torch.equal(m.y, n.y) and torch.equal(m.total, n.total) and m.y is a and m.total is b
    with pytest.raises(g.RFP2Error):
        g.rfp2_rms_norm(a, weight, residual=b, total=b, y=b)
    with pytest.raises(g.RFP2Error):
        g.rfp2_rms_norm(a[:49], weight, y=a[1:])


def test_codes_at_half_integers(g):
    """Blocks of whole numbers whose largest is 254: odd values lie between two codes and go away from zero; the
    neighbours of such values on both sides go to their own code.  Any factor of the row and any weight that
    is a power of two leave the codes alone."""
    import torch
    r = np.random.default_rng(12)
    x = r.integers(-254, 255, (64, 256)).astype(np.float32)
    x.reshape(64, 8, 32)[:, :, 5] = 254 * np.where(r.random((64, 8)) < 0.5, -1, 1)
    x[1::3] = np.nextafter(x[1::3], np.float32(0))
    x[2::3] = np.nextafter(x[2::3], np.sign(x[2::3]) * np.float32(1e9))
    x.reshape(64, 8, 32)[:, :, 5] = 254
    x *= np.exp2(r.integers(-20, 20, (64, 1))).astype(np.float32)
    weight = np.repeat(np.exp2(r.integers(-3, 4, 8)), 32).astype(np.float32)
    n = g.rfp2_rms_norm(torch.from_numpy(x).cuda(), torch.from_numpy(weight).cuda(), eps=1e-12, want="q8")
    np.testing.assert_array_equal(n.q.cpu().numpy(), plain.codes(x, weight))


@pytest.mark.parametrize("K", [64, 1001, 4096])
@pytest.mark.parametrize("size", [1e-40, 1e-30, 1e-20, 1e15, 1e25, 3e37])
def test_rows_of_any_size(g, K, size):
    """Squares that leave fp32's range, above and below; eps small beside them, and not."""
    x = made(5, K, "float32", 13).clamp_(-3, 3).mul_(size)
    weight = 1.0 + 0.3 * made(1, K, "float32", 14)[0]
    for eps in (1e-6, 1e-37):
        n = g.rfp2_rms_norm(x, weight, eps=eps, want="y")
        ref = plain.norm(x.double().cpu().numpy(), weight.double().cpu().numpy(), eps)
        # values below 2^-126 and reciprocals above 2^126 keep fewer digits
        bound = np.abs(ref) * (2.0 ** -17 if size < 1e-35 or size > 1e37 else 33 * plain.U) + 2.0 ** -148
        assert np.all(np.abs(n.y.double().cpu().numpy() - ref) <= bound), eps


def test_rows_of_zeros_infinities_and_nan(g):
    import torch
    x = made(6, 128, "float32", 15)
    x[0] = 0
    x[1, 40] = float("inf")
    x[2, 99] = float("nan")
    x[3, :32] = 0
    weight = torch.ones(128, device="cuda")
    n = g.rfp2_rms_norm(x, weight, want="both")
    assert not n.y[0].any() and not n.q[0].any() and not n.d[0].any()
    # an infinity takes everything else of its row to zero, and is none itself
    assert bool(n.y[1, 40].isnan()) and int(n.y[1].count_nonzero()) == 1 and bool(n.y[2].isnan().all())
    values = n.q.view(6, 4, 32).float() * n.d[..., None]
    assert bool(values[1, 1].isnan().all()) and not values[1, [0, 2, 3]].any()
    assert bool(values[2].isnan().all()) and not values[3, 0].any()
    check(x[3:], weight, g.Norm(n.y[3:], n.q[3:], n.d[3:], None))


def test_blocks_feed_the_gemv(g):
    """q and d are what rfp2_gemv_q8 takes: the same as quantising y, but for codes at the border of two."""
    import torch
    K, M = 1024, 64
    W = g.rfp2_pack_weights(made(M, K, "float32", 16, 0.03))
    x = made(4, K, "float32", 17)
    n = g.rfp2_rms_norm(x, torch.ones(K, device="cuda"), want="both")
    q, d = g.rfp2_quantize_act(n.y)
    assert int((q != n.q).sum()) <= 4 and float((d - n.d).abs().max() / d.max()) < 2 ** -20
    a, b = g.rfp2_gemv_q8(W, M, K, n.q, n.d), g.rfp2_gemv_q8(W, M, K, q, d)
    assert float((a - b).norm() / b.norm()) < 1e-3


def test_nothing_to_do_and_refusals(g):
    import torch
    x, w = made(4, 64, "float32"), torch.ones(64, device="cuda")
    n = g.rfp2_rms_norm(x[:0], w, want="both")
    assert n.y.shape == (0, 64) and n.q.shape == (0, 64) and n.d.shape == (0, 2)
    for call in (lambda: g.rfp2_rms_norm(x, w, eps=0.0), lambda: g.rfp2_rms_norm(x, w, eps=float("nan")),
                 lambda: g.rfp2_rms_norm(x[:, :40], w[:40].clone(), want="q8")):
        with pytest.raises((g.RFP2Error, ValueError)):
            call()
    for call in (lambda: g.rfp2_rms_norm(x, w[:32]), lambda: g.rfp2_rms_norm(x, w, residual=x[:2]),
                 lambda: g.rfp2_rms_norm(x, w, residual=x.half()), lambda: g.rfp2_rms_norm(x, w, want="z"),
                 lambda: g.rfp2_rms_norm(x[:, ::2], w[:32]), lambda: g.rfp2_rms_norm(x, w, want="q8", q=torch.empty((4, 32), dtype=torch.int8, device="cuda")),
                 lambda: g.rfp2_rms_norm(x[0], w), lambda: g.rfp2_rms_norm(x, w, total=x.clone())):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: g.rfp2_rms_norm(x.double(), w), lambda: g.rfp2_rms_norm(x.cpu(), w)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(RuntimeError, match="gradient"):
        g.rfp2_rms_norm(x, w.clone().requires_grad_())
    with torch.no_grad():
        g.rfp2_rms_norm(x, w.clone().requires_grad_())

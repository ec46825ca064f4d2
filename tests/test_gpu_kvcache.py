"""The Q8 paged cache (rfp2_kv_write, rfp2_kv_read): codes and scales equal the definition's bit for bit
where k is not rotated; rotated keys may sit one code away where the float64 quotient is within the
rotation's error of a boundary."""
import numpy as np
import pytest

import _attention as plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import gemm_rocmfp2_mul_gb300 as g
    g.build()
    g.lib()
    return g


def _tensor(a, dtype):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).to(getattr(torch, dtype))


def _draw(kind, shape, seed):
    r = np.random.default_rng(seed)
    x = r.standard_normal(shape).astype(np.float32)
    if kind == "wide":      # channels of very different sizes, down to subnormal blocks
        x *= np.exp2(r.integers(-140, 60, shape[:-1] + (shape[-1] // 32,)).astype(np.float32)).repeat(32, -1)
    elif kind == "ties":    # quotients at and beside half-integers
        b = x.reshape(*shape[:-1], -1, 32)
        n = r.integers(-126, 126, b.shape) + 0.5
        d = np.exp2(r.uniform(-3, 3, b.shape[:-1] + (1,))).astype(np.float32)
        b[:] = (n * d).astype(np.float32)
        b[..., 0] = (127 * d)[..., 0]
        bump = r.integers(-2, 3, b.shape).astype(np.int32)
        b[:] = (b.view(np.int32) + bump).view(np.float32)
    elif kind == "zeros":
        x[r.random(shape) < 0.9] = 0.0
        x[:, ::2] = 0.0
    return x


@pytest.mark.parametrize("kind", ["normal", "wide", "ties", "zeros"])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("T,H,D,page", [(1, 1, 32, 1), (9, 8, 128, 16), (37, 3, 96, 7), (70, 5, 64, 64), (6, 2, 256, 33)])
def test_codes_and_scales_are_the_definitions(g, T, H, D, page, dtype, kind):
    import torch
    pages = T // page + 3
    cache = g.rfp2_kv_alloc(pages, H, page, D)
    k, v = (_tensor(_draw(kind, (T, H, D), 5 * T + D + i), dtype) for i in range(2))
    slots = np.random.default_rng(T).permutation(pages * page)[:T].astype(np.int64)
    if T > 4:
        slots[2] = -1
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    g.rfp2_kv_write(cache, k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), dev_status=st)
    assert int(st) == 0
    got = [t.cpu().numpy() for t in cache]
    kept = slots >= 0
    p, o = slots[kept] // page, slots[kept] % page
    for x, codes, scales in ((k, *got[:2]), (v, *got[2:])):
        q, d = plain.quantise(x.float().numpy()[kept])
        np.testing.assert_array_equal(codes[p, :, o], q)
        np.testing.assert_array_equal(scales[p, :, o], d)
        # what no token was written to is untouched
        codes[p, :, o] = 0
        scales[p, :, o] = 0
        assert not codes.any() and not scales.any()
    # read back: the product code * scale, rounded once
    for out in ("float32", "bfloat16", "float16"):
        rk, rv = g.rfp2_kv_read(cache, torch.from_numpy(slots).cuda(), dtype=getattr(torch, out))
        for x, y in ((k, rk), (v, rv)):
            q, d = plain.quantise(x.float().numpy())
            with np.errstate(invalid="ignore"):
                ref = (q.astype(np.float32) * np.repeat(d, 32, -1)).astype(np.float32)
            ref[~kept] = 0.0
            ref = torch.from_numpy(ref).to(getattr(torch, out))
            np.testing.assert_array_equal(y.float().cpu().numpy(), ref.float().numpy())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,T,H,D,R", [("float32", 20, 4, 128, 128), ("bfloat16", 65, 2, 96, 64),
                                           ("float16", 3, 5, 64, 34), ("bfloat16", 7, 1, 256, 2)])
def test_rotated_keys(g, dtype, T, H, D, R, interleaved):
    """The rotated value is off by at most 5e-7 (|a| + |b|) (see the rotation's tests), so the scale by
    that and two roundings, and the code is the float64 one or, within that of a boundary, its neighbour."""
    import torch
    page = 16
    cache = g.rfp2_kv_alloc(T // page + 2, H, page, D)
    k, v = (_tensor(_draw("normal", (T, H, D), R + i), dtype) for i in range(2))
    pos = np.random.default_rng(1).integers(0, 100000, T).astype(np.int32)
    f, _ = g.rfp2_rope_frequencies(R)
    slots = np.arange(T, dtype=np.int64) + 3
    g.rfp2_kv_write(cache, k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), torch.from_numpy(pos).cuda(), f,
                    interleaved=interleaved, factor=1.2)
    p, o = slots // page, slots % page
    kc, ks, vc, vs = (t.cpu().numpy()[p, :, o] for t in cache)
    q, d = plain.quantise(v.float().numpy())
    np.testing.assert_array_equal(vc, q)
    np.testing.assert_array_equal(vs, d)
    x = plain.rope(k.double().numpy(), pos, f.cpu().numpy(), interleaved=interleaved, factor=1.2)
    b = x.reshape(T, H, -1, 32)
    top = np.abs(b).max(-1)
    off = 1.2 * 5e-7 * 2 * np.abs(k.float().numpy()).max()
    assert np.all(np.abs(ks * 127.0 - top) <= off + 2.0 ** -22 * top)
    t = b / (top / 127)[..., None]
    away = np.abs(kc.reshape(b.shape) - t)
    slack = 127 * 2 * off / top + 127 * 2.0 ** -22
    assert np.all(away <= 0.5 + slack[..., None])


def test_unaligned_and_strided_rows(g):
    import torch
    T, H, D, page = 11, 3, 64, 8
    r = np.random.default_rng(0)
    for dtype in ("float32", "bfloat16"):
        whole = _tensor(r.standard_normal((T, 2 * H * D + 9)).astype(np.float32), dtype).cuda()
        k = whole[:, 1: 1 + H * D].unflatten(1, (H, D))
        v = whole[:, 5 + H * D: 5 + 2 * H * D].unflatten(1, (H, D))
        slots = torch.arange(T, device="cuda")
        f, _ = g.rfp2_rope_frequencies(64)
        pos = torch.arange(T, dtype=torch.int32, device="cuda")
        for rope in ({}, {"positions": pos, "inv_freq": f}, {"positions": pos, "inv_freq": f, "interleaved": True}):
            a, b = (g.rfp2_kv_alloc(3, H, page, D) for _ in range(2))
            g.rfp2_kv_write(a, k, v, slots, **rope)
            g.rfp2_kv_write(b, k.contiguous(), v.contiguous(), slots, **rope)
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_values_that_are_not_finite(g):
    """A block with an infinity or a NaN reads back as NaN; its neighbours are not touched by it."""
    import torch
    k = torch.ones((4, 1, 64), device="cuda")
    k[0, 0, 3] = float("nan")
    k[1, 0, 40] = float("inf")
    k[2, 0, 31] = -float("inf")
    k[2, 0, 30] = float("nan")
    cache = g.rfp2_kv_alloc(1, 1, 4, 64)
    slots = torch.arange(4, device="cuda")
    g.rfp2_kv_write(cache, k, k, slots)
    for x in g.rfp2_kv_read(cache, slots):
        nan = torch.isnan(x[:, 0].unflatten(1, (2, 32)))
        assert torch.equal(nan.all(-1), nan.any(-1))
        assert nan.all(-1).tolist() == [[True, False], [False, True], [True, False], [False, False]]
        assert bool((x[~torch.isnan(x)] == 1.0).all())


def test_slots_outside_the_cache(g):
    """Nothing is written or read there: the status says so and a read gives NaN."""
    import torch
    cache = g.rfp2_kv_alloc(2, 1, 4, 32)
    x = torch.ones((5, 1, 32), device="cuda")
    slots = torch.tensor([8, -2, 3, 2 ** 62, -1], device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    g.rfp2_kv_write(cache, x, x, slots, dev_status=st)
    assert int(st) == 7
    assert int(cache[0].ne(0).sum()) == 32 and bool((cache[0].view(8, 32)[3] == 127).all())
    st.zero_()
    k, v = g.rfp2_kv_read(cache, slots, dev_status=st)
    assert int(st) == 7
    for y in (k, v):
        y = y[:, 0]
        assert bool(torch.isnan(y[[0, 1, 3]]).all()) and bool((y[2] == 1).all()) and bool((y[4] == 0).all())


def test_refusals(g):
    import torch
    cache = g.rfp2_kv_alloc(2, 2, 4, 64)
    k = torch.zeros((3, 2, 64), device="cuda")
    slots = torch.arange(3, device="cuda")
    f, _ = g.rfp2_rope_frequencies(64)
    bad = [(TypeError, dict(slots=slots.int())), (ValueError, dict(k=k[:, :1])), (ValueError, dict(slots=slots[:2])),
           (ValueError, dict(v=k.half())), (TypeError, dict(k=k.double(), v=k.double())),
           (TypeError, dict(cache=(cache[0].int(), *cache[1:]))), (ValueError, dict(cache=(cache[0], cache[1][:1], *cache[2:])))]
    for error, change in bad:
        args = {"cache": cache, "k": k, "v": k, "slots": slots, **change}
        with pytest.raises(error):
            g.rfp2_kv_write(**args)
    for change, status in ((dict(inv_freq=f), 1), (dict(positions=slots.int()), 1),
                           (dict(positions=slots.int(), inv_freq=torch.zeros(33, device="cuda")), 2)):
        with pytest.raises(g.RFP2Error) as e:
            g.rfp2_kv_write(cache, k, k, slots, **change)
        assert e.value.status == status
    odd = (torch.zeros((2, 2, 4, 48), dtype=torch.int8, device="cuda"), torch.zeros((2, 2, 4, 1), device="cuda")) * 2
    with pytest.raises(g.RFP2Error) as e:
        g.rfp2_kv_read(odd, slots)
    assert e.value.status == 2
    with pytest.raises(ValueError):
        g.rfp2_kv_read(cache, slots, k=k[:2])
    with pytest.raises(TypeError):
        g.rfp2_kv_read(cache, slots, k=k.half(), v=k)
    assert g.rfp2_kv_read(cache, slots[:0])[0].shape == (0, 2, 64)
    g.rfp2_kv_write(cache, k[:0], k[:0], slots[:0])

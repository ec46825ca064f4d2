"""The attention operators' host side: frequencies, workspace sizes and the checks that need no GPU."""
import ctypes as C
import math

import numpy as np
import pytest


@pytest.fixture(scope="module")
def g():
    import gemm_rocmfp2_mul_gb300 as g
    g.build()
    g.lib()
    return g


@pytest.mark.parametrize("R,base", [(2, 10000.0), (64, 10000.0), (128, 500000.0), (96, 1e6)])
def test_frequencies(g, R, base):
    plain, factor = g.rfp2_rope_frequencies(R, base, device="cpu")
    want = base ** (-np.arange(0, R, 2) / R)
    np.testing.assert_array_equal(plain.numpy(), want.astype(np.float32))
    assert factor == 1.0
    linear, _ = g.rfp2_rope_frequencies(R, base, "linear", stretch=4.0, device="cpu")
    np.testing.assert_array_equal(linear.numpy(), (want / 4).astype(np.float32))
    if R > 2:
        # the larger base leaves the fastest pair alone and divides the slowest by the stretch
        larger, _ = g.rfp2_rope_frequencies(R, base, "base", stretch=4.0, device="cpu")
        assert larger[0] == 1.0 and abs(float(larger[-1]) / (want[-1] / 4) - 1) < 1e-6
    ramp, factor = g.rfp2_rope_frequencies(R, base, "ramp", stretch=8.0, trained=4096.0, device="cpu")
    assert abs(factor - (0.1 * math.log(8.0) + 1.0)) < 1e-6
    turns = 4096.0 * want / (2 * math.pi)
    np.testing.assert_array_equal(ramp.numpy()[turns >= 32], want[turns >= 32].astype(np.float32))
    np.testing.assert_array_equal(ramp.numpy()[turns <= 1], (want / 8)[turns <= 1].astype(np.float32))
    between = (turns > 1) & (turns < 32)
    assert np.all(ramp.numpy()[between] <= want[between]) and np.all(ramp.numpy()[between] >= want[between] / 8)
    assert np.all(np.diff(ramp.numpy()) <= 0)


def test_frequency_refusals(g):
    for kw, status in ((dict(R=3), 2), (dict(R=0), 2), (dict(R=64, base=0.0), 1), (dict(R=64, base=float("nan")), 1),
                       (dict(R=64, scaling="linear", stretch=-1.0), 1), (dict(R=64, scaling="ramp", fast=1.0, slow=1.0), 1),
                       (dict(R=64, scaling="ramp", trained=0.0), 1), (dict(R=2, scaling="base", stretch=2.0), 2)):
        with pytest.raises(g.RFP2Error) as e:
            g.rfp2_rope_frequencies(device="cpu", **kw)
        assert e.value.status == status
    with pytest.raises(KeyError):
        g.rfp2_rope_frequencies(64, scaling="unknown", device="cpu")


def test_checks_come_before_any_launch(g):
    """Every refusal below returns before the library touches the GPU; `p` is never read."""
    L = g.lib()
    EINVAL, ESHAPE, EALIGN, EWORKSPACE = 1, 2, 3, 9
    p, odd = C.c_void_p(4096), C.c_void_p(4097)

    def rope(x=p, dtype=0, T=1, H=1, D=64, pos=p, f=p, R=64, flags=0, out=p):
        return L.rfp2_rope(x, dtype, T, H, D, D, D, pos, f, R, 1.0, flags, out, D, D, None)

    assert rope(T=0) == 0 and rope(H=0, x=None) == 0
    assert [rope(x=None), rope(out=None), rope(pos=None), rope(f=None), rope(dtype=3), rope(flags=4), rope(T=-1)] == [EINVAL] * 7
    assert [rope(R=63), rope(R=66), rope(R=-2), rope(D=65), rope(D=1 << 17), rope(T=1 << 40)] == [ESHAPE] * 6
    assert [rope(x=odd), rope(out=odd, dtype=1), rope(pos=odd), rope(f=odd)] == [EALIGN] * 4

    def write(k=p, v=p, dtype=0, T=1, slots=p, pos=None, f=None, R=0, flags=0, kc=p, pages=1, heads=1, page=1, D=32):
        return L.rfp2_kv_write(k, v, dtype, T, D, D, D, D, slots, pos, f, R, 1.0, flags, kc, p, p, p, pages, heads, page, D,
                               None, None)

    assert write(T=0) == 0
    assert [write(k=None), write(v=None), write(slots=None), write(kc=None), write(dtype=-1), write(flags=2), write(T=-1),
            write(pos=p), write(f=p)] == [EINVAL] * 9
    assert [write(D=48), write(D=288), write(D=0), write(pages=0), write(page=0), write(heads=0), write(pages=1 << 41),
            write(pos=p, f=p, R=34), write(pos=p, f=p, R=31)] == [ESHAPE] * 9
    assert [write(k=odd), write(slots=C.c_void_p(4100)), write(kc=C.c_void_p(4104))] == [EALIGN] * 3

    def read(kc=p, T=1, dtype=0, slots=p, k=p, v=p, D=32):
        return L.rfp2_kv_read(kc, p, p, p, 1, 1, 1, D, slots, T, dtype, k, v, None, None)

    assert read(T=0) == 0 and read(k=None, v=None) == 0
    assert [read(kc=None), read(slots=None), read(dtype=7), read(T=-1)] == [EINVAL] * 4
    assert read(D=33) == ESHAPE and read(k=C.c_void_p(4100)) == EALIGN

    def attn(q=p, dtype=0, B=1, nq=1, Hq=4, D=64, kc=p, pages=8, heads=2, page=16, table=p, width=4, stride=4, lens=p,
             window=0, softcap=0.0, out=p, lse=p, ws=p, size=1 << 40):
        return L.rfp2_attn_decode(q, dtype, B, nq, Hq, D, D, D, D, kc, p, p, p, pages, heads, page, table, width, stride, lens,
                                  1.0, window, softcap, out, lse, ws, size, None, None)

    assert [attn(q=None), attn(kc=None), attn(table=None), attn(lens=None), attn(out=None), attn(dtype=5), attn(window=-1),
            attn(softcap=-1.0)] == [EINVAL] * 8
    assert [attn(B=0), attn(nq=0), attn(Hq=3), attn(Hq=0), attn(D=80), attn(D=320), attn(pages=0), attn(page=0), attn(width=0),
            attn(stride=3), attn(width=1 << 30), attn(pages=1 << 31), attn(nq=1 << 20)] == [ESHAPE] * 13
    assert [attn(ws=None), attn(size=0)] == [EWORKSPACE] * 2
    assert [attn(kc=C.c_void_p(4104)), attn(q=odd), attn(ws=C.c_void_p(4112)), attn(lens=odd), attn(table=odd)] == [EALIGN] * 5


def test_workspace_size_grows_with_nothing_it_should_not(g):
    n = g.rfp2_attn_decode_workspace_bytes
    assert n(1, 1, 8, 8, 128) > 0
    assert n(0, 1, 8, 8, 128) == 0 and n(1, 1, 9, 8, 128) == 0

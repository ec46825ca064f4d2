"""Edges of the attention operators' arguments that the host decides, without a GPU."""
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


def test_no_tokens_to_write_with_a_rotation(g):
    """An empty tensor has no address: with T = 0 no pointer is looked at, of positions neither."""
    p = C.c_void_p(4096)
    for positions, inv_freq in ((None, p), (p, None), (p, p), (None, None)):
        assert g.lib().rfp2_kv_write(None, None, 0, 0, 64, 64, 64, 64, None, positions, inv_freq, 64, 1.0, 0, p, p, p, p,
                                     1, 1, 1, 64, None, None) == 0


@pytest.mark.parametrize("kw", [dict(prompt=0), dict(new=0), dict(prompt=16, new=0), dict(new=-1), dict(batch=0)])
def test_the_example_needs_a_prompt_and_new_tokens(kw):
    """Before any work on the GPU: its trial step writes the token after the prompt, which a cache for the prompt
    alone has no page for."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_layer.py")
    spec = importlib.util.spec_from_file_location("decode_layer", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    with pytest.raises(ValueError, match="are needed"):
        example.run(**{**dict(prompt=4, new=4), **kw})


def attn_decode(g, q, out, lse, B=2, nq=3, Hq=4, D=64, strides=None, dtype=0, page=16, width=4, heads=2):
    """The status of a call whose arrays are addresses that nothing looks at."""
    p = C.c_void_p(1 << 40)
    strides = strides or (nq * Hq * D, Hq * D, D)
    return g.lib().rfp2_attn_decode(C.c_void_p(q), dtype, B, nq, Hq, D, *strides, p, p, p, p, 8, heads, page, p, width, width, p, 1.0, 0,
                                    0.0, C.c_void_p(out), C.c_void_p(lse), p, 1 << 40, None, None)


def test_overlaps_of_queries_and_outputs_are_refused(g):
    """A row of q is read before the same row of out is written, but not before any other."""
    q, row = 1 << 30, 64 * 4
    rows = 2 * 3 * 4
    far = 1 << 35
    assert attn_decode(g, q, q + 16, far) == 1                                  # the same rows, moved
    assert attn_decode(g, q, q + (rows - 1) * row, far) == 1                    # the last row of q
    assert attn_decode(g, q, q - (rows - 1) * row, far) == 1                    # the first
    assert attn_decode(g, q, q, far, strides=(64, 2 * 4 * 64, 2 * 64)) == 1     # the same memory in another order
    assert attn_decode(g, q, q, far, nq=1, strides=(8 * 64, 0, 64)) == 1        # out runs into the second sequence's q
    assert attn_decode(g, q, far, q + rows * row - 4) == 1                      # lse over q
    assert attn_decode(g, q, far, far + 4 * rows) == 1                          # and over out
    assert attn_decode(g, q, far, far - 4) == 1


def test_the_line_ends_before_32_bits_do(g):
    """Places on the line of tiles are 32-bit numbers, to which a unit's gap of 4 is added on the way: a line of
    2^31 - 4 places and more is refused (it is (table_width + 5) * heads for pages of 16)."""
    for line, heads in ((2 ** 31 - 2, 33), (2 ** 31 - 3, 95), (2 ** 31 - 4, 932)):
        assert line % heads == 0
        assert attn_decode(g, 1 << 30, 1 << 35, 1 << 36, B=1, nq=1, Hq=heads, heads=heads, page=16, width=line // heads - 5) == 2


@pytest.mark.parametrize("R,base,stretch,trained,fast,slow", [(128, 10000.0, 8.0, 4096.0, 32.0, 1.0), (64, 500000.0, 4.0, 8192.0, 32.0, 1.0),
                                                              (96, 10000.0, 16.0, 2048.0, 20.0, 2.5)])
def test_the_ramp_between_its_ends(g, R, base, stretch, trained, fast, slow):
    """f (keep + (1 - keep) / stretch), keep = (trained f / 2 pi - slow) / (fast - slow) within [0, 1], in double and
    rounded once: libm's last places may fall either way at a float's boundary, so half a float's place and 1e-14."""
    got, _ = g.rfp2_rope_frequencies(R, base, "ramp", stretch=stretch, trained=trained, fast=fast, slow=slow, device="cpu")
    between = 0
    for i, x in enumerate(got.tolist()):
        f = base ** (-2 * i / R)
        keep = min(1.0, max(0.0, (trained * f / (2 * math.pi) - slow) / (fast - slow)))
        between += 0.0 < keep < 1.0
        want = f * (keep + (1 - keep) / stretch)
        assert abs(x - want) <= 0.5 * float(np.spacing(np.float32(want))) + 1e-14 * want
    assert between >= 5         # the case has a ramp

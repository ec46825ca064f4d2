"""Edges of the attention operators' arguments that the host decides, without a GPU."""
import ctypes as C

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

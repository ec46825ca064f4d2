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

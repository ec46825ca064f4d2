"""The decode layer of examples/: the products, rotation, cache and attention together, a prompt and then
tokens from a replayed graph, against the layer in float64."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("prompt,new,batch", [(300, 20, 2), (1, 3, 1), (17, 40, 8)])
def test_decode_layer(prompt, new, batch):
    """Activations and cache in blocks of 8 bits: a value is off by at most half a step, its block's largest
    over 254, uniformly: with the largest of 32 normal values near 2.1 deviations that is 2.1 / 254 / sqrt(3)
    = 0.5 % of a deviation.  It enters four times (two products, keys, values; the prompt's products take
    bf16 instead), the scores' part scaled by |s| of order 1: 2 % covers their sum for every token."""
    import gemm_rocmfp2_mul_gb300 as g
    g.build()
    spec = importlib.util.spec_from_file_location("decode_layer", os.path.join(ROOT, "examples", "decode_layer.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    layer, inputs, y = example.run(prompt, new, batch)
    ref = example.reference(layer, inputs)
    off = (y.double() - ref).norm(dim=-1) / ref.norm(dim=-1)
    assert int(layer.status) == 0
    assert layer.lens.tolist() == [prompt + new] * batch
    assert float(off.max()) < 0.02, off.max()

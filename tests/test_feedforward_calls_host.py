"""Python calls of the feed-forward operators that are refused before the library or a GPU is needed."""
import pytest


def test_buffers_for_what_is_not_wanted():
    """A buffer that is passed is filled; one that would not be is refused, not left as it was."""
    import torch
    import gemm_rocmfp2_mul_gb300 as g
    x, w = torch.zeros((4, 64)), torch.ones(64)
    y, q, d = torch.zeros((4, 64)), torch.zeros((4, 64), dtype=torch.int8), torch.zeros((4, 2))
    for kw in (dict(want="q8", y=y), dict(want="q8", y=y, q=q, d=d), dict(want="y", q=q), dict(want="y", d=d),
               dict(y=y, dtype=torch.bfloat16), dict(want="both", y=y, dtype=torch.float16)):
        with pytest.raises(ValueError):
            g.rfp2_rms_norm(x, w, **kw)
    with pytest.raises(ValueError):
        g.rfp2_moe_combine(torch.zeros((4, 2, 64)), torch.ones((4, 2)), out=y, dtype=torch.float16)

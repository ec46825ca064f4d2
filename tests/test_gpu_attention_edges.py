"""The attention operators at the edges of their arguments: nothing to do, tensors elsewhere, memory in common."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import gemm_rocmfp2_mul_gb300 as g
    g.build()
    g.lib()
    return g


def test_no_tokens_and_no_pairs_to_write(g):
    """No token, rotated or not, is nothing to write; frequencies of no pair turn nothing, as in rfp2_rope."""
    import torch
    cache, same = (g.rfp2_kv_alloc(2, 2, 4, 64) for _ in range(2))
    k, v = torch.randn((2, 3, 2, 64), device="cuda")
    slots = torch.arange(3, device="cuda")
    positions = torch.arange(3, dtype=torch.int32, device="cuda")
    f, _ = g.rfp2_rope_frequencies(64)
    none = {t: torch.empty(0, dtype=t, device="cuda") for t in (torch.int32, torch.int64, torch.float32)}
    for no_slots, no_positions in ((slots[:0], positions[:0]), (none[torch.int64], none[torch.int32])):
        for frequencies in (f, f[:0], none[torch.float32]):
            g.rfp2_kv_write(cache, k[:0], v[:0], no_slots, no_positions, frequencies)
    assert not any(t.any() for t in cache)
    g.rfp2_kv_write(same, k, v, slots)
    for no_frequencies in (f[:0], none[torch.float32]):
        cache[0].zero_()
        g.rfp2_kv_write(cache, k, v, slots, positions, no_frequencies)
        assert all(torch.equal(a, b) for a, b in zip(cache, same)) and bool(cache[0].any())

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


def test_tensors_of_another_device_are_refused(g):
    """The library launches on the current device: tensors elsewhere would be read there by their addresses.
    (Tensors without memory stand for those of a second GPU: no call below can come to a launch.)"""
    import torch

    class Elsewhere(torch.Tensor):
        @staticmethod
        def __new__(cls, *shape, dtype=torch.float32):
            strides = [1]
            for n in shape[:0:-1]:
                strides.insert(0, strides[0] * n)
            return torch.Tensor._make_wrapper_subclass(cls, shape, strides=strides, dtype=dtype,
                                                       device=f"cuda:{torch.cuda.current_device() + 1}")

        @classmethod
        def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
            raise AssertionError(f"{func} of a tensor without memory")

    x = Elsewhere(3, 2, 64)
    positions, f, slots = Elsewhere(3, dtype=torch.int32), Elsewhere(32), Elsewhere(3, dtype=torch.int64)
    cache = tuple(Elsewhere(2, 2, 4, n, dtype=t) for n, t in ((64, torch.int8), (2, torch.float32)) * 2)
    q, lse = Elsewhere(3, 1, 2, 64), Elsewhere(3, 1, 2)
    table, lens, workspace = Elsewhere(3, 2, dtype=torch.int32), positions, Elsewhere(1 << 20, dtype=torch.uint8)
    W, y = Elsewhere(16, 20, dtype=torch.uint8), Elsewhere(3, 16)
    calls = [lambda: g.rfp2_rope(x, positions, f, out=x), lambda: g.rfp2_kv_write(cache, x, x, slots),
             lambda: g.rfp2_kv_read(cache, slots, k=x, v=x), lambda: g.rfp2_attn_decode_workspace(q, 2),
             lambda: g.rfp2_attn_decode(q, cache, table, lens, out=q, lse=lse, workspace=workspace),
             lambda: g.rfp2_gemv(W, 16, 64, y, y=y, workspace=workspace),
             lambda: g.rfp2_pack_weights(y, out=W)]
    for call in calls:
        with pytest.raises(ValueError, match="current device"):
            call()

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


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_a_gradient_goes_through_the_rotation(g, interleaved, inverse):
    """The rotation is linear: its gradient is the transpose, which is the rotation back by the same factor; the
    gradient's gradient is the rotation itself.  Against the call itself (its own tests check it against the
    formula) and against a difference, exact for a linear map up to the rounding of 256 terms of up to 8 in
    fp32."""
    import torch
    r = torch.Generator(device="cuda").manual_seed(3)
    x, gy, step = (torch.randn((5, 2, 64), generator=r, device="cuda") for _ in range(3))
    positions = torch.arange(5, dtype=torch.int32, device="cuda") * 77
    f, _ = g.rfp2_rope_frequencies(48)
    how = dict(interleaved=interleaved, inverse=inverse, factor=1.25)
    leaf = x.clone().requires_grad_()
    y = g.rfp2_rope(leaf, positions, f, **how)
    assert torch.equal(y.detach(), g.rfp2_rope(x, positions, f, **how))
    grad_out = gy.clone().requires_grad_()
    (gx,) = torch.autograd.grad(y, leaf, grad_out, create_graph=True)
    assert torch.equal(gx.detach(), g.rfp2_rope(gy, positions, f, **{**how, "inverse": not inverse}))
    difference = ((g.rfp2_rope(x + step, positions, f, **how).double() - g.rfp2_rope(x, positions, f, **how).double()) * gy).sum()
    assert abs(float(difference - (gx.detach().double() * step).sum())) <= 640 * 8 * 2.0 ** -22
    (ggx,) = torch.autograd.grad(gx, grad_out, x)
    assert torch.equal(ggx, g.rfp2_rope(x, positions, f, **how))
    # of a sum: a gradient without strides of its own
    y = g.rfp2_rope(leaf, positions, f, **how)
    y.sum().backward()
    assert torch.equal(leaf.grad, g.rfp2_rope(torch.ones_like(x), positions, f, **{**how, "inverse": not inverse}))


def test_in_place_and_gradients(g):
    """out= drops no gradient in silence; a tensor that a call writes has another version, so that autograd knows."""
    import torch
    f, _ = g.rfp2_rope_frequencies(64)
    positions = torch.arange(3, dtype=torch.int32, device="cuda")
    leaf = torch.randn((3, 2, 64), device="cuda", requires_grad=True)
    for out in (leaf, torch.empty((3, 2, 64), device="cuda")):
        with pytest.raises(RuntimeError, match="gradient"):
            g.rfp2_rope(leaf, positions, f, out=out)
        with torch.no_grad():
            g.rfp2_rope(leaf, positions, f, out=out)
    x = leaf.detach().clone()
    kept = leaf * x                      # autograd keeps x
    g.rfp2_rope(x, positions, f, out=x)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        kept.sum().backward()
    cache = g.rfp2_kv_alloc(2, 2, 4, 64)
    slots = torch.arange(3, device="cuda")
    q, lse = torch.randn((1, 1, 2, 64), device="cuda"), torch.empty((1, 1, 2), device="cuda")
    out, k, v = torch.empty_like(q), torch.empty_like(x), torch.empty_like(x)
    table, lens = torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    written = (*cache, k, v, out, lse)
    before = [t._version for t in written]
    g.rfp2_kv_write(cache, x, x, slots)
    g.rfp2_kv_read(cache, slots, k=k, v=v)
    g.rfp2_attn_decode(q, cache, table, lens, out=out, lse=lse)
    assert all(t._version > n for t, n in zip(written, before))
    with torch.inference_mode():         # where versions are not kept
        inside = x.clone()
        g.rfp2_rope(inside, positions, f, out=inside)
    g.rfp2_rope(inside, positions, f, out=inside)


def test_queries_and_outputs_in_common_memory(g):
    """In place, row by row, and in the gaps between the rows of q: the same results as apart."""
    import torch
    r = torch.Generator(device="cuda").manual_seed(5)
    B, nq, Hq, Hkv, D, page, pages = 3, 2, 8, 2, 64, 16, 400
    cache = g.rfp2_kv_alloc(pages, Hkv, page, D)
    for t in cache:
        t.copy_(torch.randint(-127, 128, t.shape, generator=r, device="cuda") if t.dtype == torch.int8 else
                torch.rand(t.shape, generator=r, device="cuda") / 60)
    table = torch.randperm(pages - 1, generator=r, device="cuda").int().view(B, -1)
    lens = torch.tensor([2100, 17, 0], dtype=torch.int32, device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        q = torch.randn((B, nq, Hq, D), generator=r, device="cuda").to(dtype)
        out, lse = g.rfp2_attn_decode(q, cache, table, lens)
        here = q.clone()
        for _ in range(3):
            here.copy_(q)
            same, lse2 = g.rfp2_attn_decode(here, cache, table, lens, out=here)
            assert same.data_ptr() == here.data_ptr() and torch.equal(same, out) and torch.equal(lse2, lse)
        n = nq * Hq * D
        arena = torch.zeros((B, 5 * n), device="cuda", dtype=dtype)
        between = arena[:, :n].unflatten(1, (nq, Hq, D))
        between.copy_(q)
        gap = arena[0, n: 4 * n].view(B, nq, Hq, D)
        inside, _ = g.rfp2_attn_decode(between, cache, table, lens, out=gap)
        assert inside.data_ptr() == gap.data_ptr() and torch.equal(inside, out) and torch.equal(between, q)
        with pytest.raises(g.RFP2Error) as e:
            g.rfp2_attn_decode(between, cache, table, lens, out=arena.view(-1)[2 * n + D: 5 * n + D].view(B, nq, Hq, D))
        assert e.value.status == 1


@pytest.mark.parametrize("T,H,D,turned", [(3000, 1, 32, 0), (3000, 1, 32, 32), (16417, 2, 64, 64), (200001, 1, 32, 0), (1500001, 1, 32, 2)])
def test_many_tokens_to_write_and_read(g, T, H, D, turned):
    """More tokens than a CTA's table holds, than the CTAs take at once, odd ones: each is where its slot says, the
    same as when it is written by itself."""
    import torch
    r = torch.Generator(device="cuda").manual_seed(T)
    page = 16
    whole, parts = (g.rfp2_kv_alloc(-(-T // page) + 1, H, page, D) for _ in range(2))
    k, v = torch.randn((2, T, H, D), generator=r, device="cuda")
    slots = torch.randperm(T, generator=r, device="cuda")
    slots[:: 97] = -1
    rotation = ()
    if turned:
        rotation = (torch.randint(0, 9999, (T,), generator=r, device="cuda", dtype=torch.int32), g.rfp2_rope_frequencies(turned)[0])
    g.rfp2_kv_write(whole, k, v, slots, *rotation)
    for a in range(0, T, 999):
        b = min(a + 999, T)
        g.rfp2_kv_write(parts, k[a:b], v[a:b], slots[a:b], *(t if t.numel() != T else t[a:b] for t in rotation))
    assert all(torch.equal(x, y) for x, y in zip(whole, parts))
    kept = slots >= 0
    rk, rv = g.rfp2_kv_read(whole, slots)
    if not turned:
        assert float((rk - k)[kept].abs().max()) <= float(k.abs().max()) / 253
    assert float((rv - v)[kept].abs().max()) <= float(v.abs().max()) / 253
    assert not rk[~kept].any() and not rv[~kept].any()


def test_no_sequences(g):
    """A batch of none, as a server between requests has, is nothing to do; what else is wrong is still said."""
    import torch
    cache = g.rfp2_kv_alloc(2, 2, 4, 64)
    q = torch.empty((0, 1, 4, 64), device="cuda")
    table, lens = (torch.empty(s, dtype=torch.int32, device="cuda") for s in ((0, 3), (0,)))
    for workspace in (None, torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")):
        out, lse = g.rfp2_attn_decode(q, cache, table, lens, workspace=workspace)
        assert out.shape == (0, 1, 4, 64) and lse.shape == (0, 1, 4)
    with pytest.raises(ValueError):
        g.rfp2_attn_decode(q, cache, table, torch.zeros(1, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError):
        g.rfp2_attn_decode(q, cache, table.long(), lens)

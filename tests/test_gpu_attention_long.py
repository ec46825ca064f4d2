"""Decode attention where a warp has many tiles: long stretches of one sequence, several short sequences one
after another, and both, against the formula in float64 (computed by torch on the GPU, a sequence at a time).

Bounds as in test_gpu_attention_range.py, with fp32 sums over a stretch and then over the stretches."""
import math

import pytest

pytestmark = pytest.mark.gpu
HALF_ULP = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}


@pytest.fixture(scope="module")
def g():
    import gemm_rocmfp2_mul_gb300 as g
    g.build()
    g.lib()
    return g


def make(B, nq, Hq, Hkv, D, page, lens, dtype, seed, shared=False, positive=False):
    """q, cache, table, lens; shared: every sequence's table starts with the same pages."""
    import torch
    r = torch.Generator(device="cuda").manual_seed(seed)
    lens = torch.as_tensor(lens, dtype=torch.int32).expand(B).contiguous()
    held = [-(-int(n) // page) for n in lens]
    pages, width = (max(held) if shared else sum(held)) + 1, max(max(held), 1)
    order = torch.randperm(pages, generator=r, device="cuda").int()
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = order[:n] if shared else order[at: at + n]
        at += n
    shape = (pages, Hkv, page)
    kc, vc = (torch.randint(-127, 128, shape + (D,), generator=r, device="cuda").to(torch.int8) for _ in range(2))
    ks, vs = (torch.exp(0.4 * torch.randn(shape + (D // 32,), generator=r, device="cuda")) / 60 for _ in range(2))
    if positive:                # and of another mean for each head and place, up to 2 * 31 + 60
        place = torch.arange(D, dtype=torch.int8, device="cuda") % 32
        vc = (vc.int().abs() % 60 + 1).to(torch.int8) + 2 * place
        vs *= torch.exp2(torch.arange(Hkv, device="cuda") / Hkv)[:, None, None]
    q = torch.randn((B, nq, Hq, D), generator=r, device="cuda").to(getattr(torch, dtype))
    return q, (kc, ks, vc, vs), table, lens.cuda()


def definition(q, cache, table, lens, window=0):
    """out, sum p|v| / sum p, lse and the largest scale sum|q k| of each row, float64."""
    import torch
    B, nq, Hq, D = q.shape
    kc, ks, vc, vs = cache
    Hkv, page = kc.shape[1:3]
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    size, lse, most = out.clone(), torch.full((B, nq, Hq), -math.inf, dtype=torch.float64, device="cuda"), 0.0
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            continue
        j = torch.arange(n, device="cuda")
        p, o = table[b, j // page].long(), j % page
        for h in range(Hkv):
            k, v = (c[p, h, o].double() * s[p, h, o].double().repeat_interleave(32, -1) for c, s in ((kc, ks), (vc, vs)))
            x = q[b].double().view(nq, Hkv, -1, D)[:, h]
            s = torch.einsum("igd,jd->igj", x, k) * D ** -0.5
            end = n - nq + 1 + torch.arange(nq, device="cuda")[:, None]
            seen = (j < end) & ((j >= end - window) if window else True)
            s = s.masked_fill(~seen[:, None], -math.inf)
            w = torch.softmax(s, -1).nan_to_num(0.0)
            here = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            out[b, :, here] = w @ v
            size[b, :, here] = w @ v.abs()
            lse[b, :, here] = torch.logsumexp(s, -1)
            most = max(most, float((x.abs() @ k.abs().T).max()) * D ** -0.5)
    return out, size, lse, most


def judge(state, out, lse, dtype, window=0):
    ref, size, ref_lse, most = definition(*state, window=window)
    n = float(state[3].max())
    ds = 2.0 ** -19 * most
    share = 2 * ds + 2.0 ** -19 + n * 2.0 ** -23 + (0.0 if dtype == "float32" else 2.0 ** -15)
    bound = size * share + HALF_ULP[dtype] * ref.abs() + (2.0 ** -25 if dtype == "float16" else 0.0)
    err = (out.double() - ref).abs()
    assert bool(out.isfinite().all()) and bool((err <= bound).all()), float((err / bound.clamp(min=1e-30)).max())
    empty = ref_lse.isinf()
    assert bool((lse[empty] == -math.inf).all()) and bool((out[empty] == 0).all())
    off = (lse.double() - ref_lse).abs()[~empty]
    assert bool((off <= ds + 2.0 ** -20 + n * 2.0 ** -24 + 2.0 ** -22 * ref_lse[~empty].abs()).all()), float(off.max())


def run(g, state, window=0):
    import torch
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = g.rfp2_attn_decode(*state, window=window, dev_status=st)
    assert int(st) == 0
    return out, lse


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("B,Hq,Hkv,D,page,keys,window", [
    (64, 8, 8, 32, 16, 4000, 0), (64, 64, 8, 64, 64, 4000, 0), (48, 40, 8, 64, 17, 3000, 0), (40, 128, 8, 128, 16, 2500, 0),
    (64, 32, 8, 64, 16, 4000, 1500), (24, 16, 8, 256, 17, 1500, 0)])
def test_long_stretches(g, B, Hq, Hkv, D, page, keys, window, dtype):
    """Twenty to seventy tiles a warp, of one sequence or of two or three."""
    import torch
    r = torch.Generator().manual_seed(B + D)
    lens = torch.randint(keys // 2, keys, (B,), generator=r)
    lens[B // 2] = 0
    state = make(B, 1, Hq, Hkv, D, page, lens, dtype, seed=page)
    judge(state, *run(g, state, window), dtype, window)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("B,nq,Hq,Hkv,D,page,window", [
    (600, 1, 8, 8, 64, 16, 0), (700, 1, 64, 4, 32, 7, 0), (300, 3, 32, 16, 128, 16, 0), (600, 1, 32, 8, 64, 64, 50), (200, 1, 8, 8, 256, 24, 0)])
def test_several_sequences_a_warp(g, B, nq, Hq, Hkv, D, page, window, dtype):
    """Hundreds of sequences of 0 to 200 keys and a long one among them: a warp ends one, has some whole and
    begins another."""
    import torch
    r = torch.Generator().manual_seed(B)
    lens = torch.randint(0, 200, (B,), generator=r)
    lens[::7] = 0
    lens[B // 3] = 5000
    state = make(B, nq, Hq, Hkv, D, page, lens, dtype, seed=nq + D)
    judge(state, *run(g, state, window), dtype, window)


@pytest.mark.parametrize("dtype,Hq,most", [("float16", 8, 2.0 ** -16), ("float16", 64, 2.0 ** -16), ("bfloat16", 64, 2.0 ** -15),
                                           ("float32", 32, 2.0 ** -20)])
def test_sums_of_long_rows_are_not_cut_off(g, dtype, Hq, most):
    """Some 1700 tiles a warp of positive values.  What cutting off takes from a sum has one sign, about
    2^-25 of it a tile, 2^-14 in the end.  Roundings to nearest cancel: N = 2048 Hq outputs, each off by up to
    h of itself (half a unit: 2^-8, 2^-11, 2^-24), have a mean error of deviation h / sqrt(3 N), four
    of which are 2^-15.3 for bf16 of 64 heads and 2^-16.8 for f16 of 8."""
    B, Hkv, D, keys = 64, 8, 32, 131072
    state = make(B, 1, Hq, Hkv, D, 64, keys, dtype, seed=5, shared=True, positive=True)
    out, lse = run(g, state)
    judge(state, out, lse, dtype)
    ref = definition(*state)[0]
    bias = float(((out.double() - ref) / ref).mean())
    assert abs(bias) <= most, bias

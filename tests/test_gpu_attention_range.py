"""Decode attention over values, weights and queries of any size, each output judged by what goes into it.

Bounds, from the formula.  A score is off by at most ds = 2^-19 scale sum|q k| (as in test_gpu_attention.py),
so a weight by a factor within 1 +- (ds + 2^-21).  A weight times a value's scale is an fp32 product, and it
enters whole for fp32 outputs; for 16-bit ones to 16 bits: the first 8 cut off, so that less than 2^-7 is
left, and that rounded to 8, 2^-8 of it: 2^-15.  The sums are fp32's: n 2^-23.  Every term is relative to
size = sum p|v| / sum p of the output itself, whatever other outputs of its row are, and half a unit in the
last place of the result is added.  A weight below 2^-126 of the largest is nothing (fp32's range)."""
import numpy as np
import pytest

import _attention as plain
from test_gpu_attention import Case, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import gemm_rocmfp2_mul_gb300 as g
    g.build()
    g.lib()
    return g


def half_ulp(ref, dtype):
    """Half a unit in the last place of `dtype` at each |ref|."""
    bits, least = {"float32": (24, -149), "bfloat16": (8, -133), "float16": (11, -24)}[dtype]
    with np.errstate(divide="ignore"):
        e = np.where(ref == 0, -1000.0, np.floor(np.log2(np.abs(ref))))
    return np.exp2(np.maximum(e - bits, least - 1.0))


def judge(c, out, lse, **kw):
    q = c.q.double().numpy()
    ref, ref_lse = plain.attention(q, c.k, c.v, c.lens, c.scale, **kw)
    size, _ = plain.attention(q, c.k, [np.abs(v) for v in c.v], c.lens, c.scale, **kw)
    B, nq, Hq, D = q.shape
    most = np.zeros((B, 1, Hq, 1))
    for b in range(B):
        for h in range(Hq if len(c.k[b]) else 0):
            most[b, 0, h, 0] = (np.abs(c.k[b][:, h // (Hq // c.k[b].shape[1])]) @ np.abs(q[b, :, h]).T).max()
    ds = 2.0 ** -19 * c.scale * most
    n = float(np.max(c.lens))
    share = 2 * ds + 2.0 ** -19 + n * 2.0 ** -23 + (0.0 if c.dtype == "float32" else 2.0 ** -15)
    bound = size * share + half_ulp(ref, c.dtype)
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    err = np.abs(out - ref)
    assert np.isfinite(out).all() and np.all(err <= bound), (err / bound).max()
    seen = np.isfinite(ref_lse)
    off = np.abs(lse - ref_lse)[seen]
    room = np.broadcast_to(ds[..., 0], lse.shape)[seen] + 2.0 ** -20 + n * 2.0 ** -24 + 2.0 ** -22 * np.abs(ref_lse[seen])
    assert np.all(off <= room), (off / room).max()


def rescale(c, by):
    """Multiply the value scales [pages, heads, page, blocks] and what the case knows of them."""
    c.vs *= by
    page = c.vs.shape[2]
    for b, n in enumerate(c.lens):
        j = np.arange(n)
        p, o = c.table[b, j // page], j % page
        c.v[b] = plain.values(c.vc[p, :, o], c.vs[p, :, o])


SHAPES = [(2, 1, 4, 2, 128, 16, [300, 77]), (1, 1, 10, 1, 64, 24, 200), (1, 3, 8, 1, 96, 16, 120), (2, 1, 2, 2, 256, 33, [90, 41])]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("apart", [10, 20, 40])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "h%d_%d_D%d" % (s[2], s[3], s[4]))
def test_blocks_of_a_head_that_differ(g, shape, apart, dtype):
    """Value scales 2^apart between the blocks of a head: the same blocks for every key, and others for each."""
    r = np.random.default_rng(apart)
    D = shape[4]
    for same in (True, False):
        c = Case(*shape, dtype=dtype, seed=apart)
        size = c.vs.shape if not same else (D // 32,)
        rescale(c, np.exp2(-apart * r.integers(0, 2, size) + (0 if same else -3 * r.integers(0, 2, size))).astype(np.float32))
        if dtype == "float16":      # whose own range would hide the small ones
            rescale(c, np.float32(2.0 ** (apart // 3)))
        judge(c, *_run(g, c))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("Hq,Hkv,D", [(4, 4, 128), (16, 2, 64), (16, 1, 128), (3, 1, 256)])
def test_one_key_is_its_value(g, Hq, Hkv, D, dtype):
    c = Case(40, 1, Hq, Hkv, D, 16, 1, dtype=dtype, seed=D + Hq)
    r = np.random.default_rng(1)
    rescale(c, np.exp2(-r.integers(0, 12, c.vs.shape)).astype(np.float32))
    judge(c, *_run(g, c))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("Hq", [2, 16])
def test_small_weights_count_where_the_large_have_no_value(g, Hq, dtype):
    """Peaked scores, and codes that are 0 for most (key, block)s: an output may rest on weights far below
    the largest."""
    c = Case(1, 1, Hq, 1, 128, 16, 160, dtype=dtype, seed=3, spread=5.0)
    r = np.random.default_rng(2)
    c.vc *= (r.random(c.vs.shape) < 0.05).astype(np.int8).repeat(32, -1)
    rescale(c, np.float32(1.0))
    if dtype == "float16":
        rescale(c, np.float32(2.0 ** 10))
    judge(c, *_run(g, c))


@pytest.mark.parametrize("Hq", [4, 8, 16])
def test_values_of_extreme_size(g, Hq):
    for e in (-90, 100):
        c = Case(2, 1, Hq, 1, 64, 16, [50, 200], seed=4)
        rescale(c, np.float32(2.0 ** e))
        judge(c, *_run(g, c))


@pytest.mark.parametrize("keys", [-100, 0, 100])
@pytest.mark.parametrize("dtype,tiny,huge", [("float32", -120, 100), ("float32", -60, 90), ("bfloat16", -120, 115)])
def test_tiny_and_huge_queries_of_one_key_head(g, dtype, tiny, huge, keys):
    """Rows of q far below 1 beside rows far above it, on keys of any size: scores of 0, of order 1, and as large
    as fp32 holds, side by side."""
    import torch
    c = Case(1, 2, 8, 2, 64, 16, 90, dtype=dtype, seed=7)
    size = torch.tensor([tiny, huge, 0, tiny, 0, huge, tiny, huge]).double().exp2().view(1, 1, 8, 1)
    size = torch.minimum(size, torch.tensor(2.0 ** (120 - keys)).double())     # whose scores stay finite
    c.q = (c.q.double() * size).to(c.q.dtype)
    c.ks *= np.float32(2.0 ** keys)
    c.k = [k * 2.0 ** keys for k in c.k]
    judge(c, *_run(g, c))

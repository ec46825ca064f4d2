"""Decode attention over the paged Q8 cache (rfp2_attn_decode) against the formula in float64, on the
values that the cache holds.

Tolerances, from the formula.  A score is a sum of products of q and exact codes: with q in two pieces of
11 bits (residual 2^-22), fp32 sums inside blocks, over blocks, times the scale, it is off by at most
ds = 2^-19 scale sum|q k| (and a soft cap of 2 ulp adds 2^-21 cap).  Every p is then off by a factor
within 1 +- (ds + 2^-21) of the reference's, numerator and denominator alike, and fp32 sums over n keys
add n 2^-24.  With 16-bit activations q is exact, and p times a value's scale is rounded to 11 bits.
A weight below 2^-40 of the largest may be lost altogether (an exponent that underflows).
So |out - ref| <= (sum p|v| / sum p)(2 ds + 2^-19 + n 2^-23 [+ 2^-10 for 16 bits]) + n 2^-40 max|v| + half
a unit of the output's last place, and |lse - ref| <= ds + 2^-20 + n 2^-24 + 2^-22 |lse|."""
import numpy as np
import pytest

import _attention as plain

pytestmark = pytest.mark.gpu
HALF_ULP = {"float32": 0.0, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}


@pytest.fixture(scope="module")
def g():
    import gemm_rocmfp2_mul_gb300 as g
    g.build()
    g.lib()
    return g


class Case:
    """A cache of shuffled pages in which everything that no sequence holds is NaN, and a table whose
    unused places are garbage."""

    def __init__(self, B, nq, Hq, Hkv, D, page, lens, dtype="float32", seed=0, spread=1.0, v_spread=0.0):
        import torch
        r = np.random.default_rng(seed)
        self.lens = np.broadcast_to(np.asarray(lens, np.int32), (B,)).copy()
        held = [-(-int(n) // page) for n in self.lens]
        pages, width = sum(held) + 2, max(max(held), 1) + 1
        order = r.permutation(pages)
        self.table = r.choice([-1, pages, 2 ** 31 - 1, -2 ** 31], (B, width)).astype(np.int32)
        shape = (pages, Hkv, page, D)
        self.kc, self.vc = (r.integers(-127, 128, shape).astype(np.int8) for _ in range(2))
        self.ks, self.vs = (np.full(shape[:3] + (D // 32,), np.nan, np.float32) for _ in range(2))
        self.k, self.v, at = [], [], 0
        for b in range(B):
            n = int(self.lens[b])
            mine = order[at: at + held[b]]
            at += held[b]
            self.table[b, : held[b]] = mine
            j = np.arange(n)
            p, o = mine[j // page] if n else j, j % page
            size = (n, Hkv, D // 32)
            self.ks[p, :, o] = np.exp(0.5 * r.standard_normal(size)) * spread / 60
            self.vs[p, :, o] = np.exp(0.5 * r.standard_normal(size)) * np.exp2(v_spread * r.standard_normal((n, Hkv, 1))) / 60
            self.k.append(plain.values(self.kc[p, :, o], self.ks[p, :, o]))
            self.v.append(plain.values(self.vc[p, :, o], self.vs[p, :, o]))
        self.q = torch.from_numpy(r.standard_normal((B, nq, Hq, D)).astype(np.float32)).to(getattr(torch, dtype))
        self.dtype, self.scale = dtype, D ** -0.5

    def device(self):
        import torch
        cache = tuple(torch.from_numpy(t).cuda() for t in (self.kc, self.ks, self.vc, self.vs))
        return self.q.cuda(), cache, torch.from_numpy(self.table).cuda(), torch.from_numpy(self.lens).cuda()

    def check(self, out, lse, window=0, softcap=0.0, scale=None, lens=None):
        scale = self.scale if scale is None else scale
        lens = self.lens if lens is None else lens
        q = self.q.double().numpy()
        ref, ref_lse = plain.attention(q, self.k, self.v, lens, scale, window, softcap)
        size, _ = plain.attention(q, self.k, [np.abs(v) for v in self.v], lens, scale, window, softcap)
        B, nq, Hq, D = q.shape
        most = np.zeros((B, 1, Hq, 1))
        for b in range(B):
            if len(self.k[b]):
                for h in range(Hq):
                    most[b, 0, h, 0] = np.nanmax(np.abs(self.k[b][:, h // (Hq // self.k[b].shape[1])]) @ np.abs(q[b, :, h]).T)
        ds = 2.0 ** -19 * abs(scale) * most + 2.0 ** -21 * softcap
        n = float(np.max(lens))
        share = 2 * ds + 2.0 ** -19 + n * 2.0 ** -23 + (0.0 if self.dtype == "float32" else 2.0 ** -10)
        lost = n * 2.0 ** -40 * max([float(np.nanmax(np.abs(v))) for v in self.v if v.size] or [0.0])
        bound = size * share + lost + HALF_ULP[self.dtype] * np.abs(ref) + (2.0 ** -25 if self.dtype == "float16" else 0.0)
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        assert np.array_equal(np.isnan(out), np.isnan(ref)) and np.all(np.isfinite(out))
        err = np.abs(out - ref)
        assert np.all(err <= bound), (err / np.maximum(bound, 1e-30)).max()
        empty = np.isinf(ref_lse)
        assert np.array_equal(lse == -np.inf, empty) and np.all(out[empty] == 0.0)
        off = np.abs(lse[~empty] - ref_lse[~empty])
        room = np.broadcast_to(ds[..., 0], lse.shape)[~empty] + 2.0 ** -20 + n * 2.0 ** -24 + 2.0 ** -22 * np.abs(ref_lse[~empty])
        assert np.all(off <= room), (off / room).max()


def _run(g, c, **kw):
    import torch
    q, cache, table, lens = c.device()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = g.rfp2_attn_decode(q, cache, table, lens, dev_status=st, **kw)
    assert int(st) == 0
    return out, lse


SHAPES = [
    # B, nq, Hq, Hkv, D, page, lens
    (1, 1, 1, 1, 32, 1, 1),
    (1, 1, 8, 1, 64, 16, 15),
    (3, 1, 32, 8, 128, 16, [1, 17, 300]),
    (2, 1, 8, 8, 128, 64, [64, 65]),
    (2, 1, 40, 8, 128, 32, [1000, 31]),
    (5, 1, 16, 2, 64, 7, [0, 6, 7, 8, 501]),
    (2, 1, 5, 5, 96, 17, [250, 33]),
    (1, 1, 16, 1, 128, 128, 700),
    (1, 1, 34, 2, 160, 48, 555),
    (2, 1, 4, 2, 192, 16, [400, 129]),
    (1, 1, 6, 2, 224, 5, 333),
    (3, 1, 14, 2, 256, 33, [100, 0, 512]),
    (9, 1, 4, 4, 32, 256, [0, 1, 255, 256, 257, 3, 511, 0, 40]),
]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "B%d_q%d_h%d_%d_D%d_p%d" % s[:6])
def test_one_new_token(g, shape, dtype):
    c = Case(*shape, dtype=dtype, seed=sum(shape[:6]))
    c.check(*_run(g, c))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("window,softcap", [(0, 0.0), (0, 5.0), (1, 0.0), (37, 0.0), (128, 20.0), (100000, 0.0)])
def test_several_tokens_windows_and_soft_caps(g, window, softcap, dtype):
    """Queries that see no key (fewer keys than queries), one key, part of a tile."""
    c = Case(6, 5, 12, 2, 64, 24, [0, 2, 5, 6, 100, 700], dtype=dtype, seed=window)
    c.check(*_run(g, c, window=window, softcap=softcap), window=window, softcap=softcap)


@pytest.mark.parametrize("page", [1, 7, 16, 24, 64])
def test_pages_that_the_window_has_left(g, page):
    """Under a window, a sequence's old pages may belong to others: their table entries are not looked at."""
    window, nq = 50, 2
    c = Case(3, nq, 4, 2, 64, page, [200, 49, 333], seed=page)
    for b, n in enumerate(c.lens):
        first = max(0, int(n) - nq + 1 - window)
        c.table[b, : first // page] = [-1, 2 ** 31 - 1, -5][b]
        c.k[b][:first] = c.v[b][:first] = np.nan     # the formula does not look at them either
    c.check(*_run(g, c, window=window), window=window)


def test_many_columns(g):
    """Queries and heads of a key head beyond one tile of columns."""
    c = Case(2, 9, 14, 2, 128, 16, [400, 30], seed=5)
    c.check(*_run(g, c))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_long_context_is_split_and_joined(g, dtype):
    c = Case(1, 1, 4, 1, 64, 64, 40000, dtype=dtype, seed=2)
    c.check(*_run(g, c))
    c = Case(3, 1, 2, 1, 128, 16, [9000, 1, 5000], dtype=dtype, seed=3)
    c.check(*_run(g, c))


def test_many_short_sequences(g):
    r = np.random.default_rng(0)
    c = Case(1500, 1, 2, 1, 32, 4, r.integers(0, 12, 1500), seed=9)
    c.check(*_run(g, c))


@pytest.mark.parametrize("spread", [0.0, 8.0, 400.0])
def test_scores_of_any_size(g, spread):
    """Equal scores, peaked ones, and a softmax that is one key."""
    c = Case(2, 1, 8, 2, 64, 16, [300, 77], seed=4, spread=spread)
    c.check(*_run(g, c))


@pytest.mark.parametrize("dtype", ["float32", "float16"])
def test_value_scales_of_any_size(g, dtype):
    """Values whose scales differ by many powers of two between tokens, and tiny or zero ones."""
    c = Case(2, 1, 8, 2, 64, 16, [300, 77], seed=4, dtype=dtype, v_spread=4.0)
    c.check(*_run(g, c))
    c = Case(1, 1, 4, 1, 64, 16, 100, seed=6)
    c.vs *= np.float32(2.0 ** -100)
    c.v = [v * 2.0 ** -100 for v in c.v]
    c.check(*_run(g, c))
    c.vs[:] = 0.0
    c.v = [v * 0.0 for v in c.v]
    c.check(*_run(g, c))


def test_lse_of_one_key_is_its_score(g):
    """Near 0 as well: no constant of the kernel's own may round it.  The score's own bound ds (above) and
    the roundings of the way to base 2 and back, 2^-21 of it."""
    for D, Hq, Hkv, small in ((128, 4, 4, 2.0 ** -10), (64, 16, 2, 2.0 ** -14), (256, 5, 1, 1.0)):
        c = Case(3, 1, Hq, Hkv, D, 16, 1, seed=11)
        c.vs[:] = np.float32(1 / 60)
        c.q = c.q * small
        _, lse = _run(g, c)
        q = c.q.double().numpy()[:, 0].reshape(3, Hkv, Hq // Hkv, D)
        k = np.stack([k[0] for k in c.k])[:, :, None]
        s, size = ((x * k).sum(-1).reshape(3, Hq) * c.scale for x in (q, np.abs(q) * np.sign(k)))
        err = np.abs(lse.double().cpu().numpy()[:, 0] - s)
        assert (err <= 2.0 ** -19 * size + 2.0 ** -21 * np.abs(s)).all(), (err / np.abs(s)).max()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
def test_lse_of_one_key_under_a_cap(g, dtype):
    """cap tanh(s / cap): the score's bound ds, and 2^-20 of the result for the reciprocal, the products, the
    tangent's two units in the last place and the way to base 2 and back.  A cap of 2^60 and more is none."""
    import torch
    c = Case(3, 1, 8, 4, 128, 16, 1, seed=12, dtype=dtype)
    c.vs[:] = np.float32(1 / 60)
    c.q = c.q * torch.tensor([2.0 ** -12, 2.0 ** -4, 1, 8, 2.0 ** -12, 2.0 ** -4, 1, 8]).to(c.q.dtype).view(8, 1)
    q = c.q.double().numpy()[:, 0].reshape(3, 4, 2, 128)
    k = np.stack([k[0] for k in c.k])[:, :, None]
    s, size = ((x * k).sum(-1).reshape(3, 8) * c.scale for x in (q, np.abs(q) * np.sign(k)))
    for cap in (30.0, 0.5, 1000.0):
        _, lse = _run(g, c, softcap=cap)
        want = cap * np.tanh(s / cap)
        err = np.abs(lse.double().cpu().numpy()[:, 0] - want)
        assert (err <= 2.0 ** -19 * size + 2.0 ** -20 * np.abs(want)).all(), (cap, (err / np.abs(want)).max())
    plain_out, plain_lse = _run(g, c)
    for cap in (2.0 ** 60, 3e38, float("inf")):
        out, lse = _run(g, c, softcap=cap)
        assert torch.equal(out, plain_out) and torch.equal(lse, plain_lse)


def test_queries_of_any_size(g):
    import torch
    for size in (2.0 ** -120, 2.0 ** 100):
        c = Case(1, 1, 8, 2, 64, 16, 90, seed=7)
        c.q = c.q * torch.tensor([size, 1, 0, size, 1, 1, size, 0]).float().view(1, 1, 8, 1)
        c.ks /= np.float32(size)
        c.k = [k / size for k in c.k]
        if size < 1:     # only the small queries' scores stay finite
            c.q[:, :, [1, 4, 5]] = 0
        c.check(*_run(g, c))


def test_nan_and_infinity_where_they_are_visible(g):
    """A visible key that is not finite spoils the rows that see it and no others."""
    c = Case(2, 3, 4, 2, 64, 16, [60, 60], seed=1)
    b, j = 0, 58                       # seen by queries 1 and 2 of sequence 0
    c.ks[c.table[b, j // 16], 1, j % 16, 0] = np.nan
    out, lse = _run(g, c)
    spoiled = np.isnan(out.cpu().numpy()).all(-1)
    assert np.array_equal(spoiled, np.isnan(out.cpu().numpy()).any(-1))
    assert np.array_equal(spoiled, np.isnan(lse.cpu().numpy()))
    want = np.zeros((2, 3, 4), bool)
    want[0, 1:, 2:] = True             # heads 2 and 3 read key head 1
    assert np.array_equal(spoiled, want)
    c = Case(1, 1, 2, 1, 64, 16, 40, seed=1)
    c.vs[c.table[0, 1], 0, 3, 1] = np.inf
    out, lse = _run(g, c)
    assert not bool(out[..., 32:].isfinite().any()) and bool(out[..., :32].isfinite().all()) and bool(lse.isfinite().all())


def test_strides_and_scale(g):
    import torch
    c = Case(3, 2, 8, 2, 64, 16, [40, 41, 300], seed=8, dtype="bfloat16")
    q, cache, table, lens = c.device()
    wide = torch.zeros((3, 8, 2, 67), dtype=q.dtype, device="cuda")
    wide[..., 3:] = q.transpose(1, 2)
    wide_table = torch.full((3, 99), -7, dtype=torch.int32, device="cuda")
    wide_table[:, 5: 5 + table.shape[1]] = table
    out, lse = g.rfp2_attn_decode(wide[..., 3:].transpose(1, 2), cache, wide_table[:, 5: 5 + table.shape[1]], lens, scale=0.3)
    c.check(out, lse, scale=0.3)


def test_workspace_serves_call_after_call(g):
    """One workspace, calls of many sizes in a row and on a stream of its own: the same bits as with a
    new one each time."""
    import torch
    cases = [Case(*s, seed=i) for i, s in enumerate(SHAPES + [(1, 1, 4, 1, 64, 64, 20000)])]
    state = [c.device() for c in cases]
    alone = [g.rfp2_attn_decode(*s) for s in state]
    size = max(g.rfp2_attn_decode_workspace_bytes(*s[0].shape[:3], s[1][0].shape[1], s[0].shape[3]) for s in state)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
        for _ in range(3):
            again = [g.rfp2_attn_decode(*s, workspace=ws) for s in state]
        stream.synchronize()
    for a, b in zip(alone, again):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_cache_beyond_32_bit_offsets(g):
    """Codes past 4 GiB: the last pages of a large cache hold the sequence."""
    import torch
    c = Case(1, 1, 8, 2, 128, 64, 500, seed=3)
    q, cache, table, lens = c.device()
    pages = 265000                     # x 2 heads x 64 x 128 bytes = 4.3 GB of codes
    shift = pages - cache[0].shape[0]
    big = tuple(torch.zeros((pages,) + t.shape[1:], dtype=t.dtype, device="cuda") for t in cache)
    for t, s in zip(big, cache):
        t[shift:] = s
    held = -(-500 // 64)
    table = table.clone()
    table[:, :held] += shift
    assert big[0].numel() > 2 ** 32
    c.check(*g.rfp2_attn_decode(q, big, table, lens))
    slots = (table[0, :1].long() * 64 + 63)
    k, v = g.rfp2_kv_read(big, slots)
    assert torch.equal(k[0].double().cpu(), torch.from_numpy(c.k[0][63]).float().double())
    g.rfp2_kv_write(big, v, k, slots)
    k2, v2 = g.rfp2_kv_read(big, slots)
    # the values of a block of codes quantise back to within one rounding of themselves
    assert torch.allclose(k2, v, rtol=0, atol=float(v.abs().max()) / 200) and torch.allclose(v2, k, rtol=0, atol=float(k.abs().max()) / 200)
    del big


def test_pages_and_lengths_outside_the_cache(g):
    """The rows that need them are NaN and the status says so; the others are right."""
    import torch
    c = Case(4, 1, 4, 2, 64, 16, [50, 50, 50, 50], seed=2)
    q, cache, table, lens = c.device()
    table[1, 2] = cache[0].shape[0]
    lens[2] = -1
    lens[3] = table.shape[1] * 16 + 1
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = g.rfp2_attn_decode(q, cache, table, lens, dev_status=st)
    assert int(st) == 7
    assert bool(out[1:].isnan().all()) and bool(lse[1:].isnan().all())
    c.q, c.k, c.v = c.q[:1], c.k[:1], c.v[:1]
    c.check(out[:1], lse[:1], lens=c.lens[:1])


def test_the_sum_of_two_halves(g):
    """Attention over a cache equals that over its two halves joined by their lse: what lse is for."""
    import torch
    c = Case(1, 1, 8, 2, 64, 16, 320, seed=12)
    q, cache, table, lens = c.device()
    out, lse = g.rfp2_attn_decode(q, cache, table, lens)
    half = torch.full_like(lens, 160)
    a, la = g.rfp2_attn_decode(q, cache, table, half)
    b, lb = g.rfp2_attn_decode(q, cache, table[:, 10:], half)
    joined = torch.logaddexp(la.double(), lb.double())
    assert float((joined - lse.double()).abs().max()) < 1e-5
    mix = (torch.exp(la.double() - joined)[..., None] * a.double() + torch.exp(lb.double() - joined)[..., None] * b.double())
    assert float((mix - out.double()).abs().max()) < 1e-5


def test_refusals(g):
    import torch
    c = Case(2, 1, 4, 2, 64, 16, [5, 6])
    q, cache, table, lens = c.device()
    for error, change in [(TypeError, dict(q=q.double())), (TypeError, dict(lens=lens.long())), (TypeError, dict(table=table.long())),
                          (ValueError, dict(lens=lens[:1])), (ValueError, dict(q=q[0])), (ValueError, dict(table=table[:1])),
                          (ValueError, dict(out=torch.empty((2, 1, 4, 32), device="cuda"))),
                          (ValueError, dict(lse=torch.empty((2, 1, 3), device="cuda"))),
                          (TypeError, dict(out=torch.empty((2, 1, 4, 64), device="cuda").half())),
                          (TypeError, dict(workspace=torch.zeros(1 << 20, device="cuda")))]:
        with pytest.raises(error):
            g.rfp2_attn_decode(**{"q": q, "cache": cache, "table": table, "lens": lens, **change})
    for change, status in ((dict(q=q[:, :, :3]), 2), (dict(window=-1), 1), (dict(softcap=-1.0), 1), (dict(softcap=float("nan")), 1),
                           (dict(workspace=torch.zeros(8, dtype=torch.uint8, device="cuda")), 9), (dict(q=q[:, :0]), 2)):
        with pytest.raises(g.RFP2Error) as e:
            g.rfp2_attn_decode(**{"q": q, "cache": cache, "table": table, "lens": lens, **change})
        assert e.value.status == status

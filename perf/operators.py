"""Cases of the attention operators that stand between the block-quantised products of a decoder layer.

Three operators, each with the sizes it meets in use:
  rope   rotary positions of the query and key heads (rfp2_rope)
  kv     new keys and values written to the paged cache as Q8 blocks and read back
         (rfp2_kv_write, rfp2_kv_read), with the keys rotated on the way in some cases
  attn   attention of the newest tokens of each sequence over that cache (rfp2_attn_decode)

A cache is four tensors: key codes int8 [pages, heads, page, D], key scales fp32
[pages, heads, page, D/32], and the same two for values.  A value is code * scale, with
scale = max|a| / 127 over 32 neighbouring values and code = round-half-away(a / scale).
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # One decode step of four sequences: the query heads of a 4096-wide layer, fp32 as the GEMV returns them.
        {"name": "rope_step", "op": "rope", "T": 4, "H": 32, "D": 128, "R": 128, "dtype": "f32",
         "interleaved": False, "inverse": False, "top": 4096, "stretch": 1.0},
        # A 2048-token prompt chunk of a 5120-wide layer deep in a context stretched eightfold.
        {"name": "rope_prompt", "op": "rope", "T": 2048, "H": 40, "D": 128, "R": 128, "dtype": "bf16",
         "interleaved": False, "inverse": False, "top": 1000000, "stretch": 8.0},
        # The gradient through a partly rotated, interleaved head on a long ragged batch.
        {"name": "rope_grad", "op": "rope", "T": 16383, "H": 20, "D": 192, "R": 64, "dtype": "f16",
         "interleaved": True, "inverse": True, "top": 32768, "stretch": 1.0},
        # One new token of eight sequences, fp32 from the GEMV.
        {"name": "kv_step", "op": "kv", "T": 8, "H": 8, "D": 128, "page": 16, "dtype": "f32", "R": 0,
         "interleaved": False, "top": 4096, "skip": 0.0},
        # A long prompt: keys rotated and both quantised as they are written, then read for a dense prefill.
        {"name": "kv_prompt", "op": "kv", "T": 16384, "H": 8, "D": 128, "page": 64, "dtype": "bf16", "R": 128,
         "interleaved": False, "top": 131072, "skip": 0.0},
        # Padded ragged prompts: odd counts, a head of three blocks, pages of 17, some tokens not kept.
        {"name": "kv_ragged", "op": "kv", "T": 4999, "H": 5, "D": 96, "page": 17, "dtype": "f16", "R": 64,
         "interleaved": True, "top": 9000, "skip": 0.06},
        # One user, a short context: latency.
        {"name": "attn_one", "op": "attn", "B": 1, "nq": 1, "Hq": 32, "Hkv": 8, "D": 128, "len": 1000, "page": 16,
         "dtype": "f32", "window": 0, "softcap": 0.0, "empty": False, "lens_seed": 1},
        # A decode step of sixteen sequences of mixed lengths.
        {"name": "attn_step", "op": "attn", "B": 16, "nq": 1, "Hq": 32, "Hkv": 8, "D": 128, "len": 8192, "page": 16,
         "dtype": "f32", "window": 0, "softcap": 0.0, "empty": False, "lens_seed": 2},
        # One user with a very long context: the length has to be split.
        {"name": "attn_long", "op": "attn", "B": 1, "nq": 1, "Hq": 40, "Hkv": 8, "D": 128, "len": 131072, "page": 64,
         "dtype": "bf16", "window": 0, "softcap": 0.0, "empty": False, "lens_seed": 3},
        # A full server: 64 sequences, a million cached tokens in all.
        {"name": "attn_batch", "op": "attn", "B": 64, "nq": 1, "Hq": 64, "Hkv": 8, "D": 128, "len": 32768, "page": 64,
         "dtype": "bf16", "window": 0, "softcap": 0.0, "empty": False, "lens_seed": 4},
        # Verifying five drafted tokens a sequence under a sliding window and a soft cap; some sequences are empty.
        {"name": "attn_verify", "op": "attn", "B": 12, "nq": 5, "Hq": 16, "Hkv": 2, "D": 64, "len": 5000, "page": 48,
         "dtype": "f16", "window": 1024, "softcap": 30.0, "empty": True, "lens_seed": 5},
        # A key head for every query head, wide heads, odd pages: nothing is shared between heads.
        {"name": "attn_wide", "op": "attn", "B": 7, "nq": 1, "Hq": 16, "Hkv": 16, "D": 256, "len": 3001, "page": 33,
         "dtype": "bf16", "window": 0, "softcap": 0.0, "empty": False, "lens_seed": 6},
    ]


def _log(rng, lo, hi):
    """A size spread evenly over its logarithm; large ones are odd, so that they end inside a tile."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n | 1 if n > 1000 else n


def draw(rng):
    op = rng.choice(["rope", "kv", "attn", "attn"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op == "rope":
        D = rng.choice([32, 64, 128, 128, 160, 192, 256])
        H = rng.choice([1, 5, 8, 20, 32, 40])
        R = rng.choice([D, D, D // 2])
        return {"op": op, "T": _log(rng, 1, min(16384, (1 << 26) // (H * D))), "H": H, "D": D, "R": R, "dtype": dtype,
                "interleaved": rng.random() < 0.5, "inverse": rng.random() < 0.3, "top": _log(rng, 100, 1000000),
                "stretch": rng.choice([1.0, 1.0, 4.0, 16.0])}
    if op == "kv":
        D = rng.choice([32, 64, 96, 128, 128, 160, 192, 256])
        H = rng.choice([1, 2, 5, 8])
        R = rng.choice([0, D, D // 2])
        # Rotated keys are read back in 16 bits: a rotation that is one unit in the last place off can move a code.
        if R and dtype == "f32":
            dtype = "bf16"
        return {"op": op, "T": _log(rng, 1, 16384), "H": H, "D": D, "page": rng.choice([1, 8, 16, 17, 32, 48, 64, 128, 256]),
                "dtype": dtype, "R": R, "interleaved": rng.random() < 0.5, "top": _log(rng, 100, 1000000),
                "skip": rng.choice([0.0, 0.0, 0.1])}
    D = rng.choice([32, 64, 128, 128, 160, 224, 256])
    Hkv = rng.choice([1, 2, 4, 5, 8])
    group = rng.choice([1, 2, 4, 5, 7, 8, 16])
    nq = rng.choice([1, 1, 1, 2, 4, 5, 8])
    B = _log(rng, 1, 64)
    most = max(1, min(131072, (1 << 30) // (B * Hkv * D), (1 << 28) // (B * nq * Hkv * group),
                      (1 << 33) // (B * nq * Hkv * group * D)))
    return {"op": op, "B": B, "nq": nq, "Hq": Hkv * group, "Hkv": Hkv, "D": D, "len": _log(rng, 1, most),
            "page": rng.choice([1, 8, 16, 17, 32, 48, 64, 128, 256]), "dtype": dtype,
            "window": rng.choice([0, 0, 0, _log(rng, 1, 8192)]), "softcap": rng.choice([0.0, 0.0, 30.0]),
            "empty": rng.random() < 0.3, "lens_seed": rng.randrange(1 << 20)}


def _lens(case):
    """The sequences' lengths: anything up to the longest, which is there; some are empty where the case says so."""
    rng = random.Random(case["lens_seed"])
    lens = [1 + int(rng.random() * case["len"]) for _ in range(case["B"])]
    lens = [min(n, case["len"]) for n in lens]
    if case["empty"]:
        lens = [0 if rng.random() < 0.2 else n for n in lens]
    lens[rng.randrange(case["B"])] = case["len"]
    return lens


def _frequencies(R, stretch):
    """Rotary frequencies fp32 [R/2]; a context stretched s-fold turns its slow pairs s times slower."""
    f = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    if stretch > 1.0:
        turns = 4096.0 * f / (2.0 * math.pi)
        keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
        f = f * keep + f / stretch * (1.0 - keep)
    return f.float().cuda()


def _normal(shape, g, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    D, dtype = case["D"], DTYPES[case["dtype"]]
    if case["op"] == "rope":
        T, H = case["T"], case["H"]
        # Heads as the layer's product leaves them: a token's row holds more than the rotated heads.
        rows = _normal((T, (H + 2) * D), g, dtype)
        x = rows[:, : H * D].view(T, H, D)
        positions = torch.randint(0, case["top"], (T,), generator=g, device="cuda", dtype=torch.int32)
        return {**case, "x": x, "positions": positions, "inv_freq": _frequencies(case["R"], case["stretch"]),
                "factor": 1.0 + 0.1 * math.log(case["stretch"]), "out": torch.empty((T, H, D), device="cuda", dtype=dtype)}
    if case["op"] == "kv":
        T, H, page = case["T"], case["H"], case["page"]
        # Channels differ in size, a few by much, as keys do.
        wide = torch.exp(0.5 * _normal((2, 1, H, D), g))
        wide[0, :, :, :: 31] *= 8.0
        rows = torch.stack([(_normal((T, H, D), g) * wide[i]) for i in range(2)], 1).to(dtype)
        pages = (T if T <= 64 else -(-T // page)) + 3
        order = torch.randperm(pages, generator=g, device="cuda")
        t = torch.arange(T, device="cuda")
        if T <= 64:
            slots = order[t] * page + torch.randint(0, page, (T,), generator=g, device="cuda")
        else:
            slots = order[t // page] * page + t % page
        slots = torch.where(torch.rand((T,), generator=g, device="cuda") < case["skip"], -1, slots)
        cache = tuple(torch.zeros((pages, H, page, n), device="cuda", dtype=d)
                      for n, d in ((D, torch.int8), (D // 32, torch.float32)) * 2)
        positions = torch.randint(0, case["top"], (T,), generator=g, device="cuda", dtype=torch.int32)
        return {**case, "k": rows[:, 0], "v": rows[:, 1], "slots": slots, "cache": cache, "positions": positions,
                "inv_freq": _frequencies(case["R"], 1.0) if case["R"] else None,
                "k_out": torch.empty((T, H, D), device="cuda", dtype=dtype),
                "v_out": torch.empty((T, H, D), device="cuda", dtype=dtype)}
    B, nq, Hq, Hkv, page = case["B"], case["nq"], case["Hq"], case["Hkv"], case["page"]
    lens = _lens(case)
    held = [-(-n // page) for n in lens]
    pages, width = sum(held) + 1, max(max(held), 1)
    order = torch.randperm(pages, generator=g, device="cuda").int()
    # The table's unused places hold -1.
    first = torch.tensor([sum(held[:b]) for b in range(B)], device="cuda")[:, None]
    used = torch.arange(width, device="cuda")[None, :]
    table = torch.where(used < torch.tensor(held, device="cuda")[:, None],
                        order[(first + used).clamp(max=pages - 1)], -1).int()

    def codes():
        return (_normal((pages, Hkv, page, D), g) * 42.0).clamp_(-127.0, 127.0).round_().to(torch.int8)

    def scales(size):
        return torch.exp(0.4 * _normal((pages, Hkv, page, D // 32), g)) * (size / 42.0)

    cache = (codes(), scales(1.0), codes(), scales(0.7))
    return {**case, "q": _normal((B, nq, Hq, D), g, dtype), "cache": cache, "table": table,
            "lens": torch.tensor(lens, device="cuda", dtype=torch.int32),
            "out": torch.empty((B, nq, Hq, D), device="cuda", dtype=dtype),
            "lse": torch.empty((B, nq, Hq), device="cuda", dtype=torch.float32), "workspace": None}


# -- the plain forms: elementary operations in 32 bits, rounded once at the end -----------------------------------


def _angles(positions, inv_freq):
    """cos, sin of position * frequency [T, R/2]; what the 32-bit product loses is carried along, so that
    long contexts keep their angles."""
    p, f = positions.float()[:, None], inv_freq[None, :]
    a = p * f
    cp, cf = 4097.0 * p, 4097.0 * f
    ph, fh = cp - (cp - p), cf - (cf - f)
    pl, fl = p - ph, f - fh
    rest = ((ph * fh - a) + ph * fl + pl * fh) + pl * fl
    c, s = torch.cos(a), torch.sin(a)
    return c - s * rest, s + c * rest


def _rotated(x, positions, inv_freq, interleaved, inverse=False, factor=1.0):
    """x [T, H, D] in 32 bits with its first 2 * len(inv_freq) values rotated."""
    n = inv_freq.shape[0]
    x = x.float()
    c, s = (t[:, None, :] * factor for t in _angles(positions, inv_freq))
    if inverse:
        s = -s
    head, rest = x[..., : 2 * n], x[..., 2 * n:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        turned = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = head[..., :n], head[..., n:]
        turned = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([turned, rest], -1)


def _written(x, codes, scales, page, row):
    """x [T, H, D] quantised into the cache at page `page`, place `row`."""
    T, H, D = x.shape
    a = x.reshape(T, H, D // 32, 32)
    d = a.abs().amax(-1) / 127.0
    t = a / torch.where(d == 0.0, 1.0, d)[..., None]
    whole = torch.trunc(t)
    q = whole + torch.sign(t) * ((t - whole).abs() >= 0.5)
    codes[page, :, row] = q.clamp(-127.0, 127.0).to(torch.int8).reshape(T, H, D)
    scales[page, :, row] = d


def _held(codes, scales):
    """The values that codes [..., D] and scales [..., D/32] stand for, in 32 bits."""
    return (codes.float().unflatten(-1, (-1, 32)) * scales[..., None]).flatten(-2)


def _plain_kv(s):
    kept = s["slots"] >= 0
    slots = s["slots"][kept]
    page, row = slots // s["page"], slots % s["page"]
    k = s["k"].float()
    if s["R"]:
        k = _rotated(k, s["positions"], s["inv_freq"], s["interleaved"])
    kq, kd, vq, vd = s["cache"]
    _written(k[kept], kq, kd, page, row)
    _written(s["v"].float()[kept], vq, vd, page, row)
    s["k_out"].zero_()
    s["v_out"].zero_()
    s["k_out"][kept] = _held(kq[page, :, row], kd[page, :, row]).to(s["k_out"].dtype)
    s["v_out"][kept] = _held(vq[page, :, row], vd[page, :, row]).to(s["v_out"].dtype)
    return {"k": s["k_out"], "v": s["v_out"]}


def _plain_attn(s):
    B, nq, Hq, Hkv, D = s["B"], s["nq"], s["Hq"], s["Hkv"], s["D"]
    kq, kd, vq, vd = s["cache"]
    at = s["table"].clamp(min=0).long()
    k, v = (_held(q[at], d[at]).transpose(1, 2).reshape(B, Hkv, -1, D) for q, d in ((kq, kd), (vq, vd)))
    q = s["q"].float().view(B, nq, Hkv, Hq // Hkv, D).transpose(1, 2).reshape(B, Hkv, -1, D)
    x = torch.matmul(q, k.transpose(-1, -2)) * D ** -0.5
    if s["softcap"]:
        x = s["softcap"] * torch.tanh(x / s["softcap"])
    x = x.view(B, Hkv, nq, Hq // Hkv, -1)
    j = torch.arange(x.shape[-1], device=x.device)
    end = s["lens"][:, None] - nq + 1 + torch.arange(nq, device=x.device)
    seen = j < end[..., None]
    if s["window"]:
        seen = seen & (j >= end[..., None] - s["window"])
    x = torch.where(seen[:, None, :, None, :], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, -1, p.shape[-1]), v).view(B, Hkv, nq, -1, D)
    o = torch.where(total > 0.0, o / total, 0.0)
    lse = (torch.log(total) + top)[..., 0]
    s["out"].copy_(o.transpose(1, 2).reshape(B, nq, Hq, D))
    s["lse"].copy_(lse.transpose(1, 2).reshape(B, nq, Hq))
    return {"out": s["out"], "lse": s["lse"]}


def run(s):
    if own:
        import gemm_rocmfp2_mul_gb300 as g
        if s["op"] == "rope":
            return g.rfp2_rope(s["x"], s["positions"], s["inv_freq"], out=s["out"], interleaved=s["interleaved"],
                               inverse=s["inverse"], factor=s["factor"])
        if s["op"] == "kv":
            if s["R"]:
                g.rfp2_kv_write(s["cache"], s["k"], s["v"], s["slots"], positions=s["positions"],
                                inv_freq=s["inv_freq"], interleaved=s["interleaved"])
            else:
                g.rfp2_kv_write(s["cache"], s["k"], s["v"], s["slots"])
            k, v = g.rfp2_kv_read(s["cache"], s["slots"], k=s["k_out"], v=s["v_out"])
            return {"k": k, "v": v}
        if s["workspace"] is None:
            s["workspace"] = g.rfp2_attn_decode_workspace(s["q"], s["Hkv"])
        out, lse = g.rfp2_attn_decode(s["q"], s["cache"], s["table"], s["lens"], window=s["window"],
                                      softcap=s["softcap"], out=s["out"], lse=s["lse"], workspace=s["workspace"])
        return {"out": out, "lse": lse}
    if s["op"] == "rope":
        s["out"].copy_(_rotated(s["x"], s["positions"], s["inv_freq"], s["interleaved"], s["inverse"], s["factor"]))
        return s["out"]
    return _plain_kv(s) if s["op"] == "kv" else _plain_attn(s)


def work(case):
    D, size = case["D"], SIZE[case["dtype"]]
    if case["op"] == "rope":
        T, H, R = case["T"], case["H"], case["R"]
        return {"bytes": 2 * T * H * D * size + 4 * T + 2 * R, "flops": 3 * T * H * R}
    row = D + D // 8  # codes and scales of one key or value
    if case["op"] == "kv":
        T, H = case["T"], case["H"]
        # Read both, write their rows, read the rows, write both.
        return {"bytes": 4 * T * H * (D * size + row) + 16 * T + (4 * T + 2 * case["R"] if case["R"] else 0),
                "flops": 8 * T * H * D + 3 * T * H * case["R"]}
    B, nq, Hq, Hkv, window = (case[n] for n in ("B", "nq", "Hq", "Hkv", "window"))
    keys = pairs = 0
    for n in _lens(case):
        ends = [n - nq + 1 + i for i in range(nq)]
        seen = [(max(0, e - window) if window else 0, max(0, e)) for e in ends]
        pairs += sum(e - b for b, e in seen if e > b)
        keys += max(0, max(e for _, e in seen) - min(b for b, _ in seen))
    tables = 4 * B + 4 * -(-keys // case["page"])
    return {"bytes": keys * Hkv * 2 * row + B * nq * Hq * (2 * D * size + 4) + tables, "flops": 4 * pairs * Hq * D}


# -- the definitions in 64 bits -------------------------------------------------------------------------------------


def _turn64(x, positions, inv_freq, interleaved, sign, factor):
    y = x.double().clone()
    n = inv_freq.numel()
    theta = sign * torch.outer(positions.double(), inv_freq.double())
    turn = torch.polar(torch.full_like(theta, factor), theta)[:, None, :]
    if interleaved:
        z = torch.view_as_complex(y[..., : 2 * n].unflatten(-1, (n, 2)).contiguous()) * turn
        y[..., : 2 * n] = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(y[..., :n].contiguous(), y[..., n: 2 * n].contiguous()) * turn
        y[..., :n], y[..., n: 2 * n] = z.real, z.imag
    return y


def _blocks64(x):
    b = x.double().unflatten(-1, (-1, 32))
    step = b.abs().max(-1, keepdim=True).values / 127
    n = torch.floor(b.abs() / step.masked_fill(step == 0, 1.0) + 0.5)
    return (torch.sign(b) * n * step).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _turn64(s["x"], s["positions"], s["inv_freq"], s["interleaved"], -1.0 if s["inverse"] else 1.0, s["factor"])
    if case["op"] == "kv":
        k = s["k"].double()
        if case["R"]:
            k = _turn64(k, s["positions"], s["inv_freq"], s["interleaved"], 1.0, 1.0)
        lost = (s["slots"] < 0)[:, None, None]
        return {"k": _blocks64(k).masked_fill(lost, 0.0), "v": _blocks64(s["v"]).masked_fill(lost, 0.0)}
    B, nq, Hq, Hkv, D = (case[n] for n in ("B", "nq", "Hq", "Hkv", "D"))
    out = torch.zeros((B, nq, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, nq, Hq), -math.inf, dtype=torch.float64, device="cuda")
    kq, kd, vq, vd = s["cache"]
    for b, n in enumerate(_lens(case)):
        ends = [n - nq + 1 + i for i in range(nq)]
        if ends[-1] <= 0:
            continue
        begin = max(0, min(ends) - case["window"]) if case["window"] else 0
        j = torch.arange(begin, n, device="cuda")
        page, row = s["table"][b, j // case["page"]].long(), j % case["page"]
        # [n, Hkv, D]: each code times the scale of its block
        k = kq[page, :, row].double() * kd[page, :, row].double().repeat_interleave(32, -1)
        v = vq[page, :, row].double() * vd[page, :, row].double().repeat_interleave(32, -1)
        for i, e in enumerate(ends):
            first = max(0, e - case["window"]) if case["window"] else 0
            if e <= first:
                continue
            q = s["q"][b, i].double().view(Hkv, Hq // Hkv, D)
            x = torch.einsum("hgd,jhd->hgj", q, k[first - begin: e - begin]) / math.sqrt(D)
            if case["softcap"]:
                x = torch.tanh(x / case["softcap"]) * case["softcap"]
            lse[b, i] = torch.logsumexp(x, -1).reshape(Hq)
            out[b, i] = torch.einsum("hgj,jhd->hgd", torch.softmax(x, -1), v[first - begin: e - begin]).reshape(Hq, D)
    return {"out": out, "lse": lse}

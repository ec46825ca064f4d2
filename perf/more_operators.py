"""Cases of the feed-forward half of a decoder layer: what stands around the products of its (routed) experts.

Four operators, each with the sizes it meets in use:
  norm     root-mean-square norm after the residual's addition, in an activation type and/or in the
           Q8 blocks of the GEMVs (rfp2_rms_norm)
  route    the experts of each token and their weights, from the router's logits (rfp2_moe_route)
  experts  the routed experts' products on ROCmFP2 weights for any number of tokens, with bias and
           gated activation (rfp2_moe_gemm)
  combine  the weighted sum of a token's experts, plus the residual (rfp2_moe_combine)

ROCmFP2 weights: ten bytes per 32 weights, selectors of the levels {-4, -1, 1, 4} in eight bytes and
two UE4M3 scales, one per 16 weights.  Q8 blocks: value = code * d per 32, d = max|y| / 127,
code = round-half-away(y / d), of the values before any rounding.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # A decode step of four sequences of a 4096-wide layer: the GEMVs' fp32, quantised for the next GEMV.
        {"name": "norm_step", "op": "norm", "T": 4, "K": 4096, "dtype": "f32", "wtype": "f32", "residual": True,
         "want": "q8", "pad": 0},
        # A long prompt of a 5120-wide layer: the norm before a prefill product.
        {"name": "norm_prompt", "op": "norm", "T": 16384, "K": 5120, "dtype": "bf16", "wtype": "bf16",
         "residual": True, "want": "y", "pad": 0},
        # A ragged batch with padding behind its last sequence: values for the router, blocks for the experts.
        {"name": "norm_ragged", "op": "norm", "T": 4999, "K": 1376, "dtype": "f16", "wtype": "f32",
         "residual": False, "want": "both", "pad": 57},
        # A decode step: four tokens over 256 experts.
        {"name": "route_step", "op": "route", "T": 4, "E": 256, "top_k": 8, "dtype": "f32", "scoring": "softmax",
         "bias": False, "groups": 1, "keep": 1, "group_top": 1, "renormalise": True, "scale": 1.0, "masked": 0.0,
         "pad": 0},
        # A long prompt: sigmoid scores, a balancing bias, four of eight groups.
        {"name": "route_prompt", "op": "route", "T": 16384, "E": 256, "top_k": 8, "dtype": "f32",
         "scoring": "sigmoid", "bias": True, "groups": 8, "keep": 4, "group_top": 2, "renormalise": True,
         "scale": 2.5, "masked": 0.0, "pad": 0},
        # An odd number of experts, some of them masked for some tokens, 16-bit logits, padded rows.
        {"name": "route_ragged", "op": "route", "T": 4999, "E": 60, "top_k": 4, "dtype": "bf16",
         "scoring": "softmax", "bias": False, "groups": 1, "keep": 1, "group_top": 1, "renormalise": False,
         "scale": 1.0, "masked": 0.3, "pad": 41},
        # Sixteen decoded tokens over 256 experts: about a hundred experts of one or two tokens each.
        {"name": "experts_step", "op": "experts", "T": 16, "E": 256, "M": 768, "K": 2048, "top_k": 8,
         "activation": "none", "bias": False, "each": False, "pad": 0},
        # A prompt chunk over 256 experts, gate and up rows in one product, padded tokens left out.
        {"name": "experts_prompt", "op": "experts", "T": 2047, "E": 256, "M": 1536, "K": 2048, "top_k": 8,
         "activation": "silu", "bias": False, "each": False, "pad": 13},
        # A long prompt over eight wide experts: thousands of tokens each.
        {"name": "experts_large", "op": "experts", "T": 8192, "E": 8, "M": 14336, "K": 4096, "top_k": 2,
         "activation": "silu", "bias": True, "each": False, "pad": 0},
        # A decode step: eight experts' rows of each of four tokens, onto the fp32 residual.
        {"name": "combine_step", "op": "combine", "T": 4, "M": 2048, "top_k": 8, "dtype": "bf16", "otype": "f32",
         "residual": True, "pad": 0},
        # A long prompt.
        {"name": "combine_prompt", "op": "combine", "T": 16384, "M": 2048, "top_k": 8, "dtype": "bf16",
         "otype": "bf16", "residual": True, "pad": 0},
        # Odd rows, slots without an expert.
        {"name": "combine_ragged", "op": "combine", "T": 4999, "M": 1001, "top_k": 3, "dtype": "f16",
         "otype": "f16", "residual": False, "pad": 300},
    ]


def _log(rng, lo, hi):
    """A size spread evenly over its logarithm; large ones are odd, so that they end inside a tile."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))
    return n | 1 if n > 1000 else n


def draw(rng):
    op = rng.choice(["norm", "route", "experts", "experts", "combine"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op == "norm":
        want = rng.choice(["y", "q8", "both"])
        K = _log(rng, 8, 16384)
        if want != "y":
            K = max(32, K // 32 * 32)
        T = _log(rng, 1, min(32768, (1 << 26) // K))
        return {"op": op, "T": T, "K": K, "dtype": dtype, "wtype": rng.choice(["f32", dtype]),
                "residual": rng.random() < 0.7, "want": want, "pad": rng.choice([0, 0, T // 16])}
    if op == "route":
        E = rng.choice([8, 16, 60, 64, 100, 128, 160, 256, 384, 512])
        groups = rng.choice([g for g in (1, 1, 2, 4, 8) if E % g == 0])
        keep = rng.randint(1, groups)
        T = _log(rng, 1, 32768)
        return {"op": op, "T": T, "E": E, "top_k": rng.choice([k for k in (1, 2, 4, 6, 8, 16) if k <= E * keep // groups]),
                "dtype": dtype, "scoring": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5,
                "groups": groups, "keep": keep, "group_top": rng.choice([1, 2]), "renormalise": rng.random() < 0.6,
                "scale": rng.choice([1.0, 2.5]), "masked": rng.choice([0.0, 0.0, 0.2]), "pad": rng.choice([0, 0, T // 16])}
    if op == "experts":
        E = rng.choice([1, 4, 8, 16, 60, 128, 256])
        K = rng.choice([256, 512, 768, 1024, 2048, 4096, 5120])
        activation = rng.choice(["none", "silu", "gelu"])
        M = rng.choice([m for m in (32, 96, 256, 768, 1440, 1536, 2048, 4096, 8192) if m * K * E <= 1 << 30])
        top_k = rng.choice([k for k in (1, 2, 4, 8) if k <= E])
        T = _log(rng, 1, min(16384, (1 << 39) // (M * K * top_k)))
        return {"op": op, "T": T, "E": E, "M": M, "K": K, "top_k": top_k, "activation": activation,
                "bias": rng.random() < 0.3, "each": rng.random() < 0.3, "pad": rng.choice([0, 0, T // 16])}
    top_k = rng.choice([1, 2, 3, 4, 6, 8])
    M = _log(rng, 16, 8192)
    T = _log(rng, 1, min(32768, (1 << 28) // (M * top_k)))
    return {"op": op, "T": T, "M": M, "top_k": top_k, "dtype": dtype, "otype": rng.choice(["f32", dtype]),
            "residual": rng.random() < 0.7, "pad": rng.choice([0, 0, T // 16])}


def _normal(shape, g, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    T, op = case["T"], case["op"]
    s = dict(case)
    if op == "norm":
        K, dtype = case["K"], DTYPES[case["dtype"]]
        # Channels differ in size, a few by much, as a residual stream's do; tokens too.
        wide = torch.exp(0.4 * _normal((1, K), g))
        wide[:, :: 97] *= 12.0
        size = torch.exp(0.5 * _normal((T, 1), g))
        x = _normal((T, K), g) * size
        x[T - case["pad"]:] = 0.0
        s["x"] = x.to(dtype)
        s["residual"] = None
        if case["residual"]:
            rest = _normal((T, K), g) * wide
            rest[T - case["pad"]:] = 0.0
            s["residual"] = rest.to(dtype)
            s["total"] = torch.empty((T, K), device="cuda", dtype=dtype)
        s["weight"] = (1.0 + 0.3 * _normal((K,), g)).to(DTYPES[case["wtype"]])
        s["y"] = torch.empty((T, K), device="cuda", dtype=dtype) if case["want"] != "q8" else None
        q8 = case["want"] != "y"
        s["q"] = torch.empty((T, K), device="cuda", dtype=torch.int8) if q8 else None
        s["d"] = torch.empty((T, K // 32), device="cuda") if q8 else None
        return s
    if op == "route":
        E = case["E"]
        x = 1.5 * _normal((T, E), g) + 0.7 * _normal((1, E), g)
        x[torch.rand((T, E), generator=g, device="cuda") < case["masked"]] = -math.inf
        x[T - case["pad"]:] = -math.inf
        s["logits"] = x.to(DTYPES[case["dtype"]])
        s["bias"] = 0.1 * _normal((E,), g) if case["bias"] else None
        s["ids"] = torch.empty((T, case["top_k"]), device="cuda", dtype=torch.int32)
        s["weights"] = torch.empty((T, case["top_k"]), device="cuda")
        return s
    top_k = case["top_k"]
    if op == "experts":
        E, M, K = case["E"], case["M"], case["K"]
        # Selectors are as good as random; scales span the size that weights of a K-wide row have.
        W = torch.randint(0, 256, (E, M, K // 32, 10), generator=g, device="cuda", dtype=torch.uint8)
        W[..., 8:] = W[..., 8:] % 16 + 8
        # Some experts are liked better than others; a token's experts are distinct.
        liked = _normal((T, E), g) + 0.7 * _normal((1, E), g)
        s["ids"] = torch.sort(liked, dim=1, descending=True).indices[:, :top_k].int().contiguous()
        s["ids"][T - case["pad"]:] = -1
        s["W"] = W
        s["X"] = _normal((T, top_k, K) if case["each"] else (T, K), g, torch.bfloat16)
        s["bias"] = 0.5 * _normal((E, M), g) if case["bias"] else None
        s["Y"] = torch.empty((T, top_k, M if case["activation"] == "none" else M // 2), device="cuda", dtype=torch.bfloat16)
        s["workspace"] = None
        return s
    M = case["M"]
    s["x"] = _normal((T, top_k, M), g, DTYPES[case["dtype"]])
    w = torch.exp(_normal((T, top_k), g))
    s["weights"] = w / w.sum(1, keepdim=True)
    s["ids"] = torch.randint(0, 64, (T, top_k), generator=g, device="cuda", dtype=torch.int32)
    lost = torch.randint(0, T * top_k, (case["pad"],), generator=g, device="cuda")
    s["ids"].view(-1)[lost] = -1
    otype = DTYPES[case["otype"]]
    s["residual"] = _normal((T, M), g, otype) if case["residual"] else None
    s["out"] = torch.empty((T, M), device="cuda", dtype=otype)
    return s


# -- the plain forms: elementary operations in 32 bits, rounded once at the end; in 64 where a choice is at stake ----


def _plain_norm(s):
    x = s["x"]
    if s["residual"] is not None:
        s["total"].copy_(x.float() + s["residual"].float())
        x = s["total"]
    found = {} if s["residual"] is None else {"total": x}
    if s["y"] is not None:
        v = x.float()
        r = 1.0 / torch.sqrt((v * v).sum(-1, keepdim=True) / s["K"] + 1e-6)
        found["y"] = s["y"].copy_(v * r * s["weight"].float())
    if s["q"] is not None:
        # Which code is nearest is decided in 64 bits: the factor of the row drops out.
        v = x.double()
        u = (v * s["weight"].double()).unflatten(-1, (-1, 32))
        top = u.abs().amax(-1, keepdim=True)
        t = 127.0 * u / torch.where(top == 0.0, 1.0, top)
        code = torch.sign(t) * torch.floor(t.abs() + 0.5)
        r = 1.0 / torch.sqrt((v * v).sum(-1) / s["K"] + 1e-6)
        d = (top[..., 0] * r[:, None] / 127.0).float()
        found["value"] = (code.float() * d[..., None]).flatten(-2)
    return found


def _plain_route(s):
    T, E, k, G = s["T"], s["E"], s["top_k"], s["groups"]
    x = s["logits"].double()
    open_ = x > -math.inf
    if s["scoring"] == "softmax":
        top = x.amax(-1, keepdim=True)
        e = torch.exp(x - torch.where(open_.any(-1, keepdim=True), top, 0.0))
        total = e.sum(-1, keepdim=True)
        score = e / torch.where(total == 0.0, 1.0, total)
    else:
        score = 1.0 / (1.0 + torch.exp(-x))
    # Without a bias the order of the scores is that of the logits.
    value = score if s["bias"] is None else score + s["bias"].double()
    order = x if s["bias"] is None else value
    order = torch.where(open_, order, -math.inf)
    if G > 1:
        if s["group_top"] == 1:
            held = order.view(T, G, -1).amax(-1)
        else:
            part = torch.where(open_, value, -math.inf).view(T, G, -1)
            best = torch.sort(part, dim=-1, descending=True).values[..., :2]
            held = torch.where(best > -math.inf, best, 0.0).sum(-1)
            held = torch.where(best[..., 0] > -math.inf, held, -math.inf)
        first = torch.sort(held, dim=-1, descending=True, stable=True).indices[:, : s["keep"]]
        kept = (first[:, :, None] == torch.arange(G, device=x.device)).any(1)
        order = torch.where(kept.repeat_interleave(E // G, 1), order, -math.inf)
    best = torch.sort(order, dim=-1, descending=True, stable=True)
    chosen, there = best.indices[:, :k], best.values[:, :k] > -math.inf
    w = torch.where(there, score.gather(1, chosen), 0.0)
    if s["renormalise"]:
        total = w.sum(-1, keepdim=True)
        w = w / torch.where(total == 0.0, 1.0, total)
    s["ids"].copy_(torch.where(there, chosen, -1))
    s["weights"].copy_(w * s["scale"])
    return {"ids": s["ids"], "weights": s["weights"]}


def _plain_weights(W):
    """ROCmFP2 blocks [..., K/32, 10] as fp32 [..., K]."""
    shift = torch.tensor([0, 2, 4, 6], dtype=torch.uint8, device=W.device)
    code = ((W[..., :8, None] >> shift) & 3).float() * 2.0 - 3.0          # -3 -1 1 3
    level = (code * (code * code + 23.0) / 24.0).flatten(-2)              # -4 -1 1 4
    scale = W[..., 8:].contiguous().view(torch.float8_e4m3fn).float() * 0.5
    return (level.unflatten(-1, (2, 16)) * scale[..., None]).flatten(-3)


def _plain_experts(s):
    E, top_k = s["E"], s["top_k"]
    w = _plain_weights(s["W"])
    ids = s["ids"].flatten().long()
    ids, pair = torch.sort(ids, stable=True)
    kept = ids >= 0
    ids, pair = ids[kept], pair[kept]
    # Each expert's tokens side by side, all experts as long as the longest.
    count = (ids[None, :] == torch.arange(E, device=ids.device)[:, None]).sum(1)
    place = torch.arange(ids.numel(), device=ids.device) - (torch.cumsum(count, 0) - count)[ids]
    rows = torch.zeros((E, int(count.max()), s["K"]), device=ids.device)
    rows[ids, place] = (s["X"].flatten(0, 1)[pair] if s["each"] else s["X"][pair // top_k]).float()
    y = torch.bmm(rows, w.transpose(1, 2))[ids, place]
    if s["bias"] is not None:
        y = y + s["bias"][ids]
    if s["activation"] != "none":
        gate, up = y.chunk(2, -1)
        if s["activation"] == "silu":
            gate = gate / (1.0 + torch.exp(-gate))
        else:
            gate = 0.5 * gate * (1.0 + torch.tanh(0.7978845608028654 * (gate + 0.044715 * gate * gate * gate)))
        y = gate * up
    s["Y"].zero_()
    s["Y"].flatten(0, 1)[pair] = y.to(s["Y"].dtype)
    return s["Y"]


def _plain_combine(s):
    there = s["ids"] >= 0
    w = torch.where(there, s["weights"], 0.0)
    y = (w[..., None] * s["x"].float()).sum(1)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return s["out"].copy_(y)


def run(s):
    if own:
        import gemm_rocmfp2_mul_gb300 as g
        if s["op"] == "norm":
            n = g.rfp2_rms_norm(s["x"], s["weight"], eps=1e-6, residual=s["residual"], want=s["want"], y=s["y"],
                                q=s["q"], d=s["d"], total=s.get("total"))
            found = {} if n.total is None else {"total": n.total}
            if n.y is not None:
                found["y"] = n.y
            if n.q is not None:
                found["value"] = (n.q.unflatten(-1, (-1, 32)) * n.d[..., None]).flatten(-2)
            return found
        if s["op"] == "route":
            ids, weights = g.rfp2_moe_route(s["logits"], s["top_k"], scoring=s["scoring"], bias=s["bias"],
                                            groups=s["groups"], keep=s["keep"], group_top=s["group_top"],
                                            renormalise=s["renormalise"], scale=s["scale"], ids=s["ids"],
                                            weights=s["weights"])
            return {"ids": ids, "weights": weights}
        if s["op"] == "experts":
            if s["workspace"] is None:
                s["workspace"] = g.rfp2_moe_gemm_workspace(s["ids"], s["E"])
            return g.rfp2_moe_gemm(s["W"], s["E"], s["M"], s["K"], s["ids"], s["X"], bias=s["bias"],
                                   activation=s["activation"], Y=s["Y"], workspace=s["workspace"])
        return g.rfp2_moe_combine(s["x"], s["weights"], ids=s["ids"], residual=s["residual"], out=s["out"])
    return {"norm": _plain_norm, "route": _plain_route, "experts": _plain_experts, "combine": _plain_combine}[s["op"]](s)


def work(case):
    T, op = case["T"], case["op"]
    if op == "norm":
        K, size = case["K"], SIZE[case["dtype"]]
        row = K * size * (1 + 2 * case["residual"] + (case["want"] != "q8"))
        if case["want"] != "y":
            row += K + K // 8
        return {"bytes": T * row + K * SIZE[case["wtype"]], "flops": 8 * T * K}
    if op == "route":
        return {"bytes": T * case["E"] * SIZE[case["dtype"]] + 8 * T * case["top_k"] + 4 * case["E"] * case["bias"],
                "flops": 8 * T * case["E"]}
    top_k, M = case["top_k"], case["M"]
    if op == "experts":
        E, K = case["E"], case["K"]
        tokens = T - case["pad"]
        touched = E * (1.0 - (1.0 - top_k / E) ** tokens)  # if all were liked alike
        out = M if case["activation"] == "none" else M // 2
        rows = tokens * (top_k if case["each"] else 1)
        return {"bytes": touched * M * (K // 32 * 10 + 4 * case["bias"]) + 2 * rows * K + 2 * T * top_k * out + 4 * T * top_k,
                "flops": 2 * tokens * top_k * M * K}
    return {"bytes": T * M * (top_k * SIZE[case["dtype"]] + (1 + case["residual"]) * SIZE[case["otype"]]) + 8 * T * top_k,
            "flops": 2 * T * top_k * M}


# -- the definitions in 64 bits -------------------------------------------------------------------------------------


def _exact_norm(case, s):
    x, found = s["x"].double(), {}
    if s["residual"] is not None:
        x = x + s["residual"].double()
        found["total"] = x
        x = x.to(s["x"].dtype).double()  # the norm is that of the sum as it is kept
    y = x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * s["weight"].double()
    if case["want"] != "q8":
        found["y"] = y
    if case["want"] != "y":
        b = (x * s["weight"].double()).view(case["T"], -1, 32)
        most = b.abs().max(-1, keepdim=True).values
        steps = (b.abs() * 254.0 / most.clamp(min=1e-300)).add(1.0).div(2.0).floor().copysign(b)
        one = y.view(case["T"], -1, 32).abs().max(-1, keepdim=True).values / 127.0
        found["value"] = (steps * one).view(case["T"], -1)
    return found


def _exact_route(case, s):
    x = s["logits"].double()
    if case["scoring"] == "softmax":
        score = torch.softmax(x, -1).nan_to_num(0.0)
    else:
        score = torch.sigmoid(x)
    value = score.clone() if s["bias"] is None else score + s["bias"].double()
    value[x == -math.inf] = -math.inf
    rank = value if s["bias"] is not None else x.clone()
    T, E, G = case["T"], case["E"], case["groups"]
    if G > 1:
        n = min(case["group_top"], E // G)
        if n == 1:
            of_group = rank.view(T, G, -1).max(-1).values
        else:
            two = value.view(T, G, -1).topk(n, -1).values
            of_group = two.clamp(min=-1e9).masked_fill(two == -math.inf, 0.0).sum(-1)
            of_group[two[..., 0] == -math.inf] = -math.inf
        # a group is kept where fewer than `keep` groups come before it
        a, b = of_group[:, :, None], of_group[:, None, :]
        i = torch.arange(G, device=x.device)
        before = ((b > a) | ((b == a) & (i[None, :] < i[:, None]))).sum(-1)
        rank = rank.masked_fill((before >= case["keep"]).repeat_interleave(E // G, 1), -math.inf)
    ids = torch.full((T, case["top_k"]), -1, dtype=torch.int64, device=x.device)
    rank = rank.clone()
    for j in range(case["top_k"]):
        most = rank.max(-1, keepdim=True).values
        i = torch.where(rank == most, torch.arange(E, device=x.device), E).min(-1, keepdim=True).values
        ids[:, j: j + 1] = torch.where(most > -math.inf, i, -1)
        rank.scatter_(1, i, -math.inf)
    w = torch.where(ids >= 0, score.gather(1, ids.clamp(min=0)), 0.0)
    if case["renormalise"]:
        w = w / w.sum(-1, keepdim=True).clamp(min=1e-300)
    return {"ids": ids.int(), "weights": w * case["scale"]}


def _exact_experts(case, s):
    K, M, top_k = case["K"], case["M"], case["top_k"]
    levels = torch.tensor([-4.0, -1.0, 1.0, 4.0], dtype=torch.float64, device="cuda")
    X = s["X"].flatten(0, -2).double()
    Y = torch.zeros(s["Y"].shape, dtype=torch.float64, device="cuda").flatten(0, 1)
    pairs = s["ids"].flatten()
    for e in range(case["E"]):
        at = (pairs == e).nonzero()[:, 0]
        if not at.numel():
            continue
        blocks = s["W"][e].view(M, K // 32, 10)
        byte = blocks[..., :8].int()
        w = torch.empty((M, K // 32, 8, 4), dtype=torch.float64, device="cuda")
        for i in range(4):
            w[..., i] = levels[(byte // 4 ** i % 4).long()]
        b = blocks[..., 8:].int()
        scale = torch.where(b < 8, torch.ldexp((b % 8).double(), torch.tensor(-10, device="cuda")),
                            torch.ldexp((b % 8 + 8).double(), b // 8 - 11))
        w = w.view(M, K // 32, 2, 16) * scale[..., None]
        y = X[at if case["each"] else at // top_k] @ w.view(M, K).T
        if s["bias"] is not None:
            y += s["bias"][e].double()
        if case["activation"] == "silu":
            y = y[:, : M // 2] * torch.sigmoid(y[:, : M // 2]) * y[:, M // 2:]
        elif case["activation"] == "gelu":
            a = y[:, : M // 2]
            y = a * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (a + 0.044715 * a ** 3)) * y[:, M // 2:]
        Y[at] = y
    return Y.view(s["Y"].shape)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(case, s)
    if case["op"] == "route":
        return _exact_route(case, s)
    if case["op"] == "experts":
        return _exact_experts(case, s)
    y = s["x"].double() * s["weights"].double()[..., None]
    y = y.masked_fill((s["ids"] < 0)[..., None], 0.0).sum(1)
    return y if s["residual"] is None else y + s["residual"].double()

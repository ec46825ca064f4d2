"""Plain float64 forms of the feed-forward operators, written from their formulas with numpy alone."""
import numpy as np

U = 2.0 ** -24                                                       # half a step of fp32
HALF = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}
TINY = {"float32": 2.0 ** -150, "bfloat16": 2.0 ** -134, "float16": 2.0 ** -25}   # half the smallest step


def norm(s, weight, eps):
    """float64 [T, K] of the sums s (as they are kept)."""
    s = np.asarray(s, np.float64)
    with np.errstate(all="ignore"):
        r = 1.0 / np.sqrt((s * s).mean(-1, keepdims=True) + eps)
        return s * r * np.asarray(weight, np.float64)


def codes(s, weight):
    """int8 codes [T, K] of the blocks of s * weight: the nearest of 127 steps of a block's largest value, halves
    away from zero.  Products of fp32 values have 48 bits and the factors 8: exact in extended precision."""
    u = (np.asarray(s, np.longdouble) * np.asarray(weight, np.longdouble)).reshape(len(s), -1, 32)
    top = np.abs(u).max(-1, keepdims=True)
    with np.errstate(all="ignore"):
        c = np.floor(np.abs(u) / np.where(top == 0, 1, top) * 127 + 0.5)
    for k in (c + 1, c, c - 1):   # the largest step that the value reaches: 254 |u| >= (2 k - 1) top
        c = np.where((254 * np.abs(u) >= (2 * k - 1) * top) & (k > c), k, c)
    c = np.where(254 * np.abs(u) < (2 * c - 1) * top, c - 1, c)
    return np.where(top == 0, 0, np.sign(u) * c).astype(np.int8).reshape(np.shape(s))


def route(x, top_k, scoring="softmax", bias=None, groups=1, keep=1, group_top=1, renormalise=True, scale=1.0):
    """(ids [T, top_k], weights float64 [T, top_k]) of logits x [T, E], row by row."""
    x = np.asarray(x, np.float64)
    T, E = x.shape
    ids, weights = np.full((T, top_k), -1, np.int32), np.zeros((T, top_k))
    for t in range(T):
        v = x[t]
        if np.isnan(v).any() or (bias is not None and np.isnan(bias).any()) or (scoring == "softmax" and (v == np.inf).any()):
            weights[t] = np.nan
            continue
        there = v > -np.inf
        if not there.any():
            continue
        with np.errstate(over="ignore"):
            if scoring == "softmax":
                e = np.where(there, np.exp(np.where(there, v - v[there].max(), 0.0)), 0.0)
                score = e / e.sum()
            else:
                score = 1.0 / (1.0 + np.exp(-v))
        value = score if bias is None else score + np.asarray(bias, np.float64)
        order = v if bias is None else value
        there &= order > -np.inf
        if groups > 1:
            size = E // groups
            count = []
            for g in range(groups):
                of = [e for e in range(g * size, (g + 1) * size) if there[e]]
                by = value if group_top > 1 else order
                count.append(sum(sorted((by[e] for e in of), reverse=True)[:group_top]) if of else -np.inf)
            for g in sorted(range(groups), key=lambda g: (-count[g], g))[keep:]:
                there[g * size: (g + 1) * size] = False
        chosen = sorted((e for e in range(E) if there[e]), key=lambda e: (-order[e], e))[:top_k]
        n = len(chosen)
        ids[t, :n] = chosen
        w = score[chosen]
        if renormalise and n:
            l = v[chosen]
            w = np.exp(l - l.max()) if scoring == "softmax" else \
                np.exp(np.minimum(l, 0) - min(l.max(), 0.0)) / (1.0 + np.exp(-np.abs(l)))
            w = w / w.sum()
        weights[t, :n] = w * scale
    return ids, weights


def combine(y, weights, ids=None, residual=None):
    """(float64 [T, M], the sum of what goes into each)."""
    y, w = np.asarray(y, np.float64), np.asarray(weights, np.float64)[..., None]
    if ids is not None:
        y = np.where((np.asarray(ids) < 0)[..., None], 0.0, y)
    out, size = (w * y).sum(1), np.abs(w * y).sum(1)
    if residual is not None:
        out, size = out + np.asarray(residual, np.float64), size + np.abs(np.asarray(residual, np.float64))
    return out, size


def weights_of(packed):
    """float64 [..., K] of ROCmFP2 blocks uint8 [..., K/32, 10]."""
    b = np.asarray(packed)
    code = (b[..., :8, None] >> np.array([0, 2, 4, 6], np.uint8)) & 3
    level = np.array([-4.0, -1.0, 1.0, 4.0])[code].reshape(*b.shape[:-1], 32)
    e, m = (b[..., 8:] >> 3).astype(int), (b[..., 8:] & 7).astype(int)
    scale = np.where(e == 0, m * 2.0 ** -10, (8 + m) * 2.0 ** (e - 11.0))
    return (level.reshape(*b.shape[:-1], 2, 16) * scale[..., None]).reshape(*b.shape[:-2], -1)


def activation(kind, a):
    if kind == "silu":
        return a / (1.0 + np.exp(-a))
    return 0.5 * a * (1.0 + np.tanh(np.sqrt(2.0 / np.pi) * (a + 0.044715 * a ** 3)))


def experts(packed, ids, X, bias=None, kind="none"):
    """(float64 y [T, top_k, M or M/2], how far sums of fp32 may put each off)."""
    w = weights_of(packed)
    E, M, K = w.shape
    T, k = ids.shape
    X = np.asarray(X, np.float64)
    # Products are exact; the tensor cores cut each partial sum of at least 8 of them off at 2^-23 of its
    # largest term at most, and add 16 at a time to a sum cut off the same way: K / 8 cuts of the sum of sizes.
    step = K / 8 * 2.0 ** -23 + 2.0 ** -22
    out = np.zeros((T, k, M if kind == "none" else M // 2))
    off = np.zeros_like(out)
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            if e < 0:
                continue
            x = X[t, j] if X.ndim == 3 else X[t]
            z, size = w[e] @ x, np.abs(w[e]) @ np.abs(x)
            if bias is not None:
                z, size = z + bias[e], size + np.abs(bias[e])
            if kind == "none":
                out[t, j], off[t, j] = z, size * step
            else:
                g, u = np.split(z, 2)
                dg, du = np.split(size * step, 2)
                a = activation(kind, g)
                out[t, j] = a * u
                # both activations change by at most 1.13 of their argument's change; expf and tanhf 2^-21
                off[t, j] = (1.13 * dg + 2.0 ** -21 * np.abs(g)) * (np.abs(u) + du) + np.abs(a) * du + 2.0 ** -20 * np.abs(a * u)
    return out, off

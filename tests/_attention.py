"""Plain float64 forms of the attention operators, written from their formulas with numpy alone: a
loop over tokens, heads and queries, no blocking, no running softmax."""
import math

import numpy as np


def rope(x, positions, inv_freq, interleaved=False, inverse=False, factor=1.0):
    """float64 [T, H, D]: pairs rotated by position * frequency."""
    y = np.array(x, np.float64)
    n = len(inv_freq)
    theta = np.outer(np.asarray(positions, np.float64), np.asarray(inv_freq, np.float64))[:, None, :]
    c, s = factor * np.cos(theta), factor * np.sin(theta) * (-1.0 if inverse else 1.0)
    i = np.arange(n)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    u, w = y[..., a].copy(), y[..., b].copy()
    y[..., a], y[..., b] = u * c - w * s, w * c + u * s
    return y


def quantise(x):
    """Codes and scales of float32 x [..., D] in blocks of 32: scale = max|a| / 127 and
    code = round-half-away(a / scale), both quotients rounded to float32; a block that is not finite
    has codes 0 and a scale that is not finite."""
    b = np.asarray(x, np.float32).reshape(*x.shape[:-1], -1, 32)
    with np.errstate(all="ignore"):
        d = np.abs(b).max(-1) / np.float32(127.0)
        t = (b / np.where(d == 0, np.float32(1.0), d)[..., None]).astype(np.float64)
        q = np.sign(t) * np.floor(np.abs(t) + 0.5)
        q = np.where(np.isfinite(d)[..., None], np.clip(q, -127, 127), 0)
    return q.astype(np.int8).reshape(x.shape), d.astype(np.float32)


def values(codes, scales):
    """float64 values of codes [..., D] and scales [..., D/32]."""
    with np.errstate(invalid="ignore"):
        return codes.astype(np.float64) * np.repeat(scales.astype(np.float64), 32, axis=-1)


def attention(q, k, v, lens, scale, window=0, softcap=0.0):
    """out [B, nq, Hq, D] and lse [B, nq, Hq] in float64, of q [B, nq, Hq, D] over lists of k, v
    [n, Hkv, D] (one pair a sequence)."""
    B, nq, Hq, D = q.shape
    out, lse = np.zeros(q.shape), np.full((B, nq, Hq), -np.inf)
    for b in range(B):
        for i in range(nq):
            end = int(lens[b]) - nq + 1 + i
            begin = max(0, end - window) if window else 0
            if end <= begin:
                continue
            for h in range(Hq):
                hk = h // (Hq // k[b].shape[1])
                with np.errstate(all="ignore"):
                    s = scale * (k[b][begin:end, hk] @ q[b, i, h])
                    if softcap:
                        s = softcap * np.tanh(s / softcap)
                    m = s.max()
                    p = np.exp(s - m)
                    out[b, i, h] = p @ v[b][begin:end, hk] / p.sum()
                    lse[b, i, h] = m + math.log(p.sum()) if np.isfinite(m) else np.nan
    return out, lse

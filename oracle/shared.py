"""Shared-latent attention in fp64: one latent c [T][r] and one rotary key kr [T][dr] per token;
KV head h's key is [c B_k,h | kr], its value c B_v,h.  Keys and values are rebuilt in full and
textbook softmax attention runs on them (no rank-space shortcut)."""
from __future__ import annotations

import numpy as np


def e4m3_values() -> np.ndarray:
    """The 127 non-negative finite e4m3 values in ascending order (index = code)."""
    v = [m / 8.0 * 2.0 ** -6 for m in range(8)]
    v += [(1.0 + m / 8.0) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
    return np.array(v[:127])


def quantize_e4m3(c: np.ndarray) -> np.ndarray:
    """What the 8-bit form of c [..., r] stands for: per 32 ranks the smallest 2^e (e >= -100) with
    max|c| <= 448 * 2^e, and the nearest e4m3 value of c / 2^e, ties to the even code.  A group
    with a NaN or an infinity is NaN throughout."""
    c = np.asarray(c, np.float64)
    vals = e4m3_values()
    out = np.empty_like(c)
    flat, res = c.reshape(-1, 32), out.reshape(-1, 32)
    for i, g in enumerate(flat):
        if not np.all(np.isfinite(g)):
            res[i] = np.nan
            continue
        top = np.abs(g).max()
        e = 0
        if top > 0:
            e = int(np.floor(np.log2(top))) - 9
            while top > 448.0 * 2.0 ** e:
                e += 1
            e = max(e, -100)
        y = np.abs(g) / 2.0 ** e
        d = np.abs(y[:, None] - vals[None, :])
        best = d.min(axis=1)
        code = np.array([min(np.flatnonzero(row == b), key=lambda k: k % 2) for row, b in zip(d, best)])
        res[i] = np.sign(g) * vals[code] * 2.0 ** e
    return out


def rotate(kr: np.ndarray, pos: np.ndarray, theta: float) -> np.ndarray:
    """Rotate-half RoPE of kr [n][dr] at positions pos [n]; theta = 0: unchanged."""
    kr = np.asarray(kr, np.float64)
    if not theta:
        return kr
    h = kr.shape[1] // 2
    ang = np.asarray(pos, np.float64)[:, None] * theta ** (-np.arange(h) / h)
    a, b = kr[:, :h], kr[:, h:]
    return np.concatenate([a * np.cos(ang) - b * np.sin(ang), a * np.sin(ang) + b * np.cos(ang)], axis=1)


def expand(c: np.ndarray, B: np.ndarray, heads: int) -> np.ndarray:
    """Per-head rows [T][heads][d] of latents c [T][r] through B [r][heads * d]."""
    return (np.asarray(c, np.float64) @ B).reshape(len(c), heads, B.shape[1] // heads)


def attend(q, key, val, scale, visible):
    """One query head: q [d], key [T][d], val [T][dv], visible [T] bool -> (out, lse, weights)."""
    if not np.any(visible):
        return np.zeros(val.shape[1]), -np.inf, np.zeros(len(key))
    s = np.where(visible, key @ q * scale, -np.inf)
    m = s.max()
    p = np.exp(s - m)
    return p @ val / p.sum(), m + np.log(p.sum()), p / p.sum()


def attention(q, k, kr, v, scale, causal=True):
    """One sequence: q [n][Hq][dn + dr], k [m][Hkv][dn], kr [m][dr], v [m][Hkv][dv]; causal: query i
    sees keys j <= i + m - n.  Returns out [n][Hq][dv], lse [n][Hq] and the mix of |v| that bounds
    roundings of the weights, sum_t p_t |v_t|."""
    n, hq, _ = q.shape
    m, hkv = k.shape[:2]
    out, lse, mix = np.zeros((n, hq, v.shape[2])), np.full((n, hq), -np.inf), np.zeros((n, hq, v.shape[2]))
    for j in range(hq):
        h = j // (hq // hkv)
        key = np.concatenate([k[:, h], kr], axis=1)
        for i in range(n):
            seen = np.arange(m) <= i + m - n if causal else np.ones(m, bool)
            out[i, j], lse[i, j], p = attend(q[i, j], key, v[:, h], scale, seen)
            mix[i, j] = p @ np.abs(v[:, h])
    return out, lse, mix

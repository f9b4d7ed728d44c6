"""CPU oracle of the 4-bit cache (rows quantised, read back, attended to) and of
the log probabilities of given tokens.

TEST INFRASTRUCTURE ONLY, under the rules of ``dustin_oracle``: plain, float64,
no code shared with the CUDA library.  Pinned by ``tests/test_kv4_oracle.py``.
"""
from __future__ import annotations

import numpy as np

STEPS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3(byte):
    """What a scale's byte stands for (writing gives bytes up to 0x7f; a cache may
    hold any, bit 7 is the sign)."""
    byte = np.asarray(byte, dtype=np.int64)
    e, m = byte // 8 % 16, byte % 8
    x = np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7.0))
    x = np.where(byte >= 0x80, -x, x)
    return np.where(byte % 128 == 0x7f, np.nan, x)


SCALES = e4m3(np.arange(127))


def record_size(d):
    return -(-(d + d // 8) // 16) * 16


def nearest(x, values):
    """Index of the nearest of ascending values; of two equally near, the even
    one; beyond the last, the last."""
    hi = np.clip(np.searchsorted(values, x), 1, len(values) - 1)
    lo = hi - 1
    down, up = x - values[lo], values[hi] - x        # exact: few bits of one size
    return np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)


def quantise_blocks(x, exp):
    """x [..][16] (bf16 values) -> codes [..][16] (0 .. 15), scale byte [..]."""
    x = np.asarray(x, dtype=np.float64)
    y = np.abs(x) * 2.0 ** -exp
    good = np.isfinite(y).all(-1)
    y = np.where(good[..., None], y, 0.0)
    scale = nearest(y.max(-1), 6 * SCALES)           # six times: nothing is divided
    s = SCALES[scale][..., None]
    # Borders of codes times the scale, all exact: at a border to the even code.
    code = np.zeros(y.shape, dtype=np.int64)
    for i, m in enumerate((STEPS[1:] + STEPS[:-1]) / 2):
        code += (y > m * s) if i % 2 == 0 else (y >= m * s)
    code = np.where(s > 0, code, 0) + 8 * np.signbit(x)
    return np.where(good[..., None], code, 0), np.where(good, scale, 0x7f)


def quantise(k, v, k_exp=0, v_exp=0):
    """Records [..][record_size] (uint8) of rows k, v [..][d]."""
    d = k.shape[-1]
    out = np.zeros((*k.shape[:-1], record_size(d)), dtype=np.uint8)
    for part, (x, exp) in enumerate(((k, k_exp), (v, v_exp))):
        codes, scale = quantise_blocks(x.reshape(*x.shape[:-1], d // 16, 16), exp)
        codes = codes.reshape(x.shape)
        out[..., part * d // 2:(part + 1) * d // 2] = codes[..., ::2] + 16 * codes[..., 1::2]
        at = d + part * (d // 16)
        out[..., at:at + d // 16] = scale
    return out


def dequantise(rec, d, k_exp=0, v_exp=0):
    """K and V (float64 [..][d]) that records stand for."""
    out = []
    for part, exp in enumerate((k_exp, v_exp)):
        codes = rec[..., part * d // 2:(part + 1) * d // 2].astype(np.int64)
        x = np.empty((*codes.shape[:-1], d))
        x[..., ::2], x[..., 1::2] = codes & 15, codes >> 4
        n = x.astype(np.int64)
        value = STEPS[n & 7] * np.where(n >= 8, -1.0, 1.0)
        at = d + part * (d // 16)
        scale = e4m3(rec[..., at:at + d // 16])
        out.append(value * np.repeat(scale, 16, -1) * 2.0 ** exp)
    return out


def attention(q, k, v, scale, seen, kw=None, vw=None):
    """q [b][h_q][w][d]; k, v [b][h_kv][n][d]; seen: per sequence the positions
    that count, in order; the window kw, vw [b][h_kv][w][d], causal.  Returns o,
    lse and sum_j p_j |v_j|."""
    b, hq, w, d = q.shape
    group = hq // k.shape[1]
    o, spread = np.zeros(q.shape), np.zeros(q.shape)
    lse = np.full((b, hq, w), -np.inf)
    with np.errstate(invalid="ignore", over="ignore"):
        for i in range(b):
            for h in range(hq):
                for t in range(w):
                    keys, values = k[i, h // group, seen[i]], v[i, h // group, seen[i]]
                    if kw is not None:
                        keys = np.concatenate([keys, kw[i, h // group, :t + 1]])
                        values = np.concatenate([values, vw[i, h // group, :t + 1]])
                    s = keys @ q[i, h, t] * scale
                    if np.isnan(s).any() or np.isposinf(s).any():
                        o[i, h, t] = spread[i, h, t] = lse[i, h, t] = np.nan
                        continue
                    if not np.isfinite(s).any():
                        continue
                    top = s.max()
                    p = np.exp(s - top)
                    lse[i, h, t] = top + np.log(p.sum())
                    p /= p.sum()
                    o[i, h, t] = p @ values
                    spread[i, h, t] = p @ np.abs(values)
    return o, lse, spread


def logprobs(x, scale, tokens, top):
    """One row of logits [vocab] (float64): log probabilities of tokens, entropy,
    lse, ids and log probabilities of the `top` largest."""
    order = np.lexsort((np.arange(len(x)), -x))
    order = order[~np.isnan(x[order])][:top]
    ids = np.full(top, -1)
    ids[:len(order)] = order
    if np.isnan(x).any() or np.isposinf(x).any():
        nan = np.nan
        return np.full(len(tokens), nan), nan, nan, ids, np.full(top, nan)
    z = x * scale
    m = z.max()
    if np.isneginf(m):
        return (np.full(len(tokens), -np.inf), 0.0, -np.inf, ids,
                np.where(ids < 0, np.nan, -np.inf))
    lse = m + np.log(np.exp(z - m).sum())
    lp = z - lse
    p = np.exp(lp)
    entropy = -np.sum(p[p > 0] * lp[p > 0])
    inside = [lp[t] if 0 <= t < len(x) else -np.inf for t in tokens]
    return np.array(inside), entropy, lse, ids, np.where(ids < 0, np.nan, lp[ids])

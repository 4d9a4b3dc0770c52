"""The attention side of a layer in float64: the paged cache, attention over it, the gated
residual with its norms.  Written as the definitions, request by request and row by row;
shares nothing with the CUDA library."""
from __future__ import annotations

import numpy as np


def e4m3_values() -> np.ndarray:
    """The value of each E4M3 code: sign, 4 exponent bits (bias 7), 3 mantissa bits; code 127 is NaN."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = np.nan if (e, m) == (15, 7) else (m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        out[c] = -v if c & 128 else v
    return out


def kv_exponent(x: np.ndarray) -> int:
    """The smallest e in [-100, 119] with max|x| <= 448 * 2^e (NaN aside; -100 for zeros)."""
    x = np.abs(np.asarray(x, np.float64))
    most = np.max(np.where(np.isnan(x), 0.0, x))
    for e in range(-100, 119):
        if most <= 448.0 * 2.0 ** e:
            return e
    return 119


def quantise(x: np.ndarray):
    """(E4M3 values, exponent) of one vector: to the nearest value, ties to the even code, saturating."""
    x = np.asarray(x, np.float64)
    e = kv_exponent(x)
    vals = e4m3_values()[:127]                           # 0 .. 448, ascending with the code
    a = np.minimum(np.abs(x) * 2.0 ** -e, 448.0)
    a = np.where(np.isnan(a), 0.0, a)
    hi = np.searchsorted(vals, a)
    lo = np.maximum(hi - 1, 0)
    up = vals[hi] - a
    down = a - vals[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    q = np.copysign(vals[code], x)
    return np.where(np.isnan(x), np.nan, q), e


def block_attention(q, k, v, lengths, n_q: int, scale: float, causal: bool, window: int):
    """q [R*n_q][Hq][D]; k, v: one [L_r][Hkv][D] array a request.  Returns out, lse, and
    wabs [..][D] = sum_j p_j |v_j| and dots [..] = max_j scale * sum_d |q_d k_jd| over the keys
    seen, from which error bounds are derived."""
    q = np.asarray(q, np.float64)
    T, Hq, D = q.shape
    out = np.zeros((T, Hq, D))
    wabs = np.zeros((T, Hq, D))
    lse = np.full((T, Hq), -np.inf)
    dots = np.zeros((T, Hq))
    for r, L in enumerate(lengths):
        Hkv = k[r].shape[1]
        for i in range(n_q):
            p = L - n_q + i
            hi = min(L, p + 1) if causal else L
            lo = max(0, p - window + 1) if window else 0
            if hi <= lo:
                continue
            for h in range(Hq):
                kk = np.asarray(k[r][lo:hi, h * Hkv // Hq], np.float64)
                vv = np.asarray(v[r][lo:hi, h * Hkv // Hq], np.float64)
                t = r * n_q + i
                s = scale * (kk @ q[t, h])
                m = s.max()
                w = np.exp(s - m)
                out[t, h] = w @ vv / w.sum()
                wabs[t, h] = w @ np.abs(vv) / w.sum()
                lse[t, h] = m + np.log(w.sum())
                dots[t, h] = scale * (np.abs(kk) @ np.abs(q[t, h])).max()
    return out, lse, wabs, dots


def block_residual_norm(y, h, w_post=None, gate=None, w_pre=None, res_scale=1.0, eps=1e-6, P=1):
    """(h', x) of [T][H] inputs; gate [H] or one row for each P tokens."""
    y, h = np.asarray(y, np.float64), np.asarray(h, np.float64)
    if w_post is not None:
        y = np.asarray(w_post, np.float64) * y / np.sqrt((y * y).mean(1, keepdims=True) + eps)
    if gate is not None:
        g = np.asarray(gate, np.float64)
        y = y * (g if g.ndim == 1 else g[np.arange(len(y)) // P])
    h = h + res_scale * y
    x = h / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    return h, x if w_pre is None else x * np.asarray(w_pre, np.float64)

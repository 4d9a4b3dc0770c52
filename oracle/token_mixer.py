"""Pages and positions of a batch's next tokens, rotary positions, and the gated delta rule, in plain
Python and float64.  Written as the definitions, request by request and token by token; shares nothing
with the CUDA library."""
from __future__ import annotations

import math

import numpy as np


def kv_cache_plan(kv_len, n_new, n: int, ring, head, table, page: int):
    """(ring, head, table, new_len, pos, slots) after the requests have been served in their order.  Every page
    number is taken as valid; a length or count out of range refuses the request."""
    ring, table = np.array(ring), np.array(table)
    n_pages, (R, max_pages) = len(ring), table.shape
    first, count = (int(x) for x in head)
    cap = max_pages * page
    pos, slots, new_len = np.full((R, n), -1), np.full((R, n), -1), np.array(kv_len)
    asked = taken = 0
    given = []
    for r in range(R):
        L, m = int(kv_len[r]), int(n_new[r])
        if not (0 <= L <= cap and -L <= m <= n) or L + m > cap:
            continue
        held, need = -(-L // page), -(-(L + m) // page)
        if need > held:
            asked += need - held
            if asked > count:
                continue
            for i in range(held, need):
                table[r, i] = ring[(first + taken) % n_pages]
                taken += 1
        given += [int(x) for x in table[r, need:held]]
        new_len[r] = L + m
        for i in range(m):
            p = L + i
            pos[r, i], slots[r, i] = p, table[r, p // page] * page + p % page
    for i, x in enumerate(given):
        ring[(first + count + i) % n_pages] = x
    return ring, np.array([(first + taken) % n_pages, count - taken + len(given)]), table, new_len, pos, slots


def rotary_frequencies(rot: int, base: float, scaling: str = "plain", factor=1.0, original=1.0, low=1.0, high=2.0):
    """Radians a position of each pair."""
    out = []
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        if scaling == "linear":
            f = f / factor
        elif scaling == "rotations":
            s = min(1.0, max(0.0, (original * f / (2 * math.pi) - low) / (high - low)))
            f = s * f + (1 - s) * f / factor
        elif scaling == "dimensions":
            index = lambda turns: rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
            a, b = max(math.floor(index(high)), 0), min(math.ceil(index(low)), rot - 1)
            s = 1 - min(1.0, max(0.0, (i - a) / max(b - a, 0.001)))
            f = s * f + (1 - s) * f / factor
        out.append(f)
    return np.array(out)


def block_rotary(x, pos, freq, pairs: bool, mscale: float):
    """x [T][heads][D] at positions pos [T]: (turned, bound): bound [T][heads][D] is (|x0| + |x1|) * |mscale| of
    each turned element's pair, 0 of the others.  Rows of negative positions: NaN."""
    x = np.asarray(x, np.float64)
    y, bound = x.copy(), np.zeros_like(x)
    half = len(freq)
    for t, p in enumerate(pos):
        if p < 0:
            y[t] = np.nan
            continue
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if pairs else (i, i + half)
            turn = np.longdouble(p) * np.longdouble(freq[i])
            c, s = float(np.cos(turn)), float(np.sin(turn))
            y[t, :, a] = mscale * (x[t, :, a] * c - x[t, :, b] * s)
            y[t, :, b] = mscale * (x[t, :, b] * c + x[t, :, a] * s)
            bound[t, :, a] = bound[t, :, b] = abs(mscale) * (np.abs(x[t, :, a]) + np.abs(x[t, :, b]))
    return y, bound


def delta_rule(q, k, v, g, beta, S, scale: float, eps: float):
    """One request: q, k [n][Hk][Dk], v [n][Hv][Dv], g, beta [n][Hv], S [Hv][Dv][Dk] (transposed).  Returns
    (out [n][Hv][Dv], S, most [Hv][Dv]): most is the largest norm that a row of the state had plus the largest
    |v| of its row, from which error bounds are derived."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    n, Hv = g.shape
    if eps > 0:
        q = q / np.sqrt((q * q).sum(-1, keepdims=True) + eps)
        k = k / np.sqrt((k * k).sum(-1, keepdims=True) + eps)
    group = Hv // q.shape[1]
    S = np.array(S, np.float64)
    out = np.zeros(v.shape)
    most = np.sqrt((S * S).sum(-1))
    for t in range(n):
        for h in range(Hv):
            kk, qq = k[t, h // group], q[t, h // group]
            S[h] *= math.exp(g[t, h])
            S[h] += np.outer(beta[t, h] * (v[t, h] - S[h] @ kk), kk)
            out[t, h] = scale * (S[h] @ qq)
        most = np.maximum(most, np.sqrt((S * S).sum(-1)))
    return out, S, most + (np.abs(v).max(0) if n else 0.0)

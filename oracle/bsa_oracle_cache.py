"""Plain fp64 CPU oracle of the paged 8-bit key/value cache.

TEST INFRASTRUCTURE ONLY (same rule as ``bsa_oracle``): nothing on the product path
imports it; it shares no code with the CUDA path and depends on numpy only.

``resize`` (block tables and slots from request lengths), ``append`` (new keys or values
rounded to 8 bits with one power-of-two scale for each page and head) and ``forward``
(attention of each request's newest tokens over its pages) follow the definitions of
include/bsa.h one request, run and query at a time.  Stored numbers are held as the values
they stand for.  Pinned by ``tests/test_oracle_cache.py``.
"""

from __future__ import annotations

import math

import numpy as np

LARGEST = {"e4m3": 448.0, "int8": 127.0}
INT32_MIN = -2 ** 31


# ------------------------------------------------------------------------------ resize

def resize(table, kv_len, new_len, free, count: int, page: int, tokens: int):
    """(table, kv_len, free, count, cu_new, slots, status) after bsa_cache_resize."""
    table, free = np.array(table), np.array(free)
    old, new = [int(x) for x in kv_len], [int(x) for x in new_len]
    B, width = table.shape
    cu, slots = [0] * (B + 1), [-1] * tokens

    def result(status, lens, n):
        return table, np.array(lens), free, n, np.array(cu), np.array(slots, dtype=np.int64), status

    for b in range(B):
        if not (0 <= old[b] <= width * page and 0 <= new[b] <= width * page):
            return result(-1 - b, old, count)
    fresh = [max(0, n - o) for o, n in zip(old, new)]
    had, has = [-(-o // page) for o in old], [-(-n // page) for n in new]
    if sum(fresh) > tokens:
        return result(INT32_MIN, old, count)
    freed = sum(max(0, a - b) for a, b in zip(had, has))
    if count < 0 or count + freed > len(free):
        return result(INT32_MIN + 1, old, count)
    missing = sum(max(0, b - a) for a, b in zip(had, has)) - count - freed
    if missing > 0:
        return result(missing, old, count)
    for b in range(B):
        for j in range(has[b], had[b]):
            free[count] = table[b, j]
            count += 1
    for b in range(B):
        for j in range(had[b], has[b]):
            count -= 1
            table[b, j] = free[count]
    t = 0
    for b in range(B):
        cu[b] = t
        for pos in range(old[b], new[b]):
            slots[t] = int(table[b, pos // page]) * page + pos % page
            t += 1
    cu[B] = t
    return result(0, new, count)


# ------------------------------------------------------------------------------ append

def round_stored(x: float, kind: str) -> float:
    """The stored number next to x (ties to even, saturating; NaN: NaN, or 0 in int8)."""
    top = LARGEST[kind]
    if math.isnan(x):
        return 0.0 if kind == "int8" else x
    x = max(-top, min(top, x))
    if kind == "int8":
        return float(round(x))
    if x == 0.0:
        return x
    e = max(math.frexp(x)[1] - 1, -6)  # 2^e <= |x| < 2^(e+1), subnormals below 2^-6
    step = 2.0 ** (e - 3)
    return max(-top, min(top, round(x / step) * step))


def scale_for(amax: float, kind: str) -> float:
    """The smallest power of two in [2^-60, 2^60] with amax <= largest * scale."""
    s = 2.0 ** -60
    while s < 2.0 ** 60 and amax > LARGEST[kind] * s:
        s *= 2.0
    return s


def append(x, slots, cache, scale, kind: str):
    """(cache, scale) after new rows x [T, H, d]; cache [P, H, page, d] of stored values,
    scale [P, H]."""
    x, cache, scale = np.asarray(x, np.float64), np.array(cache, np.float64), np.array(scale, np.float64)
    P, H, page, d = cache.shape
    runs = []  # (page id, tokens)
    for t, slot in enumerate(int(s) for s in slots):
        if not 0 <= slot < P * page:
            continue
        if runs and runs[-1][0] == slot // page and runs[-1][1][-1] == t - 1:
            runs[-1][1].append(t)
        else:
            runs.append((slot // page, [t]))
    rnd = np.vectorize(lambda v: round_stored(v, kind), otypes=[np.float64])
    for pid, ts in runs:
        start = int(slots[ts[0]]) % page
        for h in range(H):
            rows = x[ts, h]
            fin = np.abs(rows[np.isfinite(rows)])
            s = scale_for(fin.max() if fin.size else 0.0, kind)
            if start:
                s = max(s, scale[pid, h])
                if s != scale[pid, h]:
                    cache[pid, h, :start] = rnd(cache[pid, h, :start] * (scale[pid, h] / s))
            scale[pid, h] = s
            for t in ts:
                cache[pid, h, int(slots[t]) % page] = rnd(x[t, h] / s)
    return cache, scale


# ----------------------------------------------------------------------------- forward

def forward(q, k, v, k_scale, v_scale, table, kv_len, cu_q, scale: float, window: int = -1,
            softcap: float = 0.0, sinks=None, layout=None, block: int = 0):
    """q [T, Hq, d]; k, v [P, H, page, d] of stored values, scales [P, H].  Returns (out,
    lse, weight, size): weight[t, h] = sum of |weight * value| over the keys, per element
    (what the rounding of the weights acts on), and size[t, h] = the largest
    scale * k_scale * sum |q k| over the keys (what the rounding of the scores acts on)."""
    q = np.asarray(q, np.float64)
    T, Hq, d = q.shape
    P, H, page, _ = k.shape
    G = Hq // H
    out, weight = np.zeros((T, Hq, d)), np.zeros((T, Hq, d))
    lse, size = np.full((T, Hq), -np.inf), np.zeros((T, Hq))
    for b in range(len(kv_len)):
        n = int(cu_q[b + 1]) - int(cu_q[b])
        length = min(int(kv_len[b]), table.shape[1] * page)
        for i in range(n):
            t, pos = int(cu_q[b]) + i, length - n + i
            c = np.arange(pos + 1) if pos >= 0 else np.arange(0)
            if window >= 0:
                c = c[c >= pos - window]
            ids = table[b, c // page]
            c, ids = c[(ids >= 0) & (ids < P)], ids[(ids >= 0) & (ids < P)]
            for g in range(H):
                on = np.ones(len(c), bool) if layout is None else layout[g, pos // block][c // block] == 1
                cc, pp = c[on], ids[on]
                kk = k[pp, g, cc % page] * k_scale[pp, g][:, None]
                vv = v[pp, g, cc % page] * v_scale[pp, g][:, None]
                for h in range(g * G, (g + 1) * G):
                    s = scale * (kk @ q[t, h])
                    if softcap > 0:
                        s = softcap * np.tanh(s / softcap)
                    sink = -np.inf if sinks is None else float(sinks[h])
                    top = max(s.max() if len(s) else -np.inf, sink)
                    if top == -np.inf:
                        continue
                    e = np.exp(s - top)
                    z = e.sum() + np.exp(sink - top)
                    lse[t, h] = top + np.log(z)
                    out[t, h] = (e / z) @ vv
                    weight[t, h] = (e / z) @ np.abs(vv)
                    if len(s):
                        size[t, h] = abs(scale) * (np.abs(kk) @ np.abs(q[t, h])).max()
    return out, lse, weight, size

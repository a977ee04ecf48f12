"""Plain fp64 CPU oracle of block-sparse differential attention, forward and backward.

TEST INFRASTRUCTURE ONLY (same rule as ``bsa_oracle``).  For batch b, output head h (kv head
g = h // (H / kv_heads)), query row r and map m in {0, 1}, with A(r) the active keys of the
layout of kv head g (any length L; the last block is clipped):

  s_m[c] = scale * <q[b, 2h+m, r, :], key m of c>;  key m is k[b, g, c, :] when the queries have
           d numbers, k[b, g, c, m d/2 : (m+1) d/2] when they have d / 2
  P_m    = softmax of s_m over A(r)  (0 when A(r) is empty),  O_m = P_m V
  out    = O_0 - lam O_1,  lse_m = ln sum exp s_m
and for an upstream gradient dO, by the chain rule through each softmax apart:
  dP_0 = dO V^T, dP_1 = -lam dO V^T,  dS_m = P_m * (dP_m - rowsum(P_m * dP_m)),
  dQ_m = scale dS_m K_m,  dK_m = scale dS_m^T Q_m,  dV = P_0^T dO - P_1^T (lam dO),
  dlam = -<dO, O_1>
with dK and dV summed over the heads of a kv head.  Pinned by ``tests/test_oracle_diff.py``.

``bounds`` gives elementwise error bounds of an implementation that rounds P, P_0 - lam P_1 and
dS to bf16 before their second products and results to bf16, everything else in fp32.
"""

from __future__ import annotations

import numpy as np

BF16 = 2.0 ** -8  # half a step, relative


def mask(layout_g, block, L, causal_diag):
    """Active (row, key) pairs [L, L] of one layout head [nb, nb]."""
    at = np.arange(L) // block
    on = np.asarray(layout_g)[at][:, at] == 1
    if causal_diag:
        r = np.arange(L)
        on &= ~((at[:, None] == at[None]) & (r[None] > r[:, None]))
    return on


def _parts(q, k, layout, scale, block, causal_diag, b, h, H):
    """P_m, lse_m, Q_m, K_m of both maps of output head h."""
    g = h // (H // k.shape[1])
    L, dq, d = q.shape[2], q.shape[3], k.shape[3]
    on = mask(layout[g], block, L, causal_diag)
    for m in range(2):
        cols = slice(0, d) if dq == d else slice(m * dq, (m + 1) * dq)
        qm, km = q[b, 2 * h + m], k[b, g][:, cols]
        s = np.where(on, scale * (qm @ km.T), -np.inf)
        top = s.max(1)
        e = np.exp(s - np.where(np.isfinite(top), top, 0.0)[:, None])
        z = e.sum(1)
        with np.errstate(divide="ignore"):
            lse = np.log(z) + top
        yield e / np.where(z > 0, z, 1.0)[:, None], lse, qm, km, cols


def _lam(lam, b, h):
    return lam[h] if lam.ndim == 1 else lam[b, h][:, None]


def forward(q, k, v, lam, layout, scale, block, causal_diag):
    """(out [B, H, L, d], lse [B, 2H, L], out2 = O_1)."""
    q, k, v, lam = (np.asarray(x, dtype=np.float64) for x in (q, k, v, lam))
    B, H2, L, _ = q.shape
    H, d = H2 // 2, k.shape[3]
    out, out2, lse = np.zeros((B, H, L, d)), np.zeros((B, H, L, d)), np.zeros((B, H2, L))
    for b in range(B):
        for h in range(H):
            vg = v[b, h // (H // k.shape[1])]
            for m, (p, y, _, _, _) in enumerate(_parts(q, k, layout, scale, block, causal_diag, b, h, H)):
                lse[b, 2 * h + m] = y
                o = p @ vg
                if m == 0:
                    out[b, h] = o
                else:
                    out[b, h] -= _lam(lam, b, h) * o
                    out2[b, h] = o
    return out, lse, out2


def backward(q, k, v, lam, do, layout, scale, block, causal_diag):
    """(dq, dk, dv, dlam); dlam in lam's shape."""
    q, k, v, lam, do = (np.asarray(x, dtype=np.float64) for x in (q, k, v, lam, do))
    B, H2, L, _ = q.shape
    H = H2 // 2
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    dlam = np.zeros((B, H, L))
    for b in range(B):
        for h in range(H):
            g = h // (H // k.shape[1])
            for m, (p, _, qm, km, cols) in enumerate(_parts(q, k, layout, scale, block, causal_diag, b, h, H)):
                w = do[b, h] * (1.0 if m == 0 else -_lam(lam, b, h))  # dL/dO_m
                dp = w @ v[b, g].T
                ds = p * (dp - (p * dp).sum(1, keepdims=True))
                dq[b, 2 * h + m] = scale * ds @ km
                dk[b, g][:, cols] += scale * ds.T @ qm
                dv[b, g] += p.T @ w
                if m == 1:
                    dlam[b, h] = -(do[b, h] * (p @ v[b, g])).sum(1)
    return dq, dk, dv, dlam.sum((0, 2)) if lam.ndim == 1 else dlam


def bounds(q, k, v, lam, do, layout, scale, block, causal_diag):
    """Elementwise error bounds {name: array} of the results of both functions.

    P is off by e_p relative: its exponent is a product of d numbers summed in fp32, at most
    2^-24 d sum |q k| scale off, minus a number below 16, and the exponential by 2^-22.  Then,
    with A_m = P_m |V|:
      out    2^-8 (A_0 + lam A_1) (P in bf16) + e_p of the same + 2^-8 |out|
      out2   likewise, map 1 alone
      D_1    sum |dO| (bound of out2),  D_0  sum |dO| (bound of out) + lam of D_1's
      dS     |w| P (bound of D + e_p |dP - D|) + 2^-8 |dS|
      dQ     scale (bound of dS) |K| + 2^-8 |dQ|;  dK likewise
      dV     (2^-8 |P_0 - lam P_1| + e_p (P_0 + lam P_1))^T |dO| + 2^-8 |dV|
      dlam   e_p sum P_1 |dP| (a row), summed where lam is one number a head
    and 2^-20 of each sum of magnitudes for its fp32 accumulation."""
    q, k, v, lam, do = (np.asarray(x, dtype=np.float64) for x in (q, k, v, lam, do))
    B, H2, L, _ = q.shape
    H = H2 // 2
    out, _, out2 = forward(q, k, v, lam, layout, scale, block, causal_diag)
    gq, gk, gv, _ = backward(q, k, v, lam, do, layout, scale, block, causal_diag)
    bnd = {"out": np.zeros_like(out), "out2": np.zeros_like(out), "dq": np.zeros_like(q),
           "dk": np.zeros_like(k), "dv": np.zeros_like(v), "dlam": np.zeros((B, H, L))}
    for b in range(B):
        for h in range(H):
            g = h // (H // k.shape[1])
            av, ado = np.abs(v[b, g]), np.abs(do[b, h])
            l = np.broadcast_to(_lam(lam, b, h), (L, 1))
            al = np.abs(l)
            maps = list(_parts(q, k, layout, scale, block, causal_diag, b, h, H))
            sums = [np.abs(qm) @ np.abs(km).T for _, _, qm, km, _ in maps]
            e_p = [2.0 ** -21 + 2.0 ** -24 * (q.shape[3] * abs(scale) * np.where(p > 0, s, 0).max(1, keepdims=True)
                                              + 64) for (p, *_), s in zip(maps, sums)]
            a = [p @ av for p, *_ in maps]
            bnd["out2"][b, h] = (BF16 + e_p[1] + 2.0 ** -20) * a[1] + BF16 * np.abs(out2[b, h])
            bnd["out"][b, h] = (BF16 + e_p[0] + 2.0 ** -20) * a[0] + al * (BF16 + e_p[1] + 2.0 ** -20) * a[1] \
                + BF16 * np.abs(out[b, h])
            d1 = (ado * bnd["out2"][b, h]).sum(1, keepdims=True)
            d0 = (ado * bnd["out"][b, h]).sum(1, keepdims=True) + al * d1
            dp = do[b, h] @ v[b, g].T
            adp = ado @ av.T
            w = maps[0][0] - l * maps[1][0]
            bnd["dv"][b, g] += (BF16 * np.abs(w) + (e_p[0] + 2.0 ** -20) * maps[0][0]
                                + al * (e_p[1] + 2.0 ** -20) * maps[1][0]).T @ ado
            for m, (p, _, qm, km, cols) in enumerate(maps):
                wm = np.ones_like(al) if m == 0 else al
                centre = dp - (p * dp).sum(1, keepdims=True)
                ds = wm * p * np.abs(centre)
                e = wm * p * ((d1 if m else d0) + 2.0 ** -20 * adp) + (BF16 + e_p[m] + 2.0 ** -20) * ds
                bnd["dq"][b, 2 * h + m] = abs(scale) * e @ np.abs(km)
                bnd["dk"][b, g][:, cols] += abs(scale) * e.T @ np.abs(qm)
            bnd["dlam"][b, h] = ((e_p[1] + 2.0 ** -20) * (maps[1][0] * np.maximum(np.abs(dp), 2.0 ** -4 * adp))
                                 .sum(1, keepdims=True))[:, 0]
    bnd["dq"] += BF16 * np.abs(gq)
    bnd["dk"] += BF16 * np.abs(gk)
    bnd["dv"] += BF16 * np.abs(gv)
    if lam.ndim == 1:
        bnd["dlam"] = bnd["dlam"].sum((0, 2))
    for name in ("out", "out2", "dq", "dk", "dv", "dlam"):
        bnd[name] += 2.0 ** -40
    return bnd

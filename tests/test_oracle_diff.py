"""Pins of the differential-attention oracle against things other than itself (CPU only):
the plain forward oracle, a closed form, central differences, and zero-padded queries."""

import numpy as np
import pytest

import oracle
from oracle import diff as od


def _case(B, H, kv, L, d, dq, block, rows, seed, hole=True):
    r = np.random.default_rng(seed)
    nb = -(-L // block)
    lay = (r.random((kv, nb, nb)) < 0.5).astype(np.int32)
    lay[:, np.arange(nb), np.arange(nb)] = 1
    if hole and nb > 1:
        lay[0, 1] = 0
    q, k, v = (r.standard_normal(s) for s in ((B, 2 * H, L, dq), (B, kv, L, d), (B, kv, L, d)))
    lam = r.random((B, H, L)) if rows else r.random(H)
    return q, k, v, lam, r.standard_normal((B, H, L, d)), lay


def test_is_the_difference_of_two_plain_forwards():
    B, H, L, d, block = 2, 3, 64, 8, 16
    q, k, v, lam, _, lay = _case(B, H, H, L, d, d, block, True, 1)
    out, lse, out2 = od.forward(q, k, v, lam, lay, 0.3, block, True)
    o = [oracle.forward(q[:, m::2], k, v, lay, 0.3, block, True) for m in range(2)]
    assert np.allclose(out, o[0][0] - lam[..., None] * o[1][0], atol=1e-12)
    assert np.allclose(out2, o[1][0], atol=1e-12)
    for m in range(2):
        np.testing.assert_allclose(lse[:, m::2], o[m][1], atol=1e-12)


def test_equal_maps_and_weight_one_cancel():
    q, k, v, lam, _, lay = _case(1, 2, 1, 21, 8, 8, 8, False, 2)
    q[:, 1::2] = q[:, 0::2]
    out, _, _ = od.forward(q, k, v, np.ones(2), lay, 0.5, 8, True)
    assert np.abs(out).max() < 1e-13


def test_key_halves_are_zero_padded_queries():
    q, k, v, lam, do, lay = _case(1, 2, 1, 20, 8, 4, 8, True, 3)
    wide = np.zeros((1, 4, 20, 8))
    wide[:, 0::2, :, :4], wide[:, 1::2, :, 4:] = q[:, 0::2], q[:, 1::2]
    for a, b in zip(od.forward(q, k, v, lam, lay, 0.4, 8, True), od.forward(wide, k, v, lam, lay, 0.4, 8, True)):
        np.testing.assert_allclose(a, b, atol=1e-13)
    a, b = (od.backward(x, k, v, lam, do, lay, 0.4, 8, True) for x in (q, wide))
    np.testing.assert_allclose(a[0][:, 1::2], b[0][:, 1::2, :, 4:], atol=1e-13)
    for i in (1, 2, 3):
        np.testing.assert_allclose(a[i], b[i], atol=1e-13) if i != 1 else None
    # dk of the wide queries adds their own zero half: the same numbers
    np.testing.assert_allclose(a[1], b[1], atol=1e-13)


@pytest.mark.parametrize("dq,rows,causal", [(6, False, True), (3, True, True), (6, True, False)])
def test_gradients_are_central_differences(dq, rows, causal):
    B, H, kv, L, d, block = 1, 2, 1, 11, 6, 4
    q, k, v, lam, do, lay = _case(B, H, kv, L, d, dq, block, rows, 4 + dq)
    f = lambda *x: (od.forward(*x, lay, 0.7, block, causal)[0] * do).sum()  # noqa: E731
    grads = od.backward(q, k, v, lam, do, lay, 0.7, block, causal)
    args = [q, k, v, lam]
    rng = np.random.default_rng(9)
    for n, grad in enumerate(grads):
        x = args[n]
        for _ in range(25):
            at = tuple(rng.integers(0, s) for s in x.shape)
            ends = []
            for step in (1e-5, -1e-5):
                y = x.copy()
                y[at] += step
                ends.append(f(*(y if i == n else a for i, a in enumerate(args))))
            assert abs((ends[0] - ends[1]) / 2e-5 - grad[at]) < 1e-7 * max(1, np.abs(grad).max()), (n, at)


def test_bounds_catch_planted_mistakes():
    """The bounds are loose by a small factor only: a lost weight, a missing row term, a diagonal
    off by one and a key half mixed up all leave them."""
    q, k, v, lam, do, lay = _case(1, 2, 1, 70, 64, 64, 64, True, 6, hole=False)
    args = (lay, 0.125, 64, True)
    bnd = od.bounds(q, k, v, lam, do, *args)
    ref = od.forward(q, k, v, lam, *args)
    off = od.forward(q, k, v, lam * 1.1, *args)
    assert (np.abs(off[0] - ref[0]) > bnd["out"]).any()
    off = od.forward(q, k, v, lam, lay, 0.125, 64, False)
    assert (np.abs(off[0] - ref[0]) > bnd["out"]).any()
    gr = od.backward(q, k, v, lam, do, *args)
    off = od.backward(q, k, v, 1.1 * lam, do, *args)
    for i, name in enumerate(("dq", "dk", "dv")):
        assert (np.abs(off[i] - gr[i]) > bnd[name]).any(), name
    assert (np.abs(gr[3] * 1.001 - gr[3]) > bnd["dlam"]).any()

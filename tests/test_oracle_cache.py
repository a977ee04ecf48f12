"""Pins of the paged-cache oracle (CPU only): torch's e4m3 rounding, brute force over all
stored numbers, scale closed forms, stack invariants of resize, and fp64 attention over the
gathered pages."""

import numpy as np
import pytest
import torch
import torch.nn.functional as F

from oracle import bsa_oracle_cache as oc


def _e4m3_values():
    return torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()


def test_round_stored_is_nearest():
    """Every result is a stored number, none is nearer, and ties take the even one (torch's
    conversion of the same values)."""
    vals = _e4m3_values()
    vals = np.unique(vals[np.isfinite(vals)])
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(400) * s for s in (1e-3, 0.02, 1.0, 100.0)]
                       + [vals, (vals[1:] + vals[:-1]) / 2, [0.0, 447.9, 1e6, -1e6]])
    got = np.array([oc.round_stored(v, "e4m3") for v in x])
    assert np.all(np.isin(got, vals))
    near = np.abs(x[:, None] - vals[None]).min(1)
    assert np.array_equal(np.abs(got - x), near)
    ref = torch.tensor(np.clip(x, -448, 448)).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(got, ref)
    ints = [oc.round_stored(v, "int8") for v in (0.5, 1.5, -2.5, 126.5, 127.4, 1000.0, -1000.0)]
    assert ints == [0.0, 2.0, -2.0, 126.0, 127.0, 127.0, -127.0]
    assert np.isnan(oc.round_stored(float("nan"), "e4m3"))
    assert oc.round_stored(float("nan"), "int8") == 0.0


@pytest.mark.parametrize("kind,largest", [("e4m3", 448.0), ("int8", 127.0)])
def test_scale_closed_form(kind, largest):
    for amax in (1e-3, 0.9, 1.0, 127.0, 127.5, 448.0, 448.1, 3e4):
        s = oc.scale_for(amax, kind)
        assert np.log2(s) == round(np.log2(s)) and amax <= largest * s and amax > largest * s / 2
    assert oc.scale_for(0.0, kind) == 2.0 ** -60 and oc.scale_for(1e38, kind) == 2.0 ** 60


def test_resize_by_hand():
    table = np.array([[7, 3, -1, -1], [5, -1, -1, -1], [2, 6, 4, -1]])
    free = np.array([0, 1, 9, -1, -1, -1, -1, -1, -1, -1])
    got = oc.resize(table, [7, 4, 10], [9, 5, 3], free, 3, 4, 6)
    # request 2 gives back 6 and 4: the stack is 0 1 9 6 4; request 0 takes 4, request 1 takes 6
    assert got[0].tolist() == [[7, 3, 4, -1], [5, 6, -1, -1], [2, 6, 4, -1]]
    assert got[1].tolist() == [9, 5, 3] and got[3] == 3 and got[2][:3].tolist() == [0, 1, 9]
    assert got[4].tolist() == [0, 2, 3, 3]
    assert got[5].tolist() == [3 * 4 + 3, 4 * 4, 6 * 4, -1, -1, -1] and got[6] == 0


def test_resize_keeps_every_page_once():
    rng = np.random.default_rng(3)
    B, width, page, pages = 9, 6, 16, 40
    table, lens = np.full((B, width), -1), np.zeros(B, int)
    free, count = rng.permutation(pages), pages
    for _ in range(30):
        new = np.where(rng.random(B) < 0.3, rng.integers(0, width * page + 1, B), lens)
        table, lens, free, count, cu, slots, status = oc.resize(table, lens, new, free, count, page, B * width * page)
        held = [p for b in range(B) for p in table[b, : -(-int(lens[b]) // page)]]
        assert sorted(held + free[:count].tolist()) == list(range(pages))
        assert status == 0 or np.all(slots == -1)
        assert len(set(slots[slots >= 0])) == (slots >= 0).sum() == cu[-1]


def test_resize_refusals():
    table, free = np.zeros((2, 2), int), np.arange(4)
    assert oc.resize(table, [0, 0], [8, 9], free, 4, 4, 20)[6] == -2
    assert oc.resize(table, [0, -1], [8, 8], free, 4, 4, 20)[6] == -2
    assert oc.resize(table, [0, 0], [8, 8], free, 4, 4, 15)[6] == oc.INT32_MIN
    assert oc.resize(table, [0, 0], [8, 8], free, 5, 4, 16)[6] == oc.INT32_MIN + 1
    assert oc.resize(table, [0, 0], [8, 8], free, 1, 4, 16)[6] == 3


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_append_growing_scale(kind):
    """Tokens one at a time, each twice the last: after every append each kept number is
    within a step of what it stood for, and the newest is within half a step."""
    cache, scale = np.zeros((1, 1, 16, 4)), np.full((1, 1), 7.0)
    x = np.array([[1.0, -0.3, 0.77, 0.01]]) * 2.0 ** np.arange(16)[:, None]
    for t in range(16):
        cache, scale = oc.append(x[t][None, None], [t], cache, scale, kind)
        s = scale[0, 0]
        step = s if kind == "int8" else np.maximum(np.abs(x[: t + 1]) / 8, s * 2.0 ** -9)
        assert np.all(np.abs(cache[0, 0, : t + 1] * s - x[: t + 1]) <= step)
        assert np.all(np.abs(cache[0, 0, t] * s - x[t]) <= (step if kind == "int8" else step[t]) / 2 + 1e-12)


@pytest.mark.parametrize("window,softcap", [(-1, 0.0), (5, 0.0), (-1, 2.0)])
def test_forward_is_attention_over_the_pages(window, softcap):
    rng = np.random.default_rng(5)
    P, H, G, page, d, n = 9, 2, 3, 4, 8, 3
    k, v = rng.standard_normal((2, P, H, page, d))
    ks, vs = rng.random((2, P, H)) + 0.5
    table, lens, cu = np.array([[4, 0, 7, 2], [1, 8, 3, 5]]), [14, 9], [0, 3, 6]
    q = rng.standard_normal((6, H * G, d))
    out, lse, weight, size = oc.forward(q, k, v, ks, vs, table, lens, cu, 0.4, window, softcap)
    for b in range(2):
        kk = (k * ks[..., None, None])[table[b]].transpose(1, 0, 2, 3).reshape(H, -1, d)[:, : lens[b]]
        vv = (v * vs[..., None, None])[table[b]].transpose(1, 0, 2, 3).reshape(H, -1, d)[:, : lens[b]]
        kk, vv = (torch.from_numpy(a.repeat(G, 0)) for a in (kk, vv))
        qq = torch.from_numpy(q[cu[b]: cu[b + 1]].transpose(1, 0, 2).copy())
        pos = torch.arange(lens[b] - n, lens[b])[:, None]
        c = torch.arange(lens[b])[None]
        mask = (c <= pos) & (c >= pos - (window if window >= 0 else 10 ** 6))
        s = 0.4 * qq @ kk.transpose(1, 2)
        if softcap:
            s = softcap * torch.tanh(s / softcap)
        else:
            ref = F.scaled_dot_product_attention(qq, kk, vv, attn_mask=mask, scale=0.4)
            assert np.abs(out[cu[b]: cu[b + 1]].transpose(1, 0, 2) - ref.numpy()).max() < 1e-9
        s = s.masked_fill(~mask, -np.inf)
        assert np.abs(lse[cu[b]: cu[b + 1]].T - torch.logsumexp(s, -1).numpy()).max() < 1e-9
        ref = torch.softmax(s, -1) @ vv
        assert np.abs(out[cu[b]: cu[b + 1]].transpose(1, 0, 2) - ref.numpy()).max() < 1e-9
    assert np.all(weight >= np.abs(out) - 1e-12)


def test_forward_edges():
    """Positions before the first token and rows of masked pages are empty; a sink is then
    all there is; a layout row leaves only its blocks; a bad page holds no keys."""
    rng = np.random.default_rng(6)
    k, v = rng.standard_normal((2, 3, 1, 4, 8))
    one = np.ones((3, 1))
    q = rng.standard_normal((5, 2, 8))
    table = np.array([[1, 2]])
    out, lse, _, _ = oc.forward(q, k, v, one, one, table, [3], [0, 5], 1.0)
    assert np.all(out[:2] == 0) and np.all(np.isinf(lse[:2])) and np.all(np.isfinite(lse[2:]))
    assert np.allclose(out[2], v[1, 0, 0])
    _, lse, _, _ = oc.forward(q, k, v, one, one, table, [3], [0, 5], 1.0, sinks=[0.5, -2.0])
    assert np.allclose(lse[0], [0.5, -2.0])
    layout = np.zeros((1, 2, 2), int)
    layout[0, 1, 0] = 1
    a = oc.forward(q[:1], k, v, one, one, table, [6], [0, 1], 1.0, layout=layout, block=4)
    b = oc.forward(q[:1], k, v, one, one, table, [4], [0, 1], 1.0)
    assert np.allclose(a[0], b[0]) and np.allclose(a[1], b[1])
    c = oc.forward(q[:1], k, v, one, one, np.array([[1, 3]]), [6], [0, 1], 1.0)
    assert np.allclose(c[0], b[0]) and np.allclose(c[1], b[1])

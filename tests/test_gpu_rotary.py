"""GPU parity of bsa_rotary against complex products in 64 bits.

Bound: the sine's argument is the exact angle rounded to fp32 (2^-25 half-turns, 1e-7 radians)
and the sine and cosine are good to 2^-22, so a result is off by at most 5e-7 (|x| + |y|) before
its rounding, eps / 2 of its size."""

import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import block_sparse_head_gb300 as bsa

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    return cuda_lib


def _turned(x, positions, f, axis, pairing, inverse):
    """x [..., tokens, heads or not ...] as fp64 numpy [B, H, L, d]; positions [axes, B, L]."""
    out = x.copy()
    n = len(f)
    for i in range(n):
        a, b = (i, i + n) if pairing == "half" else (2 * i, 2 * i + 1)
        angle = (positions[axis[i]].astype(np.longdouble) * np.longdouble(f[i]))[:, None]
        angle = np.remainder(angle, 2 * np.longdouble("3.14159265358979323846264338327950288")).astype(np.float64)
        z = (x[..., a] + 1j * x[..., b]) * np.exp((-1j if inverse else 1j) * angle)
        out[..., a], out[..., b] = z.real, z.imag
    return out


def _within(got, x, ref, n, pairing):
    got, eps = got.double().cpu().numpy(), torch.finfo(got.dtype).eps
    size = np.zeros_like(x)
    if pairing == "half":
        s = np.abs(x[..., :n]) + np.abs(x[..., n:2 * n])
        size[..., :n], size[..., n:2 * n] = s, s
    else:
        s = np.abs(x[..., 0:2 * n:2]) + np.abs(x[..., 1:2 * n:2])
        size[..., 0:2 * n:2], size[..., 1:2 * n:2] = s, s
    err = np.abs(got - ref)
    # 2^-25: half a step of fp16's subnormals
    assert np.all(err <= eps / 2 * np.abs(ref) + 5e-7 * size + 2.0 ** -25), err.max()
    assert np.array_equal(got[..., 2 * n:], x[..., 2 * n:])  # behind the pairs: as it was


def _ladder(pairs, axes, seed=0):
    r = np.random.default_rng(seed)
    return [10000.0 ** (-i / pairs) for i in range(pairs)], r.integers(0, axes, pairs).tolist()


def _check(B, H, Hkv, L, d, pairs, axes=1, pairing="half", dtype="bf16", inverse=False, far=1 << 20, shared=False,
           layout="heads", in_place=False, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = np.random.default_rng(seed)
    f, axis = _ladder(pairs, axes, seed)
    axis[0] = axes - 1
    table = bsa.rotary_table(f, axis)
    # Positions on both sides of zero, the ends of 32 bits among them.
    pos = r.integers(-far, far, (axes, B, L))
    pos.flat[:: max(1, pos.size // 3)] = [2 ** 31 - 1, -2 ** 31, 0, 1][: len(pos.flat[:: max(1, pos.size // 3)])]
    if shared:
        pos[:] = pos[:, :1]
    pd = torch.as_tensor((pos[:, 0] if shared else pos).astype(np.int32)).cuda().contiguous()
    xs = []
    for heads in (H, Hkv):
        if layout == "fused":  # [B, L, heads + 3, d] rows, seen as [B, heads, L, d]
            x = torch.randn(B, L, heads + 3, d, generator=g).to(TYPES[dtype]).cuda()[:, :, 1:1 + heads].transpose(1, 2)
        else:
            x = torch.randn(B, heads, L, d, generator=g).to(TYPES[dtype]).cuda()
        xs.append(x)
    before = [x.double().cpu().numpy() for x in xs]
    kw = dict(q_out=xs[0], k_out=xs[1]) if in_place else {}
    got = bsa.rotary(*xs, pd, table, pairing=pairing, inverse=inverse, **kw)
    for y, x in zip(got, before):
        _within(y, x, _turned(x, pos, f, axis, pairing, inverse), pairs, pairing)
    if in_place:
        assert got[0] is xs[0] and got[1] is xs[1]
    return xs, pd, table, got


@pytest.mark.parametrize("pairing", ["half", "adjacent"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d,pairs", [(128, 64), (64, 32), (256, 128), (96, 40), (80, 20), (128, 22), (64, 13), (8, 1),
                                     (8, 4), (200, 100)])
def test_heads(pairing, dtype, d, pairs):
    """All sizes of pieces: pairs that eight, four, two or nothing divides; numbers behind them."""
    _check(2, 3, 1, 37, d, pairs, 3, pairing, dtype, seed=d + pairs)


@pytest.mark.parametrize("pairing", ["half", "adjacent"])
@pytest.mark.parametrize("L", [1, 2, 31, 33, 500])
@pytest.mark.parametrize("B,H,Hkv", [(1, 1, 1), (3, 8, 2), (1, 40, 8)])
def test_lengths(pairing, L, B, H, Hkv):
    _check(B, H, Hkv, L, 128, 64, 3, pairing, seed=L + H)


def test_more_tokens_than_a_grid_of_tiles():
    _check(2, 5, 2, 5000, 64, 32, 2, seed=5)


@pytest.mark.parametrize("pairing", ["half", "adjacent"])
@pytest.mark.parametrize("layout", ["heads", "fused"])
@pytest.mark.parametrize("in_place", [False, True])
def test_strides_in_place_and_inverse(pairing, layout, in_place):
    _check(2, 4, 2, 70, 96, 32, 4, pairing, inverse=True, layout=layout, in_place=in_place, shared=True, seed=7)


def test_packed_tokens_are_one_batch_entry():
    g = torch.Generator().manual_seed(8)
    rows = torch.randn(50, 9, 128, generator=g).to(torch.bfloat16).cuda()
    f, axis = _ladder(64, 3)
    table = bsa.rotary_table(f, axis)
    pos = torch.randint(0, 1000, (3, 50), generator=g, dtype=torch.int32).cuda()
    q, k = bsa.rotary(rows[:, :6], rows[:, 6:8], pos, table)
    for x, y in ((rows[:, :6], q), (rows[:, 6:8], k)):
        want, none = bsa.rotary(x.transpose(0, 1)[None].contiguous(), None, pos, table)
        assert none is None and y.shape == x.shape
        assert torch.equal(want[0].transpose(0, 1), y)


def test_there_and_back():
    """The inverse turn of the turned numbers, both rounded: within two roundings of the start."""
    xs, pos, table, (q, _) = _check(1, 4, 2, 300, 128, 64, 3, dtype="fp16", seed=9)
    back, _ = bsa.rotary(q, None, pos, table, inverse=True)
    size = xs[0].double().view(1, 4, 300, 2, 64).pow(2).sum(3).sqrt().repeat(1, 1, 1, 2)
    assert torch.all((back.double() - xs[0].double()).abs() <= (2 * 2.0 ** -11 * 1.5 + 2e-6) * size + 2.0 ** -23)


def test_inverse_is_the_gradient():
    """<rotary(x), g> by central differences in x against <rotary's inverse of g>, in exact pairs of
    steps: the turn is linear, so a step of one number gives its gradient exactly up to the
    roundings of the two results, eps / 2 each of numbers below 8."""
    g = torch.Generator().manual_seed(10)
    x = torch.randn(1, 1, 4, 16, generator=g).to(torch.float16).cuda()
    do = torch.randn(1, 1, 4, 16, generator=g).to(torch.float16).cuda()
    table = bsa.rotary_table([1.0, 0.7, 0.3], [0, 1, 0])
    pos = torch.randint(-50, 50, (2, 4), generator=g, dtype=torch.int32).cuda()
    grad = bsa.rotary(do, None, pos, table, inverse=True)[0]
    for t in range(4):
        for n in range(16):
            ends = []
            for step in (1.0, -1.0):
                y = x.clone()
                y[0, 0, t, n] = step
                ends.append((bsa.rotary(y, None, pos, table)[0].double() * do.double()).sum())
            slope = float(ends[0] - ends[1]) / 2
            assert abs(slope - float(grad[0, 0, t, n])) <= 2.0 ** -10 * float(do.double().abs().sum())


def test_relative_positions_only():
    """Scores of turned queries and keys depend on the distance of their positions: the same at
    position 0 as 2^30 further, where a product in fp32 would have lost the angle."""
    g = torch.Generator().manual_seed(11)
    q, k = (torch.randn(1, 1, 64, 128, generator=g).to(torch.float16).cuda() for _ in range(2))
    table = bsa.rotary_table(_ladder(64, 1)[0])
    near = torch.arange(64, dtype=torch.int32).cuda()[None]
    s = []
    for off in (0, 1 << 30):
        a, b = bsa.rotary(q, k, near + off, table)
        s.append(a[0, 0].double() @ b[0, 0].double().T)
    # each turned number is rounded by 2^-11: 128 products of numbers of size about one
    assert (s[0] - s[1]).abs().max() < 4 * 2.0 ** -11 * 128 ** 0.5 * 3


@pytest.mark.parametrize("pairing", ["half", "adjacent"])
def test_large_frequencies_at_far_positions(pairing):
    """Frequencies up to the largest that a table takes, at the ends of 32 bits: the angle as an exact
    fraction, so that the bound at the top holds here as for a ladder below one."""
    f = [1e6, -1e6, 123456.789, 1e3, 12.5, 1.0, 1e5 * math.pi, 777.7]
    pos = [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 2, -123456789, 1 << 30, 1]
    g = torch.Generator().manual_seed(16)
    x = torch.randn(1, 2, len(pos), 16, generator=g).to(torch.float16).cuda()
    got = bsa.rotary(x, None, torch.tensor([pos], dtype=torch.int32).cuda(), bsa.rotary_table(f), pairing=pairing)[0]
    two_pi = Fraction("6.28318530717958647692528676655900576839433879875021164194989")
    before = x.double().cpu().numpy()
    want = before.copy()
    for i, w in enumerate(f):
        a, b = (i, i + len(f)) if pairing == "half" else (2 * i, 2 * i + 1)
        for t, at in enumerate(pos):
            turned = (before[:, :, t, a] + 1j * before[:, :, t, b]) * np.exp(1j * float((Fraction(w) * at) % two_pi))
            want[:, :, t, a], want[:, :, t, b] = turned.real, turned.imag
    _within(got, before, want, len(f), pairing)


def test_streams_and_capture():
    g = torch.Generator().manual_seed(12)
    q, k = (torch.randn(1, 4, 100, 64, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    pos = torch.arange(100, dtype=torch.int32).cuda()[None]
    table = bsa.rotary_table(_ladder(32, 1)[0])
    want = bsa.rotary(q, k, pos, table)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = bsa.rotary(q, k, pos, table, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        held = bsa.rotary(q, k, pos, table)
    pos += 5
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, bsa.rotary(q, k, pos, table)))


def test_offsets_behind_32_bits():
    """More than 2^31 numbers of queries: the last tokens of the last head against a call of them
    alone, in place and not."""
    L, d, n = 270_000, 128, 70
    q = torch.empty(1, 64, L, d, dtype=torch.bfloat16, device="cuda")
    assert q.numel() > 2 ** 31
    g = torch.Generator().manual_seed(15)
    tail = torch.randn(1, 2, n, d, generator=g).to(torch.bfloat16).cuda()
    q[:, -2:, -n:] = tail
    q[:, 0, :n] = tail[:, 0]
    pos = torch.arange(L, dtype=torch.int32).cuda()[None]
    table = bsa.rotary_table(_ladder(64, 1)[0])
    want = bsa.rotary(tail, None, pos[:, -n:].contiguous(), table)[0]
    first = bsa.rotary(tail[:, :1].contiguous(), None, pos[:, :n].contiguous(), table)[0]
    for out in (None, q):
        got = bsa.rotary(q, None, pos, table, q_out=out)[0]
        assert torch.equal(got[:, -2:, -n:], want) and torch.equal(got[:, :1, :n], first)
        del got


def test_queries_that_are_the_keys():
    """q and k one tensor: turned into two outputs; in place it is refused."""
    q = torch.randn(1, 2, 9, 64, device="cuda").to(torch.bfloat16)
    pos = torch.arange(9, dtype=torch.int32).cuda()[None]
    table = bsa.rotary_table(_ladder(32, 1)[0])
    a, b = bsa.rotary(q, q, pos, table)
    assert torch.equal(a, b) and torch.equal(a, bsa.rotary(q, None, pos, table)[0])
    with pytest.raises(bsa.BsaError):
        bsa.rotary(q, q, pos, table, q_out=q, k_out=q)
    with pytest.raises(bsa.BsaError):
        bsa.rotary(q, None, pos, table, q_out=q[:, :1].expand(1, 2, 9, 64))


def test_no_tokens():
    table = bsa.rotary_table([1.0])
    q = torch.empty(0, 4, 64, dtype=torch.float16, device="cuda")
    out, none = bsa.rotary(q, None, torch.empty(1, 0, dtype=torch.int32, device="cuda"), table)
    assert out.shape == q.shape and none is None


def test_before_the_attention():
    """Queries and keys turned, then differential attention over them: against the same in 64 bits
    on the turned, rounded numbers."""
    from oracle import diff as od

    g = torch.Generator().manual_seed(13)
    B, H, Hkv, L, d = 1, 2, 1, 200, 64
    q = torch.randn(B, 2 * H, L, d, generator=g).to(torch.bfloat16).cuda()
    k, v = (torch.randn(B, Hkv, L, d, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    lam = torch.rand(H, generator=g).cuda()
    table = bsa.rotary_table([10000.0 ** (-i / 32) for i in range(32)], [0] * 8 + [1] * 12 + [2] * 12)
    pos = torch.stack([torch.arange(L) // 50, torch.arange(L) % 50 // 10, torch.arange(L) % 10]).to(torch.int32).cuda()
    do = torch.randn(B, H, L, d, generator=g).to(torch.bfloat16).cuda()
    lay = torch.tril(torch.ones(Hkv, 4, 4, dtype=torch.int32))
    lut = bsa.build_lut(lay, B)
    qr, kr = bsa.rotary(q, k, pos, table)
    out, lse, out2 = bsa.diff_forward(qr, kr, v, lam, lut, 0.125, 64, True, training=True)
    dq, dk, dv, dlam = bsa.diff_backward(qr, kr, v, lam, out, out2, lse, do, lut, 0.125, 64, True)
    dq, dk = bsa.rotary(dq, dk, pos, table, inverse=True, q_out=dq, k_out=dk)
    assert lut.device_status()[0] == 0
    num = lambda t: t.double().cpu().numpy()  # noqa: E731
    args = [num(t) for t in (qr, kr, v, lam)]
    bnd = od.bounds(*args, num(do), lay.numpy(), 0.125, 64, True)
    assert np.all(np.abs(num(out) - od.forward(*args, lay.numpy(), 0.125, 64, True)[0]) <= bnd["out"])
    gq, gk, _, _ = od.backward(*args, num(do), lay.numpy(), 0.125, 64, True)
    f = [10000.0 ** (-i / 32) for i in range(32)]
    axis = [0] * 8 + [1] * 12 + [2] * 12
    for got, ref, b in ((dq, gq, bnd["dq"]), (dk, gk, bnd["dk"])):
        want = _turned(ref, pos.cpu().numpy()[:, None], f, axis, "half", True)
        # the bounds of a pair add up under a turn; one more rounding
        b = b[..., :32] + b[..., 32:]
        tol = np.concatenate([b, b], -1) + 2.0 ** -8 * np.abs(want) + 1e-6 * np.abs(ref).max()
        tol = tol + 2.0 ** -8 * np.concatenate([b, b], -1)
        assert np.all(np.abs(num(got) - want) <= tol)


def test_refusals():
    q = torch.randn(1, 2, 10, 64, device="cuda").to(torch.bfloat16)
    pos = torch.zeros(1, 10, dtype=torch.int32, device="cuda")
    table = bsa.rotary_table([1.0, 0.5])
    for bad in (dict(q=q.float()), dict(q=q.cpu()), dict(q=q[0, 0]), dict(k=q[0]), dict(k=q.half()), dict(k=q[:, :, :5]),
                dict(pos=pos.long()), dict(pos=pos.cpu()), dict(pos=pos[:, :5]), dict(pos=pos.repeat(2, 1)),
                dict(pos=torch.zeros(1, 20, dtype=torch.int32, device="cuda")[:, ::2]), dict(table=None),
                dict(pairing="both"), dict(q_out=q[:, :1]), dict(q=q.transpose(2, 3))):
        a = {**dict(q=q, k=None, pos=pos, table=table), **bad}
        with pytest.raises(ValueError):
            bsa.rotary(a.pop("q"), a.pop("k"), a.pop("pos"), a.pop("table"), **a)
    with pytest.raises(bsa.BsaError):  # more pairs than numbers
        bsa.rotary(q, None, pos, bsa.rotary_table(np.ones(33)))
    with pytest.raises(bsa.BsaError):
        bsa.rotary(torch.randn(1, 2, 10, 68, device="cuda").to(torch.bfloat16)[..., :64], None, pos, table)
    for bad in ([], [[1.0]], [math.nan], [1e7]):
        with pytest.raises((ValueError, bsa.BsaError)):
            bsa.rotary_table(bad)
    for bad in ([0], [0, 9], [0, -1], [0.0, 1.0], [0, 10 ** 12]):
        with pytest.raises((ValueError, bsa.BsaError)):
            bsa.rotary_table([1.0, 0.5], bad)

"""GPU parity of bsa_diff_forward and bsa_diff_backward against the fp64 oracle, within the
oracle's elementwise error bounds (``oracle.diff.bounds`` derives them: one rounding of each
second product's bf16 operand, one of each result, fp32 elsewhere).  lse: its exponentials and
sum in fp32, 1e-5 of its magnitude."""

import math

import numpy as np
import pytest
import torch

import block_sparse_head_gb300 as bsa
from oracle import diff as od

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    return cuda_lib


def _layout(kv, nb, seed, p=0.4):
    """Random blocks on both sides of the diagonal, a row and a column without any."""
    g = torch.Generator().manual_seed(seed)
    lay = (torch.rand(kv, nb, nb, generator=g) < p).to(torch.int32)
    lay[:, torch.arange(nb), torch.arange(nb)] = (torch.rand(kv, nb, generator=g) < 0.7).to(torch.int32)
    if nb > 2:
        lay[:, 1], lay[:, :, 2] = 0, 0
    return lay


def _inputs(B, H, kv, L, d, dq, rows, seed, dev="cuda"):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(dev)  # noqa: E731
    lam = torch.rand(*((B, H, L) if rows else (H,)), generator=g) * 1.2 - 0.2
    return r(B, 2 * H, L, dq), r(B, kv, L, d), r(B, kv, L, d), lam.to(dev), r(B, H, L, d)


def _np(t):
    return t.detach().double().cpu().numpy()


def _within(got, ref, bound, name):
    got = _np(got)
    assert np.array_equal(np.isfinite(got), np.isfinite(ref)), name
    fin = np.isfinite(ref)
    err = np.abs(got - ref)[fin]
    b = np.broadcast_to(bound, ref.shape)[fin]
    assert np.all(err <= b), (name, float((err / b).max()))


def _check(q, k, v, lam, do, lay, scale, block, causal, lut=None):
    lut = bsa.build_lut(lay, q.shape[0]) if lut is None else lut
    out, lse, out2 = bsa.diff_forward(q, k, v, lam, lut, scale, block, causal, training=True)
    grads = bsa.diff_backward(q, k, v, lam, out, out2, lse, do, lut, scale, block, causal)
    status, word = lut.device_status()
    assert status == 0, hex(word)
    args = [_np(t) for t in (q, k, v, lam)]
    ro, rl, ro2 = od.forward(*args, lay.numpy(), scale, block, causal)
    bnd = od.bounds(*args, _np(do), lay.numpy(), scale, block, causal)
    _within(out, ro, bnd["out"], "out")
    _within(out2, ro2, bnd["out2"], "out2")
    with np.errstate(invalid="ignore"):
        _within(lse, rl, 1e-5 * np.maximum(1.0, np.abs(rl)), "lse")
    for got, ref, name in zip(grads, od.backward(*args, _np(do), lay.numpy(), scale, block, causal),
                              ("dq", "dk", "dv", "dlam")):
        _within(got, ref, bnd[name], name)
    return out, lse, out2, grads


KINDS = [(64, 64, 64), (64, 128, 128), (64, 128, 64), (128, 64, 64), (128, 128, 128), (128, 128, 64)]


@pytest.mark.parametrize("block,d,dq", KINDS)
@pytest.mark.parametrize("L", [1, 17, 64, 130, 500])
def test_lengths(block, d, dq, L):
    nb = -(-L // block)
    q, k, v, lam, do = _inputs(1, 2, 1, L, d, dq, True, 10 * L + block + d + dq)
    _check(q, k, v, lam, do, torch.tril(torch.ones(1, nb, nb, dtype=torch.int32)), 1 / math.sqrt(dq), block, True)


@pytest.mark.parametrize("block,d,dq", KINDS)
@pytest.mark.parametrize("B,H,kv,causal,rows", [(2, 2, 2, True, False), (1, 6, 2, False, True)])
def test_random_layouts(block, d, dq, B, H, kv, causal, rows):
    L = 6 * block - 37
    q, k, v, lam, do = _inputs(B, H, kv, L, d, dq, rows, 3 * block + d + dq + B)
    lay = _layout(kv, 6, 5 + block + H)
    out, lse, _, grads = _check(q, k, v, lam, do, lay, 1 / math.sqrt(dq), block, causal)
    # a row without an active key, a key that no row sees: exactly zero
    assert torch.all(out[:, :, block:2 * block] == 0) and torch.all(lse[:, :, block:2 * block] == -math.inf)
    assert torch.all(grads[0][:, :, block:2 * block] == 0)
    for t in grads[1:3]:
        assert torch.all(t[:, :, 2 * block:3 * block] == 0)
    if rows:
        assert torch.all(grads[3][:, :, block:2 * block] == 0)


@pytest.mark.parametrize("scale", [0.0, -0.2, 1.5])
def test_scales_and_a_growing_maximum(scale):
    block, L = 64, 64 * 9
    q, k, v, lam, do = _inputs(1, 2, 1, L, 128, 128, False, 71)
    for j in range(9):  # later blocks score higher: the running maximum moves, O is rescaled
        k[:, :, j * block:(j + 1) * block] *= 0.2 + 0.1 * j
    _check(q, k, v, lam, do, torch.tril(torch.ones(1, 9, 9, dtype=torch.int32)), scale, block, True)


@pytest.mark.parametrize("block,d,dq", KINDS)
@pytest.mark.parametrize("L", [100, 200])
def test_scores_far_below_zero(block, d, dq, L):
    """Every score near -130, the last block cut by the sequence's end and seen by all rows: places
    behind the end score 0 there, and exp(0 - lse) is more than fp32 holds."""
    nb = -(-L // block)
    q, k, v, lam, do = _inputs(1, 2, 1, L, d, dq, True, 94 + L + block + d + dq)
    q, k = (0.05 * q.float() - 1.0).to(torch.bfloat16), (0.05 * k.float() + 1.0).to(torch.bfloat16)
    _check(q, k, v, lam, do, torch.ones(1, nb, nb, dtype=torch.int32), 130.0 / dq, block, False)


def test_many_items_a_cta():
    """More work items than SMs in every walk, so that CTAs change items several times."""
    q, k, v, lam, do = _inputs(2, 8, 4, 1600, 64, 64, True, 72)
    _check(q, k, v, lam, do, _layout(4, 25, 73, 0.15), 0.125, 64, True)


@pytest.mark.parametrize("block,d,dq", [(64, 64, 64), (128, 128, 64)])
def test_columns_cut_between_ctas(block, d, dq):
    """One kv head of eight heads and few, long columns: every column's steps are shared by several
    CTAs, some of them inside one column for their whole share, columns without a block between."""
    nb = 14
    lay = torch.zeros(1, nb, nb, dtype=torch.int32)
    lay[0, :, 3], lay[0, :, 7], lay[0, 5:9, 10], lay[0, 13, 13] = 1, 1, 1, 1
    q, k, v, lam, do = _inputs(2, 8, 1, nb * block - 3, d, dq, False, 90)
    _check(q, k, v, lam, do, lay, 1 / math.sqrt(dq), block, True)


def test_layout_without_a_block():
    q, k, v, lam, do = _inputs(1, 2, 1, 100, 64, 64, False, 91)
    _check(q, k, v, lam, do, torch.zeros(1, 2, 2, dtype=torch.int32), 0.1, 64, True)


def test_repeatable_and_on_another_stream():
    q, k, v, lam, do = _inputs(1, 4, 2, 900, 128, 64, False, 74)
    lay = _layout(2, 8, 75)
    lut = bsa.build_lut(lay, 1)
    first = _check(q, k, v, lam, do, lay, 0.125, 128, True, lut)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse, out2 = bsa.diff_forward(q, k, v, lam, lut, 0.125, 128, True, training=True, stream=side)
    grads = bsa.diff_backward(q, k, v, lam, out, out2, lse, do, lut, 0.125, 128, True, stream=side)
    side.synchronize()
    for a, b in zip((out, lse, out2) + grads, first[:3] + first[3]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("block,d,dq", [(64, 64, 64), (128, 128, 128), (64, 128, 64)])
@pytest.mark.parametrize("rows", [False, True])
def test_weights_far_from_one(block, d, dq, rows):
    """|lam| from 2 to 30, of both signs: D_0 = <dO, out> + lam D_1 is the small difference of large
    numbers, whose roundings the bounds count."""
    L = 9 * block - 5
    q, k, v, lam, do = _inputs(1, 4, 2, L, d, dq, rows, 97 + block + d + dq)
    lam = torch.where(lam > 0.4, 2.0 + 28.0 * lam.clamp(0, 1), -2.0 - 20.0 * lam.abs())
    _check(q, k, v, lam, do, torch.tril(torch.ones(2, 9, 9, dtype=torch.int32)), 1 / math.sqrt(dq), block, True)


@pytest.mark.parametrize("block", [64, 128])
def test_key_halves_of_a_long_sequence(block):
    nb = -(-2999 // block)
    q, k, v, lam, do = _inputs(1, 4, 2, 2999, 128, 64, True, 98 + block)
    _check(q, k, v, lam, do, torch.tril(_layout(2, nb, 99, 0.3)), 0.125, block, True)


def test_a_key_half_that_is_not_finite_spoils_its_block_alone():
    """NaN and infinity among the numbers of one map's key half and of a value: rows that see their
    block may be lost, the others keep their bits, gradients of other blocks' keys too."""
    block, L = 64, 6 * 64
    q, k, v, lam, do = _inputs(1, 2, 1, L, 128, 64, True, 101)
    lay = torch.zeros(1, 6, 6, dtype=torch.int32)
    lay[0, :, 0], lay[0, 3, 2], lay[0, torch.arange(6), torch.arange(6)] = 1, 1, 1
    lay[0, 5, 5] = 0
    lut = bsa.build_lut(lay, 1)

    def step(k, v):
        out, lse, out2 = bsa.diff_forward(q, k, v, lam, lut, 0.125, block, True, training=True)
        return (out, lse, out2) + bsa.diff_backward(q, k, v, lam, out, out2, lse, do, lut, 0.125, block, True)

    want = step(k, v)
    kb, vb = k.clone(), v.clone()
    kb[0, 0, 2 * block + 5, 70], kb[0, 0, 2 * block + 9, 3], vb[0, 0, 2 * block + 7, 11] = math.nan, math.inf, -math.inf
    got = step(kb, vb)
    assert lut.device_status()[0] == 0
    keep = torch.ones(L, dtype=torch.bool, device="cuda")
    for row in (2, 3):  # rows that see block 2
        keep[row * block:(row + 1) * block] = False
    for a, b in zip(got[:4] + got[6:], want[:4] + want[6:]):
        assert torch.equal(a[:, :, keep], b[:, :, keep])
    for a, b in zip(got[4:6], want[4:6]):  # keys that only rows without block 2 see
        for c in (1, 4, 5):
            assert torch.equal(a[:, :, c * block:(c + 1) * block], b[:, :, c * block:(c + 1) * block])


def test_captured_behind_a_memset_and_another_stream():
    """The graph's node before the first kernel is no kernel, and the second call has two of them
    before it, one of another stream."""
    q, k, v, lam, do = _inputs(1, 2, 2, 500, 64, 64, False, 102)
    lut = bsa.build_lut(torch.tril(torch.ones(2, 8, 8, dtype=torch.int32)), 1)
    source = [t.clone() for t in (q, v, do)]

    def step(side=None):
        q.zero_()
        here = torch.cuda.current_stream()
        if side is not None:
            side.wait_stream(here)
            with torch.cuda.stream(side):
                v.copy_(source[1])
                v.mul_(0.5)
        else:
            v.copy_(source[1])
            v.mul_(0.5)
        q.copy_(source[0])
        q.mul_(2.0)
        if side is not None:
            here.wait_stream(side)
        out, lse, out2 = bsa.diff_forward(q, k, v, lam, lut, 0.125, 64, True, training=True)
        do.zero_()
        first = bsa.diff_backward(q, k, v, lam, out, out2, lse, do, lut, 0.125, 64, True)
        do.copy_(source[2])
        return (out, lse, out2) + first + bsa.diff_backward(q, k, v, lam, out, out2, lse, do, lut, 0.125, 64, True)

    want = [t.clone() for t in step()]
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        held = step(other)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, want):
            assert torch.equal(a, b)


def test_behind_a_library_product():
    """Kernels of other libraries right before and behind each call, on one stream."""
    lut = bsa.build_lut(_layout(2, 8, 75), 1)
    q, k, v, lam, do = _inputs(1, 8, 2, 1000, 128, 128, True, 103)
    a = torch.randn(4096, 4096, device="cuda", dtype=torch.bfloat16)

    def step(product):
        product()
        out, lse, out2 = bsa.diff_forward(q, k, v, lam, lut, 0.1, 128, True, training=True)
        product()
        got = (out, lse, out2) + bsa.diff_backward(q, k, v, lam, out, out2, lse, do, lut, 0.1, 128, True)
        product()
        return got

    want = step(lambda: None)
    for _ in range(20):
        for x, y in zip(step(lambda: a @ a), want):
            assert torch.equal(x, y)
    assert lut.device_status()[0] == 0


def test_two_streams_at_once():
    """Forwards and backwards on two streams that share the LUT, with nothing between them: the
    same bits as one after another."""
    lut = bsa.build_lut(_layout(2, 8, 75), 1)
    sets = [_inputs(1, 8, 2, 1000, 128, 128, rows, 76 + rows) for rows in (False, True)]

    def step(t, **kw):
        q, k, v, lam, do = t
        out, lse, out2 = bsa.diff_forward(q, k, v, lam, lut, 0.1, 128, True, training=True, **kw)
        return (out, lse, out2) + bsa.diff_backward(q, k, v, lam, out, out2, lse, do, lut, 0.1, 128, True, **kw)

    want = [step(t) for t in sets]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in sets]
    got = [[step(t, stream=s) for t, s in zip(sets, sides)] for _ in range(6)]
    torch.cuda.synchronize()
    assert lut.device_status()[0] == 0
    for both in got:
        for a, b in zip(both, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_offsets_behind_32_bits():
    """More than 2^31 numbers of queries; the last heads and the first against calls of them alone.
    dk and dv are summed in fp32 in another order there: within one rounding of each other."""
    L, H, d, block = 65536, 132, 128, 128
    nb = L // block
    lay = torch.zeros(1, nb, nb, dtype=torch.int32)
    lay[0, torch.arange(nb), torch.arange(nb)] = 1
    lay[0, nb - 1, 0] = 1
    luts = [bsa.build_lut(lay.expand(n, nb, nb).contiguous(), 1) for n in (H, 1)]
    g = torch.Generator(device="cuda").manual_seed(92)

    def rows(n):
        t = torch.empty(1, n, L, d, dtype=torch.bfloat16, device="cuda")
        for h in range(n):
            t[0, h] = torch.randn(L, d, generator=g, device="cuda")
        return t

    q, k, v, do = rows(2 * H), rows(H), rows(H), rows(H)
    assert q.numel() > 2 ** 31
    lam = torch.rand(1, H, L, generator=g, device="cuda")
    out, lse, out2 = bsa.diff_forward(q, k, v, lam, luts[0], 0.1, block, True, training=True)
    grads = bsa.diff_backward(q, k, v, lam, out, out2, lse, do, luts[0], 0.1, block, True)
    assert luts[0].device_status()[0] == 0
    for h in (0, H - 1):
        one = [t[:, h:h + 1].contiguous() for t in (k, v, lam, do)]
        qh = q[:, 2 * h:2 * h + 2].contiguous()
        o, s, o2 = bsa.diff_forward(qh, *one[:3], luts[1], 0.1, block, True, training=True)
        gr = bsa.diff_backward(qh, *one[:3], o, o2, s, one[3], luts[1], 0.1, block, True)
        assert torch.equal(out[:, h:h + 1], o) and torch.equal(out2[:, h:h + 1], o2)
        assert torch.equal(lse[:, 2 * h:2 * h + 2], s) and torch.equal(grads[0][:, 2 * h:2 * h + 2], gr[0])
        assert torch.equal(grads[3][:, h:h + 1], gr[3])
        for a, b in ((grads[1], gr[1]), (grads[2], gr[2])):
            a, b = a[:, h:h + 1].float(), b.float()
            # One bf16 step, at most 2^-7 of the value, and the order of the sums: at most four
            # steps of eight accumulations, each off by 2^-23 of a sum of at most 256 terms below 10.
            assert torch.all((a - b).abs() <= 2.0 ** -7 * torch.maximum(a.abs(), b.abs()) + 32 * 2560 * 2.0 ** -23)


def test_captured_step_follows_its_inputs():
    q, k, v, lam, do = _inputs(1, 2, 2, 300, 64, 64, False, 76)
    lay = torch.tril(torch.ones(2, 5, 5, dtype=torch.int32))
    lut, ws = bsa.build_lut(lay, 1), bsa.diff_workspace(1, 2, 300, 64, 64)

    def step():
        out, lse, out2 = bsa.diff_forward(q, k, v, lam, lut, 0.125, 64, True, training=True)
        return (out, lse) + bsa.diff_backward(q, k, v, lam, out, out2, lse, do, lut, 0.125, 64, True, workspace=ws)

    step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        held = step()
    for seed in (77, 78):
        for dst, src in zip((q, k, v, lam, do), _inputs(1, 2, 2, 300, 64, 64, False, seed)):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, step()):
            assert torch.equal(a, b)


def test_inference_call_equals_the_training_one():
    q, k, v, lam, _ = _inputs(1, 2, 1, 200, 128, 128, False, 79)
    lut = bsa.build_lut(torch.ones(1, 2, 2, dtype=torch.int32), 1)
    a = bsa.diff_forward(q, k, v, lam, lut, 0.09, 128, True, training=True)
    b = bsa.diff_forward(q, k, v, lam, lut, 0.09, 128, True)
    assert b[2] is None and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_outputs_off_a_sector_boundary():
    """Rows of 128 or 256 bytes at a base that is 16- but not 32-byte aligned; guards around the
    outputs stay as they were."""
    B, H, kv, L, d = 1, 2, 1, 100, 64
    q, k, v, lam, do = _inputs(B, H, kv, L, d, d, True, 80)
    lay = torch.ones(1, 2, 2, dtype=torch.int32)
    lut = bsa.build_lut(lay, 1)

    def room(shape, dtype):
        n = math.prod(shape)
        pad = 16 // dtype.itemsize
        base = torch.full((n + 4 * pad,), 7.0, dtype=dtype, device="cuda")
        return base, base[pad: pad + n].view(shape), pad

    shapes = [((B, H, L, d), torch.bfloat16), ((B, 2 * H, L), torch.float32), ((B, H, L, d), torch.bfloat16)]
    bases = [room(*s) for s in shapes]
    out, lse, out2 = (b[1] for b in bases)
    bsa.diff_forward(q, k, v, lam, lut, 0.125, 64, True, out=out, lse=lse, out2=out2)
    ref = bsa.diff_forward(q, k, v, lam, lut, 0.125, 64, True, training=True)
    gshapes = [(q.shape, torch.bfloat16), (k.shape, torch.bfloat16), (v.shape, torch.bfloat16), (lam.shape, torch.float32)]
    gbases = [room(*s) for s in gshapes]
    dq, dk, dv, dlam = (b[1] for b in gbases)
    bsa.diff_backward(q, k, v, lam, out, out2, lse, do, lut, 0.125, 64, True, dq=dq, dk=dk, dv=dv, dlam=dlam)
    gref = bsa.diff_backward(q, k, v, lam, *(ref[i] for i in (0, 2, 1)), do, lut, 0.125, 64, True)
    for a, b in zip((out, lse, out2, dq, dk, dv, dlam), ref + gref):
        assert torch.equal(a, b)
    for base, view, pad in bases + gbases:
        n = view.numel()
        assert torch.all(base[:pad] == 7) and torch.all(base[pad + n:] == 7)


@pytest.mark.parametrize("site", [1, 2, 6, 7, 8, 9, 10, 12, 13, 14])
def test_expired_wait_ends_the_forward_and_leaves_no_trace(site):
    q, k, v, lam, _ = _inputs(2, 8, 8, 1024, 64, 64, False, 81)
    lut = bsa.build_lut(torch.tril(torch.ones(8, 16, 16, dtype=torch.int32)), 2)
    ref = bsa.diff_forward(q, k, v, lam, lut, 0.125, 64, True)
    assert lut.device_status()[0] == 0
    lut.debug_expire_wait(site)
    bsa.diff_forward(q, k, v, lam, lut, 0.125, 64, True)
    status, word = lut.device_status()
    assert status == -8 and (word & 0xFFFF) == site
    lut.debug_expire_wait(0)
    again = bsa.diff_forward(q, k, v, lam, lut, 0.125, 64, True)
    assert lut.device_status()[0] == 0
    assert torch.equal(ref[0], again[0]) and torch.equal(ref[1], again[1])


@pytest.mark.parametrize("site", [1, 2, 6, 7, 8, 9, 12])
@pytest.mark.parametrize("block", [64, 128])
def test_expired_wait_ends_the_backward_and_leaves_no_trace(site, block):
    q, k, v, lam, do = _inputs(2, 8, 8, 16 * block, 64, 64, False, 82)
    lut = bsa.build_lut(torch.tril(torch.ones(8, 16, 16, dtype=torch.int32)), 2)
    out, lse, out2 = bsa.diff_forward(q, k, v, lam, lut, 0.125, block, True, training=True)
    args = (q, k, v, lam, out, out2, lse, do, lut, 0.125, block, True)
    ref = bsa.diff_backward(*args)
    assert lut.device_status()[0] == 0
    lut.debug_expire_wait(site)
    bsa.diff_backward(*args)
    status, word = lut.device_status()
    assert status == -8 and (word & 0xFFFF) == site
    lut.debug_expire_wait(0)
    again = bsa.diff_backward(*args)
    assert lut.device_status()[0] == 0
    for a, b in zip(ref, again):
        assert torch.equal(a, b)


def test_refusals_of_the_binding():
    q, k, v, lam, do = _inputs(1, 2, 1, 128, 64, 64, False, 83)
    lut = bsa.build_lut(torch.ones(1, 2, 2, dtype=torch.int32), 1)

    def f(q=q, k=k, v=v, lam=lam, lut=lut, block=64, **kw):
        return bsa.diff_forward(q, k, v, lam, lut, 0.1, block, True, **kw)

    for bad in (dict(q=q[:, :3]), dict(q=q.float()), dict(q=q.cpu()), dict(k=k.transpose(2, 3)), dict(v=v[:, :, :64]),
                dict(lam=lam.double()), dict(lam=lam[:1]), dict(lam=lam.view(1, 2)), dict(q=q[0]),
                dict(out=torch.empty(1, 2, 128, 64, device="cuda")), dict(lse=torch.empty(1, 2, 128, device="cuda"))):
        with pytest.raises(ValueError):
            f(**bad)
    with pytest.raises(bsa.BsaError):
        f(block=128)  # the layout has two blocks
    with pytest.raises(bsa.BsaError):
        f(lut=bsa.build_lut(torch.ones(2, 2, 2, dtype=torch.int32), 1))
    with pytest.raises(bsa.BsaError):
        f(lut=bsa.build_lut(torch.ones(1, 2, 2, dtype=torch.int32), 2))
    with pytest.raises(bsa.BsaError):
        f(lut=bsa.build_lut(torch.ones(1, 2, 2, dtype=torch.int32), 1, upload=False))
    out, lse, out2 = f(training=True)
    with pytest.raises(bsa.BsaError):
        bsa.diff_backward(q, k, v, lam, out, out2, lse, do, lut, 0.1, 64, True,
                          workspace=torch.empty(1024, dtype=torch.uint8, device="cuda"))

"""The table of rotary frequencies (host only) against exact arithmetic, and the argument checks of
bsa_rotary, which come back before any device work."""

import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest

import block_sparse_head_gb300 as bsa
from block_sparse_head_gb300 import binding

A = 1 << 20
# 2 pi to 60 digits
TWO_PI = Fraction("6.28318530717958647692528676655900576839433879875021164194989")


@pytest.fixture(scope="module")
def lib():
    return bsa.load_library()


def _table(lib, f, axis=None):
    f = np.asarray(f, np.float64)
    out = np.zeros((f.size, 2), np.uint64)
    a = None if axis is None else np.asarray(axis, np.int32)
    status = lib.bsa_rotary_table(f.ctypes.data, None if a is None else a.ctypes.data, f.size, out.ctypes.data)
    return status, out


def test_table_is_the_fraction_of_a_turn(lib):
    """Within three roundings to 53 bits: of 2 pi, of the quotient and of its fraction (2^-52 of the
    quotient), and the last place of the 64-bit fraction."""
    f = [0.0, 1.0, -1.0, 2 * math.pi, math.pi, -math.pi, 1e6, -1e6, 123.456, 1e-9] + \
        [10000.0 ** (-i / 64) for i in range(64)]
    status, out = _table(lib, f)
    assert status == 0 and np.all(out[:, 1] == 0)
    for x, t in zip(f, out[:, 0]):
        off = (Fraction(int(t), 2 ** 64) - Fraction(x) / TWO_PI) % 1
        off = min(off, 1 - off)
        assert off <= abs(Fraction(x) / TWO_PI) / 2 ** 51 + Fraction(1, 2 ** 62), x


def test_table_is_within_a_place_of_its_64_bits(lib):
    """The largest frequencies too, whose turns have 18 bits before the point: two roundings to 2^-64,
    half a place each, and the second double's own (2^-53 of 2^-36 turns, 2^-106 of 2 pi: nothing)."""
    r = np.random.default_rng(3)
    f = [1e6, -1e6, 999999.9, 123456.789, 1e3, 1.0, -1.0, math.pi, -3 * math.pi, 1e5 * math.pi, 5e-324, 1e-30, 0.0,
         -0.0] + (10.0 ** r.uniform(-12, 6, 500) * r.choice([-1, 1], 500)).tolist() + \
        [10000.0 ** (-i / 64) for i in range(64)]
    for at in range(0, len(f), 128):
        status, out = _table(lib, f[at:at + 128])
        assert status == 0
        for x, t in zip(f[at:], out[:, 0]):
            off = (Fraction(int(t), 2 ** 64) - Fraction(x) / TWO_PI) % 1
            assert min(off, 1 - off) <= Fraction(1, 2 ** 64) + Fraction(1, 2 ** 80), x


def test_table_axes_and_refusals(lib):
    status, out = _table(lib, [1.0, 0.5, 0.25], [2, 0, 7])
    assert status == 0
    assert (out[:, 1] & 0xFFFFFFFF).tolist() == [2, 0, 7] and np.all(out[:, 1] >> 32 == 0)
    assert _table(lib, [1.0], [8])[0] == -2 and _table(lib, [1.0], [-1])[0] == -2
    for bad in (math.inf, math.nan, 1.1e6, -2e6):
        assert _table(lib, [0.5, bad])[0] == -6
    assert _table(lib, np.ones(129))[0] == -2
    x = np.ones(2)
    assert lib.bsa_rotary_table(None, None, 2, x.ctypes.data) == -1
    assert lib.bsa_rotary_table(x.ctypes.data, None, 2, None) == -1
    assert lib.bsa_rotary_table(x.ctypes.data, None, 0, x.ctypes.data) == -2


def test_arguments(lib):
    names = ["q", "qo", "H", "qb", "qh", "qt", "qob", "qoh", "qot", "k", "ko", "Hk", "kb", "kh", "kt", "kob", "koh",
             "kot", "pos", "pa", "pb", "table", "pairs", "axes", "pairing", "inverse", "B", "L", "d", "dtype"]
    good = dict(zip(names, [A, A + 4096, 4, 512, 128, 64, 512, 128, 64, A, A + 4096, 2, 512, 128, 64, 512, 128, 64, A, 8,
                            0, A, 32, 1, 0, 0, 1, 8, 64, 0]))

    def f(**kw):
        return lib.bsa_rotary(binding._ROTARY_ARGS.pack(*{**good, **kw}.values()), None)

    for n in ("q", "qo", "k", "ko", "pos", "table"):
        assert f(**{n: 0}) == -1, n
    for n in ("q", "qo", "k", "ko", "table"):
        assert f(**{n: A + 8}) == -5, n
    assert f(pos=A + 2) == -5
    for n in ("qb", "qh", "qt", "qob", "qoh", "qot", "kb", "kh", "kt", "kob", "koh", "kot"):
        assert f(**{n: 68}) == -5, n
    for kw, want in [(dict(d=0), -2), (dict(d=60), -2), (dict(d=264), -2), (dict(pairs=0), -2), (dict(pairs=33), -2),
                     (dict(axes=0), -2), (dict(axes=9), -2), (dict(B=-1), -2), (dict(L=-1), -2), (dict(L=1 << 30), -2),
                     (dict(H=-1), -2), (dict(Hk=65536), -2), (dict(dtype=2), -4), (dict(pairing=2), -6),
                     (dict(qo=A, qoh=256), -6), (dict(ko=A, kot=128), -6)]:
        assert f(**kw) == want, kw
    assert lib.bsa_rotary(None, None) == -1
    # nothing to do: no device is asked for
    assert f(L=0) == 0 and f(B=0) == 0 and f(H=0, Hk=0) == 0 and f(H=0, q=0, qo=0, L=0) == 0


def test_outputs_that_share_places_are_refused(lib):
    """Queries that are the keys too, turned in place (twice, or read after the turn), and outputs
    whose rows are one row."""
    names = ["q", "qo", "H", "qb", "qh", "qt", "qob", "qoh", "qot", "k", "ko", "Hk", "kb", "kh", "kt", "kob", "koh",
             "kot", "pos", "pa", "pb", "table", "pairs", "axes", "pairing", "inverse", "B", "L", "d", "dtype"]
    C, D, E = A + 4096, A + 8192, A + 12288
    good = dict(zip(names, [A, C, 4, 4096, 512, 64, 4096, 512, 64, D, E, 2, 4096, 512, 64, 4096, 512, 64, A, 8,
                            0, A, 32, 1, 0, 0, 2, 8, 64, 0]))

    def f(**kw):
        return lib.bsa_rotary(binding._ROTARY_ARGS.pack(*{**good, **kw}.values()), None)

    for kw in (dict(q=D, qo=D, ko=D), dict(ko=C), dict(k=A, qo=A), dict(q=D, ko=D), dict(qob=0), dict(qoh=0), dict(qot=0),
               dict(kob=0), dict(koh=0), dict(kot=0)):
        assert f(**kw) == -6, kw


def test_strides_of_dimensions_of_one_are_not_compared(lib):
    """In place, queries of one batch entry, head or token whose unused strides differ between input and
    output: the check goes on to the keys, which have no pointer here.  With two of them it ends at the
    queries."""
    names = ["q", "qo", "H", "qb", "qh", "qt", "qob", "qoh", "qot", "k", "ko", "Hk", "kb", "kh", "kt", "kob", "koh",
             "kot", "pos", "pa", "pb", "table", "pairs", "axes", "pairing", "inverse", "B", "L", "d", "dtype"]
    good = dict(zip(names, [A, A, 2, 4096, 512, 64, 4096, 512, 64, 0, 0, 2, 4096, 512, 64, 4096, 512, 64, A, 8,
                            0, A, 32, 1, 0, 0, 2, 2, 64, 0]))

    def f(**kw):
        return lib.bsa_rotary(binding._ROTARY_ARGS.pack(*{**good, **kw}.values()), None)

    assert f() == -1
    for size, stride in (("B", "qob"), ("H", "qoh"), ("L", "qot")):
        for other in (8192, 0):
            assert f(**{stride: other}) == -6, stride
            assert f(**{size: 1, stride: other}) == -1, stride

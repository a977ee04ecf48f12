"""Argument checks of the differential-attention calls: they come back before any device work,
so they are tested without a GPU (fake, aligned pointers that are never dereferenced)."""

import ctypes

import pytest
import torch

import block_sparse_head_gb300 as bsa

A = 1 << 20


@pytest.fixture(scope="module")
def lib():
    return bsa.load_library()


@pytest.fixture(scope="module")
def lut():
    return bsa.build_lut(torch.ones(2, 3, 3, dtype=torch.int32), 2, upload=False)


SIZES = (("B", 2), ("H", 4), ("kv", 2), ("L", 150), ("d", 128), ("dq", 128), ("rows", 0))
ERRORS = [(dict(block=32), -6), (dict(block=0), -6), (dict(d=96), -6), (dict(d=256), -6), (dict(dq=32), -6),
          (dict(d=64, dq=32), -6), (dict(d=64, dq=128), -6), (dict(scale=float("nan")), -6),
          (dict(scale=float("inf")), -6), (dict(scale=3e38), -6), (dict(B=0), -2), (dict(B=1), -2), (dict(H=0), -2),
          (dict(H=3), -2), (dict(kv=1), -2), (dict(kv=0), -2), (dict(L=0), -2), (dict(L=128), -2), (dict(L=193), -2),
          (dict(L=-5), -2), (dict(block=128), -2), (dict(H=1 << 30), -2), (dict(), -9)]


def test_forward(lib, lut):
    names = ("q", "k", "v", "lam", "lut", "out", "lse", "out2")

    def f(**kw):
        ptrs = [kw.get(n, lut.handle if n == "lut" else A) for n in names]
        return lib.bsa_diff_forward(*ptrs, *(kw.get(n, x) for n, x in SIZES), kw.get("scale", 0.1),
                                    kw.get("block", 64), 1, None)

    for n in names[:7]:
        assert f(**{n: None}) == -1, n
    for n in ("q", "k", "v", "out", "out2"):
        assert f(**{n: A + 8}) == -5, n
    for n in ("lam", "lse"):
        assert f(**{n: A + 2}) == -5, n
    for kw, want in ERRORS:
        assert f(**kw) == want, kw
    rect = bsa.build_lut(torch.ones(2, 3, 4, dtype=torch.int32), 2, upload=False)
    assert f(lut=rect.handle) == -2


def test_backward(lib, lut):
    names = ("q", "k", "v", "lam", "out", "out2", "lse", "dout", "lut", "dq_out", "dk", "dv", "dlam", "ws")

    def f(**kw):
        ptrs = [kw.get(n, lut.handle if n == "lut" else A) for n in names]
        return lib.bsa_diff_backward(*ptrs, kw.get("bytes", 1 << 40), *(kw.get(n, x) for n, x in SIZES),
                                     kw.get("scale", 0.1), kw.get("block", 64), 1, None)

    for n in names:
        assert f(**{n: None}) == -1, n
    for n in ("q", "k", "v", "out", "out2", "dout", "dq_out", "dk", "dv", "ws"):
        assert f(**{n: A + 8}) == -5, n
    for n in ("lam", "lse", "dlam"):
        assert f(**{n: A + 2}) == -5, n
    for kw, want in ERRORS:
        assert f(**kw) == want, kw


def test_workspace(lib):
    n = ctypes.c_int64()
    assert lib.bsa_diff_workspace(1, 1, 1, 64, 64, None) == -1
    for bad in ((0, 1, 1), (1, 0, 1), (1, 1, 0), (1 << 15, 1 << 15, 1 << 10), (1, 1, 1 << 30)):
        assert lib.bsa_diff_workspace(*bad, 64, 64, ctypes.byref(n)) == -2
    for bad in ((96, 64), (64, 32)):
        assert lib.bsa_diff_workspace(1, 1, 1, *bad, ctypes.byref(n)) == -6


def test_cache_forward(lib):
    from block_sparse_head_gb300 import binding

    names = ("q", "lam", "table", "kv_len", "cu_q", "out", "lse", "status", "ws")

    def f(**kw):
        cache = binding._CACHE.pack(A, A, A, A, 64, kw.get("kv", 2), 64, kw.get("d", 128), 2)
        ptrs = [kw.get(n, A) for n in names]
        sizes = [kw.get(n, x) for n, x in (("B", 2), ("max_pages", 4), ("T", 2), ("heads", 4), ("dq", 128), ("max_q", 1),
                                           ("rows", 0), ("dtype", 0))]
        return lib.bsa_cache_diff_forward(cache, *ptrs, kw.get("bytes", 1 << 30), *sizes, 256, 256,
                                          kw.get("scale", 0.1), None, None)

    for n in names:
        if n != "status":
            assert f(**{n: None}) == -1, n
    for n in ("q", "out", "ws"):
        assert f(**{n: A + 8}) == -5, n
    for n in ("lam", "lse", "status", "table"):
        assert f(**{n: A + 2}) == -5, n
    for kw, want in [(dict(dq=32), -6), (dict(dq=256), -6), (dict(d=64, dq=32), -6), (dict(d=64), -6), (dict(heads=3), -2),
                     (dict(heads=0), -2), (dict(heads=-4), -2), (dict(heads=130, kv=2), -2), (dict(heads=1 << 30), -2),
                     (dict(dtype=2), -4), (dict(T=-1), -2), (dict(B=0), -2), (dict(max_q=0), -2),
                     (dict(scale=float("inf")), -6)]:
        assert f(**kw) == want, kw

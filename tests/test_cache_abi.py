"""Argument checks of the cache calls: they come back before any device work, so they are
tested without a GPU (fake, aligned pointers that are never dereferenced)."""

import ctypes

import numpy as np
import pytest
import torch

import block_sparse_head_gb300 as bsa
from block_sparse_head_gb300 import binding

A = 1 << 20


@pytest.fixture(scope="module")
def lib():
    return bsa.load_library()


def _cache(**kw):
    return binding._CACHE.pack(*(0 if x is None else x for x in _fields(kw)))


def _fields(kw):
    return (kw.get("k", A), kw.get("v", A), kw.get("k_scale", A), kw.get("v_scale", A),
                         kw.get("n_pages", 64), kw.get("kv_heads", 2), kw.get("page", 64),
                         kw.get("d", 128), kw.get("cache_dtype", 2))


CACHE_ERRORS = [(dict(k=None), -1), (dict(v=None), -1), (dict(k_scale=None), -1), (dict(v_scale=None), -1),
                (dict(page=8), -6), (dict(page=48), -6), (dict(page=256), -6), (dict(page=0), -6),
                (dict(d=96), -6), (dict(d=256), -6), (dict(cache_dtype=0), -4), (dict(cache_dtype=4), -4),
                (dict(n_pages=0), -2), (dict(kv_heads=0), -2), (dict(n_pages=1 << 25), -2),
                (dict(k=A + 8), -5), (dict(v=A + 4), -5), (dict(k_scale=A + 2), -5)]


def test_resize(lib):
    names = ("table", "kv_len", "new_len", "free", "count", "len_out", "count_out", "cu", "slots", "status")

    def f(**kw):
        return lib.bsa_cache_resize(*(kw.get(n, A) for n in names), kw.get("B", 4), kw.get("max_pages", 8),
                                    kw.get("n_pages", 64), kw.get("page", 64), kw.get("tokens", 128), None)

    for n in names:
        assert f(**{n: None}) == -1, n
        assert f(**{n: A + 2}) == -5, n
    assert f(page=8) == -6 and f(page=33) == -6 and f(page=256) == -6
    assert f(B=0) == -2 and f(B=8193) == -2 and f(max_pages=0) == -2 and f(n_pages=0) == -2
    assert f(tokens=-1) == -2 and f(max_pages=1 << 25) == -2 and f(n_pages=1 << 25) == -2


def test_append(lib):
    def f(**kw):
        c = _cache(**{n: kw[n] for n in kw if n in ("k", "v", "k_scale", "v_scale", "n_pages", "kv_heads",
                                                    "page", "d", "cache_dtype")})
        strides = [kw.get(n, 256) for n in ("kt", "kh", "vt", "vh")]
        return lib.bsa_cache_append(c, kw.get("xk", A), kw.get("xv", A), kw.get("slots", A),
                                    kw.get("T", 5), kw.get("dtype", 0), *strides, None)

    for kw, status in CACHE_ERRORS:
        assert f(**kw) == status, kw
    for n in ("xk", "xv", "slots"):
        assert f(**{n: None}) == -1, n
    assert f(xk=A + 8) == -5 and f(xv=A + 2) == -5 and f(slots=A + 2) == -5
    for n in ("kt", "kh", "vt", "vh"):
        assert f(**{n: 252}) == -5, n
    assert f(dtype=2) == -4 and f(dtype=-1) == -4 and f(T=-1) == -2
    assert f(T=0, xk=None, xv=None, slots=None) == 0  # nothing to do
    assert lib.bsa_cache_append(None, A, A, A, 5, 0, 256, 256, 256, 256, None) == -1


def test_forward(lib):
    lut = bsa.build_lut(np.ones((2, 8, 8), np.int32), 1, upload=False)
    need = ctypes.c_int64()
    # the size depends on the device, which is not there: any large one passes the check
    big = 1 << 40

    def f(**kw):
        c = _cache(**{n: kw[n] for n in kw if n in ("k", "v", "k_scale", "v_scale", "n_pages", "kv_heads",
                                                    "page", "d", "cache_dtype")})
        x = binding._CACHE_ARGS.pack(kw.get("window", -1), kw.get("softcap", 0.0), kw.get("sinks", 0),
                                     kw["lut"].value if "lut" in kw else 0, kw.get("block", 64))
        ptrs = [kw.get(n, A) for n in ("q", "table", "kv_len", "cu_q", "out", "lse", "status", "workspace")]
        return lib.bsa_cache_forward(c, *ptrs, big, kw.get("B", 3), kw.get("max_pages", 8),
                                     kw.get("T", 9), kw.get("heads", 8), kw.get("max_q", 4), kw.get("dtype", 0),
                                     kw.get("qt", 1024), kw.get("qh", 128),
                                     ctypes.c_float(kw.get("scale", 0.1)), x, None)

    for kw, status in CACHE_ERRORS:
        assert f(**kw) == status, kw
    for n in ("q", "table", "kv_len", "cu_q", "out", "lse", "workspace"):
        assert f(**{n: None}) == -1, n
    assert f(status=None, T=-1) == -2       # may be left out
    for n in ("q", "out", "workspace"):
        assert f(**{n: A + 8}) == -5, n
    for n in ("table", "kv_len", "cu_q", "lse", "status", "sinks"):
        assert f(**{n: A + 2}) == -5, n
    assert f(qt=1020) == -5 and f(qh=4) == -5
    assert f(dtype=3) == -4
    assert f(B=0) == -2 and f(T=-1) == -2 and f(max_pages=0) == -2 and f(max_q=0) == -2
    assert f(max_pages=(1 << 23) + 1) == -2 and f(T=(1 << 29) + 1) == -2    # positions past 2^29
    assert f(B=1 << 30, kv_heads=4) == -2
    assert f(heads=7) == -2 and f(heads=0) == -2 and f(heads=258) == -2 and f(max_pages=1 << 25) == -2
    assert f(scale=3e38) == -6 and f(softcap=3e38) == -6 and f(scale=1e20, softcap=1e-30) == -6
    assert f(scale=float("nan")) == -6 and f(softcap=-1.0) == -6 and f(softcap=float("inf")) == -6
    assert f(lut=lut.handle, block=32) == -6
    assert f(lut=lut.handle, max_pages=9) == -2          # the block table outgrows the layout
    assert f(lut=lut.handle, kv_heads=4) == -2           # one layout row for each kv head
    assert f(lut=lut.handle) == -9                       # never uploaded
    assert lib.bsa_cache_workspace(8, 2, 96, 1, ctypes.byref(need)) == -6
    assert lib.bsa_cache_workspace(8, 3, 128, 1, ctypes.byref(need)) == -2
    assert lib.bsa_cache_workspace(8, 2, 128, 0, ctypes.byref(need)) == -2
    assert lib.bsa_cache_workspace(8, 2, 128, 1, None) == -1


def test_binding_refuses_host_tensors():
    """The binding's own checks, before the library is called."""
    kc = torch.zeros(4, 2, 16, 64, dtype=torch.int8)
    sc = torch.ones(4, 2)
    i = torch.zeros(3, dtype=torch.int32)
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="k_cache"):
        bsa.cache_append(x, x, i, kc, kc, sc, sc)
    with pytest.raises(ValueError, match="k_cache"):
        bsa.cache_append(x, x, i, kc.float(), kc, sc, sc)
    with pytest.raises(ValueError, match="k_cache"):
        bsa.cache_forward(x, kc, kc, sc, sc, i[None], i[:1], i[:2], 1.0)
    with pytest.raises(ValueError, match="block_table"):
        bsa.cache_resize(i, i, i, i, i[:1], 16, 4)

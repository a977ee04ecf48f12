"""Limits of the cache calls' packed tokens (2^29): larger calls, whose 32-bit indexes would wrap
around, come back before any device work.  CPU only: fake pointers, never dereferenced."""

import pytest

import block_sparse_head_gb300 as bsa
from block_sparse_head_gb300 import binding

A = 1 << 20
SHAPE = -2
TOO_MANY = [(1 << 29) + 1, 2 ** 31 - 200_001, 2 ** 31 - 1]


@pytest.fixture(scope="module")
def lib():
    return bsa.load_library()


@pytest.mark.parametrize("tokens", TOO_MANY)
def test_resize_tokens(lib, tokens):
    assert lib.bsa_cache_resize(*[A] * 10, 4, 8, 64, 64, tokens, None) == SHAPE


@pytest.mark.parametrize("T", TOO_MANY)
def test_append_tokens(lib, T):
    cache = binding._CACHE.pack(A, A, A, A, 64, 2, 64, 128, 2)
    assert lib.bsa_cache_append(cache, A, A, A, T, 0, 256, 128, 256, 128, None) == SHAPE

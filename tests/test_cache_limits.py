"""Limits of the cache calls' packed tokens (2^29): larger calls, whose 32-bit indexes would wrap
around, come back before any device work.  CPU only: fake pointers, never dereferenced."""

import pytest

import block_sparse_head_gb300 as bsa

A = 1 << 20
SHAPE = -2
TOO_MANY = [(1 << 29) + 1, 2 ** 31 - 200_001, 2 ** 31 - 1]


@pytest.fixture(scope="module")
def lib():
    return bsa.load_library()


@pytest.mark.parametrize("tokens", TOO_MANY)
def test_resize_tokens(lib, tokens):
    assert lib.bsa_cache_resize(*[A] * 10, 4, 8, 64, 64, tokens, None) == SHAPE

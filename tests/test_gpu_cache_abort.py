"""The failure path of the cache's attention kernels, driven without a fault or a hang: waits at
one site, or one role, give up at once (``Lut.debug_expire_wait``), the call records a site in its
status word and every role of every CTA returns; the next call, with a zeroed workspace and the
knob off, gives the same bits as before."""

import math
import time

import numpy as np
import pytest
import torch

import block_sparse_head_gb300 as bsa

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    return cuda_lib


class Call:
    """Requests of `lens` tokens each, `n` queries each; the layout lists every block for the rows
    of the queries."""

    def __init__(self, lens, n, G, H, d, page=128):
        g = torch.Generator(device="cuda").manual_seed(d + G + n)
        held = [-(-x // page) for x in lens]
        P = sum(held)
        self.kc, self.vc = (torch.randint(-90, 91, (P, H, page, d), generator=g, device="cuda", dtype=torch.int8)
                            for _ in range(2))
        self.ks, self.vs = torch.full((2, P, H), 2.0 ** -6, device="cuda").unbind(0)
        self.table = torch.full((len(lens), max(held)), -1, **I32)
        at = 0
        for b, k in enumerate(held):
            self.table[b, :k] = torch.arange(at, at + k, **I32)
            at += k
        self.q = torch.randn(n * len(lens), G * H, d, generator=g, device="cuda").to(torch.float16)
        self.lens = torch.tensor(lens, **I32)
        self.cu = torch.arange(0, n * len(lens) + 1, n, **I32)
        nb = max(held) * page // 128
        rows = {(x - i - 1) // 128 for x in lens for i in range(n)}
        layout = np.zeros((H, nb, nb), np.int32)
        layout[:, sorted(rows)] = 1
        self.lut = bsa.build_lut(layout, 1)
        self.n, self.scale = n, 1 / math.sqrt(d)
        self.ws = bsa.cache_workspace(G * H, H, d, n)

    def __call__(self, status=None):
        out, lse, _ = bsa.cache_forward(self.q, self.kc, self.vc, self.ks, self.vs, self.table, self.lens, self.cu,
                                        self.scale, max_q=self.n, lut=self.lut, block=128, workspace=self.ws,
                                        status=status)
        return out, lse

    def check_site(self, site, words=None, ways=2):
        """With `site` given up on, a call's status (and the workspace's, the other way to it) is
        one of `words` (0x10000 | site)."""
        words = words or [0x10000 | site]
        ref = self()
        assert bsa.cache_status(self.ws) == 0
        assert torch.all(torch.isfinite(ref[0])) and torch.all(torch.isfinite(ref[1]))
        self.lut.debug_expire_wait(site)
        try:
            status = torch.full((1,), -1, **I32)
            self(status)
            assert int(status[0]) in words, hex(int(status[0]))
            self.ws.zero_()
            if ways == 2:
                self()
            assert ways == 1 or bsa.cache_status(self.ws) in words, hex(bsa.cache_status(self.ws))
        finally:
            self.lut.debug_expire_wait(0)
        self.ws.zero_()
        got = self()
        assert bsa.cache_status(self.ws) == 0
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


@pytest.mark.parametrize("G,d", [(8, 128), (16, 128), (4, 64), (9, 64)])
def test_decode_producer_gives_up(G, d):
    """One request and kv head over all CTAs, each with more stages of 256 keys than its ring
    holds (3 of d = 128, 6 of 64): none comes to the end of a segment before the wait."""
    Call([1 << 19], 1, G, 1, d).check_site(1)


@pytest.mark.parametrize("site", [6, 16])
@pytest.mark.parametrize("G,n,d", [(4, 1, 128), (4, 4, 128), (9, 1, 64)])
def test_decode_wait_gives_up(G, n, d, site):
    """Whole and cut units, several segments a CTA: consumers that wait for a stage, and that meet
    in a join."""
    Call([3000, 130, 9000, 257] * 8, n, G, 4, d).check_site(site)


@pytest.mark.parametrize("d", [128, 64])
def test_decode_copier_gives_up(d):
    """The values' copier leaves; the producer's wait for its own copies has one limit for all stages
    (4 s), the call returns after it."""
    begin = time.monotonic()
    Call([3000, 130, 9000, 257], 1, 4, 4, d).check_site(2)
    assert time.monotonic() - begin < 14  # two calls that give up


@pytest.mark.parametrize("G,H,d", [(4, 4, 128), (1, 3, 64)])
@pytest.mark.parametrize("site,others", [(6, [1, 2, 7, 9]), (7, [1, 2, 6, 8, 9, 11, 12]), (17, [17])])
def test_tile_role_is_missing(G, H, d, site, others):
    """The kernel for many rows with one role gone: products of the scores, of the values, or the
    look-ups.  All that wait for it run out of tries (four seconds), with products in flight and
    weights being written; whole and cut units."""
    begin = time.monotonic()
    Call([6000, 300, 20000, 1290], 200, G, H, d).check_site(site, [0x10000 | x for x in others], ways=1)
    assert time.monotonic() - begin < 20

"""Keys of the paged 8-bit cache that weigh little beside others of their row: they have to
count in the output as the formula says, because they may be all there is of it.

Bound of an output element (d = 128, n keys), all from the formula's fp64 values:
  * scores off by (d + 16) 2^-24 max|s| (fp32 sum of exact products) and base-2 exponent and
    logarithm by 2^-20, together delta; twice that on a weight (numerator and normaliser), and
    2^-11 for its rounding to fp16 and n 2^-23 for the fp32 sums, acting on sum w|v|;
  * a weight that is subnormal in fp16 is off by 2^-25 in units in which the row's largest
    weight times V scale (`top`) is at least 2^7: by 2^-32 top, times |stored value|, summed;
  * the output rounded once: eps / 2 |out|.
"""

import math

import numpy as np
import pytest
import torch

from oracle import bsa_oracle_cache as oc
from test_gpu_cache import Case, TYPES

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    return cuda_lib


def _formula(c, scale):
    """out, lse, sum w|v|, size, and top * sum |stored value|, of a case with one request."""
    d, n = c.d, c.news[0]
    L = c.lens[0]
    pos = np.arange(L)
    ids, at = c.table[0, pos // c.page], pos % c.page
    stored = [x.float().double().cpu().numpy()[ids, :, at] for x in (c.kc, c.vc)]      # [L, H, d]
    ks, vs = (x.double().cpu().numpy()[ids] for x in (c.ks, c.vs))                     # [L, H]
    q = c.q[:n].double().cpu().numpy()
    Hq = q.shape[1]
    G = Hq // c.H
    out, weight, small = (np.zeros((n, Hq, d)) for _ in range(3))
    lse, size = np.zeros((n, Hq)), np.zeros((n, Hq))
    for h in range(Hq):
        g = h // G
        k, v8 = stored[0][:, g] * ks[:, g, None], stored[1][:, g]
        s = scale * q[:, h] @ k.T
        s[pos[None] > (L - n + np.arange(n))[:, None]] = -np.inf
        top = s.max(1, keepdims=True)
        lse[:, h] = top[:, 0] + np.log(np.exp(s - top).sum(1))
        w = np.exp(s - lse[:, h, None])
        wv = w * vs[None, :, g]
        out[:, h], weight[:, h] = wv @ v8, wv @ np.abs(v8)
        small[:, h] = wv.max(1, keepdims=True) * ((w > 0).astype(float) @ np.abs(v8))
        size[:, h] = (scale * np.abs(q[:, h]) @ np.abs(k).T).max(1)
    return out, lse, weight, size, small


def _check(c):
    n, scale = c.news[0], 1 / math.sqrt(c.d)
    out, lse = (x[:n].double().cpu().numpy() for x in c.run(scale))
    ro, rl, weight, size, small = _formula(c, scale)
    keys = c.lens[0]
    delta = (c.d + 16) * 2.0 ** -24 * size + 2.0 ** -20
    tol = (torch.finfo(TYPES[c.dtype]).eps / 2 * np.abs(ro)
           + (2.0 ** -11 + 2 * delta[..., None] + keys * 2.0 ** -23) * weight + 2.0 ** -32 * small)
    # From 65520, half a step past the largest number 65504 = 2047 * 2^5, fp16 rounds to infinity.
    past = (np.abs(ro) - tol >= 65520.0) if c.dtype == "fp16" else np.zeros(ro.shape, bool)
    assert np.all(out[past] == np.sign(ro[past]) * np.inf)
    bad = ~past & (np.abs(out - ro) > tol)
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[0], out[bad][0], ro[bad][0], tol[bad][0])
    assert np.all(np.abs(lse - rl) <= delta + keys * 2.0 ** -24 + 2.0 ** -22 * (1 + np.abs(rl)))


CASES = [(1, 4, 1, "e4m3", "bf16"), (4, 4, 1, "int8", "fp16"), (40, 4, 1, "e4m3", "fp16"),
         (1, 4, 2, "int8", "bf16"), (130, 1, 1, "int8", "bf16"), (1, 128, 1, "e4m3", "fp16")]


@pytest.mark.parametrize("n,G,H,kind,dtype", CASES)
@pytest.mark.parametrize("bits", [20, 24, 27])
def test_dominant_key_without_values(n, G, H, kind, dtype, bits):
    """The first key (a model's attention sink) leads every other by 2^bits and has no values:
    the outputs are those of the long tail behind it."""
    c = Case([2500], [n], G, H, 128, 64, kind, dtype, seed=bits)
    T = c.q.shape[0]
    g = torch.Generator().manual_seed(1)
    c.q = (1 + 0.1 * torch.randn(T, G * H, 128, generator=g)).to(TYPES[dtype]).cuda()
    page = int(c.table[0, 0])
    top = 64 if kind == "int8" else 0x68  # 64 in e4m3
    c.kc.view(torch.uint8)[page] = 0
    c.kc.view(torch.uint8)[page, :, 0] = top
    c.vc.view(torch.uint8)[page, :, 0] = 0
    # 64 ks sum(q) / sqrt(d), sum(q) about 128, is the lead over scores about 0
    c.ks[page] = bits * math.log(2) * math.sqrt(128) / (64 * 128)
    c.ks[torch.as_tensor(c.table[0, 1:])] *= 0.3
    _check(c)


@pytest.mark.parametrize("n,G,H,kind,dtype", CASES)
@pytest.mark.parametrize("bits", [20, 24])
def test_one_large_value_scale(n, G, H, kind, dtype, bits):
    """One page holds an outlier: its V scale is 2^bits of the others', its values zero but for
    one column of one token.  The other columns are those of all other pages."""
    c = Case([1500], [n], G, H, 128, 64, kind, dtype, seed=bits + 1)
    page = int(c.table[0, 5])
    c.vc.view(torch.uint8)[page] = 0
    c.vc.view(torch.uint8)[page, :, 7, 9] = 127 if kind == "int8" else 0x7E  # the largest number
    c.vs[page] *= 2.0 ** bits
    _check(c)

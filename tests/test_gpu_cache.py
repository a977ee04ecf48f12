"""GPU parity of the paged 8-bit cache (bsa_cache_resize, bsa_cache_append,
bsa_cache_forward) against the fp64 oracle.

resize and append are compared exactly: whole numbers, and stored numbers that are one
rounding of an exact quotient.

Bounds of the forward, from its roundings (n keys, head dim d; the oracle returns
weight = sum w|v| and size = max |scale| k_scale sum |q k| of each row):
  * a score is an fp32 sum of d exact products, then a few fp32 products: off by at most
    (d + 16) 2^-24 size; the soft-cap's tanh adds 2^-20 cap, base-2 exponent and logarithm
    (ex2/lg2 approximations) 2^-20.  Call the sum delta.
  * a weight is then off by 2 delta relative (numerator and normaliser), by 2^-11 for its
    rounding to fp16 and by n 2^-23 for the fp32 sums, all acting on `weight`; weights so
    small that they are subnormal in fp16 are off by 2^-25 of the largest, together at most
    n 2^-25 largest max(v_scale);
  * the output is rounded once: eps / 2 |out|.
  * lse is off by delta + n 2^-24 + 2^-22 (1 + |lse|).
"""

import math

import numpy as np
import pytest
import torch

import block_sparse_head_gb300 as bsa
from oracle import bsa_oracle_cache as oc

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
CACHE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
I32 = dict(dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    return cuda_lib


def ints(x):
    return torch.as_tensor(np.asarray(x, np.int32), device="cuda")


# ------------------------------------------------------------------------------ resize

def _resize(table, lens, new, free, count, page, tokens, in_place):
    t, l, f, c = ints(table), ints(lens), ints(free), ints([count])
    lo, co = (l, c) if in_place else (torch.full_like(l, -7), torch.full_like(c, -7))
    cu, slots, status = bsa.cache_resize(t, l, ints(new), f, c, page, tokens, kv_len_out=lo, free_count_out=co)
    return t, lo, f, co, cu, slots, status


def _check_resize(got, ref):
    table, lens, free, count, cu, slots, status = ref
    for name, g, r in zip(("table", "lens", "free", "count", "cu", "slots", "status"), got,
                          (table, lens, free, [count], cu, slots, [status])):
        assert np.array_equal(g.cpu().numpy(), np.asarray(r)), name


@pytest.mark.parametrize("B,width,page", [(1, 3, 16), (7, 5, 32), (33, 9, 64), (1000, 4, 128), (1025, 3, 16),
                                          (8192, 2, 16)])
@pytest.mark.parametrize("in_place", [True, False])
def test_resize_random(B, width, page, in_place):
    """Growing, shrinking, ending and idle requests in one call, several calls in a row."""
    rng = np.random.default_rng(B + page)
    pages = B * width + 5
    table, lens = np.full((B, width), -1), np.zeros(B, int)
    free, count = rng.permutation(pages), pages
    for step in range(3):
        new = np.where(rng.random(B) < 0.6, rng.integers(0, width * page + 1, B), lens)
        new = np.where(rng.random(B) < 0.2, 0, new)
        tokens = int(np.maximum(new - lens, 0).sum()) + step
        ref = oc.resize(table, lens, new, free, count, page, tokens)
        assert ref[-1] == 0
        _check_resize(_resize(table, lens, new, free, count, page, tokens, in_place), ref)
        table, lens, free, count = ref[:4]


@pytest.mark.parametrize("in_place", [True, False])
def test_resize_refusals_change_nothing(in_place):
    table, free = np.arange(6).reshape(2, 3), np.arange(10, 20)
    cases = [([5, 5], [48, 33], 1, 128),       # pages are missing
             ([5, 5], [49, 6], 9, 128),        # a length over max_pages * page
             ([5, -2], [6, 6], 9, 128),        # an old length below 0
             ([5, 5], [6, -1], 9, 128),
             ([5, 5], [40, 40], 9, 69),        # one token more than the capacity
             ([5, 5], [6, 6], -1, 128), ([5, 5], [6, 6], 11, 128),  # a count that cannot be
             ([48, 48], [0, 0], 5, 128)]       # more pages given back than there are
    for lens, new, count, tokens in cases:
        ref = oc.resize(table, lens, new, free, count, 16, tokens)
        assert ref[-1] != 0
        _check_resize(_resize(table, lens, new, free, count, 16, tokens, in_place), ref)


def test_resize_no_tokens():
    """A call that only gives pages back, with no room for tokens."""
    table, free = np.arange(6).reshape(2, 3), np.full(10, -1)
    ref = oc.resize(table, [40, 17], [1, 0], free, 0, 16, 0)
    _check_resize(_resize(table, [40, 17], [1, 0], free, 0, 16, 0, True), ref)


# ------------------------------------------------------------------------------ append

def _stored(cache):
    return cache.float().double().cpu().numpy()


def _empty_cache(P, H, page, d, kind, seed):
    """Random stored numbers and power-of-two scales, as earlier appends leave them."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(P, H, page, d, generator=g) * oc.LARGEST[kind] / 4.2
    x = (x.round() if kind == "int8" else x).clamp(-oc.LARGEST[kind], oc.LARGEST[kind]).to(CACHE[kind])
    s = torch.exp2(torch.randint(-9, -4, (P, H), generator=g).float())
    return x.cuda(), s.cuda()


def _check_append(kind, page, d, H, dtype, runs, seed, spread=1.0, pad=2, mutate=None, copies=1):
    """runs: (page id, first offset, tokens) of each run, in packed order; copies: times that
    the call has every head, for a large call that the oracle does one copy of."""
    P = max(r[0] for r in runs) + 3
    kc, ks = _empty_cache(P, H, page, d, kind, seed)
    vc, vs = _empty_cache(P, H, page, d, kind, seed + 1)
    slots = [pid * page + off + i for pid, off, n in runs for i in range(n)] + [-1] * pad
    T = len(slots)
    g = torch.Generator().manual_seed(seed + 2)
    rows = torch.randn(T, 3 * H, d, generator=g) * torch.exp(spread * torch.randn(T, 1, 1, generator=g))
    rows = rows.to(TYPES[dtype])
    if mutate is not None:
        slots = mutate(rows, slots)
    dev = rows.cuda()
    k, v = dev[:, H: 2 * H], dev[:, 2 * H:]  # strided, as a projection's output is split
    ref = [oc.append(x.double().cpu().numpy(), slots, _stored(c), s.double().cpu().numpy(), kind)
           for x, c, s in ((k, kc, ks), (v, vc, vs))]
    if copies > 1:
        k, v, kc, vc, ks, vs = (x.repeat(*[copies if i == 1 else 1 for i in range(x.dim())])
                                for x in (k, v, kc, vc, ks, vs))
    bsa.cache_append(k, v, ints(slots), kc, vc, ks, vs)
    for (rc, rs), c, s, name in zip(ref, (kc, vc), (ks, vs), "kv"):
        assert np.array_equal(s.double().cpu().numpy(), np.tile(rs, (1, copies))), name
        assert np.array_equal(_stored(c), np.tile(rc, (1, copies, 1, 1)), equal_nan=True), name


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("page,d,H", [(16, 64, 3), (32, 128, 1), (64, 128, 2), (128, 64, 5), (128, 128, 1)])
def test_append_runs(kind, dtype, page, d, H):
    """Whole pages, a page's middle, its last slot, single tokens, a chunk over several
    pages that starts and ends inside one; pages without new tokens keep their bytes."""
    runs = [(5, 0, page), (0, 0, 1), (2, page - 1, 1), (7, 3, page - 7), (1, page // 2, page // 2),
            (9, 0, page), (3, 0, 5), (11, 1, 1)]
    _check_append(kind, page, d, H, dtype, runs, seed=page + d + H)


@pytest.mark.parametrize("page,d,heads,kind,dtype", [
    (16, 64, 8, "e4m3", "bf16"), (32, 128, 8, "int8", "fp16"), (64, 64, 8, "e4m3", "fp16"),
    (128, 64, 8, "int8", "bf16"), (64, 64, 40, "int8", "fp16"), (64, 128, 40, "e4m3", "bf16"),
    (128, 64, 40, "e4m3", "fp16"), (128, 128, 40, "int8", "bf16")])
def test_append_many_rows(page, d, heads, kind, dtype):
    """Calls of thousands of token rows, where a CTA takes 16 or 64 tokens: runs of one and two
    tokens one after the other, long ones across the CTAs' borders, numbers that are not finite."""
    runs = [(i, int(o), 1 + i % 2) for i, o in enumerate(np.random.default_rng(page).integers(0, page - 1, 70))]
    runs += [(70, 0, page), (73, 0, page), (71, 5, page - 5), (72, 0, 3), (74, page // 2, page // 2)]
    runs += [(75 + i, 0, page) for i in range(max(1, 256 // page))] + [(100, 0, 7), (101, page - 2, 2)]

    def mutate(rows, slots):
        rows[3, :, 1] = float("inf")
        rows[150, :, 2] = float("-inf")
        rows[180, :, 3] = float("nan")
        slots[50] = -1
        return slots
    _check_append(kind, page, d, 1, dtype, runs, seed=page + d, pad=5, mutate=mutate, copies=heads)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_append_spread_magnitudes(kind):
    """Scales that grow by many powers of two, all-zero pages, the ends of the range."""
    def mutate(rows, slots):
        rows[0] = 0
        rows[1] *= 1e-6
        rows[2] *= 1e30
        rows[3] = 0
        rows[4] *= 1e-30
        return slots
    _check_append(kind, 16, 64, 2, "bf16", [(0, 0, 1), (1, 0, 1), (2, 0, 1), (3, 4, 1), (4, 0, 1), (5, 8, 8)],
                  seed=3, spread=4.0, mutate=mutate)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_append_infinities_and_nan(kind):
    def mutate(rows, slots):
        rows[0, :, 5] = float("inf")
        rows[1, :, 6] = float("-inf")
        rows[2, :, 7] = float("nan")
        rows[20] = float("inf")          # a run without a finite number
        return slots
    _check_append(kind, 16, 64, 2, "fp16", [(0, 0, 16), (2, 3, 4), (3, 0, 1)], seed=4, mutate=mutate)


def test_append_skips_slots_out_of_range():
    def mutate(rows, slots):
        slots[1] = -5
        slots[2] = 10 ** 6
        slots[20] = 2 ** 31 - 1
        return slots
    _check_append("e4m3", 16, 128, 2, "bf16", [(1, 0, 1), (0, 0, 2), (2, 0, 16), (5, 0, 1), (6, 0, 1)],
                  seed=5, pad=0, mutate=mutate)


def test_append_twice_is_once():
    """The same tokens again change nothing: the scale stays, kept numbers stay."""
    kc, ks = _empty_cache(4, 2, 16, 64, "int8", 1)
    vc, vs = _empty_cache(4, 2, 16, 64, "int8", 2)
    x = torch.randn(9, 2, 64, device="cuda", dtype=torch.float16) * 50
    slots = ints([7, 8, 9, 10, 11, 12, 13, 14, 15])
    bsa.cache_append(x, x, slots, kc, vc, ks, vs)
    first = [t.clone() for t in (kc, vc, ks, vs)]
    bsa.cache_append(x, x, slots, kc, vc, ks, vs)
    assert all(torch.equal(a, b) for a, b in zip(first, (kc, vc, ks, vs)))


# ----------------------------------------------------------------------------- forward

class Case:
    def __init__(self, lens, news, G=4, H=2, d=128, page=64, kind="e4m3", dtype="bf16", seed=0, pad=3,
                 scales="any", vscale_spread=0):
        rng = np.random.default_rng(seed)
        self.kind, self.dtype, self.page, self.d, self.H = kind, dtype, page, d, H
        self.lens, self.news = list(lens), list(news)
        self.cu = np.concatenate([[0], np.cumsum(news)])
        held = [-(-n // page) for n in lens]
        P, width = sum(held) + 4, max(max(held), 1)
        order = rng.permutation(P)
        self.table = np.full((len(lens), width), -1)
        at = 0
        for b, n in enumerate(held):
            self.table[b, :n] = order[at: at + n]
            at += n
        self.kc, _ = _empty_cache(P, H, page, d, kind, seed)
        self.vc, _ = _empty_cache(P, H, page, d, kind, seed + 1)
        base = 4.2 / oc.LARGEST[kind]
        f = (lambda: base * rng.uniform(0.5, 2.0, (P, H))) if scales == "any" else \
            (lambda: 2.0 ** np.round(np.log2(base) + rng.integers(-1, 2, (P, H))))
        self.ks = torch.tensor(f(), dtype=torch.float32).cuda()
        self.vs = torch.tensor(f() * 2.0 ** rng.integers(-vscale_spread, 1, (P, H)), dtype=torch.float32).cuda()
        # what the cache holds behind the lengths, and in pages of nobody, is garbage
        bad = torch.full((d,), 0x7F if kind == "e4m3" else 0x80, dtype=torch.uint8).cuda()
        for b, n in enumerate(lens):
            if n % page:
                for c in (self.kc, self.vc):
                    c.view(torch.uint8)[self.table[b, held[b] - 1], :, n % page:] = bad
        for s in (self.ks, self.vs):
            s[torch.as_tensor(order[at:])] = float("nan")
        g = torch.Generator().manual_seed(seed + 9)
        T = int(self.cu[-1]) + pad
        self.q = (torch.randn(T, G * H, d, generator=g)).to(TYPES[dtype]).cuda()

    def run(self, scale=None, **kw):
        scale = 1 / math.sqrt(self.d) if scale is None else scale
        T, Hq = self.q.shape[:2]
        out = torch.full((T, Hq, self.d), 77.0, dtype=self.q.dtype, device="cuda")
        lse = torch.full((T, Hq), 77.0, device="cuda")
        kw.setdefault("max_q", max(max(self.news), 1))
        kw.setdefault("status", torch.full((1,), -1, **I32))
        _, _, status = bsa.cache_forward(self.q, self.kc, self.vc, self.ks, self.vs, ints(self.table),
                                         ints(self.lens), ints(self.cu), scale, out=out, lse=lse, **kw)
        assert int(status[0]) == 0, hex(int(status[0]))
        return out, lse

    def check(self, scale=None, layout=None, block=64, **kw):
        scale = 1 / math.sqrt(self.d) if scale is None else scale
        lut = None if layout is None else bsa.build_lut(layout, 1)
        out, lse = self.run(scale, lut=lut, block=block if lut else None, **kw)
        n = int(self.cu[-1])
        assert torch.all(out[n:] == 77) and torch.all(lse[n:] == 77)  # rows behind the last request
        sinks = kw.get("sinks")
        opts = dict(window=-1 if kw.get("window") is None else kw["window"], softcap=kw.get("softcap", 0.0),
                    sinks=None if sinks is None else sinks.double().cpu().numpy(), layout=layout, block=block)
        kc, vc = (np.nan_to_num(_stored(c)) for c in (self.kc, self.vc))
        ro, rl, weight, size = oc.forward(
            self.q[:n].double().cpu().numpy(), kc, vc, self.ks.double().cpu().numpy(),
            self.vs.double().cpu().numpy(), self.table, self.lens, self.cu, scale, **opts)
        o, z = out[:n].double().cpu().numpy(), lse[:n].double().cpu().numpy()
        assert np.all(np.isfinite(o))
        assert np.array_equal(np.isinf(rl), np.isinf(z)) and np.all(o[np.isinf(rl)] == 0)
        keys = max(max(self.lens), 1)
        delta = (self.d + 16) * 2.0 ** -24 * size + opts["softcap"] * 2.0 ** -20 + 2.0 ** -20
        largest = oc.LARGEST[self.kind] * np.nanmax(self.vs.double().cpu().numpy())
        tol = (torch.finfo(self.q.dtype).eps / 2 * np.abs(ro)
               + (2.0 ** -11 + 2 * delta[..., None] + keys * 2.0 ** -23) * weight + keys * 2.0 ** -25 * largest)
        bad = np.abs(o - ro) > tol
        assert not bad.any(), (bad.sum(), np.argwhere(bad)[0], np.abs(o - ro).max(), tol[bad][0])
        fin = np.isfinite(rl)
        ltol = delta + keys * 2.0 ** -24 + 2.0 ** -22 * (1 + np.abs(rl))
        off = np.abs(z[fin] - rl[fin])
        assert np.all(off <= ltol[fin]), off.max()


LENS = [1, 2, 15, 16, 17, 63, 64, 65, 128, 257, 1000]


@pytest.mark.parametrize("G,H,d,page,kind,dtype", [
    (1, 3, 128, 64, "e4m3", "bf16"), (4, 2, 128, 64, "e4m3", "bf16"), (8, 1, 64, 16, "int8", "fp16"),
    (3, 2, 64, 32, "e4m3", "fp16"), (7, 1, 128, 16, "int8", "bf16"), (16, 1, 128, 128, "e4m3", "bf16"),
    (9, 2, 64, 128, "int8", "bf16"), (2, 4, 128, 32, "int8", "fp16"), (1, 2, 64, 128, "e4m3", "bf16"),
    (32, 1, 128, 64, "e4m3", "bf16"), (128, 1, 64, 64, "e4m3", "bf16"), (20, 1, 128, 16, "int8", "bf16")])
def test_decode_lengths(G, H, d, page, kind, dtype):
    """One query a request at lengths around the page and tile sizes."""
    Case(LENS, [1] * len(LENS), G, H, d, page, kind, dtype, seed=G + d).check()


@pytest.mark.parametrize("G,H,d,page,kind,dtype", [
    (4, 2, 128, 64, "e4m3", "bf16"), (1, 2, 128, 16, "int8", "bf16"), (5, 1, 64, 32, "e4m3", "fp16"),
    (8, 2, 64, 128, "int8", "bf16"), (16, 1, 128, 128, "e4m3", "fp16"), (3, 1, 128, 64, "e4m3", "bf16")])
def test_several_queries(G, H, d, page, kind, dtype):
    """Requests without queries, drafts, chunks longer than a tile, a whole prompt at once."""
    Case([40, 9, 300, 200, 131, 257, 64], [0, 1, 4, 70, 131, 129, 17], G, H, d, page, kind, dtype, seed=d).check()


@pytest.mark.parametrize("max_q", [1, 40])
@pytest.mark.parametrize("d,kind", [(128, "e4m3"), (64, "int8")])
def test_many_short_units(max_q, d, kind):
    """A dozen units and more for every CTA, most of them a step long, some without a key."""
    rng = np.random.default_rng(d)
    lens = rng.integers(0, 150, 130)
    news = [int(rng.integers(0, min(n, 12) + 2)) for n in lens]
    Case(lens, news, 4, 16, d, 32, kind, "bf16", seed=d).check(max_q=max_q, sinks=torch.randn(64, device="cuda"))


@pytest.mark.parametrize("max_q", [1, 2, 16, 1000])
def test_max_q_is_only_a_hint(max_q):
    Case([300, 20, 77], [5, 1, 40], 4, 1, seed=2).check(max_q=max_q)


@pytest.mark.parametrize("news", [[1, 1, 1], [3, 1, 2], [150, 40, 9]])
@pytest.mark.parametrize("opts", [dict(window=0), dict(window=70), dict(softcap=3.0), dict(sinks=True),
                                  dict(window=33, softcap=20.0, sinks=True)])
def test_options(news, opts):
    c = Case([520, 40, 130], news, 4, 2, seed=7)
    if opts.get("sinks"):
        opts = dict(opts, sinks=torch.randn(8, device="cuda") * 3)
    c.check(**opts)


@pytest.mark.parametrize("news", [[1, 1, 1, 1], [2, 4, 3, 1], [200, 70, 64, 5]])
@pytest.mark.parametrize("page,block", [(16, 64), (32, 128), (64, 64), (128, 64), (64, 128), (128, 128)])
def test_layout(news, page, block):
    """Random layouts with empty rows; queries whose rows differ; blocks smaller and larger
    than a page."""
    c = Case([700, 100, 64, 129], news, 2, 3, 64 if page == 32 else 128, page, seed=page + block)
    nb = -(-c.table.shape[1] * page // block)
    rng = np.random.default_rng(1)
    layout = (rng.random((3, nb, nb)) < 0.5).astype(np.int32)
    layout[1, nb // 2] = 0
    layout[2, 0] = 0
    c.check(layout=layout, block=block)
    c.check(layout=layout, block=block, window=150, softcap=10.0, sinks=torch.randn(6, device="cuda"))


@pytest.mark.parametrize("block", [64, 128])
def test_layout_rows_inside_a_tile(block):
    """One query head a kv head: 128 rows would reach over two layout rows of 64 queries."""
    c = Case([500, 333], [300, 130], 1, 2, page=64, seed=block)
    nb = -(-c.table.shape[1] * 64 // block)
    layout = (np.random.default_rng(2).random((2, nb, nb)) < 0.5).astype(np.int32)
    c.check(layout=layout, block=block)


def test_layout_above_the_diagonal_is_not_seen():
    """A full layout is the dense call: keys after the query are not attended."""
    c = Case([333, 70], [40, 1], 2, 2, seed=3)
    layout = np.ones((2, 6, 6), np.int32)
    a, b = c.run(), c.run(lut=bsa.build_lut(layout, 1), block=64)
    assert torch.equal(a[1][:41], b[1][:41])
    c.check(layout=layout)


@pytest.mark.parametrize("news", [[1, 1, 1], [4, 3, 40]])
def test_pages_that_are_not_there(news):
    """Pages outside [0, n_pages) hold no keys; a request of such pages alone is empty."""
    c = Case([300, 130, 64], news, 4, 1, page=32, seed=5)
    c.table[0, 2] = -1
    c.table[0, 5] = 10 ** 6
    c.table[1] = -3
    c.check()
    c.check(sinks=torch.randn(4, device="cuda"))


@pytest.mark.parametrize("news", [[3, 1, 2], [70, 1, 20]])
def test_more_queries_than_tokens(news):
    c = Case([2, 0, 0], news, 4, 2, seed=6)
    c.check()
    c.check(sinks=torch.randn(8, device="cuda"))


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 40])
@pytest.mark.parametrize("news", [[3, 1, 2], [70, 1, 20]])
def test_window_wider_than_anything(news, window):
    """The widest window masks nothing, negative positions included."""
    c = Case([2, 500, 0], news, 4, 2, seed=26)
    a, b = c.run(), c.run(window=window)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c.check(window=window)


@pytest.mark.parametrize("news", [[1, 1], [1, 60]])
def test_nan_in_places_that_are_masked(news):
    """NaN keys and values before the window, of one request's single query; NaN keys that a
    query does not see yet."""
    c = Case([300, 200], news, 4, 2, page=16, seed=27)
    nan = torch.full((128,), 0x7F, dtype=torch.uint8, device="cuda")
    for pos in (0, 17, 200):
        for x in (c.kc, c.vc):
            x.view(torch.uint8)[c.table[0, pos // 16], :, pos % 16] = nan
    if news[1] > 1:  # keys of the newest token: seen by the last query alone
        c.kc.view(torch.uint8)[c.table[1, 199 // 16], :, 199 % 16] = nan
        out, lse = c.run(window=50)
        n = int(c.cu[-1])
        assert torch.all(torch.isnan(lse[n - 1])) and torch.all(torch.isfinite(lse[: n - 1]))
        assert torch.all(torch.isfinite(out[: n - 1]))
    else:
        c.check(window=50)


def test_zero_requests_queries_and_tokens():
    """No packed tokens at all, and requests none of which has a query."""
    c = Case([50, 20], [1, 0], 4, 2, seed=28)
    for T, cu in ((0, [0, 0, 0]), (3, [0, 0, 0]), (3, [1, 1, 1])):
        q = c.q[:1].repeat(max(T, 1), 1, 1)[:T]
        out, lse = torch.full_like(q, 5.0), torch.full((T, 8), 5.0, device="cuda")
        for max_q in (1, 40):
            _, _, status = bsa.cache_forward(q, c.kc, c.vc, c.ks, c.vs, ints(c.table), ints(c.lens), ints(cu), 0.1,
                                             max_q=max_q, out=out, lse=lse)
            assert int(status[0]) == 0 and torch.all(out == 5) and torch.all(lse == 5)
        bsa.cache_append(q[:, :2], q[:, :2], ints([-1] * T), c.kc.view(torch.float8_e4m3fn), c.vc, c.ks, c.vs)


def test_calls_side_by_side():
    """Calls of both kinds on two streams at once, each with a workspace of its own."""
    cs = [Case([9000, 300], [1, 1], 4, 2, seed=29), Case([2000, 900], [300, 50], 4, 2, seed=30)]
    refs = [c.run() for c in cs]
    args = [[ints(c.table), ints(c.lens), ints(c.cu)] for c in cs]
    ws = [bsa.cache_workspace(8, 2, 128, max(c.news)) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[], []]
    for _ in range(10):
        for i, c in enumerate(cs):
            with torch.cuda.stream(streams[i]):
                outs[i].append(bsa.cache_forward(c.q, c.kc, c.vc, c.ks, c.vs, *args[i], 1 / math.sqrt(c.d),
                                                 max_q=max(c.news), workspace=ws[i]))
    torch.cuda.synchronize()
    for i, c in enumerate(cs):
        n = int(c.cu[-1])
        assert bsa.cache_status(ws[i]) == 0
        for out, lse, status in outs[i]:
            assert status is None
            assert torch.equal(out[:n], refs[i][0][:n]) and torch.equal(lse[:n], refs[i][1][:n])


def test_one_workspace_for_all_shapes():
    """A workspace made for the largest call serves smaller ones of other head counts."""
    ws = bsa.cache_workspace(32, 1, 128, 1000)
    for G, H, d, news in ((4, 2, 128, [1, 1]), (8, 1, 64, [2, 1]), (1, 3, 128, [1, 200]), (32, 1, 64, [1, 1])):
        c = Case([6000, 5000], news, G, H, d, 64, seed=G)
        ref, got = c.run(), c.run(workspace=ws)
        assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])


@pytest.mark.parametrize("max_q", [1, 40])
def test_status_in_the_workspace(max_q):
    """Without a status word of its own a call leaves the workspace's as it is, or notes a wait
    that gave up; with one it does not touch the workspace's."""
    c = Case([500, 300], [1, 1], 4, 2, seed=31)
    ws = bsa.cache_workspace(8, 2, 128, max_q)
    for word in (0, 0x10010):
        ws[:4].view(torch.int32).fill_(word)
        ref = c.run(max_q=max_q, workspace=ws)
        assert bsa.cache_status(ws) == word
        out, lse, status = bsa.cache_forward(c.q, c.kc, c.vc, c.ks, c.vs, ints(c.table), ints(c.lens), ints(c.cu),
                                             1 / math.sqrt(c.d), max_q=max_q, workspace=ws)
        assert status is None and bsa.cache_status(ws) == word
        assert torch.equal(out[:2], ref[0][:2]) and torch.equal(lse[:2], ref[1][:2])


def test_length_past_the_table():
    """kv_len counts as at most max_pages * page."""
    c = Case([128, 64], [1, 5], 2, 1, seed=8)
    c.lens = [1000, 64]
    c.check()


@pytest.mark.parametrize("news", [[1, 1], [4, 100]])
def test_strided_queries(news):
    """Queries taken out of a fused projection's rows."""
    c = Case([200, 180], news, 4, 2, seed=9)
    T = c.q.shape[0]
    rows = torch.randn(T, 3 * 8 + 5, 128, device="cuda").to(torch.bfloat16)
    rows[:, 3: 11] = c.q
    c.q = rows[:, 3: 11]
    c.check()
    c.q = rows.transpose(0, 1).contiguous().transpose(0, 1)[:, 3: 11]  # heads outermost
    c.check()


@pytest.mark.parametrize("lens,news,G,H", [([40000], [1], 8, 1), ([30000, 1, 700], [1, 1, 1], 4, 2),
                                           ([9000, 8000], [4, 3], 4, 1), ([5000, 4100], [40, 30], 4, 1),
                                           ([6000], [1], 128, 1)])
def test_long_axis_is_split(lens, news, G, H):
    """Few rows over a long axis: work is split over the keys and joined."""
    Case(lens, news, G, H, page=128, seed=11).check()


def test_many_requests():
    """More work items than the GPU takes at a time, of very different lengths."""
    rng = np.random.default_rng(4)
    lens = [int(x) for x in np.exp(rng.uniform(0, np.log(900), 400))]
    Case(lens, [1] * 400, 2, 2, 64, 16, "int8", seed=12).check()


@pytest.mark.parametrize("news", [[1, 1], [3, 50]])
def test_growing_scores(news):
    """Each page scores above the one before by more than any fixed reference allows."""
    c = Case([700, 300], news, 4, 1, page=32, seed=13)
    for b, n in enumerate(c.lens):
        ids = torch.as_tensor(c.table[b, : -(-n // 32)])
        c.ks[ids] *= 1.3 ** torch.arange(len(ids), device="cuda")[:, None]
    c.check()


@pytest.mark.parametrize("news", [[1, 1], [2, 33]])
def test_value_scales_far_apart(news):
    """Pages whose V scales differ by 2^20: weights are relative to weight times scale."""
    Case([500, 200], news, 4, 2, page=16, seed=14, vscale_spread=20).check()


@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
@pytest.mark.parametrize("news", [[1, 1], [2, 33]])
def test_scales(scale, news):
    Case([500, 77], news, 4, 2, page=16, seed=15).check(scale=scale)


@pytest.mark.parametrize("news", [[1, 1], [2, 33]])
def test_large_and_small_queries(news):
    """bf16 queries far outside fp16's range, each head another."""
    c = Case([500, 77], news, 4, 2, seed=16)
    c.q *= torch.exp2(torch.tensor([-100.0, -40, -14, 0, 15, 40, 90, 100], device="cuda"))[None, :, None]
    c.ks *= 0
    c.ks += 2.0 ** -60
    # heads whose scores vanish and heads that pick one key: both exact up to the roundings
    c.check(scale=2.0 ** -40)


def test_same_answers_every_time():
    """No atomics whose order changes results: two calls give the same bits."""
    for news in ([1, 1, 1], [40, 3, 9]):
        c = Case([3000, 20000, 57], news, 8, 1, seed=17)
        a, b = c.run(), c.run()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_refusals():
    c = Case([30], [1], 4, 2)
    with pytest.raises(ValueError, match="sinks"):
        c.run(sinks=torch.zeros(2, device="cuda"))
    with pytest.raises(ValueError, match="block"):
        bsa.cache_forward(c.q, c.kc, c.vc, c.ks, c.vs, ints(c.table), ints(c.lens), ints(c.cu), 0.1,
                          lut=bsa.build_lut(np.ones((2, 1, 1), np.int32), 1))
    with pytest.raises(ValueError, match="contiguous"):
        bsa.cache_forward(c.q, c.kc.transpose(1, 2).contiguous().transpose(1, 2), c.vc, c.ks, c.vs, ints(c.table),
                          ints(c.lens), ints(c.cu), 0.1)
    with pytest.raises(bsa.BsaError) as e:
        c.run(workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    assert e.value.status == -11


# -------------------------------------------------------------------------- all together

def _model_step(tok_k, tok_v, state, slots, cu, q, scale, max_q, lut, ws=None):
    bsa.cache_append(tok_k, tok_v, slots, state["kc"], state["vc"], state["ks"], state["vs"])
    return bsa.cache_forward(q, state["kc"], state["vc"], state["ks"], state["vs"], state["table"], state["lens"],
                             cu, scale, max_q=max_q, lut=lut, block=64 if lut else None, workspace=ws)


@pytest.mark.parametrize("use_layout", [False, True])
def test_serving_loop_in_a_graph(use_layout):
    """Prompts in one eager step, then decode steps replayed from one captured graph while
    the requests grow over page borders, one ends and its pages go to another."""
    H, G, d, page, B, width = 2, 4, 128, 16, 3, 16
    P = 30
    rng = np.random.default_rng(0)
    g = torch.Generator().manual_seed(0)
    st = dict(kc=torch.zeros(P, H, page, d, dtype=torch.float8_e4m3fn, device="cuda"),
              vc=torch.zeros(P, H, page, d, dtype=torch.float8_e4m3fn, device="cuda"),
              ks=torch.zeros(P, H, device="cuda"), vs=torch.zeros(P, H, device="cuda"),
              table=torch.full((B, width), -1, **I32), lens=torch.zeros(B, **I32),
              free=ints(rng.permutation(P)), count=ints([P]))
    layout = np.tril(rng.random((H, 4, 4)) < 0.7).astype(np.int32) | np.eye(4, dtype=np.int32)
    lut = bsa.build_lut(layout, 1) if use_layout else None
    host = dict(table=st["table"].cpu().numpy(), lens=np.zeros(B, int), free=st["free"].cpu().numpy(), count=P,
                kc=np.zeros((P, H, page, d)), vc=np.zeros((P, H, page, d)), ks=np.zeros((P, H)), vs=np.zeros((P, H)))
    scale = 1 / math.sqrt(d)

    def rows(T, heads):
        return torch.randn(T, heads, d, generator=g).to(torch.bfloat16)

    def check(new, tokens, k, v, q, cu, out, lse):
        host["table"], host["lens"], host["free"], host["count"], rcu, slots, status = oc.resize(
            host["table"], host["lens"], new, host["free"], host["count"], page, tokens)
        assert status == 0 and np.array_equal(cu.cpu().numpy(), rcu)
        assert np.array_equal(st["table"].cpu().numpy(), host["table"])
        assert np.array_equal(st["lens"].cpu().numpy(), host["lens"])
        for x, c, s in ((k, "kc", "ks"), (v, "vc", "vs")):
            host[c], host[s] = oc.append(x.double().numpy(), slots, host[c], host[s], "e4m3")
            assert np.array_equal(_stored(st[c]), host[c]) and np.array_equal(st[s].double().cpu().numpy(), host[s])
        n = rcu[-1]
        ro, rl, weight, size = oc.forward(q[:n].double().numpy(), host["kc"], host["vc"], host["ks"], host["vs"],
                                          host["table"], host["lens"], rcu, scale,
                                          layout=layout if use_layout else None, block=64)
        delta = (d + 16) * 2.0 ** -24 * size + 2.0 ** -20
        tol = (2.0 ** -8 * np.abs(ro) + (2.0 ** -11 + 2 * delta[..., None] + 256 * 2.0 ** -23) * weight
               + 256 * 2.0 ** -25 * 448 * host["vs"].max())
        assert np.all(np.abs(out[:n].double().cpu().numpy() - ro) <= tol)
        fin = np.isfinite(rl)
        assert np.all(np.abs(lse[:n].double().cpu().numpy() - rl)[fin] <= (delta + 2e-5 + 1e-6 * np.abs(rl))[fin])

    # prompts
    new, tokens = [70, 1, 100], 180
    k, v, q = rows(tokens, H), rows(tokens, H), rows(tokens, G * H)
    cu, slots, status = bsa.cache_resize(st["table"], st["lens"], ints(new), st["free"], st["count"], page, tokens)
    out, lse, _ = _model_step(k.cuda(), v.cuda(), st, slots, cu, q.cuda(), scale, 100, lut)
    check(new, tokens, k, v, q, cu, out, lse)

    # decode steps from a graph with fixed addresses
    want = torch.zeros(B, **I32)
    dk, dv, dq = (torch.zeros(B, n, d, dtype=torch.bfloat16, device="cuda") for n in (H, H, G * H))

    def step():
        cu, slots, status = bsa.cache_resize(st["table"], st["lens"], want, st["free"], st["count"], page, B)
        return cu, status, _model_step(dk, dv, st, slots, cu, dq, scale, 1, lut)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want.copy_(st["lens"])
        step()  # nothing grows: a warm-up that changes nothing
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cu, status, (out, lse, ok) = step()
    for i in range(20):
        new = [int(x) + 1 for x in host["lens"]]
        if i == 5:
            new[2] = 0                       # ends; its pages go to the others
        elif i > 5 and i < 9:
            new[2] = 0
        k, v, q = rows(B, H), rows(B, H), rows(B, G * H)
        dk.copy_(k)
        dv.copy_(v)
        dq.copy_(q)
        want.copy_(ints(new))
        graph.replay()
        assert int(status[0]) == 0 and int(ok[0]) == 0
        check(new, B, k, v, q, cu, out, lse)


def test_on_a_stream_of_its_own():
    """Calls on a side stream with memory of their own, while the default stream is busy."""
    c = Case([3000, 700], [1, 1], 4, 2, seed=20)
    ref = c.run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    busy = torch.randn(4096, 4096, device="cuda")
    args = [ints(c.table), ints(c.lens), ints(c.cu)]
    torch.cuda.synchronize()
    for _ in range(20):
        busy = busy @ busy * 1e-3
    out, lse, status = bsa.cache_forward(c.q, c.kc, c.vc, c.ks, c.vs, *args, 1 / math.sqrt(c.d), max_q=1, stream=s)
    s.synchronize()
    assert int(status[0]) == 0
    assert torch.equal(out[:2], ref[0][:2]) and torch.equal(lse[:2], ref[1][:2])


def test_two_graphs_share_a_workspace():
    """Two captured calls with one workspace, replayed one after the other."""
    cs = [Case([3000, 700], [1, 1], 4, 2, seed=21), Case([100, 9000], [1, 1], 4, 2, seed=22)]
    ws = bsa.cache_workspace(8, 2, 128, 1)
    refs = [c.run() for c in cs]
    graphs, outs = [], []
    for c in cs:
        args = [ints(c.table), ints(c.lens), ints(c.cu)]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(bsa.cache_forward(c.q, c.kc, c.vc, c.ks, c.vs, *args, 1 / math.sqrt(c.d), max_q=1,
                                          workspace=ws))
        graphs.append((graph, args))
    for _ in range(5):
        for graph, _ in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for (out, lse, _), ref in zip(outs, refs):
        assert torch.equal(out[:2], ref[0][:2]) and torch.equal(lse[:2], ref[1][:2])


def test_offsets_past_32_bits():
    """A cache of more than 2^32 numbers; the pages in use are its last ones."""
    H, page, d = 8, 128, 128
    P = (1 << 32) // (H * page * d) + 40
    kc, vc = (torch.zeros(P, H, page, d, dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((P, H), float("nan"), device="cuda") for _ in range(2))
    x = torch.randn(300, H, d, device="cuda", dtype=torch.float16)
    table = ints([[P - 1, P - 7, P - 3]])
    lens, slots = ints([0]), None
    free, count = ints(list(range(4)) + [0] * (P - 4)), ints([4])
    slots = torch.cat([(table[0, j] * page + torch.arange(min(page, 300 - j * page), device="cuda")).int()
                       for j in range(3)])
    bsa.cache_append(x, x, slots, kc, vc, ks, vs)
    small = [t[P - 8:].clone() for t in (kc, vc, ks, vs)]
    for n in (1, 33):
        q = torch.randn(n, 2 * H, d, device="cuda", dtype=torch.float16)
        cu, lens = ints([0, n]), ints([300])
        a = bsa.cache_forward(q, kc, vc, ks, vs, table, lens, cu, 0.1, max_q=n)
        b = bsa.cache_forward(q, *small, table - (P - 8), lens, cu, 0.1, max_q=n)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        assert torch.all(torch.isfinite(a[0]))
    # the stored numbers against the values
    got = kc[P - 1].float() * ks[P - 1][:, None, None]
    assert torch.all((got - x[:128].transpose(0, 1).float()).abs() <= ks[P - 1][:, None, None] / 2)

"""GPU parity of bsa_cache_diff_forward against the fp64 oracle: out = O_0 - lam O_1 of the
oracle's O for the query heads 2h and 2h + 1.

Bounds: those of the cache's forward (test_gpu_cache) for each O before its rounding, the
second's times |lam|, and one rounding of the difference, eps / 2 |out|."""

import math

import numpy as np
import pytest
import torch

import block_sparse_head_gb300 as bsa
from oracle import bsa_oracle_cache as oc
from test_gpu_cache import LENS, Case, _stored, ints
from test_gpu_cache_abort import Call

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cuda_lib):
    return cuda_lib


class DiffCase(Case):
    """G: query heads of a kv head, two maps for each output head; split: queries of d / 2."""

    def __init__(self, lens, news, G=4, H=2, split=False, rows=True, seed=0, **kw):
        super().__init__(lens, news, G, H, seed=seed, **kw)
        if split:
            self.q = self.q[..., : self.d // 2].contiguous()
        T, Hq, self.dq = self.q.shape
        g = torch.Generator().manual_seed(seed + 5)
        self.lam = (torch.rand(*((T, Hq // 2) if rows else (Hq // 2,)), generator=g) * 1.3 - 0.2).cuda()

    def run(self, scale=None, **kw):
        scale = 1 / math.sqrt(self.dq) if scale is None else scale
        T, Hq = self.q.shape[:2]
        out = torch.full((T, Hq // 2, self.d), 77.0, dtype=self.q.dtype, device="cuda")
        lse = torch.full((T, Hq), 77.0, device="cuda")
        kw.setdefault("max_q", max(max(self.news), 1))
        kw.setdefault("status", torch.full((1,), -1, dtype=torch.int32, device="cuda"))
        _, _, status = bsa.cache_diff_forward(self.q, self.lam, self.kc, self.vc, self.ks, self.vs, ints(self.table),
                                              ints(self.lens), ints(self.cu), scale, out=out, lse=lse, **kw)
        assert int(status[0]) == 0, hex(int(status[0]))
        return out, lse

    def check(self, scale=None, layout=None, block=64, **kw):
        scale = 1 / math.sqrt(self.dq) if scale is None else scale
        lut = None if layout is None else bsa.build_lut(layout, 1)
        out, lse = self.run(scale, lut=lut, block=block if lut else None, **kw)
        n = int(self.cu[-1])
        assert torch.all(out[n:] == 77) and torch.all(lse[n:] == 77)  # rows behind the last request
        sinks = kw.get("sinks")
        opts = dict(window=-1 if kw.get("window") is None else kw["window"], softcap=kw.get("softcap", 0.0),
                    sinks=None if sinks is None else sinks.double().cpu().numpy(), layout=layout, block=block)
        kc, vc = (np.nan_to_num(_stored(c)) for c in (self.kc, self.vc))
        q = self.q[:n].double().cpu().numpy()
        if self.dq != self.d:  # each map's queries before its own key half, zero before the other
            wide = np.zeros(q.shape[:2] + (self.d,))
            wide[:, 0::2, : self.dq], wide[:, 1::2, self.dq:] = q[:, 0::2], q[:, 1::2]
            q = wide
        ro, rl, weight, size = oc.forward(q, kc, vc, self.ks.double().cpu().numpy(), self.vs.double().cpu().numpy(),
                                          self.table, self.lens, self.cu, scale, **opts)
        lam = self.lam.double().cpu().numpy()
        lam = np.broadcast_to(lam if lam.ndim == 1 else lam[:n], (n, ro.shape[1] // 2))[..., None]
        ref = ro[:, 0::2] - lam * ro[:, 1::2]
        o, z = out[:n].double().cpu().numpy(), lse[:n].double().cpu().numpy()
        assert np.all(np.isfinite(o))
        assert np.array_equal(np.isinf(rl), np.isinf(z))
        keys = max(max(self.lens), 1)
        delta = (self.d + 16) * 2.0 ** -24 * size + opts["softcap"] * 2.0 ** -20 + 2.0 ** -20
        largest = oc.LARGEST[self.kind] * np.nanmax(self.vs.double().cpu().numpy())
        each = (2.0 ** -11 + 2 * delta[..., None] + keys * 2.0 ** -23) * weight + keys * 2.0 ** -25 * largest
        tol = torch.finfo(self.q.dtype).eps / 2 * np.abs(ref) + each[:, 0::2] + np.abs(lam) * each[:, 1::2]
        bad = np.abs(o - ref) > tol
        assert not bad.any(), (bad.sum(), np.argwhere(bad)[0], np.abs(o - ref).max(), tol[bad][0])
        fin = np.isfinite(rl)
        ltol = delta + keys * 2.0 ** -24 + 2.0 ** -22 * (1 + np.abs(rl))
        off = np.abs(z[fin] - rl[fin])
        assert np.all(off <= ltol[fin]), off.max()


@pytest.mark.parametrize("G,H,split,kw", [
    (2, 3, False, dict(d=128, page=64)), (4, 2, True, dict(d=128, page=64, dtype="fp16")),
    (8, 1, False, dict(d=64, page=16, kind="int8", dtype="fp16")), (6, 2, False, dict(d=64, page=32)),
    (16, 1, True, dict(d=128, page=128, kind="int8")), (10, 1, False, dict(d=64, page=128)),
    (32, 1, True, dict(d=128, page=64)), (128, 1, False, dict(d=64, page=64)),
    (24, 1, False, dict(d=128, page=16, kind="int8"))])
@pytest.mark.parametrize("rows", [False, True])
def test_decode_lengths(G, H, split, kw, rows):
    """One query a request at lengths around the page and tile sizes."""
    DiffCase(LENS, [1] * len(LENS), G, H, split, rows, seed=G + H, **kw).check()


@pytest.mark.parametrize("G,H,split,kw", [
    (4, 2, False, dict(d=128, page=64)), (2, 2, True, dict(d=128, page=16, kind="int8")),
    (6, 1, False, dict(d=64, page=32, dtype="fp16")), (8, 2, False, dict(d=64, page=128, kind="int8")),
    (16, 1, True, dict(d=128, page=128, dtype="fp16"))])
def test_several_queries(G, H, split, kw):
    """Requests without queries, drafts, chunks longer than a tile, a whole prompt at once."""
    DiffCase([40, 9, 300, 200, 131, 257, 64], [0, 1, 4, 70, 131, 129, 17], G, H, split, seed=G, **kw).check()


@pytest.mark.parametrize("max_q", [1, 40])
@pytest.mark.parametrize("split", [False, True])
def test_many_short_units(max_q, split):
    """A dozen units and more for every CTA, most of them a step long, some without a key."""
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 150, 130)
    news = [int(rng.integers(0, min(n, 12) + 2)) for n in lens]
    DiffCase(lens, news, 4, 16, split, page=32, seed=4).check(max_q=max_q, sinks=torch.randn(64, device="cuda"))


@pytest.mark.parametrize("news", [[1, 1, 1], [3, 1, 2], [150, 40, 9]])
@pytest.mark.parametrize("opts", [dict(window=0), dict(window=70), dict(softcap=3.0), dict(sinks=True),
                                  dict(window=33, softcap=20.0, sinks=True)])
def test_options(news, opts):
    c = DiffCase([520, 40, 130], news, 4, 2, seed=7)
    if opts.get("sinks"):
        opts = dict(opts, sinks=torch.randn(8, device="cuda") * 3)
    c.check(**opts)


@pytest.mark.parametrize("news", [[1, 1, 1, 1], [200, 70, 64, 5]])
@pytest.mark.parametrize("page,block", [(16, 64), (128, 64), (64, 128)])
def test_layout(news, page, block):
    """Random layouts with empty rows."""
    c = DiffCase([700, 100, 64, 129], news, 2, 3, page == 64, page=page, seed=page + block)
    nb = -(-c.table.shape[1] * page // block)
    layout = (np.random.default_rng(1).random((3, nb, nb)) < 0.5).astype(np.int32)
    layout[1, nb // 2] = 0
    layout[2, 0] = 0
    c.check(layout=layout, block=block, window=150)


@pytest.mark.parametrize("news", [[1], [9], [300]])
def test_cut_units_are_joined(news):
    """Few units over many CTAs: every row is joined from pieces."""
    DiffCase([6000], news, 8, 1, True, rows=False, seed=8).check()


@pytest.mark.parametrize("B", [30, 60, 100])
@pytest.mark.parametrize("n,d", [(1, 128), (4, 128), (4, 64)])
def test_units_cut_into_few_pieces(B, n, d):
    """One to five partial results a unit, of 4 rows and of 16."""
    DiffCase([900 - 7 * i for i in range(B)], [n] * B, 4, 1, d=d, page=32, seed=B + n + d).check(
        max_q=n, sinks=torch.randn(4, device="cuda"))


@pytest.mark.parametrize("news", [[3, 1, 2], [70, 1, 20]])
def test_more_queries_than_tokens(news):
    c = DiffCase([2, 0, 0], news, 4, 2, seed=6)
    c.check()
    out, lse = c.run()
    empty = torch.isinf(lse[:, 0::2]) & torch.isinf(lse[:, 1::2])
    assert bool(empty.any()) and torch.all(out[empty] == 0)


@pytest.mark.parametrize("news", [[1, 1], [4, 60]])
def test_strided_queries_and_a_workspace_of_its_own(news):
    """Rows of a fused projection; one workspace for calls of both kinds, which leave it fit for
    each other."""
    c = DiffCase([700, 90], news, 4, 2, True, seed=9)
    ref = c.run()
    T, Hq, dq = c.q.shape
    fused = torch.randn(T, 2 * Hq + 3, dq, device="cuda").to(c.q.dtype)
    fused[:, 2: 2 + Hq] = c.q
    c.q = fused[:, 2: 2 + Hq]
    ws = bsa.cache_workspace(Hq, c.H, c.d, max(news))
    for _ in range(2):
        got = c.run(workspace=ws, status=torch.zeros(1, dtype=torch.int32, device="cuda"))
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
        plain = torch.randn(T, Hq, c.d, device="cuda").to(c.q.dtype)
        bsa.cache_forward(plain, c.kc, c.vc, c.ks, c.vs, ints(c.table), ints(c.lens), ints(c.cu), 0.1,
                          max_q=max(news), workspace=ws)
    assert bsa.cache_status(ws) == 0


def test_a_captured_decode_step_follows_its_lengths():
    c = DiffCase([300, 90, 11], [1, 1, 1], 4, 2, seed=10, pad=0)
    lens, table, cu = ints(c.lens), ints(c.table), ints(c.cu)
    ws = bsa.cache_workspace(8, 2, 128, 1)
    call = lambda: bsa.cache_diff_forward(c.q, c.lam, c.kc, c.vc, c.ks, c.vs, table, lens, cu, 0.1,  # noqa: E731
                                          max_q=1, workspace=ws)
    call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        held = call()
    for new in ([299, 64, 3], [17, 0, 1]):
        lens.copy_(ints(new))
        graph.replay()
        torch.cuda.synchronize()
        want = call()
        assert torch.equal(held[0], want[0]) and torch.equal(held[1], want[1])
    assert bsa.cache_status(ws) == 0


def test_a_serving_step():
    """Pages for new tokens, the tokens' keys and values, their queries' attention: the calls as a
    step makes them, against the oracle on what the cache holds."""
    P, Hkv, H, page, d, B = 40, 2, 4, 16, 128, 3
    i32 = dict(dtype=torch.int32, device="cuda")
    kc = torch.zeros(P, Hkv, page, d, dtype=torch.float8_e4m3fn, device="cuda")
    vc = torch.zeros_like(kc)
    ks, vs = torch.ones(2, P, Hkv, device="cuda").unbind(0)
    table, kv_len = torch.full((B, 12), -1, **i32), torch.zeros(B, **i32)
    free, count = torch.arange(P, **i32), torch.tensor([P], **i32)
    g = torch.Generator(device="cuda").manual_seed(12)
    for new, T in (([70, 9, 33], 115), ([71, 10, 34], 3), ([71, 14, 35], 5)):
        k, v = (torch.randn(T, Hkv, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
        q = torch.randn(T, 2 * H, d // 2, generator=g, device="cuda").to(torch.bfloat16)
        lam = torch.rand(T, H, generator=g, device="cuda")
        cu, slots, status = bsa.cache_resize(table, kv_len, ints(new), free, count, page, T)
        bsa.cache_append(k, v, slots, kc, vc, ks, vs)
        out, lse, st = bsa.cache_diff_forward(q, lam, kc, vc, ks, vs, table, kv_len, cu, 0.125)
        assert int(status[0]) == 0 and int(st[0]) == 0
        n = int(cu[-1])
        wide = np.zeros((n, 2 * H, d))
        qn = q[:n].double().cpu().numpy()
        wide[:, 0::2, :64], wide[:, 1::2, 64:] = qn[:, 0::2], qn[:, 1::2]
        ro, rl, weight, size = oc.forward(wide, _stored(kc), _stored(vc), ks.double().cpu().numpy(),
                                          vs.double().cpu().numpy(), table.cpu().numpy(), kv_len.tolist(),
                                          cu.cpu().numpy(), 0.125)
        ln = lam[:n].double().cpu().numpy()[..., None]
        ref = ro[:, 0::2] - ln * ro[:, 1::2]
        delta = 144 * 2.0 ** -24 * size + 2.0 ** -20
        each = (2.0 ** -11 + 2 * delta[..., None] + 71 * 2.0 ** -23) * weight + 71 * 2.0 ** -25 * 8
        tol = 2.0 ** -8 * np.abs(ref) + each[:, 0::2] + ln * each[:, 1::2]
        assert np.all(np.abs(out[:n].double().cpu().numpy() - ref) <= tol)
        assert np.all(np.abs(lse[:n].double().cpu().numpy() - rl) <= delta + 2.0 ** -20 * (1 + np.abs(rl)))


class DiffCall(Call):
    """test_gpu_cache_abort's calls, as two maps of G / 2 heads a kv head."""

    def __call__(self, status=None):
        lam = torch.linspace(0.1, 0.9, self.q.shape[1] // 2, device="cuda")
        out, lse, _ = bsa.cache_diff_forward(self.q, lam, self.kc, self.vc, self.ks, self.vs, self.table, self.lens,
                                             self.cu, self.scale, max_q=self.n, lut=self.lut, block=128,
                                             workspace=self.ws, status=status)
        return out, lse


@pytest.mark.parametrize("site", [6, 16])
@pytest.mark.parametrize("G,n,d", [(4, 1, 128), (4, 4, 128), (10, 1, 64)])
def test_decode_wait_gives_up(G, n, d, site):
    DiffCall([3000, 130, 9000, 257] * 8, n, G, 4, d).check_site(site)


@pytest.mark.parametrize("site,others", [(6, [1, 2, 7, 9]), (7, [1, 2, 6, 8, 9, 11, 12]), (17, [17])])
def test_tile_role_is_missing(site, others):
    DiffCall([6000, 300, 20000, 1290], 200, 4, 4, 128).check_site(site, [0x10000 | x for x in others], ways=1)


def test_no_tokens():
    c = DiffCase([40], [0], 4, 2, pad=0, seed=13)
    out, lse = c.run(max_q=1)
    assert out.shape == (0, 4, 128) and lse.shape == (0, 8)


def test_refusals():
    c = DiffCase([40], [1], 4, 2, seed=11)
    for bad in (dict(q=c.q[:, :3]), dict(q=c.q.float()), dict(q=c.q.cpu()), dict(q=c.q[0]), dict(lam=c.lam.double()),
                dict(lam=c.lam[:, :1]), dict(lam=c.lam[0, :1]), dict(lam=c.lam.cpu()), dict(lam=None)):
        a = {**dict(q=c.q, lam=c.lam), **bad}
        with pytest.raises(ValueError):
            bsa.cache_diff_forward(a["q"], a["lam"], c.kc, c.vc, c.ks, c.vs, ints(c.table), ints(c.lens), ints(c.cu), 0.1)
    with pytest.raises(bsa.BsaError):  # neither d nor d / 2
        bsa.cache_diff_forward(c.q[..., :32], c.lam, c.kc, c.vc, c.ks, c.vs, ints(c.table), ints(c.lens), ints(c.cu), 0.1)
    with pytest.raises(ValueError):
        bsa.cache_diff_forward(c.q, c.lam, c.kc, c.vc, c.ks, c.vs, ints(c.table), ints(c.lens), ints(c.cu), 0.1,
                               sinks=torch.zeros(4, device="cuda"))

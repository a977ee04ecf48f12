"""Workloads of differential attention and of rotary positions with several axes, with
their plain forms.

Four operators:

* ``diff_forward``: the difference of two block-sparse softmax maps over one value matrix,
  ``out = (P_0 - lam P_1) V``, over the active blocks of a layout;
* ``diff_forward`` and ``diff_backward`` together, a training step's attention: gradients of
  queries, keys, values and of the weight ``lam``;
* ``cache_diff_forward``: the same difference for each request's newest tokens over a paged
  8-bit key/value cache;
* ``rotary``: rotation of queries and keys by positions on one to four axes (text; time,
  height and width of images and video), and its inverse, which is its gradient.

``run`` computes them in elementary torch operations, or, where ``own`` is true, through
the framework's entry points.
"""

import math

import torch

own = False

QMAX = {"e4m3": 448.0, "int8": 127.0}
CACHE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------------- the cases

def listed():
    return [
        # A short sequence of a small model: latency of one forward.
        dict(name="forward-512", op="forward", B=1, heads=4, kv_heads=4, L=512, d=64, dq=64, block=64,
             layout="window", lam="head"),
        # Prefill of a long context under the band-and-stride layout, keys shared by groups of heads.
        dict(name="forward-16384", op="forward", B=1, heads=16, kv_heads=4, L=16384, d=128, dq=128, block=128,
             layout="strided", lam="head"),
        # A small training step, a key half for each map, ragged last block.
        dict(name="train-333", op="train", B=2, heads=2, kv_heads=1, L=333, d=128, dq=64, block=64,
             layout="causal", lam="token"),
        # An odd length, small heads, the window-and-global layout, one weight a token.
        dict(name="train-2999", op="train", B=2, heads=8, kv_heads=8, L=2999, d=64, dq=64, block=64,
             layout="window", lam="token"),
        # An ordinary long training sequence with grouped heads.
        dict(name="train-8192", op="train", B=1, heads=16, kv_heads=4, L=8192, d=128, dq=128, block=128,
             layout="strided", lam="head"),
        # One request's decode step with a short history: latency.
        dict(name="decode-1x1000", op="cache", B=1, new=1, old=999, ragged=False, heads=16, kv_heads=8, d=128, dq=128,
             page=64, cache="e4m3", dtype="bf16", window=-1, layout="", lam="token"),
        # A batch of requests of many lengths: throughput of the ordinary decode step.
        dict(name="decode-64x8192", op="cache", B=64, new=1, old=8191, ragged=True, heads=16, kv_heads=8, d=128,
             dq=128, page=64, cache="e4m3", dtype="bf16", window=-1, layout="", lam="token"),
        # Four draft tokens verified at once, a key half for each map, int8, small pages, a window.
        dict(name="verify-16x4096", op="cache", B=16, new=4, old=4096, ragged=True, heads=16, kv_heads=8, d=128,
             dq=64, page=16, cache="int8", dtype="fp16", window=1000, layout="", lam="head"),
        # A chunk of a long prompt against what is cached so far.
        dict(name="chunk-1x2048", op="cache", B=1, new=2048, old=14336, ragged=False, heads=16, kv_heads=8, d=128,
             dq=128, page=64, cache="e4m3", dtype="bf16", window=-1, layout="", lam="token"),
        # One token each of 64 requests, packed rows of a fused projection, three axes on one ladder.
        dict(name="rotary-decode-64", op="rotary", packed=True, B=1, L=64, heads=32, kv_heads=8, d=128,
             pairs="16,24,24", ladder="shared", pairing="half", dtype="bf16", inverse=False, far=1 << 20),
        # Queries and keys of a long training sequence.
        dict(name="rotary-train-16384", op="rotary", packed=False, B=1, L=16384, heads=32, kv_heads=8, d=128,
             pairs="64", ladder="shared", pairing="half", dtype="bf16", inverse=False, far=16384),
        # Gradients through the positions of a clip of 13 x 30 x 52 patches, one ladder an axis.
        dict(name="rotary-video-backward", op="rotary", packed=False, B=2, L=20280, heads=16, kv_heads=16, d=128,
             pairs="22,21,21", ladder="axis", pairing="adjacent", dtype="bf16", inverse=True, far=64),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["forward", "train", "train", "cache", "cache", "rotary"])
    if op == "rotary":
        pairs, ladder = rng.choice([("16,24,24", "shared"), ("64", "shared"), ("22,21,21", "axis"), ("8,12,12", "axis"),
                                    ("32", "shared")])
        packed = rng.random() < 0.4
        return dict(op=op, packed=packed, B=1 if packed else rng.randint(1, 3), L=_log(rng, 1, 12000),
                    heads=rng.choice([1, 4, 16, 32]), kv_heads=rng.choice([1, 2, 8]),
                    d=rng.choice([128, 256] if pairs != "32" and pairs != "8,12,12" else [64, 96, 128]), pairs=pairs,
                    ladder=ladder, pairing=rng.choice(["half", "adjacent"]), dtype=rng.choice(["bf16", "fp16"]),
                    inverse=rng.random() < 0.4, far=rng.choice([64, 8192, 1 << 20]))
    d = rng.choice([64, 128])
    dq = rng.choice([64, d])
    lam = rng.choice(["head", "token"])
    if op == "cache":
        kv_heads = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 1, 2, 3, 4])
        case = dict(op=op, page=rng.choice([16, 32, 64, 128]), d=d, dq=dq, cache=rng.choice(["e4m3", "int8"]),
                    dtype=rng.choice(["bf16", "fp16"]), kv_heads=kv_heads, heads=kv_heads * group, lam=lam,
                    ragged=rng.random() < 0.7, window=rng.choice([-1, -1, 0, 777]),
                    layout=rng.choice(["", "", "strided", "window"]))
        kind = rng.choice(["decode", "decode", "verify", "chunk"])
        if kind == "chunk":
            return dict(case, B=_log(rng, 1, 4), new=_log(rng, 17, 1000), old=_log(rng, 1, 6000))
        B = _log(rng, 1, 64)
        return dict(case, B=B, new=1 if kind == "decode" else rng.randint(2, 8),
                    old=_log(rng, 1, min(60000, 2 * 10 ** 6 // (B * kv_heads))))
    kv_heads = rng.choice([1, 2, 4])
    return dict(op=op, B=rng.randint(1, 2), heads=kv_heads * rng.choice([1, 2, 4]), kv_heads=kv_heads,
                L=_log(rng, 1, 3500), d=d, dq=dq, block=rng.choice([64, 128]),
                layout=rng.choice(["causal", "strided", "window", "holes"]), lam=lam)


def _layout(case, nb):
    """Layouts [kv_heads, nb, nb]: everything up to the diagonal; a band of 8 blocks with every
    16th column; a window of 4 blocks with the first column; and random blocks, also after
    the diagonal, with rows and columns that have none."""
    i, j = torch.arange(nb)[:, None], torch.arange(nb)[None, :]
    if case["layout"] == "holes":
        g = torch.Generator().manual_seed(31 * nb + case["kv_heads"])
        on = torch.rand(case["kv_heads"], nb, nb, generator=g) < 0.4
        if nb > 2:
            on[:, 1], on[:, :, 2] = False, False
        return on.to(torch.int32).contiguous()
    if case["layout"] == "strided":
        on = (j <= i) & ((j > i - 8) | (j % 16 == 15))
    elif case["layout"] == "window":
        on = (j <= i) & ((j > i - 4) | (j == 0))
    else:
        on = j <= i
    return on.to(torch.int32)[None].repeat(case["kv_heads"], 1, 1).contiguous()


def _allowed(case, layout):
    """Elementwise mask [kv_heads, L, L]: the layout's blocks, causal inside diagonal ones."""
    L, b = case["L"], case["block"]
    r = torch.arange(L, device=layout.device)
    on = layout.bool().repeat_interleave(b, 1)[:, :L].repeat_interleave(b, 2)[:, :, :L]
    return on & ~((r[:, None] // b == r[None] // b) & (r[None] > r[:, None]))


def _lengths(case):
    """Old lengths and new tokens of each request; one set for a case, so that its outputs
    have one shape."""
    g = torch.Generator().manual_seed(7919 * case["B"] + case["page"])
    B = case["B"]
    old, new = torch.full((B,), case["old"]), torch.full((B,), case["new"])
    if case["ragged"]:
        old[1:] = torch.randint(case["old"] // 4, case["old"] + 1, (B,), generator=g)[1:]
        if case["new"] > 1:
            new[1:] = torch.randint(1, case["new"] + 1, (B,), generator=g)[1:]
    return old.tolist(), new.tolist()


def _block(case):
    return 128 if case["page"] == 128 else 64


def _frequencies(case):
    """(inverse frequency, axis) of each pair. "shared": one ladder over all pairs, its rungs
    dealt to the axes in sections; "axis": every axis has a ladder of its own."""
    sections = [int(n) for n in case["pairs"].split(",")]
    total = sum(sections)
    f, axis, at = [], [], 0
    for a, n in enumerate(sections):
        for i in range(n):
            f.append(10000.0 ** (-(at / total if case["ladder"] == "shared" else i / n)))
            axis.append(a)
            at += 1
    return f, axis


def _lam(case, shape, g):
    # A head's weight in the range that its reparametrisation starts from in early to late
    # layers; a token's the sigmoid of a projection.
    if case["lam"] == "head":
        return 0.2 + 0.6 * torch.rand(case["heads"], generator=g, device="cuda")
    return torch.sigmoid(torch.randn(*shape, generator=g, device="cuda"))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "rotary":
        return _prepare_rotary(case, g)
    if case["op"] == "cache":
        return _prepare_cache(case, g)
    B, H, Hkv, L, d, dq = (case[n] for n in ("B", "heads", "kv_heads", "L", "d", "dq"))
    bf16 = torch.bfloat16
    s = dict(case=case, q=torch.randn(B, 2 * H, L, dq, generator=g, device="cuda").to(bf16),
             k=torch.randn(B, Hkv, L, d, generator=g, device="cuda").to(bf16),
             v=torch.randn(B, Hkv, L, d, generator=g, device="cuda").to(bf16),
             lam=_lam(case, (B, H, L), g))
    if case["op"] == "train":
        s["dout"] = torch.randn(B, H, L, d, generator=g, device="cuda").to(bf16)
    layout = _layout(case, -(-L // case["block"]))
    s["layout"] = layout.cuda()
    if own:  # the layout's look-up table, which a program builds once
        import block_sparse_head_gb300 as bsa

        s["lut"] = bsa.build_lut(layout, B)
    return s


def _power(e):
    """2^e in fp32 from its bits: a library's power need not be exact."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _prepare_cache(case, g):
    ints = dict(dtype=torch.int32, device="cuda")
    old, new = _lengths(case)
    B, page, Hkv, H, d, dq, kind = (case[n] for n in ("B", "page", "kv_heads", "heads", "d", "dq", "cache"))
    total = [a + n for a, n in zip(old, new)]
    held = [-(-x // page) for x in total]
    pages = sum(held) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, max(held)), -1, **ints)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = order[at: at + n]
        at += n
    caches, scales = [], []
    for _ in range(2):
        c = torch.empty(pages, Hkv, page, d, dtype=CACHE[kind], device="cuda")
        flat, step = c.view(-1), 1 << 27
        for lo in range(0, flat.numel(), step):  # stored numbers spread over the type's range
            x = torch.randn(min(step, flat.numel() - lo), generator=g, device="cuda") * (QMAX[kind] / 4.2)
            flat[lo: lo + step] = (x.round() if kind == "int8" else x).clamp(-QMAX[kind], QMAX[kind]).to(c.dtype)
        caches.append(c)
        e = torch.randint(-1, 2, (pages, Hkv), generator=g, device="cuda")
        scales.append(_power(e + round(math.log2(4.2 / QMAX[kind]))))
    T = sum(new)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s = dict(case=case, k_cache=caches[0], v_cache=caches[1], k_scale=scales[0], v_scale=scales[1], table=table,
             kv_len=torch.tensor(total, **ints), cu=torch.tensor(cu, **ints), most=max(new),
             q=torch.randn(T, 2 * H, dq, generator=g, device="cuda").to(TYPES[case["dtype"]]), lam=_lam(case, (T, H), g),
             layout=None, lut=None)
    if case["layout"]:
        layout = _layout(case, -(-table.shape[1] * page // _block(case)))
        s["layout"] = layout.cuda()
    if own:  # the layout's look-up table and the workspace, which a program makes once
        import block_sparse_head_gb300 as bsa

        if case["layout"]:
            s["lut"] = bsa.build_lut(layout, 1)
        s["workspace"] = bsa.cache_workspace(2 * H, Hkv, d, s["most"])
    return s


def _prepare_rotary(case, g):
    B, L, H, Hkv, d, dtype = (case[n] for n in ("B", "L", "heads", "kv_heads", "d", "dtype"))
    f, axis = _frequencies(case)
    axes = max(axis) + 1
    if case["packed"]:  # slices of one projection's rows
        rows = torch.randn(L, H + 2 * Hkv, d, generator=g, device="cuda").to(TYPES[dtype])
        q, k = rows[:, :H], rows[:, H: H + Hkv]
        positions = torch.randint(0, case["far"], (axes, L), generator=g, device="cuda", dtype=torch.int32)
    else:
        q = torch.randn(B, H, L, d, generator=g, device="cuda").to(TYPES[dtype])
        k = torch.randn(B, Hkv, L, d, generator=g, device="cuda").to(TYPES[dtype])
        positions = torch.randint(0, case["far"], (axes, B, L), generator=g, device="cuda", dtype=torch.int32)
    s = dict(case=case, q=q, k=k, positions=positions, axis=torch.tensor(axis, device="cuda"),
             f=torch.tensor(f, dtype=torch.float64, device="cuda"))
    if own:  # the table of frequencies, which a program makes once
        import block_sparse_head_gb300 as bsa

        s["table"] = bsa.rotary_table(f, axis)
    return s


# ------------------------------------------------------------------------- the passes

def run(state):
    return {"forward": _run_train, "train": _run_train, "cache": _run_cache,
            "rotary": _run_rotary}[state["case"]["op"]](state)


def _run_train(s):
    case = s["case"]
    B, H, Hkv, L, d, dq = (case[n] for n in ("B", "heads", "kv_heads", "L", "d", "dq"))
    scale, train = 1.0 / math.sqrt(dq), case["op"] == "train"
    if own:
        import block_sparse_head_gb300 as bsa

        out, lse, out2 = bsa.diff_forward(s["q"], s["k"], s["v"], s["lam"], s["lut"], scale, case["block"], True,
                                          training=train)
        if not train:
            return {"out": out, "lse": lse}
        dq_, dk, dv, dlam = bsa.diff_backward(s["q"], s["k"], s["v"], s["lam"], out, out2, lse, s["dout"], s["lut"],
                                              scale, case["block"], True)
        return {"out": out, "lse": lse, "dq": dq_, "dk": dk, "dv": dv, "dlam": dlam}
    G, n = H // Hkv, d // dq  # heads of a group; keys of a row: one for both maps, or one each
    q = s["q"].float().view(B, Hkv, G, 2, L, dq)
    k = s["k"].float().view(B, Hkv, 1, L, n, dq).transpose(3, 4)  # [B, Hkv, 1, n, L, dq]
    v = s["v"].float()[:, :, None]
    lam = s["lam"].view(Hkv, G, 1, 1) if case["lam"] == "head" else s["lam"].view(B, Hkv, G, L, 1)
    x = torch.matmul(q, k.transpose(4, 5)) * scale  # [B, Hkv, G, 2, L, L]
    x = x.masked_fill(~_allowed(case, s["layout"])[:, None, None], -math.inf)
    m = x.amax(5, keepdim=True)
    m = m.masked_fill(m == -math.inf, 0.0)
    p = torch.exp(x - m)
    del x
    z = p.sum(5, keepdim=True)
    lse = (m + torch.log(z)).view(B, 2 * H, L)
    p = p / z.masked_fill(z == 0, 1.0)
    w = p[:, :, :, 0] - lam * p[:, :, :, 1]  # [B, Hkv, G, L, L]
    bf16 = torch.bfloat16
    result = {"out": torch.matmul(w, v).view(B, H, L, d).to(bf16), "lse": lse}
    if not train:
        return result
    do = s["dout"].float().view(B, Hkv, G, L, d)
    dp = torch.matmul(do, v.transpose(3, 4))[:, :, :, None]  # [B, Hkv, G, 1, L, L]
    rows = (p * dp).sum(5, keepdim=True)
    ds = p * (dp - rows)
    ds[:, :, :, 1] *= -lam
    result["dv"] = torch.matmul(w.transpose(3, 4), do).sum(2).to(bf16)
    result["dq"] = (torch.matmul(ds, k) * scale).view(B, 2 * H, L, dq).to(bf16)
    dk = (torch.matmul(ds.transpose(4, 5), q) * scale).sum(2)  # [B, Hkv, 2, L, dq]
    dk = dk.sum(2) if n == 1 else dk.transpose(2, 3).reshape(B, Hkv, L, d)
    result["dk"] = dk.to(bf16)
    dlam = -rows[:, :, :, 1].reshape(B, H, L)
    result["dlam"] = dlam.double().sum((0, 2)).float() if case["lam"] == "head" else dlam
    return result


def _run_cache(s):
    case = s["case"]
    page, d, dq, Hkv, H = (case[n] for n in ("page", "d", "dq", "kv_heads", "heads"))
    scale = 1.0 / math.sqrt(dq)
    if own:
        import block_sparse_head_gb300 as bsa

        out, lse, _ = bsa.cache_diff_forward(
            s["q"], s["lam"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["kv_len"], s["cu"],
            scale, max_q=s["most"], window=case["window"], lut=s["lut"],
            block=_block(case) if s["lut"] is not None else None, workspace=s["workspace"])
        return {"out": out, "lse": lse}
    B, n, G, dev, maps = case["B"], s["most"], H // Hkv, s["q"].device, d // dq
    T = s["q"].shape[0]
    cu, kv_len = s["cu"].long(), s["kv_len"].long()
    count = cu[1:] - cu[:-1]
    i = torch.arange(n, device=dev)
    rows = (cu[:-1, None] + i[None]).clamp(max=T - 1)  # [B, n]
    q = s["q"][rows].float().view(B, n, Hkv, G, 2, dq).permute(0, 2, 4, 3, 1, 5)  # [B, Hkv, 2, G, n, dq]
    pos = (kv_len - count)[:, None] + i[None]  # [B, n]
    table, block = s["table"].clamp(min=0).long(), _block(case)
    k = (s["k_cache"][table].float() * s["k_scale"][table][..., None, None]).transpose(1, 2).flatten(2, 3)
    v = (s["v_cache"][table].float() * s["v_scale"][table][..., None, None]).transpose(1, 2).flatten(2, 3)
    N = k.shape[2]
    keys = torch.arange(N, device=dev)
    allowed = (keys <= pos[..., None])[:, None]  # [B, 1, n, N]
    if s["layout"] is not None:
        on = s["layout"][:, pos // block].transpose(0, 1)  # [B, Hkv, n, nb]
        allowed = allowed & (on.repeat_interleave(block, 3)[..., :N] > 0)
    if case["window"] >= 0:
        allowed = allowed & (keys >= pos[..., None] - case["window"])[:, None]
    v = v.masked_fill(~allowed.any(2)[..., None], 0.0)
    k = k.view(B, Hkv, N, maps, dq).transpose(2, 3)  # [B, Hkv, maps, N, dq]
    x = (torch.matmul(q.flatten(3, 4), k.transpose(3, 4)) * scale).view(B, Hkv, 2, G, n, N)
    x = x.masked_fill(~allowed[:, :, None, None], -math.inf)
    m = x.amax(5, keepdim=True)
    m = m.masked_fill(m == -math.inf, 0.0)
    x = torch.exp(x - m)
    z = x.sum(5, keepdim=True)
    lse = (m + torch.log(z))[..., 0].permute(0, 4, 1, 3, 2).reshape(B, n, 2 * H)
    x = x / z.masked_fill(z == 0, 1.0)
    lam = s["lam"][None, None].expand(B, n, H) if case["lam"] == "head" else s["lam"][rows]
    w = x[:, :, 0] - lam.view(B, n, Hkv, G).permute(0, 2, 3, 1)[..., None] * x[:, :, 1]
    o = torch.matmul(w.flatten(2, 3), v).view(B, Hkv, G, n, d).permute(0, 3, 1, 2, 4).reshape(B, n, H, d)
    t = torch.arange(T, device=dev)
    b = torch.searchsorted(cu, t, right=True) - 1
    return {"out": o[b, t - cu[b]].to(s["q"].dtype), "lse": lse[b, t - cu[b]]}


def _run_rotary(s):
    case = s["case"]
    if own:
        import block_sparse_head_gb300 as bsa

        q, k = bsa.rotary(s["q"], s["k"], s["positions"], s["table"], pairing=case["pairing"], inverse=case["inverse"])
        return {"q": q, "k": k}
    t = s["positions"][s["axis"]].double()  # [pairs, L] or [pairs, B, L]
    t = t * s["f"].view(-1, *[1] * (t.dim() - 1))
    t = t.movedim(0, -1).unsqueeze(1)  # [L, 1, pairs] or [B, 1, L, pairs]
    cos, sin = torch.cos(t).float(), torch.sin(t).float()
    if case["inverse"]:
        sin = -sin
    n = cos.shape[-1]

    def turn(x):
        y = x.float()
        if case["pairing"] == "half":
            a, b = y[..., :n], y[..., n: 2 * n]
            z = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
        else:
            a, b = y[..., 0: 2 * n: 2], y[..., 1: 2 * n: 2]
            z = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
        return torch.cat([z, y[..., 2 * n:]], -1).to(x.dtype)

    return {"q": turn(s["q"]), "k": turn(s["k"])}


# ------------------------------------------------------------------------- what it takes

def _pairs(case):
    """(query, key) pairs of all requests under one layout head, and the keys that any query sees."""
    old, new = _lengths(case)
    pairs = keys = 0
    lay = _layout(case, -(-max(a + n for a, n in zip(old, new)) // _block(case)))[0].bool() if case["layout"] else None
    block, w = _block(case), case["window"]
    for a, n in zip(old, new):
        pos = torch.arange(a, a + n)
        lo = (pos - w).clamp(min=0) if w >= 0 else torch.zeros_like(pos)
        if lay is None:
            pairs += int((pos - lo + 1).sum())
            keys += int(pos[-1] - lo[0] + 1)
            continue
        row, first = lay[pos // block].long(), torch.arange(lay.shape[1]) * block
        inside = torch.minimum(pos[:, None] + 1, first[None] + block) - torch.maximum(lo[:, None], first[None])
        inside = row * inside.clamp(min=0)
        pairs += int(inside.sum())
        keys += int(inside.amax(0).sum())
    return pairs, keys


def work(case):
    if case["op"] == "rotary":
        n = case["B"] * case["L"] * (case["heads"] + case["kv_heads"]) * case["d"]
        axes = len(case["pairs"].split(","))
        return {"bytes": 4.0 * n + 4.0 * axes * case["B"] * case["L"], "flops": 3.0 * n}
    H, Hkv, d, dq = (case[n] for n in ("heads", "kv_heads", "d", "dq"))
    if case["op"] == "cache":
        pairs, keys = _pairs(case)
        T = sum(_lengths(case)[1])
        return {"bytes": keys * Hkv * d * 2 + (keys / case["page"]) * (Hkv * 8 + 4) + T * H * (4 * dq + 2 * d + 12),
                "flops": pairs * H * (4.0 * dq + 4.0 * d)}
    B, L, b = case["B"], case["L"], case["block"]
    nb = -(-L // b)
    size = torch.full((nb,), b)
    size[-1] = L - (nb - 1) * b
    lay = _layout(case, nb)
    # a diagonal block of n rows has n (n + 1) / 2 pairs
    pairs = int((lay * size[:, None] * size[None]).sum()) - int((lay.diagonal(0, 1, 2) * (size * (size - 1) // 2)).sum())
    pairs = pairs * B * H // Hkv
    rows = B * L
    moved = rows * (2 * (2 * H * dq + 2 * Hkv * d + H * d) + 8 * H)
    moved += 4 * (rows * H if case["lam"] == "token" else H)
    if case["op"] == "forward":
        return {"bytes": float(moved), "flops": pairs * (4.0 * dq + 4.0 * d)}
    # and the upstream gradient, four gradients; two maps' scores again with their products for
    # queries and keys, one product each for dP and for the values
    moved += rows * 2 * (H * d + 2 * H * dq + 2 * Hkv * d) + 4 * (rows * H if case["lam"] == "token" else H)
    return {"bytes": float(moved), "flops": pairs * (4.0 * dq + 4.0 * d + 12.0 * dq + 4.0 * d)}


# ------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        return _exact_rotary(case, s)
    if case["op"] == "cache":
        return _exact_cache(case, s)
    B, H, Hkv, L, d, dq = (case[n] for n in ("B", "heads", "kv_heads", "L", "d", "dq"))
    f64 = dict(dtype=torch.float64, device="cuda")
    train, b = case["op"] == "train", case["block"]
    out, lse = torch.zeros(B, H, L, d, **f64), torch.zeros(B, 2 * H, L, **f64)
    gq, gk, gv = torch.zeros(B, 2 * H, L, dq, **f64), torch.zeros(B, Hkv, L, d, **f64), torch.zeros(B, Hkv, L, d, **f64)
    glam = torch.zeros(B, H, L, **f64)
    at = torch.arange(L, device="cuda")
    for kv in range(Hkv):
        hidden = s["layout"][kv][at // b][:, at // b] != 1
        hidden |= (at[:, None] // b == at // b) & (at > at[:, None])
        for batch in range(B):
            v = s["v"][batch, kv].double()
            for h in range(kv * (H // Hkv), (kv + 1) * (H // Hkv)):
                lam = s["lam"][h].double() if case["lam"] == "head" else s["lam"][batch, h].double()[:, None]
                dp = s["dout"][batch, h].double() @ v.T if train else None
                for m, weight in ((0, 1.0), (1, -lam)):
                    cols = slice(0, d) if dq == d else slice(m * dq, (m + 1) * dq)
                    q, k = s["q"][batch, 2 * h + m].double(), s["k"][batch, kv, :, cols].double()
                    x = (q @ k.T / math.sqrt(dq)).masked_fill_(hidden, -math.inf)
                    y = torch.logsumexp(x, 1)
                    lse[batch, 2 * h + m] = y
                    p = x.sub_(y.masked_fill(y == -math.inf, 0.0)[:, None]).exp_()
                    o = p @ v
                    out[batch, h] += weight * o
                    if not train:
                        continue
                    do = s["dout"][batch, h].double()
                    rows = (do * o).sum(1)
                    gv[batch, kv] += p.T @ (weight * do)
                    ds = p.mul_(dp - rows[:, None]).mul_(weight)
                    gq[batch, 2 * h + m] = ds @ k / math.sqrt(dq)
                    gk[batch, kv, :, cols] += ds.T @ q / math.sqrt(dq)
                    if m == 1:
                        glam[batch, h] = -rows
    if not train:
        return {"out": out, "lse": lse}
    return {"out": out, "lse": lse, "dq": gq, "dk": gk, "dv": gv,
            "dlam": glam.sum((0, 2)) if case["lam"] == "head" else glam}


def _exact_cache(case, s):
    page, d, dq, Hkv, H = (case[n] for n in ("page", "d", "dq", "kv_heads", "heads"))
    cu, lens = s["cu"].tolist(), s["kv_len"].tolist()
    T, block = s["q"].shape[0], _block(case)
    out = torch.zeros(T, H, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(T, 2 * H, dtype=torch.float64, device="cuda")
    for b in range(case["B"]):
        L, lo, hi = lens[b], cu[b], cu[b + 1]
        ids = s["table"][b, : -(-L // page)].long()
        pos = torch.arange(L - (hi - lo), L, device="cuda")
        c = torch.arange(L, device="cuda")
        for g in range(Hkv):
            on = c[None] <= pos[:, None]
            if case["window"] >= 0:
                on &= c[None] >= pos[:, None] - case["window"]
            if s["layout"] is not None:
                on &= s["layout"][g][pos // block][:, c // block] == 1
            k = (s["k_cache"][ids, g].double() * s["k_scale"][ids, g].double()[:, None, None]).flatten(0, 1)[:L]
            v = (s["v_cache"][ids, g].double() * s["v_scale"][ids, g].double()[:, None, None]).flatten(0, 1)[:L]
            for h in range(g * (H // Hkv), (g + 1) * (H // Hkv)):
                lam = s["lam"][h].double() if case["lam"] == "head" else s["lam"][lo:hi, h].double()[:, None]
                for m, weight in ((0, 1.0), (1, -lam)):
                    key = k if dq == d else k[:, m * dq: (m + 1) * dq]
                    x = s["q"][lo:hi, 2 * h + m].double() @ key.T / math.sqrt(dq)
                    x = torch.where(on, x, -math.inf)
                    y = torch.logsumexp(x, 1)
                    lse[lo:hi, 2 * h + m] = y
                    out[lo:hi, h] += weight * (torch.exp(x - torch.where(y == -math.inf, 0.0, y)[:, None]) @ v)
    return {"out": out, "lse": lse}


def _exact_rotary(case, s):
    """Each pair as a complex number times exp(i angle)."""
    f, axis = _frequencies(case)
    sign = -1.0 if case["inverse"] else 1.0
    n, done = len(f), {}
    for name in ("q", "k"):
        x = s[name].double().clone()
        for i in range(n):
            a, b = (i, i + n) if case["pairing"] == "half" else (2 * i, 2 * i + 1)
            angle = (sign * f[i] * s["positions"][axis[i]].double()).unsqueeze(1)
            z = torch.complex(x[..., a], x[..., b]) * torch.polar(torch.ones_like(angle), angle)
            x[..., a], x[..., b] = z.real, z.imag
        done[name] = x
    return done

"""Workloads of the serving path over a paged 8-bit key/value cache, with their plain forms.

Three operators, in the order in which a serving step calls them:

* ``cache_resize``: block tables, packed query offsets and the slot of every new token,
  from the lengths that the requests have and are to have;
* ``cache_append``: the new tokens' keys and values into the cache, 8 bits a number with
  one power-of-two scale for each page of tokens and key/value head;
* ``cache_forward``: attention of each request's newest tokens over its cache, dense or
  over the active blocks of a layout.

``run`` computes them in elementary torch operations, or, where ``own`` is true, through
the framework's entry points.
"""

import math

import torch

own = False

QMAX = {"e4m3": 448.0, "int8": 127.0}
CACHE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
LOG_LO, LOG_HI = -60, 60  # scales are powers of two in [2^-60, 2^60]


# ------------------------------------------------------------------------- the cases

def listed():
    return [
        # A decode step of a small server: each of 32 requests grows by one token.
        dict(name="resize-decode-32", op="resize", B=32, page=64, longest=8192, prefill=0, leave=0.0),
        # A mixed step of a large one: 1000 requests, some admitted with whole prompts,
        # most decoding, some leaving; pages of 16 tokens, odd counts.
        dict(name="resize-mixed-1000", op="resize", B=1000, page=16, longest=4096, prefill=60, leave=0.05),
        # One token each of 64 requests, the append of a decode step.
        dict(name="append-decode-64", op="append", B=64, new=1, old=4096, kv_heads=8, d=128, page=64,
             cache="e4m3", dtype="bf16"),
        # Ragged prompt chunks with a fused projection's strides: small pages, small heads.
        dict(name="append-ragged-1000", op="append", B=5, new=200, old=333, kv_heads=16, d=64, page=16,
             cache="int8", dtype="fp16"),
        # A prompt of 16384 tokens in one call, the largest append.
        dict(name="append-prefill-16384", op="append", B=1, new=16384, old=0, kv_heads=8, d=128, page=64,
             cache="e4m3", dtype="bf16"),
        # One request's decode step with a short history: latency.
        dict(name="decode-1x1000", op="forward", B=1, new=1, old=999, ragged=False, heads=32, kv_heads=8,
             d=128, page=64, cache="e4m3", dtype="bf16", window=-1, softcap=0.0, sinks=False, layout=""),
        # A batch of requests of many lengths: throughput of the ordinary decode step.
        dict(name="decode-64x8192", op="forward", B=64, new=1, old=8191, ragged=True, heads=32, kv_heads=8,
             d=128, page=64, cache="e4m3", dtype="bf16", window=-1, softcap=0.0, sinks=False, layout=""),
        # Few long contexts: the key axis has to be split.
        dict(name="decode-4x65536", op="forward", B=4, new=1, old=65535, ragged=False, heads=32, kv_heads=8,
             d=128, page=128, cache="e4m3", dtype="bf16", window=-1, softcap=0.0, sinks=False, layout=""),
        # Decoding under the band-and-stride block layout, one layout row for each head.
        dict(name="decode-layout-8x65536", op="forward", B=8, new=1, old=65535, ragged=True, heads=32, kv_heads=32,
             d=128, page=128, cache="e4m3", dtype="bf16", window=-1, softcap=0.0, sinks=False, layout="strided"),
        # Four draft tokens verified at once, int8 cache, small heads and pages, sinks.
        dict(name="verify-16x4096", op="forward", B=16, new=4, old=4096, ragged=True, heads=32, kv_heads=8,
             d=64, page=16, cache="int8", dtype="fp16", window=1000, softcap=30.0, sinks=True, layout=""),
        # A chunk of a long prompt against what is cached so far.
        dict(name="chunk-1x2048", op="forward", B=1, new=2048, old=14336, ragged=False, heads=32, kv_heads=8,
             d=128, page=64, cache="e4m3", dtype="bf16", window=-1, softcap=0.0, sinks=False, layout=""),
        # Chunks of several prompts under the window-and-global layout, odd lengths.
        dict(name="chunk-layout-3x1000", op="forward", B=3, new=1000, old=7001, ragged=True, heads=16, kv_heads=16,
             d=128, page=64, cache="int8", dtype="bf16", window=-1, softcap=0.0, sinks=False, layout="window"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["resize", "append", "append", "forward", "forward", "forward", "forward"])
    page = rng.choice([16, 32, 64, 128])
    if op == "resize":
        return dict(op=op, B=_log(rng, 1, 1024), page=page, longest=_log(rng, 16, 4096),
                    prefill=rng.choice([0, 3, 60]), leave=rng.choice([0.0, 0.05, 0.3]))
    case = dict(op=op, page=page, d=rng.choice([64, 128]), cache=rng.choice(["e4m3", "int8"]),
                dtype=rng.choice(["bf16", "fp16"]))
    if op == "append":
        case.update(B=_log(rng, 1, 64), kv_heads=rng.choice([1, 2, 4, 8, 16]), old=_log(rng, 1, 2000) - 1)
        new = rng.choice([1, 0])
        return dict(case, new=new or _log(rng, 2, max(2, 16384 // (case["B"] * case["kv_heads"] // 8 + 1))))
    kind = rng.choice(["decode", "decode", "verify", "chunk"])
    kv_heads = rng.choice([1, 2, 4, 8, 16])
    group = rng.choice([1, 2, 3, 4, 7, 8, 16])
    if kv_heads * group > 32:
        group = 2
    if kind == "chunk":
        B, new, old = _log(rng, 1, 4), _log(rng, 17, 1000), _log(rng, 1, 6000)
    else:
        B = _log(rng, 1, 64)
        new = 1 if kind == "decode" else rng.randint(2, 8)
        old = _log(rng, 1, min(60000, 2 * 10 ** 6 // (B * kv_heads)))
    return dict(case, B=B, new=new, old=old, ragged=rng.random() < 0.7, heads=kv_heads * group, kv_heads=kv_heads,
                window=rng.choice([-1, -1, -1, 0, 777]), softcap=rng.choice([0.0, 0.0, 30.0]),
                sinks=rng.random() < 0.3, layout=rng.choice(["", "", "strided", "window"]))


def _lengths(case):
    """Old lengths and new tokens of each request, as Python numbers; one set for a case, so
    that its outputs have one shape."""
    g = torch.Generator().manual_seed(7919 * case["B"] + case["page"])
    B = case["B"]
    if case["op"] == "resize":
        old = torch.randint(0, case["longest"] + 1, (B,), generator=g)
        new = old + 1
        admit = torch.randperm(B, generator=g)[: case["prefill"]]
        prompt = torch.randint(1, case["longest"] + 1, (B,), generator=g)
        old[admit], new[admit] = 0, prompt[admit]
        left = torch.rand(B, generator=g) < case["leave"]
        left[admit] = False
        new[left] = 0
        return old.tolist(), new.tolist()
    old, new = torch.full((B,), case["old"]), torch.full((B,), case["new"])
    if case["op"] == "append" and B > 1:
        old = torch.randint(0, 2 * case["old"] + 1, (B,), generator=g)
        if case["new"] > 1:
            new = torch.randint(1, 2 * case["new"], (B,), generator=g)
    if case["op"] == "forward" and case["ragged"]:
        # A quarter of the longest and more; the first request has the longest.
        old[1:] = torch.randint(case["old"] // 4, case["old"] + 1, (B,), generator=g)[1:]
        if case["new"] > 1:
            new[1:] = torch.randint(1, case["new"] + 1, (B,), generator=g)[1:]
    return old.tolist(), new.tolist()


def _block(case):
    return 128 if case["page"] == 128 else 64


def _layout(case, positions):
    """The repository's two causal layouts, [kv_heads, nb, nb]: a band of 8 blocks with every
    16th column, and a window of 4 blocks with the first column."""
    nb = -(-positions // _block(case))
    i, j = torch.arange(nb)[:, None], torch.arange(nb)[None, :]
    if case["layout"] == "strided":
        on = (j <= i) & ((j > i - 8) | (j % 16 == 15))
    else:
        on = (j <= i) & ((j > i - 4) | (j == 0))
    return on.to(torch.int32)[None].repeat(case["kv_heads"], 1, 1).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ints = dict(dtype=torch.int32, device="cuda")
    old, new = _lengths(case)
    B, page = case["B"], case["page"]
    if case["op"] == "resize":
        lens = [max(a, b) for a, b in zip(old, new)]
        width = -(-max(lens) // page) + 1
        tokens = -(-max(1, sum(max(0, b - a) for a, b in zip(old, new))) // 64) * 64
        held = [-(-a // page) for a in old]
        pages = sum(-(-x // page) for x in lens) + 7
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        table = torch.full((B, width), -1, **ints)
        at = 0
        for b, n in enumerate(held):
            table[b, :n] = order[at: at + n]
            at += n
        free = torch.full((pages,), -1, **ints)
        free[: pages - at] = order[at:]
        return dict(case=case, table=table, old=torch.tensor(old, **ints), new=torch.tensor(new, **ints), free=free,
                    count=torch.tensor([pages - at], **ints), tokens=tokens, lens_out=torch.empty(B, **ints),
                    count_out=torch.empty(1, **ints), cu=torch.empty(B + 1, **ints),
                    slots=torch.empty(tokens, **ints), status=torch.empty(1, **ints))

    H, d, dtype, kind = case["kv_heads"], case["d"], TYPES[case["dtype"]], case["cache"]
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
        c = torch.empty(pages, H, page, d, dtype=CACHE[kind], device="cuda")
        flat, step = c.view(-1), 1 << 27
        for lo in range(0, flat.numel(), step):  # stored numbers spread over the type's range
            x = torch.randn(min(step, flat.numel() - lo), generator=g, device="cuda") * (QMAX[kind] / 4.2)
            flat[lo: lo + step] = (x.round() if kind == "int8" else x).clamp(-QMAX[kind], QMAX[kind]).to(c.dtype)
        caches.append(c)
        e = torch.randint(-1, 2, (pages, H), generator=g, device="cuda")
        scales.append(_power(e + round(math.log2(4.2 / QMAX[kind]))))
    T = sum(new)
    state = dict(case=case, k_cache=caches[0], v_cache=caches[1], k_scale=scales[0], v_scale=scales[1], table=table,
                 kv_len=torch.tensor(total, **ints), most=max(new))
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    state["cu"] = torch.tensor(cu, **ints)
    if case["op"] == "append":
        # Keys and values are slices of one projection's rows; the last tokens of the
        # capacity are padding. The spread of the tokens varies, so scales grow now and then.
        cap = T if case["new"] == 1 else T + 3
        rows = torch.randn(cap, 4 * H, d, generator=g, device="cuda")
        rows *= torch.exp(0.5 * torch.randn(cap, 1, 1, generator=g, device="cuda"))
        rows = rows.to(dtype)
        state["k"], state["v"] = rows[:, 2 * H: 3 * H], rows[:, 3 * H:]
        slots = torch.full((cap,), -1, dtype=torch.int32)
        for b in range(B):
            p = torch.arange(old[b], total[b])
            slots[cu[b]: cu[b + 1]] = table[b].cpu()[p // page] * page + (p % page).to(torch.int32)
        state["slots"] = slots.cuda()
        state["touched"] = cap // page + 2 * B + 1  # pages that the new tokens can lie in
        return state
    heads = case["heads"]
    state["q"] = torch.randn(T, heads, d, generator=g, device="cuda").to(dtype)
    state["sinks"] = torch.randn(heads, generator=g, device="cuda") if case["sinks"] else None
    state["out"] = torch.empty_like(state["q"])
    state["lse"] = torch.empty(T, heads, device="cuda")
    state["layout"] = state["lut"] = state["workspace"] = None
    if case["layout"]:
        layout = _layout(case, table.shape[1] * page)
        state["layout"], state["listed"] = layout.cuda(), int(layout.sum(2).max())
    if own:  # the layout's look-up table and the workspace, which a program makes once
        import block_sparse_head_gb300 as bsa

        if case["layout"]:
            state["lut"] = bsa.build_lut(layout, 1)
        state["workspace"] = bsa.cache_workspace(heads, H, d, state["most"])
    return state


# ------------------------------------------------------------------------- the passes

def run(state):
    return {"resize": _run_resize, "append": _run_append, "forward": _run_forward}[state["case"]["op"]](state)


def _run_resize(s):
    page, tokens = s["case"]["page"], s["tokens"]
    if own:
        import block_sparse_head_gb300 as bsa

        bsa.cache_resize(s["table"], s["old"], s["new"], s["free"], s["count"], page, tokens, kv_len_out=s["lens_out"],
                         free_count_out=s["count_out"], cu_new=s["cu"], slots=s["slots"], status=s["status"])
        return {"table": s["table"], "lens": s["lens_out"], "free": s["free"], "count": s["count_out"], "cu": s["cu"],
                "slots": s["slots"], "status": s["status"]}
    # A request that grows takes pages from the end of (free pages, then freed ones in the
    # order of requests and pages); one that shrinks gives back those behind its new length.
    old, new, table, free, count = s["old"].long(), s["new"].long(), s["table"], s["free"], s["count"].long()
    B, width = table.shape
    dev = table.device
    had, has = (old + page - 1) // page, (new + page - 1) // page
    grow, shrink = (has - had).clamp(min=0), (had - has).clamp(min=0)
    fresh = (new - old).clamp(min=0)
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), fresh.cumsum(0)])
    before, freed_before = grow.cumsum(0) - grow, shrink.cumsum(0) - shrink
    needed, freed = grow.sum(), shrink.sum()
    short = needed - freed - count
    bad = (new < 0) | (new > width * page) | (old < 0) | (old > width * page)
    first_bad = torch.where(bad, torch.arange(B, device=dev), B).min()
    status = torch.where(first_bad < B, -1 - first_bad,
                         torch.where(cu[-1] > tokens, torch.full_like(first_bad, -2 ** 31), short.clamp(min=0)))
    ok = status == 0
    # the stack of pages: the free ones, then the freed ones
    cols = torch.arange(width, device=dev)[None]
    leaving = (cols >= has[:, None]) & (cols < had[:, None])
    at = count + freed_before[:, None] + cols - has[:, None]
    stack = torch.cat([free, torch.zeros(1, dtype=free.dtype, device=dev)])
    n = free.numel()
    stack = stack.scatter(0, torch.where(leaving & ok, at, n).clamp(max=n).flatten(), table.flatten())[:n]
    arriving = (cols >= had[:, None]) & (cols < has[:, None]) & ok
    take = (count + freed - 1 - before[:, None] - (cols - had[:, None])).clamp(0, n - 1)
    out_table = torch.where(arriving, stack[take], table)
    t = torch.arange(tokens, device=dev)
    b = torch.searchsorted(cu, t, right=True) - 1
    live = (t < cu[-1]) & ok
    b = b.clamp(0, B - 1)
    p = old[b] + t - cu[b]
    slot = out_table[b, (p // page).clamp(0, width - 1)].long() * page + p % page
    i32 = torch.int32
    # pages of the stack that were taken keep their number behind the count
    return {"table": out_table, "lens": torch.where(ok, new, old).to(i32), "free": stack,
            "count": torch.where(ok, count + freed - needed, count).to(i32), "cu": torch.where(ok, cu, 0).to(i32),
            "slots": torch.where(live, slot, -1).to(i32), "status": status.to(i32).view(1)}


def _power(e):
    """2^e in fp32 from its bits: a library's power need not be exact."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _scale_of(amax, qmax):
    """The smallest power of two s in range with amax <= qmax * s."""
    m, e = torch.frexp(amax)
    mq, eq = math.frexp(qmax)
    e = (e - eq + (m > mq).to(e.dtype)).clamp(LOG_LO, LOG_HI)
    e = torch.where(amax > 0, e, torch.full_like(e, LOG_LO))
    return _power(e)


def _run_append(s):
    case = s["case"]
    page = case["page"]
    if own:
        import block_sparse_head_gb300 as bsa

        bsa.cache_append(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
        return {"k": s["k_cache"], "v": s["v_cache"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    # A page's run of new tokens begins where the page changes; tokens before it are kept.
    slots, M, qmax = s["slots"].long(), s["touched"], QMAX[case["cache"]]
    live = slots >= 0
    pid = torch.where(live, slots // page, -1)
    first = live & (pid != torch.cat([pid.new_full((1,), -1), pid[:-1]]))
    run_of = torch.where(live, first.cumsum(0) - 1, M)  # number of the token's run; M: padding
    pages = pid.new_zeros(M + 1).scatter(0, run_of, pid.clamp(min=0))[:M]
    start = pid.new_zeros(M + 1).scatter(0, torch.where(first, run_of, M), torch.where(first, slots % page, 0))[:M]
    used = (torch.arange(M, device=slots.device) <= first.sum() - 1)[:, None]
    offs = torch.arange(page, device=slots.device)
    H, d = case["kv_heads"], case["d"]

    def one(x, cache, scale):
        x = x.float()
        a = torch.where(x.isfinite(), x.abs(), 0).amax(2)  # [T, H]
        amax = a.new_zeros(M + 1, H).scatter_reduce(0, run_of[:, None].expand(-1, H), a, "amax")[:M]
        was = torch.where((start > 0)[:, None], scale[pages], 0)
        now = torch.maximum(was, _scale_of(amax, qmax))
        y = cache[pages].float() * torch.where(was > 0, was / now, 1.0)[:, :, None, None]
        kept = (offs[None] < start[:, None])[:, None, :, None]
        back = cache[pages].float()
        y = torch.where(kept, y, back)
        z = x / now[run_of.clamp(max=M - 1)][:, :, None]
        y = torch.cat([y.transpose(1, 2), y.new_zeros(1, page, H, d)])  # [M + 1, page, H, d]
        y[run_of, slots % page] = z
        y = y[:M].transpose(1, 2)
        y = (y.round() if case["cache"] == "int8" else y).clamp(-qmax, qmax).to(cache.dtype)
        # Unused places of the list write page 0's row back as it is: point them at run 0.
        src = torch.where(used[:, 0], torch.arange(M, device=slots.device), 0)
        cache.view(torch.uint8)[pages[src]] = y.view(torch.uint8)[src]
        scale[pages[src]] = now[src]

    one(s["k"], s["k_cache"], s["k_scale"])
    one(s["v"], s["v_cache"], s["v_scale"])
    return {"k": s["k_cache"], "v": s["v_cache"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _run_forward(s):
    case = s["case"]
    page, d, H, heads = case["page"], case["d"], case["kv_heads"], case["heads"]
    scale = 1.0 / math.sqrt(d)
    if own:
        import block_sparse_head_gb300 as bsa

        out, lse, _ = bsa.cache_forward(
            s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["kv_len"], s["cu"], scale,
            max_q=s["most"], window=case["window"], softcap=case["softcap"], sinks=s["sinks"], lut=s["lut"],
            block=_block(case) if s["lut"] is not None else None, out=s["out"], lse=s["lse"],
            workspace=s["workspace"])
        return {"out": out, "lse": lse}
    B, n, G, dev = case["B"], s["most"], heads // H, s["q"].device
    cu, kv_len = s["cu"].long(), s["kv_len"].long()
    count = cu[1:] - cu[:-1]
    i = torch.arange(n, device=dev)
    rows = (cu[:-1, None] + i[None]).clamp(max=s["q"].shape[0] - 1)  # [B, n]
    q = s["q"][rows].float().view(B, n, H, G, d).permute(0, 2, 3, 1, 4)  # [B, H, G, n, d]
    pos = (kv_len - count)[:, None] + i[None]  # [B, n]
    table = s["table"].clamp(min=0).long()
    block = _block(case)
    if s["layout"] is not None and n == 1:
        # one query a request: only the blocks that its layout row lists, [B, H, listed]
        on = s["layout"][:, pos[:, 0] // block].transpose(0, 1)
        on, at = torch.sort(on, dim=2, descending=True, stable=True)
        on, at = on[:, :, : s["listed"]] > 0, at[:, :, : s["listed"]]
        sub = block // page if page < block else 1
        keys = (at[..., None] * block + torch.arange(block, device=dev)).flatten(2)  # [B, H, N]
        pages = (at[..., None] * sub + torch.arange(sub, device=dev)).flatten(2)
        ids = torch.gather(table[:, None].expand(-1, H, -1), 2, pages.clamp(max=table.shape[1] - 1))
        hs = torch.arange(H, device=dev)[None, :, None]
        k, v = s["k_cache"][ids, hs].float(), s["v_cache"][ids, hs].float()
        k, v = k * s["k_scale"][ids, hs][..., None, None], v * s["v_scale"][ids, hs][..., None, None]
        k, v = k.flatten(2, 3), v.flatten(2, 3)
        allowed = (on.repeat_interleave(block, 2) & (keys <= pos[:, :, None]))[:, :, None]  # [B, H, 1, N]
        keys = keys[:, :, None]
    else:
        k = (s["k_cache"][table].float() * s["k_scale"][table][..., None, None]).transpose(1, 2).flatten(2, 3)
        v = (s["v_cache"][table].float() * s["v_scale"][table][..., None, None]).transpose(1, 2).flatten(2, 3)
        keys = torch.arange(k.shape[2], device=dev)[None, None, None]
        allowed = keys <= pos[:, None, :, None]  # [B, 1, n, N]
        if s["layout"] is not None:
            rows_on = s["layout"][:, (pos // block).clamp(max=s["layout"].shape[1] - 1)]  # [H, B, n, nb]
            allowed = allowed & (rows_on.transpose(0, 1).repeat_interleave(block, 3)[..., : k.shape[2]] > 0)
    if case["window"] >= 0:
        allowed = allowed & (keys >= pos[:, None, :, None] - case["window"])
    allowed = allowed[:, :, None]  # [B, H or 1, 1, n, N]
    v = v.masked_fill(~allowed.any(3).squeeze(2)[..., None], 0.0)
    x = (torch.matmul(q.flatten(2, 3), k.transpose(2, 3)) * scale).view(B, H, G, n, -1)
    if case["softcap"] > 0:
        x = case["softcap"] * torch.tanh(x / case["softcap"])
    x = x.masked_fill(~allowed, -math.inf)
    m = x.amax(4, keepdim=True)
    if s["sinks"] is not None:
        m = torch.maximum(m, s["sinks"].view(1, H, G, 1, 1))
    m = m.masked_fill(m == -math.inf, 0.0)
    x = torch.exp(x - m)
    z = x.sum(4, keepdim=True)
    if s["sinks"] is not None:
        z = z + torch.exp(s["sinks"].view(1, H, G, 1, 1) - m)
    o = torch.matmul(x.flatten(2, 3), v).view(B, H, G, n, d) / z.masked_fill(z == 0, 1.0)
    lse = (m + torch.log(z))[..., 0]
    t = torch.arange(s["q"].shape[0], device=dev)
    b = torch.searchsorted(cu, t, right=True) - 1
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n, heads, d)[b, t - cu[b]]
    return {"out": o.to(s["q"].dtype), "lse": lse.permute(0, 3, 1, 2).reshape(B, n, heads)[b, t - cu[b]]}


# ------------------------------------------------------------------------- what it takes

def _pairs(case, old, new):
    """(query, key) pairs of all requests under one layout head, and the keys that any query sees."""
    pairs = keys = 0
    lay = _layout(case, max(a + n for a, n in zip(old, new)))[0].bool() if case["layout"] else None
    block, w = _block(case), case["window"]
    for a, n in zip(old, new):
        pos = torch.arange(a, a + n)
        lo = (pos - w).clamp(min=0) if w >= 0 else torch.zeros_like(pos)
        if lay is None:
            pairs += int((pos - lo + 1).sum())
            keys += int(pos[-1] - lo[0] + 1)
            continue
        row, first = lay[pos // block].long(), torch.arange(lay.shape[1]) * block
        inside = (torch.minimum(pos[:, None] + 1, first[None] + block) - torch.maximum(lo[:, None], first[None])).clamp(min=0)
        pairs += int((row * inside).sum())
        keys += int((row * inside).amax(0).sum())
    return pairs, keys


def work(case):
    old, new = _lengths(case)
    page = case["page"]
    if case["op"] == "resize":
        grown = sum(max(0, -(-b // page) - -(-a // page)) for a, b in zip(old, new))
        freed = sum(max(0, -(-a // page) - -(-b // page)) for a, b in zip(old, new))
        tokens = sum(max(0, b - a) for a, b in zip(old, new))
        # lengths in and out, offsets, a page read and written for each that moves, a slot
        # for each new token and the page that it continues
        return {"bytes": 4.0 * (4 * case["B"] + 2 * (grown + freed) + tokens + case["B"]), "flops": 0}
    H, d = case["kv_heads"], case["d"]
    if case["op"] == "append":
        T = sum(new)
        runs = sum(-(-(a + n) // page) - a // page for a, n in zip(old, new))
        return {"bytes": T * H * d * 2 * (2 + 1) + T * 4 + runs * H * 2 * 8, "flops": 4.0 * T * H * d}
    pairs, keys = _pairs(case, old, new)
    T, heads = sum(new), case["heads"]
    return {"bytes": keys * H * d * 2 + (keys / page) * (H * 8 + 4) + T * heads * (4 * d + 4),
            "flops": 4.0 * pairs * heads * d}


# ------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    if case["op"] == "resize":
        return None  # whole numbers
    s = prepare(case, seed)
    page, d, H = case["page"], case["d"], case["kv_heads"]
    if case["op"] == "append":
        slots, out, qmax = s["slots"].tolist(), {}, QMAX[case["cache"]]
        runs = []
        for t, slot in enumerate(slots):
            if slot < 0:
                continue
            if runs and runs[-1][0] == slot // page:
                runs[-1][2].append(t)
            else:
                runs.append([slot // page, slot % page, [t]])
        for name in ("k", "v"):
            cache, scale, x = s[name + "_cache"].double(), s[name + "_scale"].double(), s[name].double()
            for p, start, at in runs:
                rows = x[at[0]: at[-1] + 1].transpose(0, 1)  # [H, tokens, d]
                top = rows.abs().amax((1, 2))
                m, e = torch.frexp(top.clamp(min=2.0 ** -200) / qmax)  # in [1/2, 1) times 2^e
                e = (e - (m == 0.5).to(e.dtype)).clamp(LOG_LO, LOG_HI).tolist()
                need = torch.tensor([math.ldexp(1.0, i) for i in e], dtype=top.dtype, device=top.device)
                now = torch.maximum(need, scale[p]) if start else need
                if start:
                    kept = cache[p, :, :start] * (scale[p] / now)[:, None, None]
                    cache[p, :, :start] = _stored(kept, case["cache"])
                cache[p, :, start: start + len(at)] = _stored(rows / now[:, None, None], case["cache"])
                scale[p] = now
            out[name], out[name + "_scale"] = cache, scale
        return out
    heads, G = case["heads"], case["heads"] // H
    cu, lens = s["cu"].tolist(), s["kv_len"].tolist()
    out, lse = s["q"].double(), s["lse"].double()
    block = _block(case)
    for b in range(case["B"]):
        L, n = lens[b], cu[b + 1] - cu[b]
        if n == 0:
            continue
        ids = s["table"][b, : -(-L // page)].long()
        pos = torch.arange(L - n, L, device="cuda")
        c = torch.arange(L, device="cuda")
        for h in range(H):
            on = c[None] <= pos[:, None]
            if case["window"] >= 0:
                on &= c[None] >= pos[:, None] - case["window"]
            if s["layout"] is not None:
                on &= s["layout"][h][pos // block][:, c // block] == 1
            k = (s["k_cache"][ids, h].double() * s["k_scale"][ids, h].double()[:, None, None]).flatten(0, 1)[:L]
            v = (s["v_cache"][ids, h].double() * s["v_scale"][ids, h].double()[:, None, None]).flatten(0, 1)[:L]
            for r in range(h * G, (h + 1) * G):
                x = s["q"][cu[b]: cu[b + 1], r].double() @ k.T / math.sqrt(d)
                if case["softcap"] > 0:
                    x = case["softcap"] * torch.tanh(x / case["softcap"])
                x = torch.where(on, x, -math.inf)
                y = torch.logsumexp(x, 1)
                if s["sinks"] is not None:
                    y = torch.logaddexp(y, s["sinks"][r].double())
                out[cu[b]: cu[b + 1], r] = torch.exp(x - torch.where(y == -math.inf, 0.0, y)[:, None]) @ v
                lse[cu[b]: cu[b + 1], r] = y
    return {"out": out, "lse": lse}


def _stored(x, kind):
    """x, |x| <= the type's largest value, rounded to the nearest stored number, ties to even."""
    if kind == "int8":
        return torch.round(x)
    e = (torch.frexp(x)[1] - 1).clamp(min=-6)
    step = torch.pow(2.0, e - 3).float().double()  # to the power of two next to it
    return torch.round(x / step) * step

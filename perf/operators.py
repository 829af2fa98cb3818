"""What is measured of the operators that serve many requests from an 8-bit, paged KV cache.

Four operators are run one after the other in a serving step:

- rope    rotary positions of a packed batch: half or interleaved pairs, all or part of the head,
          frequencies scaled for long contexts, and the transposed rotation (the gradient)
- plan    block table, slot map, positions and write runs of a batch, from request lengths
- append  the new tokens' K and V rows written to 8-bit pages with one scale per page and head
- attend  attention of the new tokens over each request's pages

`run` makes the framework's calls where `own` is true and computes the same in elementary torch
operations where it is false. `exact` restates the definitions in 64 bits.

Head shapes are those of the framework's workloads: 32 or 64 query heads on 8 KV heads of 128, and
4 heads on 1 KV head of 64.
"""
import math
import random

import torch

own = False

E4M3_MAX, INT8_MAX = 448.0, 127.0
SCALE_FLOOR = 2.0 ** -100


# ---- cases -------------------------------------------------------------------------------------
def listed():
    return [
        # one decode step of 16 requests: Q and K heads of a fused QKV buffer rotated in one call
        dict(name="rope-decode-16", op="rope", tokens=16, heads=40, extra=8, dim=128, rot=128,
             style="half", scaling="llama3", transpose=False, far=131072),
        # a prefill of 16K tokens with YaRN frequencies
        dict(name="rope-prefill-16k", op="rope", tokens=16384, heads=40, extra=8, dim=128, rot=128,
             style="half", scaling="yarn", transpose=False, far=1000000),
        # the gradient of an interleaved rotation of half the head, odd sizes
        dict(name="rope-part-grad", op="rope", tokens=1001, heads=5, extra=0, dim=64, rot=32,
             style="interleaved", scaling="linear", transpose=True, far=40000),
        # one decode step's bookkeeping
        dict(name="plan-decode-16", op="plan", batch=16, page=64, ctx=16384, prefill=0, long=0, pad=0),
        # a mixed step: most requests decode, some bring a prompt; a padded token buffer
        dict(name="plan-mixed-256", op="plan", batch=256, page=16, ctx=8192, prefill=24, long=1024,
             pad=77),
        # one decode step's rows into pages that hold earlier rows
        dict(name="append-decode-16", op="append", batch=16, page=64, ctx=16384, prefill=0, long=0,
             heads=8, dim=128, kind="e4m3"),
        # prompts of 16K tokens in all
        dict(name="append-prefill-16k", op="append", batch=4, page=64, ctx=0, prefill=4, long=4096,
             heads=8, dim=128, kind="e4m3"),
        # a ragged mixed step in int8
        dict(name="append-mixed-int8", op="append", batch=33, page=32, ctx=999, prefill=5, long=701,
             heads=1, dim=64, kind="int8"),
        # one request, one token, a short cache: latency
        dict(name="attend-short-int8", op="attend", batch=1, new=1, kv=501, ragged=False, q=4, kvh=1,
             dim=64, page=16, kind="int8"),
        # a decode step of 16 requests of very different lengths
        dict(name="attend-decode-16", op="attend", batch=16, new=1, kv=16384, ragged=True, q=32,
             kvh=8, dim=128, page=64, kind="e4m3"),
        # a decode step over one context of a million tokens
        dict(name="attend-decode-1m", op="attend", batch=1, new=1, kv=1048577, ragged=False, q=32,
             kvh=8, dim=128, page=64, kind="e4m3"),
        # a query chunk of 256 tokens after a 128K context
        dict(name="attend-chunk-128k", op="attend", batch=1, new=256, kv=131328, ragged=False, q=64,
             kvh=8, dim=128, page=64, kind="e4m3"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "plan", "append", "attend", "attend"])
    page = rng.choice([16, 32, 64, 128])
    kind = rng.choice(["e4m3", "int8"])
    heads, dim = rng.choice([(8, 128), (8, 128), (1, 64), (2, 64), (5, 128)])
    if op == "rope":
        dim = rng.choice([64, 128])
        h = rng.choice([1, 5, 8, 24, 40])
        return dict(op=op, tokens=_log(rng, 1, 16384), heads=h, extra=rng.choice([0, 0, 3, 8]),
                    dim=dim, rot=rng.choice([r for r in (16, 32, 48, 64, 96, 128) if r <= dim]),
                    style=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "ntk", "yarn", "llama3"]),
                    transpose=rng.random() < 0.3, far=_log(rng, 100, 2000000))
    if op == "plan":
        b = _log(rng, 1, 512)
        pre = rng.randint(0, min(b, 24))
        return dict(op=op, batch=b, page=page, ctx=_log(rng, 1, 20000), prefill=pre,
                    long=_log(rng, 2, 1024) if pre else 0, pad=rng.choice([0, 0, 1, 300]))
    if op == "append":
        b = _log(rng, 1, 64)
        pre = rng.randint(0, min(b, 4))
        return dict(op=op, batch=b, page=page, ctx=_log(rng, 1, 16384), prefill=pre,
                    long=_log(rng, 2, 4096) if pre else 0, heads=heads, dim=dim, kind=kind)
    g = rng.choice([1, 2, 4, 4, 8, 8, 3, 7])
    if rng.random() < 0.6:  # decode, or a few drafted tokens
        b, new = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 5])
        kv = max(new, _log(rng, 1, min(1048576, 8 * 1048576 // (b * heads))))
    else:                   # a query chunk or a prompt's next piece
        b, new = rng.choice([1, 1, 2, 3]), _log(rng, 17, 1024)
        g = rng.choice([2, 4, 8])
        top = 16 * 1048576 // (b * new * heads * g) * 128
        kv = new + _log(rng, 1, max(2, min(131072, top)))
    return dict(op=op, batch=b, new=new, kv=kv, ragged=rng.random() < 0.6, q=g * heads, kvh=heads,
                dim=dim, page=page, kind=kind)


def work(case):
    """Bytes and operations that a pass cannot do without: each input read once, each output
    written once; two operations for a product and its sum."""
    if case["op"] == "rope":
        n = case["tokens"] * case["heads"] * case["dim"]
        return {"bytes": 4 * n + 4 * case["tokens"], "flops": 3 * n * case["rot"] / case["dim"]}
    if case["op"] in ("plan", "append"):
        ctx, new = _lengths(case)
        page, n, b = case["page"], sum(new), case["batch"]
        added = sum(-(-(c + t) // page) - -(-c // page) for c, t in zip(ctx, new))
        if case["op"] == "plan":
            return {"bytes": 4 * (4 * b + 2 * added + 2 * n), "flops": n}
        touched = sum(-(-(c + t) // page) - c // page for c, t in zip(ctx, new) if t)
        rows = n * case["heads"] * case["dim"]
        return {"bytes": 2 * (3 * rows + 8 * touched * case["heads"]) + 4 * n, "flops": 4 * rows}
    lens, new = _kv_lengths(case), case["new"]
    rows = case["batch"] * new * case["q"]
    # row t of a request sees len - new + t + 1 keys
    pairs = sum(new * n - new * (new - 1) // 2 for n in lens) * case["q"]
    return {"bytes": 2 * sum(lens) * case["kvh"] * (case["dim"] + 4 / case["page"])
            + rows * (4 * case["dim"] + 4),
            "flops": 4 * case["dim"] * pairs}


# ---- inputs ------------------------------------------------------------------------------------
def _lengths(case):
    """(cached tokens, new tokens) of each request of a step, the same for every seed so that the
    sizes are the case's: the first `prefill` requests bring up to `long` tokens, the others one."""
    rng = random.Random(17)
    b, pre = case["batch"], case["prefill"]
    ctx = [rng.randint(max(0, case["ctx"] // 2), case["ctx"]) for _ in range(b)]
    even = pre == b
    new = [(case["long"] if even else rng.randint(1, case["long"])) if i < pre else 1
           for i in range(b)]
    return ctx, new


def _kv_lengths(case):
    rng = random.Random(29)
    n, t = case["kv"], case["new"]
    if not case["ragged"]:
        return [n] * case["batch"]
    return [n if i == 0 else rng.randint(min(n, max(t, n // 16)), n) for i in range(case["batch"])]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 1000003 + 5)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _frequencies(rot, scaling):
    """Inverse frequencies and the factor on cosine and sine of the case's scaling."""
    theta, args = 5.0e5, {"none": {}, "linear": dict(factor=4.0), "ntk": dict(factor=8.0),
                          "yarn": dict(factor=32.0, orig_len=32768, beta_fast=32.0, beta_slow=1.0),
                          "llama3": dict(factor=8.0, orig_len=8192, low_freq=1.0, high_freq=4.0)}[scaling]
    if own:
        from block_sparse_long_rope_b200 import star

        return star.star_rope_frequencies(rot, theta, scaling, **args)
    f = [theta ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        return [x / 4.0 for x in f], 1.0
    if scaling == "ntk":  # a larger base: the slowest pair turns `factor` times slower
        base = theta * 8.0 ** (rot / (rot - 2.0))
        return [base ** (-2.0 * i / rot) for i in range(rot // 2)], 1.0
    if scaling == "llama3":
        out = []
        for x in f:
            turns = 8192.0 * x / (2.0 * math.pi)  # turns within the original length
            smooth = min(1.0, max(0.0, (turns - 1.0) / (4.0 - 1.0)))
            out.append((1.0 - smooth) * x / 8.0 + smooth * x)
        return out, 1.0
    if scaling == "yarn":
        def dim_of(turns):
            return rot * math.log(32768.0 / (turns * 2.0 * math.pi)) / (2.0 * math.log(theta))
        lo, hi = max(math.floor(dim_of(32.0)), 0), min(math.ceil(dim_of(1.0)), rot - 1)
        span = (hi - lo) if hi != lo else 0.001
        ramp = [min(1.0, max(0.0, (i - lo) / span)) for i in range(rot // 2)]
        return [x / 32.0 * r + x * (1.0 - r) for x, r in zip(f, ramp)], 0.1 * math.log(32.0) + 1.0
    return f, 1.0


def _rope_inputs(case, seed):
    g = _gen(seed)
    n = case["tokens"]
    buf = torch.randn(1, n, case["heads"] + case["extra"], case["dim"], device="cuda", generator=g)
    buf = buf.to(torch.bfloat16)
    pos = torch.randint(0, case["far"], (n,), device="cuda", generator=g, dtype=torch.int32)
    return buf[:, :, :case["heads"]], pos


def _plan_inputs(case, seed):
    pairs = list(zip(*_lengths(case)))
    random.Random(seed).shuffle(pairs)  # the requests in another order
    ctx, new = [c for c, _ in pairs], [t for _, t in pairs]
    page, b = case["page"], case["batch"]
    width = max(-(-(c + t) // page) for c, t in zip(ctx, new)) + 3
    have = [-(-c // page) for c in ctx]
    added = sum(-(-(c + t) // page) - h for c, t, h in zip(ctx, new, have))
    used, pool = sum(have), sum(have) + added + 5
    order = torch.randperm(pool, generator=_gen(seed), device="cuda").to(torch.int32)
    table = torch.full((b, width), -1, dtype=torch.int32)
    ids, at = order[:used].cpu(), 0
    for i, h in enumerate(have):
        table[i, :h] = ids[at:at + h]
        at += h
    # three entries of the free list were taken by earlier steps
    free = torch.cat([order[:3], order[used:]])
    return ctx, new, table.cuda(), free, pool


def _codes(x, scale, kind):
    y = x / scale
    if kind == "int8":
        return torch.clamp(torch.round(y), -INT8_MAX, INT8_MAX).to(torch.int8)
    return torch.clamp(y, -E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _scale_for(amax, kind):
    """The smallest power of two with which amax still fits the code range."""
    m, e = torch.frexp(amax / (INT8_MAX if kind == "int8" else E4M3_MAX))
    s = torch.ldexp(torch.ones_like(amax), torch.where(m > 0.5, e, e - 1))
    return torch.where(amax > 0, s, torch.zeros_like(s)).clamp_min(SCALE_FLOOR)


def _page_dtype(kind):
    return torch.int8 if kind == "int8" else torch.float8_e4m3fn


def _pages(n, heads, page, dim, kind, gen, spread):
    """Pages of normal values, their size varying with the page and head, in 8 bits with scales."""
    out = torch.empty(n, heads, page, dim, dtype=_page_dtype(kind), device="cuda")
    scales = torch.empty(n, heads, dtype=torch.float32, device="cuda")
    step = max(1, (1 << 28) // (heads * page * dim))
    for i in range(0, n, step):
        m = min(step, n - i)
        x = torch.randn(m, heads, page, dim, device="cuda", generator=gen)
        x *= torch.exp(spread * torch.randn(m, heads, 1, 1, device="cuda", generator=gen))
        s = _scale_for(x.abs().amax(dim=(2, 3)), kind)
        out[i:i + m] = _codes(x, s[:, :, None, None], kind)
        scales[i:i + m] = s
    return out, scales


def _append_inputs(case, seed):
    ctx, new = _lengths(case)
    page, h, d, kind = case["page"], case["heads"], case["dim"], case["kind"]
    g = _gen(seed)
    touched = [-(-(c + t) // page) - c // page for c, t in zip(ctx, new)]
    pool = sum(touched) + 3
    ids = torch.randperm(pool, generator=g, device="cuda").cpu().tolist()
    slots, runs, at = [], [], 0
    for c, t, n in zip(ctx, new, touched):
        pages = ids[at:at + n]
        at += n
        for i in range(t):
            p = c + i
            if i == 0 or p % page == 0:
                runs.append(len(slots))
            slots.append(pages[p // page - c // page] * page + p % page)
    n = len(slots)
    cap = min(n, n // page + 2 * case["batch"])
    runs += [n] * (cap + 1 - len(runs))
    qkv = torch.randn(n, 2 * h + 2, d, device="cuda", generator=g)
    qkv *= torch.exp(0.5 * torch.randn(n, 2 * h + 2, 1, device="cuda", generator=g))
    qkv = qkv.to(torch.bfloat16)
    kp, ks = _pages(pool, h, page, d, kind, g, 0.3)
    vp, vs = _pages(pool, h, page, d, kind, g, 0.3)
    return qkv[:, 2:2 + h], qkv[:, 2 + h:], _ints(slots), _ints(runs), kp, vp, ks, vs


def _attend_inputs(case, seed):
    lens = _kv_lengths(case)
    page, b, t = case["page"], case["batch"], case["new"]
    g = _gen(seed)
    need = [-(-n // page) for n in lens]
    pool = sum(need) + 1
    ids = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    table = torch.full((b, max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = ids[at:at + n]
        at += n
    kp, ks = _pages(pool, case["kvh"], page, case["dim"], case["kind"], g, 0.2)
    vp, vs = _pages(pool, case["kvh"], page, case["dim"], case["kind"], g, 0.2)
    q = torch.randn(b * t, case["q"], case["dim"], device="cuda", generator=g).to(torch.bfloat16)
    return q, lens, table, kp, vp, ks, vs


def prepare(case, seed):
    if own:
        from block_sparse_long_rope_b200 import star
    s = {"case": case}
    if case["op"] == "rope":
        s["x"], s["pos"] = _rope_inputs(case, seed)
        s["y"] = torch.empty(s["x"].shape, dtype=torch.bfloat16, device="cuda")
        s["freq"], s["mscale"] = _frequencies(case["rot"], case["scaling"])
    elif case["op"] == "plan":
        ctx, new, s["table"], s["free"], _ = _plan_inputs(case, seed)
        n, b, page = sum(new), case["batch"], case["page"]
        cap = n + case["pad"]
        runs = min(cap, cap // page + 2 * b)
        s.update(total=n, ctx=_ints(ctx), new=_ints(new), begin=_ints([3]))
        s.update(cu=torch.zeros(b + 1, dtype=torch.int32, device="cuda"),
                 pos=torch.zeros(cap, dtype=torch.int32, device="cuda"),
                 slot=torch.zeros(cap, dtype=torch.int32, device="cuda"),
                 runs=torch.zeros(runs + 1, dtype=torch.int32, device="cuda"),
                 kv=torch.zeros(b, dtype=torch.int32, device="cuda"), next=_ints([0]))
        if own:
            s["ws"] = star.alloc_workspace(star.star_batch_plan_workspace_bytes(b))
    elif case["op"] == "append":
        (s["k"], s["v"], s["slot"], s["runs"], s["kp"], s["vp"], s["ks"],
         s["vs"]) = _append_inputs(case, seed)
        if own:
            s["ws"] = star.alloc_workspace(256)
    else:
        s["q"], s["lens"], s["table"], s["kp"], s["vp"], s["ks"], s["vs"] = _attend_inputs(case, seed)
        b, t = case["batch"], case["new"]
        s["cu"], s["kv"] = _ints([i * t for i in range(b + 1)]), _ints(s["lens"])
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(case["q"], b * t, dtype=torch.float32, device="cuda")
        if own:
            s["ws"] = star.alloc_workspace(star.star_kv8_attend_workspace_bytes(
                b, b * t, case["q"], case["kvh"], case["dim"], t))
    return s


# ---- one pass ----------------------------------------------------------------------------------
def run(state):
    case = state["case"]
    return {"rope": _run_rope, "plan": _run_plan, "append": _run_append,
            "attend": _run_attend}[case["op"]](state, case)


def _run_rope(s, case):
    if own:
        from block_sparse_long_rope_b200 import star

        star.star_rope_scaled(s["x"], s["y"], s["freq"], mscale=s["mscale"], pos=s["pos"],
                              interleaved=case["style"] == "interleaved",
                              transpose=case["transpose"])
        return s["y"]
    x, rot = s["x"], case["rot"]
    # angles of far positions need 64 bits
    ang = s["pos"].double()[:, None] * torch.tensor(s["freq"], dtype=torch.float64, device="cuda")
    c = (torch.cos(ang) * s["mscale"]).float()[None, :, None]
    z = (torch.sin(ang) * (-s["mscale"] if case["transpose"] else s["mscale"])).float()[None, :, None]
    xf = x.float()
    y = torch.empty(x.shape, dtype=torch.float32, device="cuda")
    if case["style"] == "half":
        a, b = xf[..., :rot // 2], xf[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * z, b * c + a * z
    else:
        a, b = xf[..., 0:rot:2], xf[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * z, b * c + a * z
    y[..., rot:] = xf[..., rot:]
    return y.to(torch.bfloat16)


def _run_plan(s, case):
    page = case["page"]
    if own:
        from block_sparse_long_rope_b200 import star

        star.star_batch_plan(s["ctx"], s["new"], s["free"], s["begin"], page, s["table"], s["cu"],
                             s["pos"], s["slot"], s["runs"], s["kv"], s["next"], s["ws"])
        return {k: s[k] for k in ("cu", "pos", "slot", "runs", "kv", "table", "next")}
    ctx, new, n, cap = s["ctx"].long(), s["new"].long(), s["total"], s["pos"].numel()
    cu = torch.cat([torch.zeros_like(new[:1]), torch.cumsum(new, 0)])
    kv = ctx + new
    have, need = (ctx + page - 1) // page, (kv + page - 1) // page
    first = torch.cumsum(need - have, 0) - (need - have) + s["begin"].long()
    col = torch.arange(s["table"].shape[1], device="cuda")[None]
    fresh = (col >= have[:, None]) & (col < need[:, None])
    at = (first[:, None] + col - have[:, None]).clamp(0, s["free"].numel() - 1)
    table = torch.where(fresh, s["free"][at], s["table"])
    tok = torch.arange(n, device="cuda")
    req = torch.searchsorted(cu[1:], tok, right=True)
    p = ctx[req] + tok - cu[req]
    slot = table[req, p // page].long() * page + p % page
    pos = torch.zeros(cap, dtype=torch.int32, device="cuda")
    pos[:n] = p.int()
    slots = torch.full((cap,), -1, dtype=torch.int32, device="cuda")
    slots[:n] = slot.int()
    touched = torch.where(new > 0, (kv - 1) // page - ctx // page + 1, torch.zeros_like(new))
    base = torch.cumsum(touched, 0) - touched
    where = base[req] + p // page - ctx[req] // page
    runs = torch.full((s["runs"].numel(),), n, dtype=torch.int64, device="cuda")
    runs = runs.scatter_reduce(0, where, tok, "amin")
    nxt = s["begin"] + (need - have).sum().int()
    return {"cu": cu.int(), "pos": pos, "slot": slots, "runs": runs.int(), "kv": kv.int(),
            "table": table, "next": nxt.int()}


def _run_append(s, case):
    if own:
        from block_sparse_long_rope_b200 import star

        star.star_kv8_append(s["k"], s["v"], s["slot"], s["runs"], s["kp"], s["vp"], s["ks"],
                             s["vs"], s["ws"])
        return {k: s[k] for k in ("kp", "vp", "ks", "vs")}
    kind, page, slot = case["kind"], case["page"], s["slot"].long()
    at, row = slot // page, slot % page
    first = torch.full((s["ks"].shape[0],), page, dtype=torch.int64, device="cuda")
    first = first.scatter_reduce(0, at, row, "amin")  # lowest row written to each page
    touched, fresh = (first < page)[:, None], (first == 0)[:, None]
    below = (torch.arange(page, device="cuda") < first[:, None])[:, None, :, None] & touched[..., None, None]
    for x, pages, scales in ((s["k"], s["kp"], s["ks"]), (s["v"], s["vp"], s["vs"])):
        x = x.float()
        amax = torch.zeros_like(scales).scatter_reduce(
            0, at[:, None].expand(-1, scales.shape[1]), x.abs().amax(2), "amax")
        new = torch.maximum(_scale_for(amax, kind), torch.where(fresh, torch.zeros_like(scales), scales))
        new = torch.where(touched, new, scales)
        # rows written before this call keep their values under a grown scale
        had = pages.float()
        had = torch.where(below, had * (scales / new)[..., None, None], had)
        pages.copy_(_codes(had, torch.ones_like(new)[..., None, None], kind))
        pages.view(torch.uint8)[at, :, row] = _codes(x, new[at][:, :, None], kind).view(torch.uint8)
        scales.copy_(new)
    return {k: s[k] for k in ("kp", "vp", "ks", "vs")}


def _run_attend(s, case):
    if own:
        from block_sparse_long_rope_b200 import star

        star.star_kv8_attend(s["q"], s["cu"], s["kv"], s["table"], s["kp"], s["vp"], s["ks"],
                             s["vs"], s["o"], s["ws"], case["new"], case["kv"], lse=s["lse"])
        return {"o": s["o"], "lse": s["lse"]}
    t, d, h = case["new"], case["dim"], case["kvh"]
    g = case["q"] // h
    o, lse = torch.empty_like(s["q"]), torch.empty_like(s["lse"])
    for i, n in enumerate(s["lens"]):
        q = s["q"][i * t:(i + 1) * t].float().view(t, h, g, d).permute(1, 2, 0, 3).reshape(h, g * t, d)
        k, v = _dequantised(s, i, n, case["page"], torch.float32)
        x = torch.matmul(q, k.transpose(1, 2)) / math.sqrt(d)
        hidden = torch.arange(n, device="cuda")[None, :] > n - t + torch.arange(t, device="cuda")[:, None]
        x = x.view(h, g, t, n).masked_fill_(hidden, -math.inf).view(h, g * t, n)
        m = x.amax(2, keepdim=True)
        m = torch.where(m == -math.inf, torch.zeros_like(m), m)
        e = torch.exp(x - m)
        z = e.sum(2, keepdim=True)
        y = torch.matmul(e, v) / torch.where(z > 0, z, torch.ones_like(z))
        o[i * t:(i + 1) * t] = y.view(h, g, t, d).permute(2, 0, 1, 3).reshape(t, h * g, d).to(o.dtype)
        lse[:, i * t:(i + 1) * t] = (m + torch.log(z)).view(h * g, t)
    return {"o": o, "lse": lse}


def _dequantised(s, i, n, page, dtype, heads=slice(None)):
    ids = s["table"][i, :-(-n // page)].long()
    out = []
    for pages, scales in ((s["kp"], s["ks"]), (s["vp"], s["vs"])):
        x = pages.view(torch.uint8)[ids][:, heads].view(pages.dtype).to(dtype) * scales[ids][:, heads, None, None].to(dtype)
        x = x.transpose(0, 1)
        out.append(x.reshape(x.shape[0], -1, x.shape[3])[:, :n])
    return out


# ---- the definitions in 64 bits ----------------------------------------------------------------
def exact(case, seed):
    return {"rope": _exact_rope, "plan": _exact_plan, "append": _exact_append,
            "attend": _exact_attend}[case["op"]](case, seed)


def _exact_rope(case, seed):
    x, pos = _rope_inputs(case, seed)
    global own
    was, own = own, False
    try:
        freq, scale = _frequencies(case["rot"], case["scaling"])
    finally:
        own = was
    half = case["rot"] // 2
    turn = torch.polar(torch.full((pos.numel(), half), scale, dtype=torch.float64, device="cuda"),
                       pos.double()[:, None] * torch.tensor(freq, dtype=torch.float64, device="cuda"))
    if case["transpose"]:
        turn = turn.conj()
    y = x.double().clone()
    if case["style"] == "half":
        i, j = slice(0, half), slice(half, 2 * half)
    else:
        i, j = slice(0, 2 * half, 2), slice(1, 2 * half, 2)
    z = torch.complex(x[..., i].double(), x[..., j].double()) * turn[None, :, None]
    y[..., i], y[..., j] = z.real, z.imag
    return y


def _exact_plan(case, seed):
    ctx, new, table, free, _ = _plan_inputs(case, seed)
    table, free, page = table.cpu().tolist(), free.cpu().tolist(), case["page"]
    cu, pos, slot, runs, kv, nxt = [0], [], [], [], [], 3
    for b, (c, t) in enumerate(zip(ctx, new)):
        for j in range(-(-c // page), -(-(c + t) // page)):
            table[b][j] = free[nxt]
            nxt += 1
        for p in range(c, c + t):
            if p == c or p % page == 0:
                runs.append(len(pos))
            pos.append(p)
            slot.append(table[b][p // page] * page + p % page)
        cu.append(len(pos))
        kv.append(c + t)
    n = len(pos)
    cap = n + case["pad"]
    pos += [0] * (cap - n)
    slot += [-1] * (cap - n)
    runs += [n] * (min(cap, cap // page + 2 * case["batch"]) + 1 - len(runs))
    return {"cu": _ints(cu), "pos": _ints(pos), "slot": _ints(slot), "runs": _ints(runs),
            "kv": _ints(kv), "table": _ints(table), "next": _ints([nxt])}


def _nearest_code(y, kind):
    """The nearest value that the 8-bit type holds, ties to even, saturating."""
    if kind == "int8":
        return torch.clamp(torch.round(y), -INT8_MAX, INT8_MAX)
    e = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -30))).clamp_min(-6.0)
    step = torch.exp2(e - 3.0)
    return torch.clamp(torch.round(y / step) * step, -E4M3_MAX, E4M3_MAX)


def _exact_append(case, seed):
    k, v, slot, runs, kp, vp, ks, vs = _append_inputs(case, seed)
    kind, page = case["kind"], case["page"]
    top = INT8_MAX if kind == "int8" else E4M3_MAX
    slot, runs = slot.cpu().tolist(), runs.cpu().tolist()
    out = []
    for x, pages, scales in ((k, kp, ks), (v, vp, vs)):
        x, got, sc = x.double(), pages.double(), scales.double()
        for a, b in zip(runs, runs[1:]):
            if a == b:
                continue
            at, row = slot[a] // page, slot[a] % page
            part = x[a:b].transpose(0, 1)                     # [heads, rows, dim]
            big = part.abs().amax(dim=(1, 2)).cpu().tolist()
            for h, m in enumerate(big):
                s = SCALE_FLOOR if m == 0 else max(SCALE_FLOOR, 2.0 ** math.ceil(math.log2(m / top)))
                if m and m <= top * s / 2 and s > SCALE_FLOOR:
                    s /= 2
                if row > 0:
                    s = max(s, float(sc[at, h]))
                    if s != float(sc[at, h]):
                        got[at, h, :row] = _nearest_code(got[at, h, :row] * (float(sc[at, h]) / s), kind)
                sc[at, h] = s
                got[at, h, row:row + b - a] = _nearest_code(part[h] / s, kind)
        out += [got.to(pages.dtype), sc]
    return {"kp": out[0], "vp": out[2], "ks": out[1], "vs": out[3]}


def _exact_attend(case, seed):
    q, lens, table, kp, vp, ks, vs = _attend_inputs(case, seed)
    s = {"table": table, "kp": kp, "vp": vp, "ks": ks, "vs": vs}
    t, d, h = case["new"], case["dim"], case["kvh"]
    g = case["q"] // h
    o = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.full((case["q"], q.shape[0]), -math.inf, dtype=torch.float64, device="cuda")
    for i, n in enumerate(lens):
        for kh in range(h):
            k, v = (x[0] for x in _dequantised(s, i, n, case["page"], torch.float64, slice(kh, kh + 1)))
            for j in range(kh * g, (kh + 1) * g):
                x = (q[i * t:(i + 1) * t, j].double() @ k.T) / math.sqrt(d)
                late = torch.arange(n, device="cuda")[None, :] - (n - t)
                x = torch.where(late > torch.arange(t, device="cuda")[:, None],
                                torch.full_like(x, -math.inf), x)
                lse[j, i * t:(i + 1) * t] = torch.logsumexp(x, 1)
                o[i * t:(i + 1) * t, j] = torch.nan_to_num(torch.softmax(x, 1), nan=0.0) @ v
    return {"o": o, "lse": lse}

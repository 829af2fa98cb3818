"""The operators over an 8-bit paged cache against plain 64-bit forms, at the sizes and masks where
they can go wrong, one by one and as a serving step runs them together."""
import ctypes
import math
import random

import pytest
import torch

from block_sparse_long_rope_b200 import _abi, star
from tests import kv8_util as U
from tests.kv8_util import E4M3, INT8, ints

pytestmark = pytest.mark.gpu
BOUNDS = "STAR_ERR_DEVICE_BOUNDS"


def _status(ws):
    try:
        star.star_device_status(ws)
        return "STAR_OK"
    except _abi.StarError as e:
        return e.name


# ---- rotary -------------------------------------------------------------------------------------
def _rope64(x, f, m, inter, tr, pos):
    """y in float64 and |a| + |b| of each pair, spread over its elements."""
    rot = 2 * len(f)
    f = torch.tensor(list(f), dtype=torch.float64, device=x.device)
    ang = pos.double()[..., None] * f
    c, s = torch.cos(ang) * m, torch.sin(ang) * (-m if tr else m)
    c, s = (t[None, :, None] if pos.dim() == 1 else t[:, :, None] for t in (c, s))
    y, size = x.double().clone(), torch.zeros_like(x, dtype=torch.float64)
    i, j = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    a, b = x[..., i].double(), x[..., j].double()
    y[..., i], y[..., j] = a * c - b * s, b * c + a * s
    size[..., i] = size[..., j] = abs(m) * (a.abs() + b.abs())
    return y, size


def _close_rope(y, want, size):
    # correct rounding: half a bf16 step; the reference's angle is off by up to 2^-52 * 2e6 * f
    bound = 2.0 ** -8 * want.abs() + 1e-9 * size + 1e-38
    assert bool(((y.double() - want).abs() <= bound).all())


@pytest.mark.parametrize("B,S,H,D,rot,inter,tr,m,far", [
    (1, 1, 1, 64, 16, False, False, 1.0, 10), (1, 1, 40, 128, 128, False, False, 1.0, 10**6),
    (1, 257, 5, 64, 32, True, False, 1.25, 10**6), (2, 33, 3, 128, 96, False, True, 0.5, 1000),
    (3, 7, 1, 64, 48, True, True, 1.0, 2 * 10**6), (1, 1200, 8, 128, 128, True, False, 1.4, 10**5),
    (1, 2500, 2, 128, 16, False, False, -2.0, 10**6), (1, 9, 2048, 64, 64, False, False, 1.0, 50),
    (1, 3000, 2043, 128, 16, False, False, 1.0, 50)])
def test_rope_scaled(B, S, H, D, rot, inter, tr, m, far):
    g = torch.Generator().manual_seed(S + H)
    buf = torch.randn(B, S, H + 2, D + 8, generator=g).to(torch.bfloat16).cuda()
    x = buf[:, :, 1:1 + H, 8:]  # strided, 16-byte aligned
    pos = torch.randint(0, far, (B, S), generator=g, dtype=torch.int32).cuda()
    if B == 1:
        pos = pos[0]
    f, _ = star.star_rope_frequencies(rot, 5e5, "linear", 3.0)
    want, size = _rope64(x, f, m, inter, tr, pos)
    y = torch.full((B, S, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    star.star_rope_scaled(x, y, f, mscale=m, interleaved=inter, transpose=tr, pos=pos)
    _close_rope(y, want, size)
    assert torch.equal(y[..., rot:], x[..., rot:])
    # in place, the rest of the buffer untouched
    keep = buf.clone()
    star.star_rope_scaled(x, x, list(f), mscale=m, interleaved=inter, transpose=tr, pos=pos)
    assert torch.equal(x, y)
    assert torch.equal(buf[:, :, 0], keep[:, :, 0]) and torch.equal(buf[:, :, H + 1], keep[:, :, H + 1])
    assert torch.equal(buf[..., :8], keep[..., :8])


@pytest.mark.parametrize("D,S", [(64, 5), (128, 700)])
def test_rope_scaled_is_star_rope_at_its_settings(D, S):
    x = torch.randn(2, S, 6, D, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    a, b = torch.empty_like(x), torch.empty_like(x)
    f, m = star.star_rope_frequencies(D, 5e5)
    star.star_rope_scaled(x, a, f, mscale=m, pos0=900000)
    star.star_rope(x, b, 5e5, pos0=900000)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("inter", [False, True])
def test_rope_gradient(inter):
    """Transposed rotation against the formula's gradient and against differences of the forward
    call (a linear map: its values at unit vectors)."""
    D, rot, m = 64, 32, 1.5
    f, _ = star.star_rope_frequencies(rot, 1e4)
    pos = ints([12345])
    w = torch.randn(1, 1, 1, D, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).cuda()
    got = torch.empty_like(w)
    star.star_rope_scaled(w, got, f, mscale=m, interleaved=inter, transpose=True, pos=pos)
    x = torch.zeros(1, 1, 1, D, dtype=torch.float64, device="cuda", requires_grad=True)
    ang = pos.double()[:, None] * torch.tensor(list(f), dtype=torch.float64, device="cuda")
    i, j = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    a, b = x[..., i], x[..., j]
    c, s = m * torch.cos(ang), m * torch.sin(ang)
    loss = ((a * c - b * s) * w[..., i].double()).sum() + ((b * c + a * s) * w[..., j].double()).sum()
    (loss + (x[..., rot:] * w[..., rot:].double()).sum()).backward()
    assert bool(((got.double() - x.grad).abs() <= 2.0 ** -8 * x.grad.abs() + 1e-9).all())
    eye = torch.eye(D, device="cuda").to(torch.bfloat16).view(1, 1, D, D)  # heads are unit vectors
    cols = torch.empty_like(eye)
    star.star_rope_scaled(eye, cols, f, mscale=m, interleaved=inter, pos=pos)
    slope = (cols.double()[0, 0] * w.double()[0, 0]).sum(1)
    # each of the two nonzero entries of a column and the result are rounded: 2^-8 each
    bound = 2.0 ** -7 * 1.01 * (cols.double()[0, 0].abs() * w.double()[0, 0].abs()).sum(1) + 1e-9
    assert bool(((got.double()[0, 0, 0] - slope).abs() <= bound).all())


def test_rope_scaled_non_finite_and_empty():
    f, _ = star.star_rope_frequencies(64, 1e4)
    x = torch.zeros(1, 3, 1, 64, dtype=torch.bfloat16, device="cuda")
    x[0, 0, 0, 0], x[0, 1, 0, 5], x[0, 2, 0, 0] = math.inf, math.nan, 1.0
    y = torch.empty_like(x)
    star.star_rope_scaled(x, y, f, pos0=0)
    assert y[0, 0, 0, 0] == math.inf and torch.isnan(y[0, 1, 0, 5])
    assert torch.isfinite(y[0, 2]).all() and float(y[0, 2, 0, 1]) == 0.0
    e = torch.empty(1, 0, 1, 64, dtype=torch.bfloat16, device="cuda")
    star.star_rope_scaled(x[:, :0], x[:, :0], f)
    assert e.numel() == 0


# ---- batch plan -----------------------------------------------------------------------------------
def _plan_case(ctx, new, page, seed, pad=0, begin=2, spare=4, width=None):
    rng = random.Random(seed)
    need = [-(-(c + t) // page) for c, t in zip(ctx, new)]
    have = [-(-c // page) for c in ctx]
    width = width or max(need + [1]) + 1
    pool = list(range(sum(need) + spare + begin))
    rng.shuffle(pool)
    table = [[-1] * width for _ in ctx]
    for b, h in enumerate(have):
        for j in range(h):
            table[b][j] = pool.pop()
    return table, pool, begin


def _plan_run(ctx, new, page, table, free, begin, cap, in_place=False, ws=None):
    B = len(ctx)
    t = dict(ctx=ints(ctx), new=ints(new), free=ints(free), begin=ints([begin]), table=ints(table),
             cu=ints([9] * (B + 1)), pos=ints([9] * cap), slot=ints([9] * cap),
             runs=ints([9] * (star.star_batch_plan_runs(cap, B, page) + 1)), kv=ints([9] * B), next=ints([9]))
    if in_place:
        t["kv"], t["next"] = t["ctx"], t["begin"]
    ws = star.alloc_workspace(star.star_batch_plan_workspace_bytes(B)) if ws is None else ws
    star.star_batch_plan(t["ctx"], t["new"], t["free"], t["begin"], page, t["table"], t["cu"],
                         t["pos"], t["slot"], t["runs"], t["kv"], t["next"], ws)
    return t, ws


def _plan_want(ctx, new, page, table, free, begin, cap, run_cap):
    table = [list(r) for r in table]
    cu, pos, slot, runs, kv, nxt = [0], [], [], [], [], begin
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
    return dict(cu=cu, pos=pos + [0] * (cap - n), slot=slot + [-1] * (cap - n),
                runs=runs + [n] * (run_cap + 1 - len(runs)), kv=kv, table=table, next=[nxt])


@pytest.mark.parametrize("ctx,new,page,pad", [
    ([0], [1], 16, 0), ([0], [0], 16, 3), ([16], [1], 16, 0), ([15], [2], 16, 5),
    ([5, 0, 31, 32, 100], [1, 0, 33, 0, 1], 32, 7), ([0] * 3, [0, 64, 128], 64, 0),
    ([7] * 600, [1] * 600, 16, 0),
    ([(37 * i) % 300 for i in range(700)], [(i * i) % 5 for i in range(700)], 16, 100),
    ([3, 9000, 0], [40000, 1, 7000], 128, 11), ([1] * 4096, [2] * 4096, 64, 1)])
@pytest.mark.parametrize("in_place", [False, True])
def test_batch_plan(ctx, new, page, pad, in_place):
    table, free, begin = _plan_case(ctx, new, page, 1)
    cap = sum(new) + pad
    t, ws = _plan_run(ctx, new, page, table, free, begin, cap, in_place)
    want = _plan_want(ctx, new, page, table, free, begin, cap, t["runs"].numel() - 1)
    for k, v in want.items():
        assert t[k].cpu().tolist() == v, k
    assert _status(ws) == "STAR_OK"


@pytest.mark.parametrize("what", ["tokens", "pages", "width", "negative", "begin"])
@pytest.mark.parametrize("big", [False, True])
def test_batch_plan_refuses_a_step_that_does_not_fit(what, big):
    page, B = 16, 900 if big else 3
    ctx, new = [20] * B, [30] * B
    table, free, begin = _plan_case(ctx, new, page, 2, spare=0)
    cap = sum(new)
    if what == "tokens":
        cap -= 1
    elif what == "pages":
        free = free[:-1]
    elif what == "width":
        table = [r[:3] for r in table]
        ctx[1] = 19
        new[1] = 30
        table[1] = table[1][:3]
        ctx[-1], new[-1] = 20, 29 + 1  # needs a fourth page
    elif what == "negative":
        new[-1] = -1
    else:
        begin = -1
    t, ws = _plan_run(ctx, new, page, table, free, begin, cap)
    assert t["cu"].cpu().tolist() == [0] * (B + 1)
    assert t["slot"].cpu().tolist() == [-1] * cap and t["pos"].cpu().tolist() == [0] * cap
    assert set(t["runs"].cpu().tolist()) == {0}
    assert t["kv"].cpu().tolist() == ctx and t["next"].cpu().tolist() == [begin]
    assert t["table"].cpu().tolist() == table
    assert _status(ws) == BOUNDS and _status(ws) == "STAR_OK"
    if what in ("tokens", "negative"):  # the workspace serves the next step
        ok = [1] * B
        table, free, begin = _plan_case(ctx, ok, page, 3)
        t, _ = _plan_run(ctx, ok, page, table, free, begin, B, ws=ws)
        assert t["cu"].cpu().tolist() == list(range(B + 1))


# ---- append -----------------------------------------------------------------------------------------
def _append_check(k, v, slots, runs, kp, vp, ks, vs, status="STAR_OK", skip=()):
    """Runs the call and compares codes and scales bit by bit; runs in `skip` are left out."""
    page = kp.shape[2]
    wk, wv = U.Pages(kp), U.Pages(vp)
    wks, wvs = ks.double().cpu(), vs.double().cpu()
    keep = list(runs)
    sl = list(slots)
    for u in skip:
        sl[keep[u]] = -1
    U.append_plain(k.double().cpu(), keep, sl, wk, wks, page)
    U.append_plain(v.double().cpu(), keep, sl, wv, wvs, page)
    ws = star.alloc_workspace(256)
    star.star_kv8_append(k, v, ints(slots), ints(runs), kp, vp, ks, vs, ws)
    assert _status(ws) == status
    for got, want in ((kp, wk.values), (vp, wv.values), (ks, wks), (vs, wvs)):
        got = got.double().cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))


def _kv(n, h, d, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, 2 * h + 1, d, generator=g) * torch.exp2(torch.randint(-3, 4, (n, 1, 1), generator=g))
    x = (x * scale).to(torch.bfloat16).cuda()
    return x[:, :h], x[:, h + 1:]


@pytest.mark.parametrize("kind", [E4M3, INT8])
@pytest.mark.parametrize("page,h,d", [(16, 1, 64), (32, 3, 64), (64, 2, 128), (128, 1, 128), (128, 2, 64),
                                      (16, 8, 128)])
def test_append(kind, page, h, d):
    # fresh full page, fresh part, one row on earlier rows, a run up to the page's end
    spans = [(0, page), (0, 3), (page - 1, 1), (5, page - 5), (1, 1), (0, 1)]
    slots, runs = [], [0]
    for i, (row, n) in enumerate(spans):
        pg = [4, 0, 6, 2, 1, 5][i]
        slots += [pg * page + row + j for j in range(n)]
        runs.append(len(slots))
    runs += [len(slots)] * 3
    k, v = _kv(len(slots), h, d, page + d)
    kp, ks = U.make_pages(8, h, page, d, kind, 1)
    vp, vs = U.make_pages(8, h, page, d, kind, 2)
    _append_check(k, v, slots, runs, kp, vp, ks, vs)


@pytest.mark.parametrize("kind", [E4M3, INT8])
def test_append_extreme_values(kind):
    """Zeros, the smallest and largest numbers, maxima at the code range's edge, infinities, NaN; an
    old scale that is zero, and one that is no power of two."""
    page, h, d = 16, 1, 64
    n = 12
    x = torch.zeros(n, 1, d)
    x[1] = 2.0 ** -130
    x[2, 0, 3] = 3.0e38
    x[3, 0, :] = torch.linspace(-448, 448, d)
    x[4, 0, 0] = 449.0 * 2 ** 5 / 2 ** 5 + 3
    x[5, 0, :] = torch.linspace(-127, 127, d)
    x[6, 0, 0] = 128.0
    x[7, 0, :3] = torch.tensor([math.inf, -math.inf, 2.0])
    x[8, 0, :3] = torch.tensor([math.nan, 1.0, -3.0])
    x[9, 0, :2] = torch.tensor([math.inf, math.nan])
    x[10, 0] = torch.linspace(-3, 3, d)
    x[11, 0] = torch.linspace(-3, 3, d)
    x = x.to(torch.bfloat16).cuda()
    slots = [i * page for i in range(10)] + [10 * page + 2, 11 * page + 2]
    runs = list(range(n + 1))
    kp, ks = U.make_pages(12, h, page, d, kind, 3)
    vp, vs = kp.clone(), ks.clone()
    ks[10], ks[11] = 0.0, 0.71
    vs.copy_(ks)
    _append_check(x, x, slots, runs, kp, vp, ks, vs)


@pytest.mark.parametrize("kind", [E4M3, INT8])
def test_append_token_by_token(kind):
    """A page filled one row at a time, its scale growing, equals the plain form step by step."""
    page, h, d = 16, 2, 64
    kp, ks = U.make_pages(2, h, page, d, kind, 4)
    vp, vs = U.make_pages(2, h, page, d, kind, 5)
    for r in range(page):
        k, v = _kv(1, h, d, 100 + r, scale=1.3 ** r)
        _append_check(k, v, [page + r], [0, 1], kp, vp, ks, vs)


def test_append_leaves_out_what_does_not_fit():
    page, h, d, kind = 16, 1, 64, E4M3
    kp, ks = U.make_pages(3, h, page, d, kind, 6)
    vp, vs = U.make_pages(3, h, page, d, kind, 7)
    k, v = _kv(9, h, d, 8)
    # a page beyond the pool, a run past its page's end, a skipped run, a good one
    slots = [3 * page, 15, 0, 0, -1, page, page + 1, page + 2, page + 3]
    _append_check(k, v, slots, [0, 1, 4, 5, 9], kp, vp, ks, vs, BOUNDS, skip=(0, 1))
    # tokens outside the call's rows
    ws = star.alloc_workspace(256)
    before = kp.clone()
    star.star_kv8_append(k, v, ints(slots), ints([-2, 1, 10, 3]), kp, vp, ks, vs, ws)
    assert _status(ws) == BOUNDS
    assert torch.equal(before.view(torch.uint8), kp.view(torch.uint8))
    star.star_kv8_append(k[:0], v[:0], ints([]), ints([0]), kp, vp, ks, vs, ws)
    assert _status(ws) == "STAR_OK"


# ---- attention ----------------------------------------------------------------------------------------
def _attend_case(lens, new, Hq, Hkv, D, page, kind, seed, q_scale=1.0, spread=0.5, pad=0):
    need = [-(-n // page) for n in lens]
    pool = sum(need) + 2
    order = list(range(pool))
    random.Random(seed).shuffle(order)
    width = max(need + [1]) + 1
    table = torch.full((len(lens), width), 2 ** 30, dtype=torch.int32)  # no page: must not be read
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    kp, ks = U.make_pages(pool, Hkv, page, D, kind, seed + 1, spread)
    vp, vs = U.make_pages(pool, Hkv, page, D, kind, seed + 2, spread)
    if kind == E4M3:  # what lies behind a request's last key may hold anything
        for b, n in enumerate(lens):
            if n % page:
                pg = int(table[b, n // page])
                for p in (kp, vp):
                    p.view(torch.uint8)[pg, :, n % page:] = 0x7F
    cu = [0]
    for t in new:
        cu.append(cu[-1] + t)
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn(cu[-1] + pad, Hq, D, generator=g) * q_scale).to(torch.bfloat16).cuda()
    return q, cu, table.cuda(), kp, vp, ks, vs


def _attend(q, cu, lens, table, kp, vp, ks, vs, max_new=None, max_kv=None, ws=None, fill=0.0):
    n, Hq, D = q.shape
    new = [b - a for a, b in zip(cu, cu[1:])]
    max_new = max_new or max(new + [1])
    max_kv = max_kv or max(list(lens) + [1])
    B, Hkv = len(lens), kp.shape[1]
    if ws is None:
        ws = star.alloc_workspace(star.star_kv8_attend_workspace_bytes(B, n, Hq, Hkv, D, max_new))
    o = torch.full((n, Hq, D), fill, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((Hq, n), fill, dtype=torch.float32, device="cuda")
    star.star_kv8_attend(q, ints(cu), ints(lens), table, kp, vp, ks, vs, o, ws, max_new, max_kv, lse=lse)
    return o, lse, ws


def _wide(table, page):
    """(table, max_kv) of a call that may see 200,000 keys: more than 32 rows of a KV head then take the
    kernel of many rows whatever the lengths are."""
    pad = torch.full((table.shape[0], -(-200000 // page)), 2 ** 30, dtype=torch.int32, device="cuda")
    pad[:, :table.shape[1]] = table
    return pad, 200000


@pytest.mark.parametrize("lens,new,Hq,Hkv,D,page,kind", [
    ([1], [1], 1, 1, 64, 16, E4M3), ([1], [1], 4, 1, 64, 16, INT8), ([15], [1], 8, 1, 128, 16, E4M3),
    ([16], [1], 4, 2, 128, 32, INT8), ([17], [1], 32, 8, 128, 64, E4M3),
    ([127, 128, 129], [1, 1, 1], 7, 7, 64, 128, E4M3),
    ([255, 1, 600, 33], [1, 1, 1, 1], 24, 8, 128, 32, INT8),
    ([5000], [1], 4, 1, 64, 16, E4M3), ([70001], [1], 8, 2, 128, 64, E4M3),
    ([3000] * 40, [1] * 40, 8, 8, 64, 64, INT8),
    # several new tokens: causal among them
    ([5], [5], 1, 1, 64, 16, E4M3), ([40], [2], 4, 1, 128, 16, E4M3), ([130], [4], 8, 2, 64, 64, INT8),
    ([1000, 31], [3, 3], 15, 3, 128, 32, E4M3), ([64], [64], 4, 1, 64, 16, E4M3),
    ([300], [129], 8, 2, 128, 64, E4M3), ([900, 77], [100, 40], 16, 2, 64, 128, INT8),
    ([20000, 5, 1300], [300, 5, 17], 16, 2, 128, 64, E4M3), ([700] * 5, [33] * 5, 8, 1, 64, 16, INT8),
    ([4097], [257], 8, 1, 128, 16, E4M3), ([130, 131], [130, 1], 1, 1, 128, 32, INT8),
    ([9000], [20], 7, 1, 64, 32, E4M3), ([40000], [16], 8, 1, 128, 64, E4M3), ([60000], [34], 8, 1, 64, 64, INT8),
    ([129, 30000, 700, 5000], [18, 16, 20, 33], 8, 1, 128, 16, E4M3), ([600, 0, 2000], [600, 0, 555], 16, 8, 128, 128, INT8),
    # many query heads on one KV head
    ([1000, 40], [1, 1], 64, 1, 128, 64, E4M3), ([500], [1], 24, 1, 64, 16, INT8), ([300], [2], 96, 2, 128, 32, E4M3),
    # requests without tokens or keys, rows that see nothing
    ([10, 0, 20, 0], [1, 0, 0, 1], 4, 1, 64, 16, E4M3), ([3], [7], 4, 2, 64, 16, E4M3),
    ([0, 0], [2, 1], 8, 1, 128, 32, INT8), ([0], [40], 4, 1, 64, 16, E4M3)])
def test_attend(lens, new, Hq, Hkv, D, page, kind):
    case = _attend_case(lens, new, Hq, Hkv, D, page, kind, 7)
    q, cu, table = case[:3]
    o, lse, ws = _attend(q, cu, lens, *case[2:])
    want = U.attend_plain(q, cu, lens, *case[2:])
    U.check_attend(o, lse, want)
    assert _status(ws) == "STAR_OK"
    if max(new) * Hq // Hkv > 32:
        table, max_kv = _wide(table, page)
        o, lse, ws = _attend(q, cu, lens, table, *case[3:], max_kv=max_kv)
        U.check_attend(o, lse, want)
        assert _status(ws) == "STAR_OK"


@pytest.mark.parametrize("kind", [E4M3, INT8])
@pytest.mark.parametrize("new", [1, 6, 50])
def test_attend_peaked_scores_and_uneven_scales(kind, new):
    """Large queries (one key takes all) and page scales that differ by powers up to 2^20."""
    lens = [777, 2100]
    case = _attend_case(lens, [new, new], 8, 2, 128, 32, kind, 11, q_scale=12.0, spread=5.0)
    want = U.attend_plain(case[0], case[1], lens, *case[2:])
    for table, max_kv in ((case[2], 2100), _wide(case[2], 32)):
        o, lse, _ = _attend(case[0], case[1], lens, table, *case[3:], max_kv=max_kv)
        U.check_attend(o, lse, want)


def test_attend_flat_tail_behind_a_peak():
    """One key 2^24 times as heavy as each of 2^19 others: the tail's weight is not lost."""
    L, D, page = 1 << 19, 64, 128
    kp = torch.zeros(L // page, 1, page, D, dtype=INT8, device="cuda")
    vp = torch.full_like(kp, 1)
    ks = torch.full((L // page, 1), 1.0, device="cuda")
    kp[0, 0, 5, 0] = 127
    vp[0, 0, 5] = -128 + 28  # -100
    table = torch.arange(L // page, dtype=torch.int32, device="cuda")[None]
    q = torch.zeros(1, 1, D, dtype=torch.bfloat16, device="cuda")
    q[0, 0, 0] = 24 * math.log(2.0) * math.sqrt(D) / 127
    o, lse, _ = _attend(q, [0, 1], [L], table, kp, vp, ks, ks)
    U.check_attend(o, lse, U.attend_plain(q, [0, 1], [L], table, kp, vp, ks, ks))


def test_attend_scales_of_zero_and_extreme_queries():
    case = _attend_case([70], [1], 4, 1, 64, 16, E4M3, 13)
    q, cu, table, kp, vp, ks, vs = case
    ids = table[0, :5].long()
    vs[ids[1]] = 0.0
    ks[ids[3]] = 0.0
    q[0, 1] *= 2.0 ** -60
    q[0, 2] = 0.0
    q[0, 3] *= 2.0 ** 12
    ks *= 2.0 ** -8
    o, lse, _ = _attend(q, cu, [70], table, kp, vp, ks, vs)
    U.check_attend(o, lse, U.attend_plain(q, cu, [70], table, kp, vp, ks, vs))


def test_attend_nan_reaches_only_the_rows_that_see_it():
    q, cu, table, kp, vp, ks, vs = _attend_case([40, 40], [1, 1], 4, 1, 64, 16, E4M3, 17)
    kp.view(torch.uint8)[int(table[0, 1]), 0, 3, 7] = 0x7F
    o, lse, _ = _attend(q, cu, [40, 40], table, kp, vp, ks, vs)
    assert torch.isnan(o[0]).all() and torch.isnan(lse[:, 0]).all()
    assert torch.isfinite(o[1]).all() and torch.isfinite(lse[:, 1]).all()
    q[1, 2, 5] = math.inf
    o, _, _ = _attend(q, cu, [40, 40], table, kp, vp, ks, vs)
    assert torch.isnan(o[1, 2]).all() and torch.isfinite(o[1, 1]).all()


@pytest.mark.parametrize("new", [3, 40, 100])
def test_attend_later_nan_does_not_reach_earlier_tokens(new):
    """A new token's own NaN value row is invisible to the tokens before it."""
    L = 50 + new
    q, cu, table, kp, vp, ks, vs = _attend_case([L], [new], 4, 1, 64, 16, E4M3, 19)
    bad = L - 2  # the last but one token's row
    vp.view(torch.uint8)[int(table[0, bad // 16]), 0, bad % 16, 9] = 0xFF
    clean = vp.clone()
    clean.view(torch.uint8)[int(table[0, bad // 16]), 0, bad % 16, 9] = 0
    for tab, max_kv in ((table, L), _wide(table, 16)):
        o, lse, _ = _attend(q, cu, [L], tab, kp, vp, ks, vs, max_kv=max_kv)
        ref, _, _ = _attend(q, cu, [L], tab, kp, clean, ks, vs, max_kv=max_kv)
        assert torch.equal(o[:new - 2], ref[:new - 2])
        assert torch.isnan(o[new - 2:, :, 9]).all() and torch.isfinite(lse).all()


def test_attend_missing_pages_of_a_chunk():
    """Keys of pages that do not exist are invisible, a whole first tile of them too."""
    lens, new = [600, 300], [50, 40]
    q, cu, table, kp, vp, ks, vs = _attend_case(lens, new, 4, 1, 64, 16, E4M3, 24)
    table[0, 3], table[0, 36], table[1, 5] = -1, kp.shape[0], 2 ** 31 - 1
    table[1, :8] = -7
    want = U.attend_plain(q, cu, lens, table, kp, vp, ks, vs)
    for tab, max_kv in ((table, 600), _wide(table, 16)):
        o, lse, ws = _attend(q, cu, lens, tab, kp, vp, ks, vs, max_kv=max_kv)
        U.check_attend(o, lse, want)
        assert _status(ws) == BOUNDS and _status(ws) == "STAR_OK"


@pytest.mark.parametrize("new", [1, 30])
def test_attend_without_lse(new):
    lens = [700, 90]
    q, cu, table, *rest = _attend_case(lens, [new, new], 8, 2, 64, 32, INT8, 25)
    table, max_kv = _wide(table, 32)
    want, _, ws = _attend(q, cu, lens, table, *rest, max_kv=max_kv)
    o = torch.empty_like(want)
    star.star_kv8_attend(q, ints(cu), ints(lens), table, *rest, o, ws, new, max_kv)
    assert torch.equal(o, want)


def test_attend_bad_pages_and_lengths():
    lens, new = [100, 100, 100], [1, 1, 1]
    q, cu, table, kp, vp, ks, vs = _attend_case(lens, new, 4, 1, 64, 16, INT8, 23)
    good, _, _ = _attend(q, cu, lens, table, kp, vp, ks, vs)
    table[0, 2], table[2, 0] = -5, kp.shape[0]
    want = U.attend_plain(q, cu, lens, table, kp, vp, ks, vs)
    o, lse, ws = _attend(q, cu, lens, table, kp, vp, ks, vs)
    U.check_attend(o, lse, want)  # keys of a missing page are invisible
    assert _status(ws) == BOUNDS and _status(ws) == "STAR_OK"
    assert torch.equal(o[1], good[1])
    # lengths beyond the bounds: the request is left out
    o, lse, ws = _attend(q, cu, [100, 101, 100], table, kp, vp, ks, vs, max_kv=100, fill=3.0)
    assert _status(ws) == BOUNDS
    assert bool((o[1] == 3.0).all()) and torch.equal(o[0].double() != 3.0, torch.ones_like(o[0], dtype=torch.bool))
    o, _, ws = _attend(q, [0, 1, 0, 3], lens, table, kp, vp, ks, vs, max_new=3, fill=3.0)
    assert _status(ws) == BOUNDS
    o, _, ws = _attend(q, [0, 1, 2, 9], lens, table, kp, vp, ks, vs, max_new=9, fill=3.0)
    assert _status(ws) == BOUNDS and bool((o[2] == 3.0).all())


@pytest.mark.parametrize("new", [[2, 1, 2], [40, 3, 70]])
def test_attend_strides_padding_and_repeats(new):
    """q as heads of a fused buffer, padded rows untouched, and the same bits every time."""
    lens = [513, 40, 2000]
    q, cu, *rest = _attend_case(lens, new, 8, 2, 128, 64, E4M3, 29, pad=3)
    rest[0], max_kv = _wide(rest[0], 64)
    n = q.shape[0]
    fused = torch.zeros(n, 12, 128, dtype=torch.bfloat16, device="cuda")
    fused[:, 2:10] = q
    o, lse, ws = _attend(fused[:, 2:10], cu, lens, *rest, fill=5.0, max_kv=max_kv)
    wo, wl, ab, mag, low = U.attend_plain(q, cu, lens, *rest)
    m = cu[-1]
    U.check_attend(o[:m], lse[:, :m], (wo[:m], wl[:, :m], ab[:m], mag[:, :m], low[:m]))
    assert bool((o[cu[-1]:] == 5.0).all()) and bool((lse[:, cu[-1]:] == 5.0).all())
    for _ in range(5):
        o2, lse2, _ = _attend(q, cu, lens, *rest, ws=ws, fill=5.0, max_kv=max_kv)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("new", [1, 70])
def test_attend_on_two_streams_with_two_workspaces(new):
    lens = [20000]
    q, cu, *rest = _attend_case(lens, [new], 8, 2, 64, 64, E4M3, 31)
    want, _, _ = _attend(q, cu, lens, *rest)
    cu_t, kv_t = ints(cu), ints(lens)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs, spaces = [], []
    for s in streams:
        outs.append([torch.empty_like(want) for _ in range(8)])
        spaces.append(star.alloc_workspace(star.star_kv8_attend_workspace_bytes(1, new, 8, 2, 64, new)))
    torch.cuda.synchronize()
    for i in range(8):
        for s, o, ws in zip(streams, outs, spaces):
            star.star_kv8_attend(q, cu_t, kv_t, *rest, o[i], ws, new, 20000, stream=s)
    torch.cuda.synchronize()
    for os_ in outs:
        for o in os_:
            assert torch.equal(o, want)


def test_attend_one_workspace_for_calls_of_many_shapes():
    """Calls of other batches, row counts and kernels leave a workspace as they found it."""
    shapes = [([5000], [1], 8, 2, 64, 16, E4M3), ([900, 77, 3000], [100, 40, 20], 16, 2, 64, 128, INT8),
              ([300] * 9, [2] * 9, 32, 8, 128, 32, E4M3), ([20000], [60], 8, 1, 128, 64, E4M3),
              ([9, 4000], [7, 4], 4, 1, 64, 16, INT8), ([70001], [1], 8, 2, 128, 64, E4M3)]
    ws = star.alloc_workspace(star.star_kv8_attend_workspace_bytes(9, 200, 32, 8, 128, 100))
    for seed, (lens, new, *rest) in enumerate(shapes + shapes[::-1]):
        case = _attend_case(lens, new, *rest, 40 + seed)
        for table, max_kv in ((case[2], max(lens)), _wide(case[2], rest[3])):
            a = _attend(case[0], case[1], lens, table, *case[3:], ws=ws, max_kv=max_kv)[:2]
            b = _attend(case[0], case[1], lens, table, *case[3:], max_kv=max_kv)[:2]
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert _status(ws) == "STAR_OK"


def test_attend_many_requests():
    rng = random.Random(3)
    lens = [rng.choice([0, 1, 5, 16, 17, 100, 300]) for _ in range(4096)]
    new = [min(n, 1) for n in lens]
    case = _attend_case(lens, new, 2, 1, 64, 16, E4M3, 51)
    o, lse, ws = _attend(case[0], case[1], lens, *case[2:])
    U.check_attend(o, lse, U.attend_plain(case[0], case[1], lens, *case[2:]))
    assert _status(ws) == "STAR_OK"


@pytest.mark.parametrize("new", [1, 40])
def test_pools_beyond_32_bit_offsets(new):
    """Pages whose bytes lie more than 2^32 into the pool, for the append and both attention kernels."""
    page, h, d, kind, pages = 128, 8, 128, INT8, 36000  # 4.7 GB each for K and V
    kp = torch.empty(pages, h, page, d, dtype=kind, device="cuda")
    vp = torch.empty_like(kp)
    ks, vs = torch.zeros(pages, h, device="cuda"), torch.zeros(pages, h, device="cuda")
    ids = [pages - 1, 3, pages - 2]
    n = 300
    k, v = _kv(n, h, d, 61)
    slots = [ids[t // page] * page + t % page for t in range(n)]
    ws = star.alloc_workspace(256)
    star.star_kv8_append(k, v, ints(slots), ints([0, page, 2 * page, n]), kp, vp, ks, vs, ws)
    assert _status(ws) == "STAR_OK"
    sub = torch.tensor(ids, device="cuda")
    wk, wv = U.Pages(torch.zeros(3, h, page, d, dtype=kind)), U.Pages(torch.zeros(3, h, page, d, dtype=kind))
    sk, sv = torch.zeros(3, h, dtype=torch.float64), torch.zeros(3, h, dtype=torch.float64)
    runs, local = [0, page, 2 * page, n], list(range(n))
    U.append_plain(k.double().cpu(), runs, local, wk, sk, page)
    U.append_plain(v.double().cpu(), runs, local, wv, sv, page)
    rows = torch.arange(3 * page).view(3, 1, page, 1) < n
    for got, want in ((kp, wk), (vp, wv)):
        assert torch.equal(torch.where(rows, got[sub].double().cpu(), 0.0), torch.where(rows, want.values, 0.0))
    assert torch.equal(ks[sub].double().cpu(), sk) and torch.equal(vs[sub].double().cpu(), sv)
    q = torch.randn(new, 2 * h, d, generator=torch.Generator().manual_seed(9)).to(torch.bfloat16).cuda()
    table, max_kv = _wide(ints([ids]), page)
    o, lse, _ = _attend(q, [0, new], [n], table, kp, vp, ks, vs, max_kv=max_kv)
    small = [t[sub].contiguous() for t in (kp, vp, ks, vs)]
    U.check_attend(o, lse, U.attend_plain(q, [0, new], [n], ints([[0, 1, 2]]), *small))


def test_attend_chunk_captured_and_replayed():
    """A captured call of many new tokens follows lengths that change between replays."""
    case = _attend_case([3000, 2000], [60, 40], 8, 2, 128, 64, E4M3, 71)
    q, cu, table, kp, vp, ks, vs = case
    cu_t, kv_t = ints(cu), ints([3000, 2000])
    o, lse = torch.zeros_like(q), torch.zeros(8, 100, device="cuda")
    ws = star.alloc_workspace(star.star_kv8_attend_workspace_bytes(2, 100, 8, 2, 128, 100))
    call = lambda: star.star_kv8_attend(q, cu_t, kv_t, table, kp, vp, ks, vs, o, ws, 100, 3000, lse=lse)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for c, lens in (([0, 60, 100], [3000, 2000]), ([0, 100, 100], [2900, 0]), ([0, 1, 100], [1, 1999])):
        cu_t.copy_(ints(c))
        kv_t.copy_(ints(lens))
        for t in (kp, vp):  # NaN behind the last key must not matter: these lengths end elsewhere
            t.view(torch.uint8)[(t.view(torch.uint8) & 0x7F) == 0x7F] = 0
        graph.replay()
        U.check_attend(o, lse, U.attend_plain(q, c, lens, table, kp, vp, ks, vs))
    assert _status(ws) == "STAR_OK"


# ---- together -----------------------------------------------------------------------------------------
@pytest.mark.parametrize("kind,inter", [(E4M3, False), (INT8, True)])
def test_serving_steps_captured_and_replayed(kind, inter):
    """Prompts of three requests, then decode steps from one captured graph that plans, rotates,
    appends and attends; every step against the plain forms."""
    Hq, Hkv, D, page, B, W = 8, 2, 64, 16, 3, 8
    prompts, steps = [21, 1, 48], 20
    f, m = star.star_rope_frequencies(32, 1e4, "yarn", 4.0, 64, beta_fast=4.0, beta_slow=1.0)
    pool = 24
    free = torch.randperm(pool, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    dt = dict(dtype=kind, device="cuda")
    kp, vp = torch.zeros(pool, Hkv, page, D, **dt), torch.zeros(pool, Hkv, page, D, **dt)
    ks, vs = (torch.zeros(pool, Hkv, device="cuda") for _ in range(2))
    table = ints([[-1] * W] * B)
    length, begin = ints([0] * B), ints([0])

    class Step:
        def __init__(self, n, max_new):
            self.new = ints([0] * B)
            self.cu, self.pos, self.slot = ints([0] * (B + 1)), ints([0] * n), ints([0] * n)
            self.runs = ints([0] * (star.star_batch_plan_runs(n, B, page) + 1))
            self.qkv = torch.zeros(1, n, Hq + 2 * Hkv, D, dtype=torch.bfloat16, device="cuda")
            self.rot = torch.zeros(1, n, Hq + Hkv, D, dtype=torch.bfloat16, device="cuda")
            self.o = torch.zeros(n, Hq, D, dtype=torch.bfloat16, device="cuda")
            self.lse = torch.zeros(Hq, n, device="cuda")
            self.max_new = max_new
            self.ws = star.alloc_workspace(star.star_batch_plan_workspace_bytes(B))
            self.ws2 = star.alloc_workspace(star.star_kv8_attend_workspace_bytes(B, n, Hq, Hkv, D, max_new))

        def run(self):
            star.star_batch_plan(length, self.new, free, begin, page, table, self.cu, self.pos,
                                 self.slot, self.runs, length, begin, self.ws)
            star.star_rope_scaled(self.qkv[:, :, :Hq + Hkv], self.rot, f, m, interleaved=inter, pos=self.pos)
            star.star_kv8_append(self.rot[0, :, Hq:], self.qkv[0, :, Hq + Hkv:], self.slot, self.runs,
                                 kp, vp, ks, vs, self.ws)
            star.star_kv8_attend(self.rot[0, :, :Hq], self.cu, length, table, kp, vp, ks, vs, self.o,
                                 self.ws2, self.max_new, W * page, lse=self.lse)

    lens = [0] * B
    shadow = [U.Pages(kp), U.Pages(vp)]
    sk, sv = ks.double().cpu(), vs.double().cpu()

    def check(s, new):
        for b, t in enumerate(new):
            lens[b] += t
        assert length.cpu().tolist() == lens and _status(s.ws) == "STAR_OK" and _status(s.ws2) == "STAR_OK"
        n = sum(new)
        pos = [lens[b] - t + i for b, t in enumerate(new) for i in range(t)]
        assert s.pos.cpu().tolist()[:n] == pos
        want, size = _rope64(s.qkv[:, :n, :Hq + Hkv], f, m, inter, False, ints(pos))
        _close_rope(s.rot[:, :n], want, size)
        runs, slots = s.runs.cpu().tolist(), s.slot.cpu().tolist()
        U.append_plain(s.rot[0, :, Hq:].double().cpu(), runs, slots, shadow[0], sk, page)
        U.append_plain(s.qkv[0, :, Hq + Hkv:].double().cpu(), runs, slots, shadow[1], sv, page)
        for got, w in ((kp, shadow[0].values), (vp, shadow[1].values), (ks, sk), (vs, sv)):
            assert torch.equal(got.double().cpu(), w)
        cu = s.cu.cpu().tolist()
        want = U.attend_plain(s.rot[0, :n, :Hq], cu, lens, table, kp, vp, ks, vs)
        U.check_attend(s.o[:n], s.lse[:, :n], want)

    g = torch.Generator().manual_seed(2)
    first = Step(sum(prompts) + 5, max(prompts))
    first.new.copy_(ints(prompts))
    first.qkv.copy_(torch.randn(first.qkv.shape, generator=g).cuda())
    first.run()
    check(first, prompts)
    dec = Step(B, 1)
    # one plain run on a copy of the state sets every kernel up before the capture
    saved = [t.clone() for t in (kp, vp, ks, vs, table, length, begin)]
    dec.run()
    torch.cuda.synchronize()
    for t, c in zip((kp, vp, ks, vs, table, length, begin), saved):
        t.copy_(c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dec.run()
    for i in range(steps):
        new = [1, 1, 0 if i % 3 == 0 else 1]
        dec.new.copy_(ints(new))
        dec.qkv.copy_(torch.randn(dec.qkv.shape, generator=g).cuda())
        graph.replay()
        check(dec, new)

"""The operators over an 8-bit paged cache at the edges of what their arguments may be: scales, scores and values
over the whole range of their types, units that leave a slot idle, sizes at the top of the range."""
import math

import pytest
import torch

from block_sparse_long_rope_b200 import star
from tests import kv8_util as U
from tests.kv8_util import E4M3, INT8, ints
from tests.test_gpu_kv8 import BOUNDS, _attend, _attend_case, _status, _wide

pytestmark = pytest.mark.gpu


# ---- units that leave a slot of the chunk kernel without rows ---------------------------------------
@pytest.mark.parametrize("D,page", [(128, 64), (64, 16)])
@pytest.mark.parametrize("g", [1, 2])
def test_attend_slots_without_rows_behind_slow_ends(D, page, g):
    """Row tiles of 256 rows whose last rows meet NaN values at the causal edge (a slow way out), each
    followed by one of few rows, which leaves the other slot idle over a whole context."""
    lens, new, Hkv = [20000, 9001, 300, 12000], [300 // g, 260 // g, 300 // g, 20], 4
    q, cu, table, kp, vp, ks, vs = _attend_case(lens, new, Hkv * g, Hkv, D, page, E4M3, 79)
    max_new = max(new)
    clean, lse0, ws = _attend(q, cu, lens, table, kp, vp, ks, vs, max_new=max_new)
    U.check_attend(clean, lse0, U.attend_plain(q, cu, lens, table, kp, vp, ks, vs))
    hit = torch.zeros(q.shape[0], Hkv, D, dtype=torch.bool, device="cuda")
    for b, (L, T) in enumerate(zip(lens, new)):
        for back in range(2, T, 3):  # every third new token's value row
            t, dim, head = T - back, (7 * back) % D, back % Hkv
            at = L - back
            vp.view(torch.uint8)[int(table[b, at // page]), head, at % page, dim] = 0x7F if back % 2 else 0xFF
            hit[cu[b] + t:cu[b + 1], head, dim] = True
    hit = hit.repeat_interleave(g, 1)
    for _ in range(3):
        o, lse, _ = _attend(q, cu, lens, table, kp, vp, ks, vs, max_new=max_new, ws=ws)
        assert _status(ws) == "STAR_OK"
        assert torch.equal(torch.isnan(o), hit) and torch.equal(lse, lse0)
        assert torch.equal(o[~hit], clean[~hit])


# ---- V scales over the whole range -----------------------------------------------------------------
def _reach(cu, kv, table, kp, vp, vs):
    """What the floor of the reference adds to `low` of check_attend: the reference stays within 2^-64 of the
    request's largest V scale, so each key may be off by 2^-36 |code| times that."""
    P, Hkv, page, D = kp.shape
    out = []
    for b, L in enumerate(kv):
        ids = table[b, :-(-L // page)].long()
        top = vs[ids].double().amax(0) * 2.0 ** -64  # [Hkv]
        code = vp[ids].double().nan_to_num().abs().sum((0, 2)) * top[:, None]
        out.append(code[None].expand(cu[b + 1] - cu[b], Hkv, D))
    return torch.cat(out)


def _check_scales(lens, new, case, tables):
    q, cu, _, kp, vp, ks, vs = case
    for table, max_kv in tables:
        wo, wl, ab, mag, low = U.attend_plain(q, cu, lens, table, kp, vp, ks, vs)
        more = _reach(cu, lens, table, kp, vp, vs).repeat_interleave(q.shape[1] // kp.shape[1], 1)
        o, lse, ws = _attend(q, cu, lens, table, kp, vp, ks, vs, max_kv=max_kv)
        U.check_attend(o, lse, (wo, wl, ab, mag, low + more))
        assert _status(ws) == "STAR_OK"


@pytest.mark.parametrize("kind", [E4M3, INT8])
@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("big,tiny", [(12, -100), (70, -70), (50, -60), (0, -100), (60, -126)])
@pytest.mark.parametrize("order", ["big tiny big", "tiny big tiny", "big tiny tiny"])
def test_attend_scales_far_apart(kind, new, big, tiny, order):
    """V scales 2^60 to 2^186 apart in every order, in spans of whole tiles and of single pages."""
    lens, page = [3000, 1300], 64
    case = list(_attend_case(lens, [new, new], 8, 2, 128, page, kind, 83))
    table, vs = case[2], case[6]
    for b, L in enumerate(lens):
        n = -(-L // page)
        for j in range(n):
            word = order.split()[min(2, 3 * j // n)]
            if b == 1:  # pages take turns: both within one tile
                word = order.split()[j % 3]
            vs[int(table[b, j])] = 2.0 ** (big if word == "big" else tiny)
    _check_scales(lens, [new, new], case, [(table, 3000), _wide(table, page)])


@pytest.mark.parametrize("new", [1, 40])
def test_attend_zero_pages_from_append(new):
    """Pages of zeros as star_kv8_append writes them (scale 2^-100) behind a long flat context and before more of
    it: the outputs stay finite and right."""
    page, h, d, L, kind = 64, 2, 64, 200000, E4M3
    n = -(-L // page)
    kp, ks = U.make_pages(n, h, page, d, kind, 91)
    vp, vs = U.make_pages(n, h, page, d, kind, 92)
    ks.mul_(2.0 ** -12)  # nearly equal weights
    vs.mul_(2.0 ** 20)
    zero = list(range(0, n, 7)) + list(range(n // 2, n // 2 + 40))
    x = torch.zeros(page * len(zero), h, d, dtype=torch.bfloat16, device="cuda")
    slots = [p * page + r for p in zero for r in range(page)]
    ws = star.alloc_workspace(256)
    star.star_kv8_append(x, x, ints(slots), ints([i * page for i in range(len(zero) + 1)]), kp, vp, ks, vs, ws)
    assert _status(ws) == "STAR_OK" and bool((vs[zero] == 2.0 ** -100).all())
    q = torch.randn(new, 4, d, generator=torch.Generator().manual_seed(93)).to(torch.bfloat16).cuda()
    table = torch.randperm(n, generator=torch.Generator().manual_seed(94)).to(torch.int32).cuda()[None]
    ordered = torch.arange(n, dtype=torch.int32, device="cuda")[None]
    for t in (table, ordered):
        _check_scales([L], [new], (q, [0, new], t, kp, vp, ks, vs), [(t, L)])


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("kind", [E4M3, INT8])
def test_attend_largest_values(kind, new):
    """Values near the largest bf16 number over a long context: a sum of weights under 2^11 times them does
    not fit fp32, their average does."""
    lens, page = [20000, 17], 32
    case = list(_attend_case(lens, [new, new], 4, 1, 64, page, kind, 97, spread=0.0))
    case[6] *= 2.0 ** 116
    want = U.attend_plain(case[0], case[1], lens, *case[2:])
    assert torch.isfinite(want[0].float()).all() and float(want[0].abs().max()) > 2.0 ** 110
    for table, max_kv in ((case[2], 20000), _wide(case[2], page)):
        o, lse, _ = _attend(case[0], case[1], lens, table, *case[3:], max_kv=max_kv)
        U.check_attend(o, lse, want)


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("scale", [1.0, 1.37])
def test_attend_smallest_scales(scale, new):
    """The other end: V scales of 2^-126, the smallest normal numbers."""
    lens, page = [20000, 17], 32
    case = list(_attend_case(lens, [new, new], 4, 1, 64, page, INT8, 98, spread=0.0))
    case[6].fill_(scale * 2.0 ** -126)
    case[4].clamp_(-40, 70).add_(50)  # values of one sign: the average is as large as they are
    wo, wl, ab, mag, low = U.attend_plain(case[0], case[1], lens, *case[2:])
    for table, max_kv in ((case[2], 20000), _wide(case[2], page)):
        o, lse, _ = _attend(case[0], case[1], lens, table, *case[3:], max_kv=max_kv)
        # (o in units of 2^-126: check_attend's absolute term is far above them)
        err = (o.double() - wo).abs() * 2.0 ** 126
        ds = 16 * 2.0 ** -23 * mag.T.unsqueeze(-1)
        # and half of fp32's fixed step of 2^-149 from each of 8 warps of up to 300 parts, over a sum of weights
        # of 2^-9 at least
        bound = (2.0 ** -8 * wo + ab * (2.0 ** -11 + 2.0 ** -18 + 2 * ds)) * 2.0 ** 126 + 2400 * 2.0 ** -15
        assert bool((err <= bound).all())
        assert float(wo[~torch.isinf(wl.T)].min()) > 2.0 ** -126  # (the second request's first rows see no key)


# ---- scores so large that fp32 steps over whole numbers ----------------------------------------------
@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("size", [0, 10, 14, 20])
@pytest.mark.parametrize("sign", [1, -1])
def test_attend_huge_scores(new, size, sign):
    """Scores of up to 2^40 of either sign, one key ahead of the others by more than any rounding: its value in
    bf16 is the output. Rows differ in size, so that their maxima are rounded differently."""
    L, D, page, Hq = 5000, 64, 16, 8
    n, best = -(-L // page), 2345
    g = torch.Generator().manual_seed(101)
    flip = torch.randint(0, 2, (D,), generator=g) * 2 - 1
    # q . K is between 100 and 127 of D |q|'s for the others where it is negative, within 20 of them where not
    other = torch.randint(-20, 21, (n, 1, page, D), generator=g) if sign > 0 else \
        -flip * torch.randint(100, 128, (n, 1, page, D), generator=g)
    kp = other.to(INT8)
    kp[best // page, 0, best % page] = ((127 if sign > 0 else -60) * flip).to(INT8)
    vp = torch.randint(-127, 128, (n, 1, page, D), generator=g).to(INT8).cuda()
    rows = (1 + torch.arange(new * Hq) / (new * Hq)) * 2.0 ** (8 + size)
    q = (rows[:, None] * flip[None]).to(torch.bfloat16).view(new, Hq, D).cuda()
    one = torch.ones(n, 1, device="cuda")
    table = torch.arange(n, dtype=torch.int32, device="cuda")[None]
    want = vp[best // page, 0, best % page].to(torch.bfloat16)
    for t, max_kv in ((table, L), _wide(table, page)):
        o, lse, ws = _attend(q, [0, new], [L], t, kp.cuda(), vp, one, one, max_kv=max_kv)
        assert _status(ws) == "STAR_OK"
        assert torch.equal(o, want.expand_as(o))
        # (D products of at most 8 and 7 bits and their sum are exact; one rounding each for the factor, the
        # score and the logarithm's)
        score = q.double().abs().sum(2).T * (127 if sign > 0 else -60) / math.sqrt(D)
        assert bool(((lse.double() - score).abs() <= 2.0 ** -21 * (score.abs() + 8)).all())


@pytest.mark.parametrize("new", [1, 40])
def test_attend_maximum_that_grows_by_less_than_a_rounding(new):
    """Scores near 2^26.6 (log2 units), where fp32 steps by 8, that grow by one step or two from tile to tile:
    a weight of 2^8 above the maximum at hand must not overflow. All values are equal, and so is the output."""
    L, D, page = 64 * 1024, 64, 64
    n = L // page
    kp = torch.zeros(n, 1, page, D, dtype=INT8)
    rung = torch.arange(n) // 2  # a tile of 128 keys is two pages
    kp[:, 0, :, 0] = 100
    kp[:, 0, :, 1] = (rung % 100)[:, None].to(INT8)
    kp[:, 0, :, 2] = (rung // 100 - 2)[:, None].to(INT8)
    vp = torch.full_like(kp, 77)
    q = torch.zeros(new, 2, D, dtype=torch.bfloat16)
    size = 2.0 ** 26.6 / 1.4427 * math.sqrt(D) / 100
    q[..., 0] = size
    q[..., 1] = float(q[0, 0, 0]) * 2.0 ** -17
    q[..., 2] = float(q[0, 0, 0]) * 100 * 2.0 ** -17
    kp, vp, q = kp.cuda(), vp.cuda(), q.cuda()
    one = torch.ones(n, 1, device="cuda")
    table = torch.arange(n, dtype=torch.int32, device="cuda")[None]
    for t, max_kv in ((table, L), _wide(table, page)):
        o, lse, _ = _attend(q, [0, new], [L], t, kp, vp, one, one, max_kv=max_kv)
        assert bool((o == 77).all()) and torch.isfinite(lse).all()


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("e", [-96, -100, -110, -113, -116, -126, -130])
def test_attend_tiny_queries_on_large_keys(new, e):
    """Rows of q down to subnormal numbers, K scales that bring the scores back to ordinary sizes."""
    lens, page = [700, 90], 32
    case = list(_attend_case(lens, [new, new], 8, 2, 64, page, E4M3, 103))
    up = min(119, -e)  # (a scale that star_kv8_append can write: 2^119 for the largest bf16 numbers)
    case[0] = (case[0].double() * 2.0 ** e).to(torch.bfloat16)
    case[5] = (case[5].double().clamp(max=2.0 ** -2) * 2.0 ** up).float()
    want = U.attend_plain(case[0], case[1], lens, *case[2:])
    for table, max_kv in ((case[2], 700), _wide(case[2], page)):
        o, lse, _ = _attend(case[0], case[1], lens, table, *case[3:], max_kv=max_kv)
        U.check_attend(o, lse, want)


# ---- many tiles ------------------------------------------------------------------------------------------
def test_attend_a_prompt_among_many_decoding_requests_under_wide_bounds():
    """One request may bring 4096 tokens and any may have a million keys: with 512 requests that would be 2^31
    tiles, but the call's tokens can make only some thousands."""
    g, B, page = torch.Generator().manual_seed(109), 512, 128
    lens = torch.randint(1, 400, (B,), generator=g).tolist()
    new = [1] * B
    lens[77], new[77] = 700, 600
    q, cu, table, kp, vp, ks, vs = _attend_case(lens, new, 32, 8, 64, page, E4M3, 109)
    wide = torch.full((B, (1 << 20) // page), 2 ** 30, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    o, lse, ws = _attend(q, cu, lens, wide, kp, vp, ks, vs, max_new=4096, max_kv=1 << 20)
    U.check_attend(o, lse, U.attend_plain(q, cu, lens, table, kp, vp, ks, vs))
    assert _status(ws) == "STAR_OK"


@pytest.mark.parametrize("run,T,Hkv,g", [(1, 1024, 8, 8), (50, 4, 64, 8)])
def test_attend_offsets_that_count_tokens_many_times(run, T, Hkv, g):
    """Offsets that start again from 0 after every `run` requests make more tiles than the call's tokens can, here
    2^31 and more: the call is left out and recorded, by either kernel."""
    B, D, page, L = 4096, 64, 128, 7996 * 128 if run > 1 else 1 << 20
    cu = [(i % (run + 1)) * T for i in range(B + 1)]
    n, rows = max(cu), 16 if T * g <= 32 else 256
    good = sum(b > a for a, b in zip(cu, cu[1:]))
    assert good * Hkv * -(-T * g // rows) * ((L - T) // 128) > 1.5 * 2 ** 31
    kp, ks = U.make_pages(2, Hkv, page, D, INT8, 1)
    table = torch.full((B, L // page), 2 ** 30, dtype=torch.int32, device="cuda")
    q = torch.zeros(n, Hkv * g, D, dtype=torch.bfloat16, device="cuda")
    o, lse, ws = _attend(q, cu, [L] * B, table, kp, kp, ks, ks, max_new=T, max_kv=L, fill=3.0)
    assert _status(ws) == BOUNDS and bool((o == 3.0).all()) and bool((lse == 3.0).all())
    # the workspace serves the next call
    case = _attend_case([300], [T], Hkv * g, Hkv, D, page, INT8, 113)
    o, lse, _ = _attend(case[0], case[1], [300], *case[2:], ws=ws)
    assert _status(ws) == "STAR_OK"
    U.check_attend(o, lse, U.attend_plain(case[0], case[1], [300], *case[2:]))


# ---- rotary near the largest number ------------------------------------------------------------------
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("m", [1.0, 1.5, 2.0, -3.0, 1e30])
def test_rope_scaled_large_values(inter, m):
    """Products that leave fp32 while the rotated value does not: the correctly rounded bf16 all the same."""
    D, S = 64, 41
    f = [math.pi / 4, 0.5, 1.0, 0.25, 0.1, 1.5, 2.0, 3.0]
    x = torch.zeros(1, S, 2, D, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(107)
    x[...] = (torch.randn(x.shape, generator=g) * 2.0 ** 126).clamp(-3.3e38, 3.3e38).to(torch.bfloat16)
    x[0, :, 0, :16] = 2.97e38  # a pair of equal numbers, turned by pi / 4 at position 1: 0 and its diagonal
    y = torch.empty_like(x)
    pos = torch.arange(S, dtype=torch.int32, device="cuda")
    star.star_rope_scaled(x, y, f, mscale=m, interleaved=inter, pos=pos)
    i, j = (slice(0, 16, 2), slice(1, 16, 2)) if inter else (slice(0, 8), slice(8, 16))
    ang = pos.double()[:, None] * torch.tensor(f, dtype=torch.float64, device="cuda")
    c, s = (m * t(ang)[None, :, None] for t in (torch.cos, torch.sin))
    a, b = x[..., i].double(), x[..., j].double()
    want = x.double().clone()
    want[..., i], want[..., j] = a * c - b * s, b * c + a * s
    # from 2^128 - 2^119 on, half a step above the largest bf16 number, a value is rounded to infinity
    err = 1e-12 * abs(m) * 2.0 ** 128
    top, a = 2.0 ** 128 - 2.0 ** 119, want.abs()
    assert bool(torch.isinf(y)[a - err >= top].all()) and not torch.isnan(y).any()
    fits = a + err < top
    assert bool(((y.double() - want).abs() <= 2.0 ** -8 * a + err)[fits].all())


# ---- bounded waits ---------------------------------------------------------------------------------------
def test_both_bounded_waits_give_up():
    """The wait by the SM's clock that the chunk kernel uses ends as the one by the global timer does: the
    call lasts as long as the longer of both, 50 ms and 50 million cycles."""
    ws = star.alloc_workspace(256)
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    star.star_debug_wait_probe(ws, seconds=0.05)
    b.record()
    assert _status(ws) == "STAR_ERR_DEVICE_TIMEOUT" and _status(ws) == "STAR_OK"
    assert 49.0 < a.elapsed_time(b) < 1000.0


# ---- together with the calls on a bf16 cache ---------------------------------------------------------------
@pytest.mark.parametrize("kind", [E4M3, INT8])
def test_a_phase1_context_moved_into_pages(kind):
    """A context encoded by Phase 1, its bf16 cache (keys rotated) moved into 8-bit pages in one append per
    sequence, and new tokens that attend over both."""
    B, L, Hq, Hkv, D, page, T, theta = 2, 700, 8, 2, 128, 32, 5, 5e5
    g = torch.Generator().manual_seed(127)
    rand = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    q, k, v = rand(B, L, Hq, D), rand(B, L, Hkv, D), rand(B, L, Hkv, D)
    o = torch.empty_like(q)
    kc, vc = (torch.zeros(B, Hkv, L + 44, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws1 = star.alloc_workspace(star.star_phase1_workspace_bytes(B, L, Hq, D))
    star.star_phase1_encode(q, k, v, o, kc, vc, 256, 128, theta, ws1)
    n_pages, W = 60, 30
    kp, vp = (torch.zeros(n_pages, Hkv, page, D, dtype=kind, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(n_pages, Hkv, device="cuda") for _ in range(2))
    table, length, begin = ints([[-1] * W] * B), ints([0] * B), ints([0])
    free = torch.randperm(n_pages, generator=g).to(torch.int32).cuda()
    shadow, sk, sv = [U.Pages(kp), U.Pages(vp)], ks.double().cpu(), vs.double().cpu()
    ws = star.alloc_workspace(star.star_kv8_attend_workspace_bytes(B, B * T, Hq, Hkv, D, T))

    def plan(new):
        n = sum(new)
        t = [ints([0] * (B + 1)), ints([0] * n), ints([0] * n),
             ints([0] * (star.star_batch_plan_runs(n, B, page) + 1))]
        star.star_batch_plan(length, ints(new), free, begin, page, table, *t, length, begin, ws)
        return t

    def append(rows_k, rows_v, slot, runs):
        star.star_kv8_append(rows_k, rows_v, slot, runs, kp, vp, ks, vs, ws)
        U.append_plain(rows_k.double().cpu(), runs.cpu().tolist(), slot.cpu().tolist(), shadow[0], sk, page)
        U.append_plain(rows_v.double().cpu(), runs.cpu().tolist(), slot.cpu().tolist(), shadow[1], sv, page)

    for b in range(B):  # (a sequence's cache is [Hkv, rows, D]: its rows are a strided view)
        _, _, slot, runs = plan([L if i == b else 0 for i in range(B)])
        append(kc[b].transpose(0, 1)[:L], vc[b].transpose(0, 1)[:L], slot, runs)
    cu, pos, slot, runs = plan([T] * B)
    x = rand(1, B * T, Hq + 2 * Hkv, D)
    f, m = star.star_rope_frequencies(D, theta)
    star.star_rope_scaled(x[:, :, :Hq + Hkv], x[:, :, :Hq + Hkv], f, m, pos=pos)
    append(x[0, :, Hq:Hq + Hkv], x[0, :, Hq + Hkv:], slot, runs)
    for got, want in ((kp, shadow[0].values), (vp, shadow[1].values), (ks, sk), (vs, sv)):
        assert torch.equal(got.double().cpu(), want)
    out = torch.empty(B * T, Hq, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(Hq, B * T, device="cuda")
    star.star_kv8_attend(x[0, :, :Hq], cu, length, table, kp, vp, ks, vs, out, ws, T, W * page, lse=lse)
    assert _status(ws) == "STAR_OK" and length.cpu().tolist() == [L + T] * B
    U.check_attend(out, lse, U.attend_plain(x[0, :, :Hq], cu.cpu().tolist(), [L + T] * B, table, kp, vp, ks, vs))


# ---- many requests, and two graphs at once ------------------------------------------------------------------
@pytest.mark.parametrize("long", [1, 16, 77])
def test_attend_most_requests_of_the_largest_head(long):
    """4096 requests of D 128, whose offsets take the most shared memory beside either kernel's tiles."""
    g = torch.Generator().manual_seed(131)
    lens = torch.randint(0, 60, (4096,), generator=g).tolist()
    new = [min(1, L) for L in lens]
    lens[1234], new[1234] = 300, long
    case = _attend_case(lens, new, 2, 1, 128, 16, E4M3, 131)
    o, lse, ws = _attend(case[0], case[1], lens, *case[2:])
    assert _status(ws) == "STAR_OK"
    U.check_attend(o, lse, U.attend_plain(case[0], case[1], lens, *case[2:]))


@pytest.mark.parametrize("new", [1, 16, 70])
def test_attend_two_graphs_replayed_at_once(new):
    """Two captured calls with a workspace each, replayed on two streams at the same time."""
    lens = [9000, 700, 20000]
    q, cu, *rest = _attend_case(lens, [new] * 3, 8, 2, 128, 64, E4M3, 137)
    want, want_lse, _ = _attend(q, cu, lens, *rest)
    cu_t, kv_t = ints(cu), ints(lens)
    sides = []
    for _ in range(2):
        ws = star.alloc_workspace(star.star_kv8_attend_workspace_bytes(3, 3 * new, 8, 2, 128, new))
        o, lse = torch.zeros_like(want), torch.zeros_like(want_lse)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(5):
                star.star_kv8_attend(q, cu_t, kv_t, *rest, o, ws, new, max(lens), lse=lse)
        sides.append((torch.cuda.Stream(), graph, o, lse, ws))
    torch.cuda.synchronize()
    for _ in range(4):
        for stream, graph, *_ in sides:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, _, o, lse, ws in sides:
        assert torch.equal(o, want) and torch.equal(lse, want_lse) and _status(ws) == "STAR_OK"


def test_attend_a_slot_idle_for_longer_than_a_wait():
    """4096 requests of one token over a long shared prefix leave the second slot idle for over 2 s, the limit of a
    bounded wait; the last request, of 300 tokens, needs it."""
    B, Hkv, D, page, L, T = 4096, 8, 64, 128, 655360, 300
    kp, ks = U.make_pages(7, Hkv, page, D, INT8, 139)
    vp, vs = U.make_pages(7, Hkv, page, D, INT8, 140)
    table = (torch.arange(L // page, dtype=torch.int32, device="cuda") % 4)[None].repeat(B, 1)
    table[-1, :4] = ints([6, 4, 5, 4])
    lens, new = [L] * (B - 1) + [500], [1] * (B - 1) + [T]
    cu = list(range(B)) + [B - 1 + T]
    g = torch.Generator().manual_seed(141)
    q = torch.randn(B - 1 + T, Hkv, D, generator=g).to(torch.bfloat16).cuda()
    q[:B - 1] = q[:1]
    o, lse, ws = _attend(q, cu, lens, table, kp, vp, ks, vs)
    assert _status(ws) == "STAR_OK"
    want = U.attend_plain(q[B - 1:], [0, T], [500], table[-1:], kp, vp, ks, vs)
    U.check_attend(o[B - 1:], lse[:, B - 1:], want)
    # the other requests are all alike, whichever CTAs share them
    few = U.attend_plain(q[:1], [0, 1], [L], table[:1], kp, vp, ks, vs)
    n = B - 1
    U.check_attend(o[:n], lse[:, :n], [t.expand(n, -1, -1) if t.dim() == 3 else t.expand(-1, n) for t in few])


# ---- weights far below the largest -----------------------------------------------------------------------
@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("kind", [E4M3, INT8])
def test_attend_small_weights_at_any_maximum(kind, new):
    """Values only under weights of 2^-20 to 2^-32 of the largest, in rows whose maximum lies between -60 and 60:
    the weights keep their bits whatever the maximum is (an output in units of 1 would be 2^-36 off)."""
    L, D, page, Hq = 64, 64, 16, 8
    n = L // page
    key = torch.arange(L)
    k = torch.zeros(L, D)
    k[:, 0] = 96
    k[:, 1] = -key.float().div(4, rounding_mode="floor")  # (0 .. -15: codes of either type)
    v = torch.where((key >= 40)[:, None], torch.randint(-15, 16, (L, D), generator=torch.Generator().manual_seed(149)), 0)
    pages = lambda x: x.view(n, 1, page, D).to(kind).cuda()  # noqa: E731
    kp, vp = pages(k), pages(v.float())
    one = torch.ones(n, 1, device="cuda")
    rows = new * Hq
    q = torch.zeros(rows, D)
    q[:, 0] = torch.linspace(-60, 60, rows) * math.sqrt(D) / 96
    q[:, 1] = 1.45 * math.sqrt(D)
    q = q.to(torch.bfloat16).view(new, Hq, D).cuda()
    table = torch.arange(n, dtype=torch.int32, device="cuda")[None]
    cu, lens = [0, new], [L + new - 1]  # every row sees the first 64 keys at least
    if new > 1:  # the new tokens' own keys: far below all others
        more = -(-(new - 1) // page)
        k2 = torch.zeros(more * page, D)
        k2[:, 1] = -120
        kp = torch.cat([kp, k2.view(more, 1, page, D).to(kind).cuda()])
        vp = torch.cat([vp, torch.zeros(more, 1, page, D).to(kind).cuda()])
        one = torch.ones(n + more, 1, device="cuda")
        table = torch.arange(n + more, dtype=torch.int32, device="cuda")[None]
    want = U.attend_plain(q, cu, lens, table, kp, vp, one, one)
    for t, max_kv in ((table, max(lens)), _wide(table, page)):
        o, lse, _ = _attend(q, cu, lens, t, kp, vp, one, one, max_kv=max_kv)
        U.check_attend(o, lse, want)
        # the bound's terms by key are 2^-36 of a code: small beside these outputs
        assert float((2.0 ** -36 * want[4]).max()) < 0.1 * float(want[0].abs().amax(2).min())

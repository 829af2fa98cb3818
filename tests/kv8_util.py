"""Plain 64-bit forms of the operators over an 8-bit paged cache, and inputs for their tests."""
import math

import torch

QMAX = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}
E4M3, INT8 = torch.float8_e4m3fn, torch.int8


def ints(v, device="cuda"):
    return torch.tensor(v, dtype=torch.int32, device=device)


def nearest_code(y, kind):
    """Value of the nearest code, ties to even, saturating; y in float64 without NaN."""
    if kind == INT8:
        return torch.clamp(torch.round(y), -127.0, 127.0)
    a = y.abs().clamp(max=1e6)
    e = torch.floor(torch.log2(a.clamp_min(2.0 ** -40))).clamp_min(-6.0)
    step = torch.exp2(e - 3.0)
    return torch.sign(y) * torch.clamp(torch.round(a / step) * step, max=448.0)


def pow2_scale(amax, kind):
    """Smallest power of two with amax / scale within the codes, at least 2^-100."""
    if amax == 0:
        return 2.0 ** -100
    s = 2.0 ** math.floor(math.log2(amax / QMAX[kind]))
    while amax > QMAX[kind] * s:
        s *= 2
    while s > 2.0 ** -100 and amax <= QMAX[kind] * s / 2:
        s /= 2
    return max(s, 2.0 ** -100)


def append_plain(x, runs, slots, pages, scales, page_len):
    """Codes (as values, float64) and scales after writing x [n, H, D] (float64) in runs; modifies
    pages and scales (both float64) in place. pages: [P, H, page_len, D] code values."""
    kind = pages.kind
    vals, sc = pages.values, scales
    for a, b in zip(runs, runs[1:]):
        if a >= b or slots[a] < 0:
            continue
        pg, row = divmod(slots[a], page_len)
        for h in range(x.shape[1]):
            part = x[a:b, h]
            fin = part[torch.isfinite(part)]
            s = pow2_scale(float(fin.abs().max()) if fin.numel() else 0.0, kind)
            if row > 0:
                old = float(sc[pg, h])
                s = max(s, old)
                if s != old:
                    vals[pg, h, :row] = nearest_code(vals[pg, h, :row] * (old / s), kind)
            sc[pg, h] = s
            q = nearest_code(torch.nan_to_num(part / s, nan=0.0, posinf=1e9, neginf=-1e9), kind)
            if kind == E4M3:
                q = torch.where(torch.isnan(part), torch.full_like(q, math.nan), q)
            vals[pg, h, row:row + b - a] = q


class Pages:
    def __init__(self, pages):
        self.kind, self.values = pages.dtype, pages.double().cpu()


def make_pages(n, heads, page_len, dim, kind, seed, spread=0.5):
    """Random pages whose size varies from page to page, with power-of-two scales."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, heads, page_len, dim, generator=g)
    x = x * torch.exp2(torch.round(2 * spread * torch.randn(n, heads, 1, 1, generator=g)))
    amax = x.abs().amax(dim=(2, 3))
    s = torch.exp2(torch.ceil(torch.log2(amax / QMAX[kind])))
    y = x / s[:, :, None, None]
    c = y.round().clamp(-127, 127).to(INT8) if kind == INT8 else y.clamp(-448, 448).to(E4M3)
    return c.cuda(), s.float().cuda()


def attend_plain(q, cu, kv, table, kp, vp, ks, vs):
    """o, lse and what error bounds need: the weighted sum of |v|, the largest sum |q k| / sqrt(D) of each
    row, and the unweighted sum of |code| times the largest V scale nearby (see check_attend); in
    float64 on the tensors' device. Keys of a page that does not exist are invisible."""
    n, Hq, D = q.shape
    P, Hkv, page_len, _ = kp.shape
    g = Hq // Hkv
    dev = q.device
    o = torch.zeros(n, Hq, D, dtype=torch.float64, device=dev)
    ab = torch.zeros_like(o)
    lse = torch.full((Hq, n), -math.inf, dtype=torch.float64, device=dev)
    mag = torch.zeros(Hq, n, dtype=torch.float64, device=dev)
    low = torch.zeros_like(o)
    for b in range(len(kv)):
        T, L = cu[b + 1] - cu[b], kv[b]
        if T <= 0 or L <= 0:
            continue
        ids = table[b, :-(-L // page_len)].long()
        real = (ids >= 0) & (ids < P)
        ids = ids.clamp(0, P - 1)
        k = (kp[ids].double() * ks[ids].double()[..., None, None]).transpose(0, 1).reshape(Hkv, -1, D)[:, :L]
        v = (vp[ids].double() * vs[ids].double()[..., None, None]).transpose(0, 1).reshape(Hkv, -1, D)[:, :L]
        there = real.repeat_interleave(page_len)[:L]
        k, v = (torch.where(there[None, :, None], x, torch.zeros_like(x)) for x in (k, v))
        sc = vs[ids].double().T.repeat_interleave(page_len, 1)  # [Hkv, keys]: the reference scale's bound
        sc = torch.nn.functional.pad(sc, (0, -sc.shape[1] % 128))
        tile = sc.view(Hkv, -1, 128).amax(2, keepdim=True).expand(-1, -1, 128).reshape(Hkv, -1)[:, :L]
        tile = torch.minimum(tile * 4096, sc.amax(1, keepdim=True))[..., None]
        code = vp[ids].double().transpose(0, 1).reshape(Hkv, -1, D)[:, :L].abs().nan_to_num() * tile
        code = torch.where(there[None, :, None], code, torch.zeros_like(code))
        for h in range(Hq):
            qq = q[cu[b]:cu[b + 1], h].double()
            s = qq @ k[h // g].T / math.sqrt(D)
            key = torch.arange(L, device=dev)
            seen = (key[None] < (L - T + 1 + torch.arange(T, device=dev))[:, None]) & there[None]
            s = s.masked_fill(~seen, -math.inf)
            some = seen.any(1)
            w = torch.softmax(s[some], 1)
            rows = torch.arange(cu[b], cu[b + 1], device=dev)[some]
            o[rows, h] = w @ v[h // g]
            ab[rows, h] = w @ v[h // g].abs()
            low[rows, h] = seen[some].double() @ code[h // g]
            lse[h, rows] = torch.logsumexp(s[some], 1)
            m = (qq.abs() @ k[h // g].abs().T / math.sqrt(D)).masked_fill(~seen, 0.0)
            mag[h, cu[b]:cu[b + 1]] = m.amax(1)
    return o, lse, ab, mag, low


def check_attend(o, lse, want):
    """Error bounds of the kernel against the 64-bit form:
    - a score is an fp32 accumulation of exact products over D / 16 steps: at most
      16 * 2^-23 * sum |q k| / sqrt(D) off (`mag`), which shifts the logarithm as much and a weight by
      as much of itself;
    - a weight is rounded to fp16 (2^-11) after ex2.approx and fp32 roundings (below 2^-20 at scores
      up to a few hundred), o sums weights times values in fp32, and is rounded to bf16 (2^-8);
    - P is held as 2^11 times the weight (at least) of the largest, so a rounding is never below half of
      fp16's smallest step, 2^-25: 2^-36 of the largest weight, and of the sum, for each key that a row
      sees. The V scale enters P as the ratio to a reference scale that is some page's of the request and
      at most 2^12 times the largest of the tile of 128 keys (`low`: the sum over keys of |code| times
      that);
    - lse adds a logarithm's fp32 roundings: 2^-21 of its size."""
    wo, wl, ab, mag, low = want
    ds = 16 * 2.0 ** -23 * mag.T.unsqueeze(-1)
    bound = 2.0 ** -8 * wo.abs() + ab * (2.0 ** -11 + 2.0 ** -18 + 2 * ds) + 2.0 ** -36 * low + 1e-30
    err = (o.double() - wo).abs()
    assert not torch.isnan(o).any()
    worst = float((err / bound).max())
    assert worst <= 1.0, f"o off by {worst:.3f} of its bound"
    empty = torch.isinf(wl)
    assert torch.equal(torch.isinf(lse), empty)
    dl = (lse.double() - wl)[~empty].abs()
    lb = (16 * 2.0 ** -23 * mag + 2.0 ** -21 * (wl.abs() + 8))[~empty]
    if dl.numel():
        worst = float((dl / lb).max())
        assert worst <= 1.0, f"lse off by {worst:.3f} of its bound"

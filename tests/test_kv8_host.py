"""Host-side behaviour of the operators over an 8-bit paged cache: refusals before any launch,
workspace sizes, the run bound, and the frequencies' formulas. These run without a GPU."""
import ctypes
import itertools
import math
import random

import pytest
import torch

from block_sparse_long_rope_b200 import _abi, star
from block_sparse_long_rope_b200 import build as star_build

OK, INVALID, UNSUPPORTED, CUDA = 0, 1, 2, 3
FAKE = ctypes.c_void_p(0x10000)   # aligned, never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x10008)
ODD4 = ctypes.c_void_p(0x10002)
NULL = ctypes.c_void_p(0)


@pytest.fixture(scope="module")
def lib():
    star_build.build()
    return _abi.load()


def _s(*v):
    return (ctypes.c_int64 * len(v))(*v)


def _freqs(n, fill=1.0):
    return (ctypes.c_double * n)(*([fill] * n))


# ---- frequencies ----------------------------------------------------------------------------
def _by_formula(rot, theta, kind, factor, orig, a, b):
    f = [theta ** (-2 * i / rot) for i in range(rot // 2)]
    if kind == "linear":
        return [x / factor for x in f], 1.0
    if kind == "ntk":
        return [(theta * factor ** (rot / (rot - 2))) ** (-2 * i / rot) for i in range(rot // 2)], 1.0
    if kind == "llama3":
        out = []
        for x in f:
            wavelength = 2 * math.pi / x
            if wavelength > orig / a:
                out.append(x / factor)
            elif wavelength < orig / b:
                out.append(x)
            else:
                u = (orig / wavelength - a) / (b - a)
                out.append((1 - u) * x / factor + u * x)
        return out, 1.0
    if kind == "yarn":
        d = [rot * math.log(orig / (n * 2 * math.pi)) / (2 * math.log(theta)) for n in (a, b)]
        lo, hi = max(math.floor(d[0]), 0), min(math.ceil(d[1]), rot - 1)
        if lo == hi:
            hi += 0.001
        out = []
        for i, x in enumerate(f):
            r = min(1.0, max(0.0, (i - lo) / (hi - lo)))
            out.append(x / factor * r + x * (1 - r))
        return out, 0.1 * math.log(factor) + 1
    return f, 1.0


@pytest.mark.parametrize("rot,theta", [(128, 5e5), (64, 1e4), (32, 5e5), (16, 1e4), (2, 1e4)])
@pytest.mark.parametrize("kind,factor,orig,a,b", [
    ("none", 1.0, 0, 0, 0), ("linear", 4.0, 0, 0, 0), ("ntk", 8.0, 0, 0, 0),
    ("yarn", 32.0, 32768, 32.0, 1.0), ("yarn", 4.0, 4096, 32.0, 1.0), ("yarn", 1.0, 100, 2.0, 2.0),
    ("llama3", 8.0, 8192, 1.0, 4.0), ("llama3", 32.0, 8192, 1.0, 4.0)])
def test_frequencies(lib, rot, theta, kind, factor, orig, a, b):
    if kind == "ntk" and rot == 2:
        with pytest.raises(_abi.StarError):
            star.star_rope_frequencies(rot, theta, kind, factor)
        return
    args = dict(beta_fast=a, beta_slow=b) if kind == "yarn" else dict(low_freq=a, high_freq=b)
    got, m = star.star_rope_frequencies(rot, theta, kind, factor, orig, **args)
    want, wm = _by_formula(rot, theta, kind, factor, orig, a, b)
    assert len(got) == rot // 2
    # a handful of fp64 roundings and pow's own last bits
    for x, y in zip(got, want):
        assert abs(x - y) <= 1e-14 * abs(y)
    assert abs(m - wm) <= 1e-15 * wm


@pytest.mark.parametrize("kw", [
    dict(rot=3), dict(rot=0), dict(rot=130), dict(theta=1.0), dict(theta=float("nan")),
    dict(scaling=5), dict(scaling=-1), dict(scaling=1, factor=0.5),
    dict(scaling=1, factor=float("inf")), dict(scaling=3, orig=0.0, a=32.0, b=1.0),
    dict(scaling=3, orig=4096.0, a=1.0, b=32.0), dict(scaling=4, orig=8192.0, a=4.0, b=1.0),
    dict(scaling=4, orig=8192.0, a=4.0, b=4.0), dict(scaling=4, orig=float("nan"), a=1.0, b=4.0),
    dict(out=None)])
def test_frequency_refusals(lib, kw):
    a = dict(rot=64, theta=1e4, scaling=0, factor=8.0, orig=0.0, a=0.0, b=0.0, out=_freqs(64))
    a.update(kw)
    m = ctypes.c_double()
    assert lib.star_rope_frequencies(a["rot"], a["theta"], a["scaling"], a["factor"], a["orig"],
                                     a["a"], a["b"], a["out"], ctypes.byref(m)) == INVALID
    assert lib.star_last_error()


def test_unknown_scaling_name():
    with pytest.raises(ValueError, match="scaling"):
        star.star_rope_frequencies(64, 1e4, "cubic")


# ---- refusals ---------------------------------------------------------------------------------
def _rope(lib, **kw):
    a = dict(x=FAKE, xs=_s(800, 80, 8), y=ctypes.c_void_p(0x90000), ys=_s(800, 80, 8), pos=NULL,
             ps=0, pos0=0, B=1, S=4, H=2, D=64, rot=32, f=_freqs(64), m=1.0, inter=0, tr=0)
    a.update(kw)
    return lib.star_rope_scaled(a["x"], a["xs"], a["y"], a["ys"], a["pos"], a["ps"], a["pos0"],
                                a["B"], a["S"], a["H"], a["D"], a["rot"], a["f"], a["m"],
                                a["inter"], a["tr"], NULL)


@pytest.mark.parametrize("kw,status", [
    (dict(x=NULL), INVALID), (dict(y=ODD), INVALID), (dict(xs=None), INVALID),
    (dict(xs=_s(800, 81, 8)), INVALID), (dict(pos=ODD4), INVALID), (dict(B=-1), INVALID),
    (dict(B=65536), INVALID), (dict(H=0), INVALID), (dict(H=2049), INVALID),
    (dict(D=96), UNSUPPORTED), (dict(rot=0), INVALID), (dict(rot=24), INVALID),
    (dict(rot=80), INVALID), (dict(inter=2), INVALID), (dict(tr=-1), INVALID),
    (dict(f=None), INVALID), (dict(f=_freqs(64, float("nan"))), INVALID),
    (dict(m=float("inf")), INVALID), (dict(y=FAKE, ys=_s(800, 160, 8)), INVALID)])
def test_rope_scaled_refusals(lib, kw, status):
    assert _rope(lib, **kw) == status
    assert lib.star_last_error()


def _plan(lib, **kw):
    a = dict(ctx=FAKE, new=FAKE, B=4, free=FAKE, nf=8, begin=FAKE, page=16, table=FAKE, W=8,
             cu=FAKE, pos=FAKE, slot=FAKE, n=64, runs=FAKE, rc=12, kv=FAKE, next=FAKE, ws=FAKE,
             wsb=256)
    a.update(kw)
    return lib.star_batch_plan(a["ctx"], a["new"], a["B"], a["free"], a["nf"], a["begin"],
                               a["page"], a["table"], a["W"], a["cu"], a["pos"], a["slot"], a["n"],
                               a["runs"], a["rc"], a["kv"], a["next"], a["ws"], a["wsb"], NULL)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), INVALID), (dict(B=4097), INVALID), (dict(page=48), UNSUPPORTED),
    (dict(page=8), UNSUPPORTED), (dict(W=0), INVALID), (dict(W=2**27), INVALID),
    (dict(nf=-1), INVALID), (dict(free=NULL), INVALID), (dict(n=-1), INVALID),
    (dict(rc=11), INVALID), (dict(pos=NULL), INVALID), (dict(ctx=ODD4), INVALID),
    (dict(kv=NULL), INVALID), (dict(next=NULL), INVALID), (dict(table=NULL), INVALID),
    (dict(wsb=255), INVALID), (dict(ws=NULL), INVALID), (dict(ws=ODD), INVALID),
    (dict(n=2**30 + 1, rc=2**30), INVALID)])
def test_batch_plan_refusals(lib, kw, status):
    assert _plan(lib, **kw) == status
    assert lib.star_last_error()


def _append(lib, **kw):
    a = dict(k=FAKE, ks=_s(64, 64), v=FAKE, vs=_s(64, 64), n=8, h=2, D=64, slot=FAKE, runs=FAKE,
             rc=8, kp=FAKE, vp=FAKE, sk=FAKE, sv=FAKE, pages=4, page=16, kind=0, ws=FAKE, wsb=256)
    a.update(kw)
    return lib.star_kv8_append(a["k"], a["ks"], a["v"], a["vs"], a["n"], a["h"], a["D"], a["slot"],
                               a["runs"], a["rc"], a["kp"], a["vp"], a["sk"], a["sv"], a["pages"],
                               a["page"], a["kind"], a["ws"], a["wsb"], NULL)


@pytest.mark.parametrize("kw,status", [
    (dict(k=NULL), INVALID), (dict(v=ODD), INVALID), (dict(ks=_s(60, 64)), INVALID),
    (dict(vs=None), INVALID), (dict(n=-1), INVALID), (dict(h=0), INVALID),
    (dict(h=2049), INVALID), (dict(D=32), UNSUPPORTED), (dict(slot=NULL), INVALID),
    (dict(runs=ODD4), INVALID), (dict(rc=-1), INVALID), (dict(kp=ODD), INVALID),
    (dict(sk=NULL), INVALID), (dict(pages=0), INVALID), (dict(pages=2**28), INVALID),
    (dict(page=256), UNSUPPORTED), (dict(kind=2), INVALID), (dict(wsb=8), INVALID)])
def test_append_refusals(lib, kw, status):
    assert _append(lib, **kw) == status
    assert lib.star_last_error()


def _attend(lib, **kw):
    a = dict(q=FAKE, qs=_s(256, 64), n=4, cu=FAKE, kv=FAKE, B=4, table=FAKE, W=8, kp=FAKE, vp=FAKE,
             sk=FAKE, sv=FAKE, pages=32, page=16, kind=1, Hq=4, h=2, D=64, new=1, max_kv=128,
             o=FAKE, lse=NULL, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return lib.star_kv8_attend(a["q"], a["qs"], a["n"], a["cu"], a["kv"], a["B"], a["table"],
                               a["W"], a["kp"], a["vp"], a["sk"], a["sv"], a["pages"], a["page"],
                               a["kind"], a["Hq"], a["h"], a["D"], a["new"], a["max_kv"], a["o"],
                               a["lse"], a["ws"], a["wsb"], NULL)


@pytest.mark.parametrize("kw,status", [
    (dict(q=NULL), INVALID), (dict(o=ODD), INVALID), (dict(qs=_s(4, 64)), INVALID),
    (dict(n=-1), INVALID), (dict(cu=NULL), INVALID), (dict(kv=ODD4), INVALID),
    (dict(B=0), INVALID), (dict(B=4097), INVALID), (dict(table=NULL), INVALID),
    (dict(W=0), INVALID), (dict(pages=0), INVALID), (dict(page=24), UNSUPPORTED),
    (dict(kind=-1), INVALID), (dict(Hq=3), INVALID), (dict(Hq=0), INVALID),
    (dict(D=256), UNSUPPORTED), (dict(new=0), INVALID), (dict(max_kv=0), INVALID),
    (dict(max_kv=129), INVALID), (dict(lse=ODD4), INVALID), (dict(wsb=256), INVALID),
    (dict(new=2**25), INVALID),
    (dict(B=4096, h=2048, Hq=2048, W=2**26, max_kv=2**29, pages=2**26), INVALID)])
def test_attend_refusals(lib, kw, status):
    assert _attend(lib, **kw) == status
    assert lib.star_last_error()


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path only")
def test_valid_calls_without_device(lib):
    for call in (_rope, _plan, _append, _attend):
        assert call(lib) in (CUDA, UNSUPPORTED)
        assert lib.star_last_error()


# ---- sizes --------------------------------------------------------------------------------------
def test_run_bound(lib):
    """No step of B requests and n tokens makes more runs than star_batch_plan_runs, and small steps
    reach it."""
    for page in (16, 32):
        for B, n in itertools.product((1, 2, 3), (0, 1, 2, 15, 16, 17, 40)):
            most, rng = 0, random.Random(n)
            for _ in range(300):
                cuts = sorted(rng.randint(0, n) for _ in range(B - 1))
                new = [b - a for a, b in zip([0] + cuts, cuts + [n])]
                runs = 0
                for t in new:
                    c = rng.choice([0, 1, page - 1, page, rng.randint(0, 100)])
                    runs += len({(c + i) // page for i in range(t)})
                most = max(most, runs)
            assert most <= star.star_batch_plan_runs(n, B, page) <= max(n, 0)
    assert star.star_batch_plan_runs(34, 1, 16) == 4  # 16 + 16 + 2 can start at row 15
    assert star.star_batch_plan_runs(2**30, 4096, 16) == 2**26 + 8192
    assert star.star_batch_plan_runs(-1, 1, 16) == 0


def test_attend_workspace_bytes(lib):
    for Hq, Hkv, D, new in ((32, 8, 128, 1), (4, 1, 64, 4), (64, 8, 128, 1), (64, 8, 128, 40)):
        rows, parts = {8: (8, 1024), 16: (16, 1024)}.get(new * Hq // Hkv, (256, 320))
        if new * Hq // Hkv < 8:
            rows, parts = 8, 1024
        want = 256 + 512 * 4 + parts * rows * 8 + parts * rows * D * 4
        for B in (1, 16):
            assert star.star_kv8_attend_workspace_bytes(B, B * new, Hq, Hkv, D, new) == want
    assert star.star_kv8_attend_workspace_bytes(0, 1, 1, 1, 64, 1) == 256
    assert star.star_batch_plan_workspace_bytes(16) == 256


# ---- the binding's own checks (CPU tensors are refused before the library is reached) --------------
def _cpu_attend():
    i = lambda *v: torch.zeros(*v, dtype=torch.int32)  # noqa: E731
    return dict(q=torch.zeros(1, 4, 64, dtype=torch.bfloat16), cu_new=i(2), kv_len=i(1),
                block_table=i(1, 4), k_pages=torch.zeros(4, 2, 16, 64, dtype=torch.int8),
                v_pages=torch.zeros(4, 2, 16, 64, dtype=torch.int8), k_scale=torch.zeros(4, 2),
                v_scale=torch.zeros(4, 2), o=torch.zeros(1, 4, 64, dtype=torch.bfloat16),
                workspace=torch.zeros(256, dtype=torch.uint8), max_new=1, max_kv=64)


@pytest.mark.parametrize("change,error", [
    ({}, ValueError),                                                    # not on a CUDA device
    (dict(q=torch.zeros(1, 4, 64)), TypeError),
    (dict(q=torch.zeros(1, 4, 128, dtype=torch.bfloat16)), ValueError),
    (dict(k_pages=torch.zeros(4, 2, 16, 64, dtype=torch.uint8)), TypeError),
    (dict(v_pages=torch.zeros(4, 2, 16, 64, dtype=torch.float8_e4m3fn)), TypeError),
    (dict(v_pages=torch.zeros(5, 2, 16, 64, dtype=torch.int8)), ValueError),
    (dict(k_scale=torch.zeros(4, 3)), ValueError),
    (dict(cu_new=torch.zeros(3, dtype=torch.int32)), ValueError),
    (dict(kv_len=torch.zeros(1, dtype=torch.int64)), ValueError),
    (dict(block_table=torch.zeros(4, dtype=torch.int32)), ValueError),
    (dict(lse=torch.zeros(4, 2)), ValueError),
    (dict(workspace=torch.zeros(256, 2, dtype=torch.uint8)[:, 0]), ValueError),
    (dict(o=torch.zeros(4, 1, 64, dtype=torch.bfloat16).transpose(0, 1)), ValueError)])
def test_attend_binding_refusals(change, error):
    args = _cpu_attend()
    args.update(change)
    with pytest.raises(error):
        star.star_kv8_attend(**args)


def test_other_binding_refusals():
    bf = lambda *v: torch.zeros(*v, dtype=torch.bfloat16)  # noqa: E731
    f = [1.0] * 16
    with pytest.raises(ValueError):
        star.star_rope_scaled(bf(1, 2, 3, 64), bf(1, 2, 3, 64), f)          # CPU
    with pytest.raises(ValueError):
        star.star_rope_scaled(bf(1, 2, 3, 64), bf(1, 2, 4, 64), f)
    with pytest.raises(TypeError):
        star.star_rope_scaled(torch.zeros(1, 2, 3, 64), bf(1, 2, 3, 64), f)
    with pytest.raises(ValueError):
        star.star_rope_scaled(bf(1, 2, 3, 64), bf(1, 2, 3, 64), f, pos=torch.zeros(3, dtype=torch.int32))
    a = _cpu_attend()
    with pytest.raises(ValueError):
        star.star_kv8_append(bf(1, 2, 64), bf(2, 2, 64), a["cu_new"], a["cu_new"], a["k_pages"],
                             a["v_pages"], a["k_scale"], a["v_scale"], a["workspace"])
    with pytest.raises(ValueError):
        star.star_kv8_append(bf(1, 2, 64), bf(1, 2, 64), a["cu_new"], a["cu_new"], a["k_pages"],
                             a["v_pages"], a["k_scale"], a["v_scale"], a["workspace"])
    with pytest.raises(TypeError):
        star.star_rope_scaled(bf(1, 2, 3, 64), bf(1, 2, 3, 64), (ctypes.c_float * 16)())
    with pytest.raises(TypeError):
        star.star_rope_scaled(None, bf(1, 2, 3, 64), f)
    i = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        star.star_batch_plan(i(1), i(2), i(4), i(1), 16, a["block_table"], i(2), i(4), i(4), i(5),
                             i(1), i(1), a["workspace"])

"""The FP4 pools' format in the tests' own 64 bits, pinned; and the refusals of
the calls over them, on the CPU (no pointer here is ever dereferenced)."""
import ctypes

import pytest
import torch

import fp4_util as F
import paged_kv_cache_34_gb300 as pa
from paged_kv_cache_34_gb300 import build as pabuild

M = 0x1000000


@pytest.fixture(scope="module")
def lib():
    pabuild.build()
    return pa.library()


# ------------------------------------------------------------------ format --
def test_e4m3_is_torchs():
    b = torch.arange(127, dtype=torch.uint8)
    assert b.view(torch.float8_e4m3fn).double().tolist() == F.e4m3_values()
    x = torch.linspace(0, 500, 100003)
    want = x.clamp(max=448).to(torch.float8_e4m3fn).view(torch.uint8).long()
    assert torch.equal(F.nearest(x.double(), F.e4m3_values()), want)


def test_codes_and_their_ties():
    x = torch.tensor([0, 0.25, 0.26, 0.75, 1.25, 1.26, 1.75, 2.5, 3.5, 5, 5.01, 6, 100.0])
    assert F.nearest(x.double(), F.E2M1).tolist() == [0, 0, 1, 2, 2, 3, 4, 4, 6, 6, 7, 7, 7]


def test_a_group_by_hand():
    # largest magnitude 12, S = 0.5: 12 / 3 = 4 is an E4M3 value (0x48), w = 2
    x = torch.zeros(1, 1, 16, dtype=torch.float16)
    x[0, 0, :6] = torch.tensor([12.0, -12.0, 2.0, 0.5, -0.6, 7.0])
    code, c = F.quantise(x, torch.tensor([0.5]))
    assert c.tolist() == [[[0x48]]]
    assert code[0, 0, :7].tolist() == [7, 15, 2, 0, 9, 6, 0]  # 3.5 is a tie: 4
    assert F.values(code, c)[0, 0, :6].tolist() == [24, -24, 4, 0, -2, 16]
    # no scale, no codes; NaN counts as 0; infinities take the largest of both
    assert F.quantise(x, torch.tensor([0.0]))[0].abs().sum() == 0
    x[0, 0, 0], x[0, 0, 1] = float("nan"), float("-inf")
    code, c = F.quantise(x, torch.tensor([0.5]))
    assert c.item() == 126 and code[0, 0, :3].tolist() == [0, 15, 0]


def test_pool_layout():
    pool = torch.arange(2 * 3 * 2 * 288).reshape(2, 3, 2, 288).to(torch.uint8)
    code, c = F.get(pool, torch.tensor([21]), 64)  # block 1, offset 5 of 16: tile 0, row 5
    row = pool[1, 2, 0]
    assert code[0, 2, 6] == row[5 * 32 + 3] & 15 and code[0, 2, 7] == row[5 * 32 + 3] >> 4
    assert c[0, 2].tolist() == row[256 + 20:256 + 24].tolist()
    again = torch.zeros_like(pool)
    F.put(again, torch.arange(32), *F.get(pool, torch.arange(32), 64))
    assert torch.equal(again, pool)


# ---------------------------------------------------------------- refusals --
def write(lib, **kw):
    a = dict(k=M, v=2 * M, kvs=256, kc=3 * M, vc=4 * M, sm=5 * M, n=4, hkv=2, d=128, bs=16, nb=64,
             ks=6 * M, vs=7 * M, dtype=1)
    a.update(kw)
    p = {n: ctypes.c_void_p(a[n]) if a[n] else None
         for n in ("k", "v", "kc", "vc", "sm", "ks", "vs")}
    return lib.pa_reshape_and_cache_fp4(p["k"], p["v"], a["kvs"], p["kc"], p["vc"], p["sm"], a["n"],
                                        a["hkv"], a["d"], a["bs"], a["nb"], p["ks"], p["vs"],
                                        a["dtype"], None, None)


WRITE = [(dict(n=-1), 2), (dict(hkv=0), 2), (dict(bs=0), 2), (dict(nb=-1), 2), (dict(nb=1 << 60), 2),
         (dict(d=96), 3), (dict(d=32), 3), (dict(hkv=65537, kvs=1 << 24), 3), (dict(bs=24), 3), (dict(bs=4), 3), (dict(dtype=7), 3),
         (dict(k=0), 1), (dict(v=0), 1), (dict(kc=0), 1), (dict(vc=0), 1), (dict(sm=0), 1),
         (dict(ks=0), 1), (dict(vs=0), 1), (dict(kvs=248), 2), (dict(kvs=260), 4),
         (dict(k=M + 8), 4), (dict(kc=3 * M + 8), 4), (dict(ks=6 * M + 2), 4),
         (dict(vs=7 * M + 1), 4), (dict(sm=5 * M + 4), 4)]


@pytest.mark.parametrize("kw,status", WRITE + [(dict(n=0), 0), (dict(n=0, k=0, sm=0), 0)])
def test_write_refusals(lib, kw, status):
    assert write(lib, **kw) == status


def gather(lib, **kw):
    a = dict(ko=M, kos=256, vo=2 * M, vos=256, r=100, kc=3 * M, vc=4 * M, bt=5 * M, bts=8, mb=8,
             ctx=6 * M, rs=7 * M, s=3, mc=100, hkv=2, d=128, bs=16, nb=64, ks=8 * M, vs=9 * M,
             dtype=1)
    a.update(kw)
    p = {n: ctypes.c_void_p(a[n]) if a[n] else None
         for n in ("ko", "vo", "kc", "vc", "bt", "ctx", "rs", "ks", "vs")}
    return lib.pa_gather_cache_fp4(p["ko"], a["kos"], p["vo"], a["vos"], a["r"], p["kc"], p["vc"],
                                   p["bt"], a["bts"], a["mb"], p["ctx"], p["rs"], a["s"], a["mc"],
                                   a["hkv"], a["d"], a["bs"], a["nb"], p["ks"], p["vs"],
                                   a["dtype"], None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(r=-1), 2), (dict(mb=-1), 2), (dict(s=-1), 2), (dict(mc=-1), 2), (dict(hkv=0), 2),
    (dict(bs=0), 2), (dict(nb=-1), 2), (dict(bts=7), 2), (dict(dtype=2), 3), (dict(d=80), 3),
    (dict(bs=256), 3), (dict(s=65536), 3), (dict(hkv=65537, kos=1 << 24, vos=1 << 24), 3), (dict(kos=248), 2), (dict(vos=248), 2),
    (dict(kos=260), 4), (dict(vos=1 << 62), 2), (dict(ko=0), 1), (dict(vo=0), 1), (dict(kc=0), 1),
    (dict(vc=0), 1), (dict(bt=0), 1), (dict(ctx=0), 1), (dict(rs=0), 1), (dict(ks=0), 1),
    (dict(vs=0), 1), (dict(ko=M + 8), 4), (dict(vo=2 * M + 2), 4), (dict(kc=3 * M + 4), 4),
    (dict(bt=5 * M + 2), 4), (dict(rs=7 * M + 1), 4), (dict(s=0), 0), (dict(mc=0), 0),
    (dict(s=0, kc=0, bt=0), 0),
])
def test_gather_refusals(lib, kw, status):
    assert gather(lib, **kw) == status


def decode(lib, new=None, **kw):
    a = dict(out=M, os=8 * 128, q=2 * M, qs=8 * 128, k=0, v=0, kvs=256, kc=3 * M, vc=4 * M, sm=0,
             n=0, bt=5 * M, bts=8, mb=8, ctx=6 * M, s=3, hq=8, hkv=2, d=128, bs=16, nb=64, ks=8 * M,
             vs=9 * M, scale=0.1, mc=100, ws=0, wsb=0, dtype=1)
    a.update(kw)
    p = {n: ctypes.c_void_p(a[n]) if a[n] else None
         for n in ("out", "q", "k", "v", "kc", "vc", "sm", "bt", "ctx", "ks", "vs", "ws")}
    head = (p["out"], a["os"], p["q"], a["qs"])
    tail = (p["bt"], a["bts"], a["mb"], p["ctx"], a["s"], a["hq"], a["hkv"], a["d"], a["bs"],
            a["nb"], p["ks"], p["vs"], a["scale"], a["mc"], p["ws"], a["wsb"], a["dtype"], None,
            None)
    if new:
        return lib.pa_decode_write_fp4(*head, p["k"], p["v"], a["kvs"], p["kc"], p["vc"], p["sm"],
                                       a["n"], *tail)
    return lib.pa_decode_fp4(*head, p["kc"], p["vc"], *tail)


DECODE = [(dict(s=-1), 2), (dict(mc=-1), 2), (dict(mb=-1), 2), (dict(hkv=3), 2), (dict(nb=0), 2),
          (dict(bts=4), 2), (dict(scale=float("nan")), 2), (dict(scale=float("inf")), 2),
          (dict(d=96), 3), (dict(bs=24), 3), (dict(bs=4), 3), (dict(dtype=3), 3),
          (dict(nb=1 << 28), 3), (dict(out=0), 1), (dict(q=0), 1), (dict(kc=0), 1),
          (dict(vc=0), 1), (dict(bt=0), 1), (dict(ctx=0), 1), (dict(ks=0), 1), (dict(vs=0), 1),
          (dict(os=1016), 2), (dict(qs=1000), 2), (dict(qs=1028), 4), (dict(q=2 * M + 8), 4),
          (dict(kc=3 * M + 8), 4), (dict(ks=8 * M + 2), 4), (dict(bt=5 * M + 2), 4),
          (dict(ctx=6 * M + 2), 4),
          # beyond the schedule's 32 bits, or its prefix sums' shared memory
          (dict(s=1 << 10, mc=1 << 19), 3), (dict(mc=2**31 - 1), 3), (dict(s=8193, mc=16), 3),
          (dict(hq=65537, hkv=65537, qs=1 << 24, os=1 << 24), 3)]


@pytest.mark.parametrize("new", [False, True])
@pytest.mark.parametrize("kw,status", DECODE)
def test_decode_refusals(lib, new, kw, status):
    assert decode(lib, new, **kw) == status


def test_decode_of_nothing(lib):
    assert decode(lib, s=0) == 0 and decode(lib, True, s=0) == 0


@pytest.mark.parametrize("kw,status", [t for t in WRITE if "hkv" not in t[0] and "nb" not in t[0]])
def test_decode_write_refuses_what_the_write_refuses(lib, kw, status):
    a = dict(k=10 * M, v=11 * M, sm=12 * M, n=3)
    a.update(kw)
    if kw.get("k"):
        a["k"] = 10 * M + 8
    assert decode(lib, True, **a) == status


def test_the_plan_refuses_what_the_call_refuses(lib):
    for s, mc in ((1 << 10, 1 << 19), (4, 2**31 - 1), (8193, 16)):
        assert lib.pa_decode_fp4_plan(s, 8, 2, 128, mc, None) == 3
    for a in ((4, 8, 3, 128, 10), (-1, 8, 2, 128, 10), (4, 8, 2, 128, -1), (4, 0, 2, 128, 1)):
        assert lib.pa_decode_fp4_plan(*a, None) == 2
    assert lib.pa_decode_fp4_plan(4, 8, 2, 96, 10, None) == 3


# ------------------------------------------------------------------ python --
def z(*s, dt=torch.bfloat16):
    return torch.zeros(s, dtype=dt)


def i32(*s):
    return torch.zeros(s, dtype=torch.int32)


POOL = z(9, 2, 2, 288, dt=torch.uint8)
S2 = torch.ones(2)


def test_python_write_checks():
    good = [z(3, 2, 64), z(3, 2, 64), POOL, POOL, z(3, dt=torch.int64), S2, S2]
    bad = [(0, z(3, 2, 128)), (0, z(3, 3, 64)), (0, z(3, 2, 64).float()), (1, z(4, 2, 64)),
           (1, z(3, 3, 64)[:, :2]), (1, z(3, 2, 64).half()), (2, POOL.char()), (3, POOL[:, :1]),
           (2, z(9, 2, 2, 289, dt=torch.uint8)), (3, z(18, 2, 2, 288, dt=torch.uint8)[::2]),
           (4, z(3, dt=torch.int32)), (4, z(4, dt=torch.int64)), (5, torch.ones(3)),
           (6, S2.double()), (5, torch.ones(4)[::2])]
    for n, t in bad:
        args = list(good)
        args[n] = t
        with pytest.raises(ValueError):
            pa.pa_reshape_and_cache_fp4(*args)
    for kw, text in ((dict(d_error=z(1)), "d_error must be"), (dict(), "current CUDA device")):
        with pytest.raises(ValueError, match=text):
            pa.pa_reshape_and_cache_fp4(*good, **kw)


def test_python_gather_checks():
    good = [z(30, 2, 64), z(30, 2, 64), POOL, POOL, i32(3, 4), i32(3), i32(3), S2, S2]
    bad = [(0, z(30, 2, 128)), (0, z(30, 2, 64).float()), (1, z(31, 2, 64)), (1, z(30, 2, 64).half()),
           (2, POOL.char()), (4, i32(4, 4)), (4, i32(3, 4).long()), (4, i32(4, 3).t()), (5, i32(4)),
           (6, i32(4)), (6, i32(3).long()), (7, torch.ones(3)), (8, S2.double())]
    for n, t in bad:
        args = list(good)
        args[n] = t
        with pytest.raises(ValueError):
            pa.pa_gather_cache_fp4(*args, max_context_len=8)
    for mc, text in ((1 << 32, "max_context_len must be"), (8, "current CUDA device")):
        with pytest.raises(ValueError, match=text):
            pa.pa_gather_cache_fp4(*good, max_context_len=mc)


def test_python_decode_checks():
    good = [z(3, 8, 64), z(3, 8, 64), POOL, POOL, i32(3, 4), i32(3), S2, S2]
    bad = [(0, z(3, 8, 64).half()), (0, z(3, 4, 64)), (1, z(3, 8, 128)), (2, POOL.char()),
           (3, POOL[:, :1]), (4, i32(4, 4)), (4, i32(3, 4).long()), (4, i32(4, 3).t()), (5, i32(4)),
           (5, i32(3).long()), (6, torch.ones(3)), (7, S2.double())]
    for n, t in bad:
        args = list(good)
        args[n] = t
        with pytest.raises(ValueError):
            pa.pa_decode_fp4(*args, scale=1.0, max_context_len=8)
    for kw, text in ((dict(max_context_len=1 << 32), "max_context_len must be"),
                     (dict(workspace=z(1 << 16, dt=torch.uint8)[::2]), "workspace must be contiguous"),
                     (dict(d_error=z(1)), "d_error must be"), (dict(), "current CUDA device")):
        kw = dict(dict(scale=1.0, max_context_len=8), **kw)
        with pytest.raises(ValueError, match=text):
            pa.pa_decode_fp4(*good, **kw)
        with pytest.raises(ValueError, match=text):
            pa.pa_decode_write_fp4(*good[:2], z(3, 2, 64), z(3, 2, 64), *good[2:4],
                                   z(3, dt=torch.int64), *good[4:], **kw)
    with pytest.raises(ValueError, match="key and value"):
        pa.pa_decode_write_fp4(*good[:2], z(3, 2, 64).half(), z(3, 2, 64).half(), *good[2:4],
                               z(3, dt=torch.int64), *good[4:], scale=1.0, max_context_len=8)

"""pa_decode_shared's refusals, on the CPU: every one is decided on the host
before any CUDA call (no pointer here is ever dereferenced)."""
import ctypes

import pytest
import torch

import paged_kv_cache_34_gb300 as pa
from paged_kv_cache_34_gb300 import build as pabuild


@pytest.fixture(scope="module")
def lib():
    pabuild.build()
    return pa.library()


def call(lib, **kw):
    a = dict(out=0x100000, os=8 * 128, q=0x200000, qs=8 * 128, k=0x300000, v=0x310000, bt=0x320000,
             bts=16, mb=16, ctx=0x330000, gs=0x340000, pl=0x350000, g=2, s=4, hq=8, hkv=2, d=128,
             bs=16, nb=64, scale=0.1, mc=100, mp=50, dtype=1)
    a.update(kw)
    p = {n: ctypes.c_void_p(a[n]) if a[n] else None
         for n in ("out", "q", "k", "v", "bt", "ctx", "gs", "pl")}
    return lib.pa_decode_shared(p["out"], a["os"], p["q"], a["qs"], p["k"], p["v"], p["bt"],
                                a["bts"], a["mb"], p["ctx"], p["gs"], p["pl"], a["g"], a["s"],
                                a["hq"], a["hkv"], a["d"], a["bs"], a["nb"], a["scale"], a["mc"],
                                a["mp"], None, 0, a["dtype"], None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(g=-1), 2), (dict(mp=-1), 2), (dict(mc=-1), 2), (dict(s=-1), 2), (dict(hkv=3), 2),
    (dict(d=96), 3), (dict(bs=24), 3), (dict(bts=8), 2), (dict(scale=float("nan")), 2),
    (dict(dtype=3), 3), (dict(out=0), 1), (dict(q=0), 1), (dict(k=0), 1), (dict(bt=0), 1),
    (dict(ctx=0), 1), (dict(gs=0), 1), (dict(pl=0), 1), (dict(gs=0x340002), 4),
    (dict(pl=0x350001), 4), (dict(q=0x200008), 4), (dict(v=0x310004), 4), (dict(qs=1000), 2),
    (dict(qs=8 * 128 + 4), 4), (dict(nb=1 << 28), 3), (dict(s=0), 0),
    # beyond the schedules' 32 bits: refused (a plain decode would read other rows)
    (dict(s=1 << 10, mc=1 << 19), 3), (dict(mc=2**31 - 1), 3), (dict(mp=2**31 - 1), 3),
    (dict(s=1 << 14, g=1 << 14, mp=1 << 22), 3),
])
def test_refusals(lib, kw, status):
    assert call(lib, **kw) == status


def test_the_plan_refuses_what_the_call_refuses(lib):
    for s, g, mc, mp in ((1 << 10, 2, 1 << 19, 50), (4, 2, 2**31 - 1, 50),
                         (4, 2, 100, 2**31 - 1), (1 << 14, 1 << 14, 100, 1 << 22)):
        assert lib.pa_decode_shared_plan(s, g, 8, 2, 128, mc, mp, None) == 3
    assert lib.pa_decode_shared_plan(4, 2, 8, 3, 128, 100, 50, None) == 2
    assert lib.pa_decode_shared_plan(4, -1, 8, 2, 128, 100, 50, None) == 2


def test_python_argument_checks():
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    good = [z(3, 8, 64), z(3, 8, 64), z(9, 16, 2, 64), z(9, 16, 2, 64), i(3, 4), i(3), i(3), i(2)]
    bad = [(0, z(3, 8, 64, dt=torch.float16)), (1, z(3, 8, 128)), (2, z(9, 16, 2, 128)),
           (3, z(9, 16, 4, 64)[:, :, :2]), (4, i(4, 4)), (4, i(3, 4).long()),
           (4, i(4, 3).t()), (5, i(4)), (6, i(4)), (7, i(3)), (7, i(2).long())]
    for n, t in bad:
        args = list(good)
        args[n] = t
        with pytest.raises(ValueError, match="^(out|caches|block_table|context_lens|group_starts|"
                                             "prefix_lens)"):
            pa.pa_decode_shared(*args, scale=1.0, max_context_len=8, max_prefix_len=4)
    for kw, text in ((dict(d_error=torch.zeros(1)), "d_error must be"),
                     (dict(), "current CUDA device")):
        with pytest.raises(ValueError, match=text):
            pa.pa_decode_shared(*good, scale=1.0, max_context_len=8, max_prefix_len=4, **kw)

"""pa_rope_and_cache's refusals, on the CPU: every one is decided on the host
before any CUDA call (no pointer here is ever dereferenced)."""
import ctypes

import pytest
import torch

import paged_kv_cache_34_gb300 as pa
from paged_kv_cache_34_gb300 import build as pabuild

M = 0x1000000


@pytest.fixture(scope="module")
def lib():
    pabuild.build()
    return pa.library()


def call(lib, **kw):
    # q, k, v: views into one buffer of rows of 12 * 128 elements
    a = dict(qo=9 * M, qos=8 * 128, ko=10 * M, kos=2 * 128, q=M, qs=12 * 128, k=M + 8 * 256,
             v=M + 10 * 256, kvs=12 * 128, pos=3 * M, cs=4 * M, most=100, rot=128, il=0, qw=5 * M,
             kw=6 * M, eps=1e-6, kc=7 * M, vc=8 * M, sm=11 * M, t=4, hq=8, hkv=2, d=128, bs=16,
             nb=64, dtype=1)
    a.update(kw)
    p = {n: ctypes.c_void_p(a[n]) if a[n] else None
         for n in ("qo", "ko", "q", "k", "v", "pos", "cs", "qw", "kw", "kc", "vc", "sm")}
    return lib.pa_rope_and_cache(p["qo"], a["qos"], p["ko"], a["kos"], p["q"], a["qs"], p["k"],
                                 p["v"], a["kvs"], p["pos"], p["cs"], a["most"], a["rot"], a["il"],
                                 p["qw"], p["kw"], a["eps"], p["kc"], p["vc"], p["sm"], a["t"],
                                 a["hq"], a["hkv"], a["d"], a["bs"], a["nb"], a["dtype"], None,
                                 None)


NONE = dict(kc=0, vc=0, sm=0)


@pytest.mark.parametrize("kw,status", [
    (dict(t=0), 0), (dict(t=0, q=0, qo=0, k=0), 0), (dict(t=-1), 2), (dict(hq=0), 2),
    (dict(hkv=0), 2), (dict(rot=-16), 2), (dict(rot=144), 2), (dict(rot=24), 3), (dict(rot=8), 3),
    (dict(d=96, rot=96), 3), (dict(hq=65537), 3), (dict(hkv=65537), 3), (dict(dtype=2), 3), (dict(eps=-1.0), 2), (dict(eps=float("nan")), 2),
    (dict(eps=float("inf")), 2), (dict(most=-1), 2), (dict(bs=0), 2), (dict(nb=-1), 2),
    (dict(nb=1 << 60), 2), (dict(qo=0), 1), (dict(q=0), 1), (dict(k=0), 1), (dict(v=0), 1),
    (dict(kc=0), 1), (dict(vc=0), 1), (dict(sm=0), 1), (dict(pos=0), 1), (dict(cs=0), 1),
    (dict(ko=0, **NONE), 1), (dict(qs=8 * 128 - 8), 2), (dict(qos=1016), 2), (dict(kvs=248), 2),
    (dict(kos=248), 2), (dict(qs=12 * 128 + 4), 4), (dict(qos=8 * 128 + 4), 4),
    (dict(kos=2 * 128 + 4), 4), (dict(kvs=12 * 128 + 4), 4), (dict(qo=9 * M + 8), 4),
    (dict(ko=10 * M + 2), 4), (dict(q=M + 8), 4), (dict(kc=7 * M + 8), 4), (dict(cs=4 * M + 4), 4),
    (dict(qw=5 * M + 2), 4), (dict(kw=6 * M + 8), 4), (dict(pos=3 * M + 2), 4),
    (dict(sm=11 * M + 4), 4), (dict(qs=1 << 62), 2), (dict(qos=1 << 62), 2), (dict(kvs=1 << 62), 2),
    (dict(kos=1 << 62), 2),
    # rows that overlap: query_out over part of query, over key, over value; key_out
    # over query or query_out; another stride in place
    (dict(qo=M + 16, qos=12 * 128), 2), (dict(qo=M + 2 * 256, qos=12 * 128), 2),
    (dict(qo=M + 9 * 256, qos=12 * 128), 2), (dict(ko=M + 256, kos=12 * 128), 2),
    (dict(ko=9 * M + 256, kos=8 * 128), 2), (dict(qo=M, qos=8 * 128), 2),
    (dict(qo=M + 24 * 256, qos=12 * 128), 2), (dict(ko=M + 11 * 256, kos=12 * 128), 2),
    (dict(t=1, qo=M + 16), 2), (dict(ko=M + 10 * 256, kos=12 * 128), 2),
])
def test_refusals(lib, kw, status):
    assert call(lib, **kw) == status


@pytest.mark.parametrize("kw", [
    # what is allowed comes to the device's properties, which need a device
    dict(), NONE, dict(rot=0, pos=0, cs=0), dict(qw=0, kw=0), dict(ko=0), dict(v=0, nb=-1, **NONE),
    dict(qo=M, qos=12 * 128), dict(ko=M + 8 * 256, kos=12 * 128), dict(t=1, qo=M),
    dict(qo=M + 20 * 256 * 12, qos=12 * 128), dict(rot=48), dict(d=64, hq=16, rot=64),
])
def test_what_is_allowed(lib, kw):
    if torch.cuda.is_available():
        pytest.skip("these pointers are none")
    assert call(lib, **kw) == 6


def test_python_argument_checks():
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)  # noqa: E731
    i = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt)  # noqa: E731
    good = [z(3, 8, 64), z(3, 8, 64), z(3, 2, 64), z(3, 2, 64), z(9, 16, 2, 64), z(9, 16, 2, 64),
            i(3, dt=torch.int64), i(3), z(50, 64, dt=torch.float32)]
    bad = [(0, z(3, 8, 64, dt=torch.float16)), (0, z(3, 4, 64)), (1, z(3, 8, 64).float()),
           (2, z(4, 2, 64)), (2, z(3, 2, 128)), (2, z(3, 4, 64)[:, ::2]), (3, z(3, 4, 64)),
           (3, z(3, 3, 64)[:, :2]), (4, z(9, 16, 2, 64).half()), (5, z(9, 16, 4, 64)[:, :, :2]),
           (4, z(9, 16, 3, 64)), (6, i(3)), (6, i(4, dt=torch.int64)), (7, i(4)),
           (7, i(3, dt=torch.int64)), (8, z(50, 64)), (8, z(64, 50, dt=torch.float32).t())]
    for n, t in bad:
        args = list(good)
        args[n] = t
        with pytest.raises(ValueError, match="^(query_out|query|key|value|caches|slot_mapping|"
                                             "positions|cos_sin)"):
            pa.pa_rope_and_cache(*args)
    for kw, text in ((dict(d_error=torch.zeros(1)), "d_error must be"),
                     (dict(q_weight=z(32)), "q_weight must be"),
                     (dict(k_weight=z(64).half()), "k_weight must be"),
                     (dict(key_out=z(3, 2, 64).half()), "key_out must be"),
                     (dict(), "current CUDA device")):
        with pytest.raises(ValueError, match=text):
            pa.pa_rope_and_cache(*good, **kw)
    with pytest.raises(ValueError, match="current CUDA device"):
        pa.pa_qk_norm_rope(good[0], good[2], good[1], good[2], good[7], good[8])

"""pa_attention_varlen's refusals, on the CPU: every one is decided on the host
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
    a = dict(out=0x100000, os=8 * 128, q=0x200000, qs=8 * 128, k=0x300000, v=0x310000, ks=2 * 128,
             cu=0x400000, s=4, t=64, mx=32, hq=8, hkv=2, d=128, scale=0.1, causal=1, dtype=1)
    a.update(kw)
    p = {n: ctypes.c_void_p(a[n]) if a[n] else None for n in ("out", "q", "k", "v", "cu")}
    return lib.pa_attention_varlen(p["out"], a["os"], p["q"], a["qs"], p["k"], p["v"], a["ks"],
                                   p["cu"], a["s"], a["t"], a["mx"], a["hq"], a["hkv"], a["d"],
                                   a["scale"], a["causal"], a["dtype"], None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(s=-1), 2), (dict(t=-1), 2), (dict(mx=-1), 2), (dict(hq=0), 2), (dict(hkv=3), 2),
    (dict(hq=2, hkv=4), 2), (dict(d=96), 3), (dict(d=256), 3), (dict(dtype=2), 3),
    (dict(scale=float("nan")), 2), (dict(scale=float("inf")), 2),
    (dict(qs=8 * 128 - 8), 2), (dict(os=8 * 128 - 8), 2), (dict(ks=2 * 128 - 8), 2),
    (dict(qs=8 * 128 + 4), 4), (dict(ks=2 * 128 + 4), 4), (dict(os=8 * 128 + 4), 4),
    (dict(out=0x100008), 4), (dict(q=0x200008), 4), (dict(k=0x300008), 4), (dict(v=0x310002), 4),
    (dict(cu=0x400002), 4), (dict(out=0), 1), (dict(q=0), 1), (dict(k=0), 1), (dict(v=0), 1),
    # more pairs of query tiles x heads than a grid has blocks
    (dict(s=1 << 30, t=1 << 30, mx=1), 3),
    (dict(cu=0), 1), (dict(s=0), 0), (dict(t=0), 0), (dict(mx=0), 0),
])
def test_refusals(lib, kw, status):
    assert call(lib, **kw) == status


def test_python_argument_checks():
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)  # noqa: E731
    cu = torch.zeros(3, dtype=torch.int32)
    good = [z(10, 8, 64), z(10, 8, 64), z(10, 2, 64), z(10, 2, 64), cu]
    bad = [(0, z(9, 8, 64)), (0, z(10, 8, 64, dt=torch.float16)), (2, z(10, 2, 128)),
           (3, z(10, 2, 64, dt=torch.float32)), (3, z(10, 4, 64)[:, :2]), (2, z(9, 2, 64)),
           (1, z(10, 64, 8).transpose(1, 2)), (4, cu.long()), (4, torch.zeros(0,
                                                                         dtype=torch.int32))]
    for i, t in bad:
        args = list(good)
        args[i] = t
        with pytest.raises(ValueError, match="^(out|query|key|value|cu_seqlens)"):
            pa.pa_attention_varlen(*args, scale=1.0, max_seqlen=8)
    with pytest.raises(ValueError, match="d_error must be"):
        pa.pa_attention_varlen(*good, scale=1.0, max_seqlen=8, d_error=torch.zeros(1))
    with pytest.raises(ValueError, match="current CUDA device"):
        pa.pa_attention_varlen(*good, scale=1.0, max_seqlen=8)


def test_packed_heads_rule():
    # csrc/pa_internal.h flash_packed_heads, restated: the tile rows it fills
    def packed(group):
        for d in range(min(group, 128), 1, -1):
            if group % d == 0 and (128 // d) * d >= 112:
                return d
        return 1
    assert [packed(g) for g in (1, 2, 3, 4, 5, 8, 13, 16, 32, 64, 96, 128)] == \
        [1, 2, 3, 4, 5, 8, 13, 16, 32, 64, 32, 128]
    for g in range(1, 300):
        d = packed(g)
        assert g % d == 0 and (128 // d) * d >= 112

"""pa_build_tables' refusals, on the CPU: every one is decided on the host
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
    a = dict(bt=0x100000, stride=16, mb=16, ctx=0x200000, q=0x210000, free=0x220000, nf=0x230000,
             cap=100, out=0x240000, cu=0x250000, slots=0x260000, pos=0x270000, nfo=0x280000, s=4,
             t=64, bs=16, nb=128)
    a.update(kw)
    p = {k: ctypes.c_void_p(v) if v else None
         for k, v in a.items() if k in ("bt", "ctx", "q", "free", "nf", "out", "cu", "slots",
                                        "pos", "nfo")}
    return lib.pa_build_tables(p["bt"], a["stride"], a["mb"], p["ctx"], p["q"], p["free"],
                               p["nf"], a["cap"], p["out"], p["cu"], p["slots"], p["pos"],
                               p["nfo"], a["s"], a["t"], a["bs"], a["nb"], None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(s=-1), 2), (dict(t=-1), 2), (dict(mb=-1), 2), (dict(cap=-1), 2), (dict(nb=-1), 2),
    (dict(bs=0), 2), (dict(stride=15), 2), (dict(bs=24), 3), (dict(bs=256), 3),
    (dict(ctx=0), 1), (dict(q=0), 1), (dict(out=0), 1), (dict(cu=0), 1), (dict(nf=0), 1),
    (dict(nfo=0), 1), (dict(slots=0), 1), (dict(free=0), 1), (dict(bt=0), 1),
    (dict(ctx=0x200002), 4), (dict(slots=0x260004), 4), (dict(pos=0x270001), 4),
    (dict(out=0x200000), 2),            # in place: other CTAs still read the lengths
    (dict(out=0x200008), 2),            # partial overlap
    (dict(out=0x210004), 2), (dict(nfo=0x230000), 2),
    # any output over any input: cumulative lengths, slots, positions, table
    (dict(cu=0x200000), 2), (dict(cu=0x21000c), 2), (dict(slots=0x220000), 2),
    (dict(pos=0x100000 - 252), 2), (dict(cu=0x1000f8), 2), (dict(nfo=0x22018c), 2),
    (dict(free=0x100000), 2), (dict(ctx=0x1000fc), 2), (dict(slots=0x1fff00), 2),
])
def test_refusals(lib, kw, status):
    assert call(lib, **kw) == status


def test_python_argument_checks():
    s, t = 3, 10
    i = lambda n, dt=torch.int32: torch.zeros(n, dtype=dt)  # noqa: E731
    good = dict(block_table=torch.zeros((s, 4), dtype=torch.int32), context_lens=i(s),
                query_lens=i(s), free_blocks=i(8), num_free=i(1), context_lens_out=i(s),
                cu_seqlens_q=i(s + 1), slot_mapping=i(t, torch.int64), num_free_out=i(1))
    bad = [dict(query_lens=i(s + 1)), dict(cu_seqlens_q=i(s)), dict(slot_mapping=i(t)),
           dict(context_lens=i(s, torch.int64)), dict(query_lens=i(s, torch.int64)),
           dict(num_free=i(2)), dict(num_free_out=i(1, torch.float32)),
           dict(context_lens_out=i(2 * s)[::2]), dict(cu_seqlens_q=i(2 * s + 2)[::2]),
           dict(slot_mapping=i(2 * t, torch.int64)[::2]), dict(free_blocks=i(16)[::2]),
           dict(block_table=torch.zeros((4, s), dtype=torch.int32).t()),
           dict(block_table=torch.zeros((s + 1, 4), dtype=torch.int32))]
    for b in bad:  # refused by name, before the device is looked at
        name = "context_lens" if "context_lens" in b else next(iter(b))
        with pytest.raises(ValueError, match=f"^{name} must"):
            pa.pa_build_tables(*{**good, **b}.values(), block_size=16, num_blocks=8)
    more = dict(block_size=16, num_blocks=8)
    for kw, text in ((dict(positions=i(t + 1)), "^positions must"),
                     (dict(positions=i(t, torch.int64)), "^positions must"),
                     (dict(d_error=i(1, torch.int64)), "d_error must be"),
                     (dict(d_error=i(0)), "d_error must be"),
                     (dict(), "current CUDA device")):
        with pytest.raises(ValueError, match=text):
            pa.pa_build_tables(*good.values(), **more, **kw)

"""Sizes that the decodes refuse because positions within a row are 32-bit, on the CPU (no
pointer here is ever dereferenced)."""
import ctypes

import pytest
import torch

import paged_kv_cache_34_gb300 as pa
from test_fp4_host import M, decode, lib  # noqa: F401

# one sequence, 65536 KV heads: 2^31 elements of queries, and the most that is less
MOST = dict(s=1, mc=32, hkv=65536, d=128, bs=8, mb=8, wsb=1 << 40, ws=15 * M)


@pytest.mark.parametrize("new", [False, True])
@pytest.mark.parametrize("hq,d", [(1 << 24, 128), (1 << 25, 64), (1 << 25, 128), (1 << 30, 64)])
def test_fp4_decode_refuses_rows_past_2_31_elements(lib, new, hq, d):  # noqa: F811
    row = hq * d
    assert decode(lib, new, **dict(MOST, hq=hq, d=d, qs=row, os=row, kvs=65536 * d)) == 3
    assert lib.pa_decode_fp4_plan(1, hq, 65536, d, 32, None) == 3
    assert lib.pa_decode_fp4_plan(0, hq, 65536, d, 0, None) == 3


def test_fp4_decode_takes_shorter_rows(lib):  # noqa: F811
    if torch.cuda.is_available():
        pytest.skip("these pointers are none")
    hq = (1 << 24) - 65536
    row = hq * 128
    assert decode(lib, **dict(MOST, hq=hq, qs=row, os=row)) == 6
    assert lib.pa_decode_fp4_plan(1, hq, 65536, 128, 32, None) == 6


@pytest.mark.parametrize("hq", [1 << 24, 1 << 27])
def test_the_other_decodes_refuse_them_too(lib, hq):  # noqa: F811
    p = [ctypes.c_void_p(n * M) for n in range(1, 12)]
    row = hq * 128
    tail = (p[4], 8, 8, p[5], 1, hq, 65536, 128, 8, 64)
    for call in (lib.pa_decode_int8, lib.pa_decode_fp8):
        assert call(p[0], row, p[1], row, p[2], p[3], *tail, p[6], p[7], 0.1, 32, 0, p[8], 1 << 40,
                    1, None, None) == 3
    assert lib.pa_decode(p[0], row, p[1], row, p[2], p[3], *tail, 0.1, 32, 0, p[8], 1 << 40, 1,
                         None, None) == 3

"""What pa_rope_and_cache refuses besides the shapes of its rows, on the CPU (no pointer
here is ever dereferenced)."""
import pytest
import torch

import paged_kv_cache_34_gb300 as pa
from test_rope_host import M, NONE, call, lib  # noqa: F401

ROWS = 4 * 8 * 128 * 2  # bytes of the query rows out


@pytest.mark.parametrize("kw", [
    # positions, the table, a weight or the slots in the rows of query_out or key_out
    dict(pos=9 * M), dict(pos=9 * M + ROWS - 4), dict(cs=9 * M + 256), dict(cs=9 * M - 256),
    dict(cs=9 * M - 100 * 128 * 4 + 16), dict(qw=9 * M + 512), dict(kw=9 * M - 240),
    dict(sm=9 * M + 8), dict(sm=9 * M - 24), dict(pos=10 * M + 4), dict(qw=10 * M, **NONE),
    dict(kw=10 * M + 4 * 2 * 128 * 2 - 16), dict(cs=10 * M - 16, most=1 << 62),
    dict(t=1, pos=9 * M + 64),
])
def test_other_inputs_in_the_rows_written(lib, kw):  # noqa: F811
    assert call(lib, **kw) == 2


@pytest.mark.parametrize("kw", [
    # beside them; of inputs that are not read; without key_out
    dict(pos=9 * M + ROWS), dict(pos=9 * M - 16), dict(cs=9 * M - 100 * 128 * 4),
    dict(qw=9 * M + ROWS), dict(kw=9 * M - 256), dict(sm=9 * M + ROWS), dict(sm=9 * M - 32),
    dict(rot=0, pos=9 * M, cs=9 * M), dict(ko=0, pos=10 * M),
])
def test_other_inputs_beside_the_rows_written(lib, kw):  # noqa: F811
    if torch.cuda.is_available():
        pytest.skip("these pointers are none")
    assert call(lib, **kw) == 6


def test_python_caches_and_slots_come_together():
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)  # noqa: E731
    good = [z(3, 8, 64), z(3, 8, 64), z(3, 2, 64), z(3, 2, 64), z(9, 16, 2, 64), z(9, 16, 2, 64),
            z(3, dt=torch.int64), z(3, dt=torch.int32), z(50, 64, dt=torch.float32)]
    for gone, text in (((4,), "given together"), ((5,), "given together"), ((6,), "given together"),
                       ((4, 5), "given together"), ((4, 6), "given together"),
                       ((5, 6), "given together"), ((3,), "value must be given"),
                       ((7,), "positions must be given")):
        args = [None if n in gone else t for n, t in enumerate(good)]
        with pytest.raises(ValueError, match=text):
            pa.pa_rope_and_cache(*args, key_out=z(3, 2, 64))
    # none of them: no cache write; no table: no rotation, and no positions
    for gone in ((3, 4, 5, 6), (4, 5, 6), (7, 8), (8,)):
        args = [None if n in gone else t for n, t in enumerate(good)]
        with pytest.raises(ValueError, match="current CUDA device"):
            pa.pa_rope_and_cache(*args, key_out=z(3, 2, 64))

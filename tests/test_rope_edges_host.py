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

"""Refusals of the serving-step operators that are decided on the host, on the
CPU (no pointer here is ever dereferenced; see also the operators' own files)."""
import pytest

import test_attention_varlen_host as varlen
from test_attention_varlen_host import lib  # noqa: F401  (fixture)


@pytest.mark.parametrize("kw,status", [
    # zeros are read from behind the last row, in 32 bits
    (dict(scale=0.0, t=(1 << 30) + 1, s=1, mx=64), 3),
])
def test_attention_varlen_refusals(lib, kw, status):  # noqa: F811
    assert varlen.call(lib, **kw) == status

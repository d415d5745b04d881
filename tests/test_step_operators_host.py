"""Refusals of the serving-step operators that are decided on the host, on the
CPU (no pointer here is ever dereferenced; see also the operators' own files)."""
import pytest
import torch

import paged_kv_cache_34_gb300 as pa
import test_attention_varlen_host as varlen
import test_decode_shared_host as shared
from test_attention_varlen_host import lib  # noqa: F401  (fixture)


@pytest.mark.parametrize("kw,status", [
    # zeros are read from behind the last row, in 32 bits
    (dict(scale=0.0, t=(1 << 30) + 1, s=1, mx=64), 3),
])
def test_attention_varlen_refusals(lib, kw, status):  # noqa: F811
    assert varlen.call(lib, **kw) == status


@pytest.mark.parametrize("d,most", [(64, 14393), (128, 10211)])
def test_decode_shared_plan_refuses_batches_that_the_call_refuses(lib, d, most):  # noqa: F811
    # 12 bytes per sequence in shared memory: refused by both, before any CUDA call
    for s in (most + 1, 3 * most):
        assert lib.pa_decode_shared_plan(s, 1, 8, 2, d, 16, 16, None) == 3
        assert shared.call(lib, s=s, d=d, bs=8, qs=8 * d, os=8 * d, mc=16, mp=16) == 3
    # (PA_ERR_CUDA without a device: not refused)
    assert lib.pa_decode_shared_plan(most, 1, 8, 2, d, 16, 16, None) != 3
    assert shared.call(lib, s=most, d=d, bs=8, qs=8 * d, os=8 * d, mc=16, mp=16) != 3
    # without a prefix it is the plain decode, whose limit is its own
    assert lib.pa_decode_shared_plan(most + 1, 0, 8, 2, d, 16, 16, None) != 3


@pytest.mark.parametrize("workspace", [torch.zeros(1, dtype=torch.uint8).expand(1 << 20),
                                       torch.zeros(1 << 12, dtype=torch.uint8)[::2]])
def test_decode_shared_refuses_a_workspace_that_is_not_its_bytes(workspace):
    # its size counts elements: an expanded or strided one has other bytes behind it
    i = lambda *n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    q, pool = torch.zeros(3, 8, 64), torch.zeros(9, 16, 2, 64)
    q, pool = q.bfloat16(), pool.bfloat16()
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        pa.pa_decode_shared(q, q, pool, pool, i(3, 4), i(3), i(3), i(2), scale=1.0,
                            max_context_len=8, max_prefix_len=4, workspace=workspace)


@pytest.mark.parametrize("bound", [-1, 1 << 31, 1 << 32, (1 << 32) + 64, (1 << 63) - 1])
def test_host_bounds_beyond_32_bits_are_refused(bound):
    # passed on as they are, 2**32 would be 0: nothing to do, without a word
    i = lambda *n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    q, pool = torch.zeros(3, 8, 64).bfloat16(), torch.zeros(9, 16, 2, 64).bfloat16()
    kv = torch.zeros(3, 2, 64).bfloat16()
    with pytest.raises(ValueError, match="max_seqlen must be"):
        pa.pa_attention_varlen(q, q, kv, kv, i(2), scale=1.0, max_seqlen=bound)
    for name in ("max_context_len", "max_prefix_len"):
        bounds = dict(max_context_len=8, max_prefix_len=4)
        bounds[name] = bound
        with pytest.raises(ValueError, match=name + " must be"):
            pa.pa_decode_shared(q, q, pool, pool, i(3, 4), i(3), i(3), i(2), scale=1.0, **bounds)
        with pytest.raises(ValueError, match=name + " must be"):
            pa.pa_decode_shared_plan(3, 2, 8, 2, 64, bounds["max_context_len"],
                                     bounds["max_prefix_len"])

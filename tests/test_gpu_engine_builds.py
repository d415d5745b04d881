"""Every build of the attention tile engine on the inputs where it can go wrong
(tests/engine_builds.py names the builds and reaches them by size).  A batch's
heads repeated until a call takes the build in question give the same values
again, so the first copy is compared with attention in 64 bits and the others
with the first."""
import pytest
import torch

import test_gpu_attention_varlen as varlen
import test_gpu_decode_shared as shared
from engine_builds import first_copy, reach, shared_build, varlen_build
from gpu_util import gpu, pa, require_gpu

pytestmark = gpu

F16, BF16 = torch.float16, torch.bfloat16
NAN = float("nan")
VARLEN = pytest.mark.parametrize("build", ["single", "compact", "pairs"])
# (build, query heads, KV heads, host bound of the prefix): the rows of one tile,
# or tile pairs (32 query heads to a KV head: four sequences to a tile)
SHARED = pytest.mark.parametrize("build,hq,hkv,bound", [
    ("single", 8, 2, None), ("compact", 32, 1, None), ("pairs", 32, 1, 1 << 20)])


def call(x, build, causal=True, **kw):
    y, bound = reach(x, build)
    varlen.run(y, causal, max_seqlen=bound, **kw)
    return y


def decode(x, build, bound):
    b = x["max_prefix"] if bound is None else bound
    assert shared_build(len(x["ctx_list"]), len(x["prefix_list"]), b, x["hq"], x["hkv"]) == build
    shared.run(x, max_prefix=b)


def test_the_rules_reach_every_build():
    # the sizes of the batches of mixed lengths, of few prompts, of long ones
    require_gpu()
    assert varlen_build(16, 16000, 2000, 32, 32) == "compact"
    assert varlen_build(2, 32000, 16384, 32, 8) == "pairs"
    assert varlen_build(1, 37, 37, 8, 2) == "single"
    assert shared_build(64, 6, 9000, 64, 8) == "compact"
    assert shared_build(256, 1, 32768, 64, 8) == "pairs"
    assert shared_build(8, 1, 16384, 32, 32) == "single"


@VARLEN
def test_nan_reaches_its_own_rows_and_no_other(build):
    # a query that is NaN gives NaN (not 0), one in K to the rows that see it
    require_gpu()
    x = varlen.make([150, 300], 4, 2, 64, BF16, seed=21, packed_kv=False)
    x["q"][70, 1, 5] = NAN                 # sequence 0, token 70, head 1
    x["k"][150 + 200, 1, 9] = NAN          # sequence 1, key 200, heads 2 and 3
    y = call(x, build)
    z = first_copy(y)
    nan = torch.isnan(z["out"])
    want = torch.zeros_like(nan)
    want[70, 1] = True
    want[350:, 2:] = True
    assert torch.equal(nan, want)
    ref = varlen.make([150, 300], 4, 2, 64, BF16, seed=21, packed_kv=False)
    ref = call(ref, build)["out"][:, :4]
    assert torch.equal(z["out"][~want], ref[~want])


@SHARED
def test_nan_of_a_query_is_its_output(build, hq, hkv, bound):
    # the query of one sequence and head; every key of another one's own part
    require_gpu()
    x = shared.make([(300, [4, 70, 1, 30, 9, 200])], hq, hkv, 64, 16, BF16, seed=22)
    decode(x, build, bound)
    ref = x["out"].clone()
    x["q"][1, hq - 2, 3] = NAN
    decode(x, build, bound)
    torch.cuda.synchronize()
    want = torch.zeros(ref.shape, dtype=torch.bool, device="cuda")
    want[1, hq - 2] = True
    assert torch.equal(torch.isnan(x["out"]), want)
    assert torch.equal(x["out"][~want], ref[~want])


def test_nan_of_a_query_in_a_join_of_four_warps():
    # few rows with many own pieces each: four warps fold a row
    require_gpu()
    x = shared.make([(200, [3000, 2500])], 4, 2, 128, 16, F16, seed=23)
    x["q"][0, 1, 100] = NAN
    shared.run(x)
    torch.cuda.synchronize()
    nan = torch.isnan(x["out"])
    assert bool(nan[0, 1].all()) and int(nan.sum()) == 128
    shared.verify(x, seqs=[1])


def big(x, power):
    """Queries and keys whose scores reach 10^38, still finite in fp32."""
    for n in ("q", "k"):
        x[n].mul_(2.0 ** power)


SCALES = pytest.mark.parametrize("scale,power", [
    # (scale, power of two on q and k): no preference, whatever the scores; one
    # that brings the largest scores to a few units; the reverse, nearly one-hot
    (0.0, 0), (0.0, 58), (2.0 ** -126, 59), (-0.11, 0), (3.0, 0)])


@VARLEN
@SCALES
def test_scales(build, scale, power, dtype=BF16):
    require_gpu()
    x = varlen.make([200, 0, 129, 1], 6, 2, 64, dtype, seed=24, packed_kv=False)
    big(x, power)
    x["scale"] = scale
    varlen.verify(first_copy(call(x, build)))


@VARLEN
@pytest.mark.parametrize("scale", [0.0, -0.11, 3.0])
def test_scales_in_half_precision(build, scale):
    test_scales(build, scale, 0, F16)


@SHARED
@SCALES
def test_scales_over_a_prefix(build, hq, hkv, bound, scale, power):
    require_gpu()
    x = shared.make([(260, [5, 17, 0, 70, 1]), (40, [3])], hq, hkv, 64, 16, BF16, seed=25)
    big(dict(q=x["q"], k=x["k_pool"]), power)
    x["scale"] = scale
    decode(x, build, bound)
    shared.verify(x)


def test_the_largest_planned_batch():
    # as many sequences as the plan serves, at the smallest blocks
    require_gpu()
    x = shared.make([(9, [1] * 5000), (17, [0, 3] * 2600), (0, [2] * 11)], 2, 1, 128, 8, F16,
                    seed=26)
    assert len(x["ctx_list"]) == 10211
    shared.run(x)
    shared.verify(x, seqs=[0, 1, 31, 4999, 5000, 5001, 8192, 10199, 10200, 10210])


def test_a_bound_of_zero_means_nothing_to_do():
    # nothing is launched: no row written, cu_seqlens not looked at; any other
    # bound that is too short is reported
    require_gpu()
    x = varlen.make([5, 40], 4, 2, 64, BF16, seed=27)
    for bound, err in ((0, 0), (1, pa.DEVERR_CU_SEQLENS)):
        varlen.run(x, max_seqlen=bound)
        torch.cuda.synchronize()
        assert int(x["err"]) == err
        assert bool((x["wide"] == -3.0).all())
    x["cu"].fill_(-9)
    x["err"].zero_()
    varlen.run(x, max_seqlen=0)
    torch.cuda.synchronize()
    assert int(x["err"]) == 0

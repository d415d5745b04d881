"""Every build of the attention tile engine on the inputs where it can go wrong
(tests/engine_builds.py names the builds and reaches them by size).  A batch's
heads repeated until a call takes the build in question give the same values
again, so the first copy is compared with attention in 64 bits and the others
with the first."""
import pytest
import torch

import test_gpu_attention_varlen as varlen
import test_gpu_decode_shared as shared
from engine_builds import (first_copy, reach, runs_with_two_rows_of_a_pair, shared_build,
                           shared_runs, varlen_build)
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


PAIRS = pytest.mark.parametrize("build", ["compact", "pairs"])


@PAIRS
@pytest.mark.parametrize("n", [1, 2, 31, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300])
@pytest.mark.parametrize("hq,hkv,d,dtype", [(1, 1, 128, BF16), (8, 2, 64, F16)])
def test_lengths_in_pairs(build, n, hq, hkv, d, dtype):
    # around one tile, two tiles, and their halves
    require_gpu()
    varlen.verify(first_copy(call(varlen.make([n], hq, hkv, d, dtype, seed=n), build)))


@PAIRS
@pytest.mark.parametrize("hq,hkv,d,dtype", [
    (hq, hkv, d, (F16, BF16)[(hq + d // 64) % 2]) for hq, hkv in varlen.HEADS for d in (64, 128)])
@pytest.mark.parametrize("causal", [True, False])
def test_heads_in_pairs(build, hq, hkv, d, dtype, causal):
    require_gpu()
    x = varlen.make([130, 0, 1, 77, 256, 3, 391], hq, hkv, d, dtype, seed=hq + d)
    varlen.verify(first_copy(call(x, build, causal)), causal)


@PAIRS
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens", [[2000, 40, 1024], [0, 0, 5, 0], [640, 640, 640], [1153]])
def test_longer_prompts_in_pairs(build, causal, lens):
    require_gpu()
    x = varlen.make(lens, 4, 1, 128, F16, seed=len(lens))
    varlen.verify(first_copy(call(x, build, causal)), causal)


def test_long_prompt_in_pairs():
    require_gpu()
    x = varlen.make([5003], 8, 1, 128, F16, seed=4)
    varlen.verify(first_copy(call(x, "pairs")))


@VARLEN
@pytest.mark.parametrize("lens", [[700], [1300, 70]])
def test_rising_scores(build, lens):
    # keys that grow along the sequence: the running maximum jumps by far more
    # than the threshold from tile to tile, in some rows only
    require_gpu()
    x = varlen.make(lens, 4, 1, 128, BF16, seed=5, packed_kv=False)
    n = sum(lens)
    x["k"] = (x["k"].float() * torch.linspace(0.1, 12.0, n, device="cuda")[:, None, None]).to(BF16)
    x["q"][::3] *= 0.01
    varlen.verify(first_copy(call(x, build)))


@VARLEN
@pytest.mark.parametrize("bad", [NAN, float("inf"), torch.finfo(BF16).min])
@pytest.mark.parametrize("causal", [True, False])
def test_neighbours_may_hold_anything(build, bad, causal):
    # the sequence in between and the rows past the last one
    require_gpu()
    x = varlen.make([150, 70, 200, 257], 8, 2, 128, BF16, seed=6, pad=90, packed_kv=False)
    end = x["cu_list"][-1]
    for n in ("q", "k", "v"):
        x[n][end:] = bad
        x[n][150:220] = bad
    varlen.verify(first_copy_of(call(x, build, causal), [0, 2, 3]), causal, seqs=[0, 2, 3])


def first_copy_of(y, seqs):
    """first_copy where the other sequences' outputs are NaN, and not compared."""
    for b, n in enumerate(y["lens"]):
        if b not in seqs:
            y["out"][y["cu_list"][b]:y["cu_list"][b] + n] = 0.0
    return first_copy(y)


@VARLEN
@pytest.mark.parametrize("at,row", [(8, 32), (0, 8), (16, 24)])
def test_output_rows_on_16_bytes(build, at, row):
    # output rows that start on 16 bytes but not on 32 (by the first row, by
    # the row stride, by both)
    require_gpu()
    x = varlen.make([200, 1, 150], 8, 2, 64, F16, seed=9)
    y, bound = reach(x, build)
    t, n = 351, 8 * 64 * y["copies"]
    flat = torch.full((t * (n + row) + at,), varlen.CANARY, dtype=F16, device="cuda")
    y["out"] = flat[at:].view(t, n + row)[:, :n].view(t, 8 * y["copies"], 64)
    varlen.run(y, max_seqlen=bound)
    varlen.verify(first_copy(y))
    assert bool((flat[:at] == varlen.CANARY).all())
    assert bool((flat[at:].view(t, n + row)[:, n:] == varlen.CANARY).all())


@VARLEN
def test_bad_cu_seqlens(build):
    # entries beyond the rows; a sequence longer than the host said: reported,
    # those sequences skipped, the others whole
    require_gpu()
    x = varlen.make([100, 50, 60, 300], 4, 2, 64, BF16, seed=1, pad=10)
    y, bound = reach(x, build)
    y["cu"] = x["cu"].clone()
    y["cu"][2] = 900
    varlen.run(y, max_seqlen=bound)
    varlen.verify(first_copy(y), seqs=[0, 3], err=pa.DEVERR_CU_SEQLENS)
    assert bool((y["out"][100:210] == varlen.CANARY).all())
    if build != "pairs":                   # (whose bound no prompt here exceeds)
        y, _ = reach(dict(x, lens=[100, 50, 60, 99], err=torch.zeros_like(x["err"])), build)
        y["lens"] = x["lens"]
        varlen.run(y, max_seqlen=100)
        varlen.verify(first_copy(y), seqs=[0, 1, 2], err=pa.DEVERR_CU_SEQLENS)
        assert bool((y["out"][210:] == varlen.CANARY).all())


def replayed(calls, outs):
    """Each of `calls` (stream) once; then all at once on two streams, twenty
    times; then captured, and the graphs replayed by turns: the same bits."""
    for c in calls:
        c(None)
    torch.cuda.synchronize()
    first = [o.clone() for o in outs]
    streams = [torch.cuda.Stream() for _ in calls]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for c, s in zip(calls, streams):
            c(s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, f) for o, f in zip(outs, first))
    graphs = []
    for c, o in zip(calls, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(2):
                c(None)
        o.fill_(0)
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, f) for o, f in zip(outs, first))


@VARLEN
def test_captured_and_two_at_once(build):
    require_gpu()
    x, bx = reach(varlen.make([400, 33, 257], 8, 2, 128, BF16, seed=2), build)
    y, by = reach(varlen.make([129, 640], 8, 2, 128, BF16, seed=3), build)
    replayed([lambda s: varlen.run(x, max_seqlen=bx, stream=s),
              lambda s: varlen.run(y, max_seqlen=by, stream=s)], [x["out"], y["out"]])
    varlen.verify(first_copy(x))
    varlen.verify(first_copy(y))


@VARLEN
def test_a_wait_that_runs_out_leaves_the_next_call_whole(build):
    require_gpu()
    x, bound = reach(varlen.make([300, 200], 4, 2, 128, BF16, seed=7), build)
    pa.pa_debug_set_wait_limit_ns(1)
    try:
        varlen.run(x, max_seqlen=bound)
        torch.cuda.synchronize()
    finally:
        pa.pa_debug_set_wait_limit_ns(0)
    assert int(x["err"]) == pa.DEVERR_TIMEOUT
    x["err"].zero_()
    varlen.run(x, max_seqlen=bound)
    varlen.verify(first_copy(x))


@SHARED
@pytest.mark.parametrize("bs", [8, 32, 128])
def test_sequences_shorter_than_their_prefix(build, hq, hkv, bound, bs):
    # as in a padded batch: rows of length 0, 1 and less than the prefix
    require_gpu()
    x = shared.make([(300, [4, 0, 9, 0, 3, 1]), (40, [2, 2])], hq, hkv, 128, bs, BF16, seed=5,
                    short=[(0, 0), (1, 0), (3, 1), (4, 299), (5, 130), (6, 0)])
    decode(x, build, bound)
    shared.verify(x)


@SHARED
@pytest.mark.parametrize("p", [1, 127, 128, 129, 700])
def test_prefix_lengths_on_every_build(build, hq, hkv, bound, p):
    require_gpu()
    x = shared.make([(p, [1, 0, 5, 40, 130, 2, 17])], hq, hkv, 64 if p % 2 else 128, 16, F16,
                    seed=p)
    decode(x, build, bound)
    shared.verify(x)


@SHARED
def test_bad_groups_and_prefix_lengths(build, hq, hkv, bound):
    require_gpu()
    for starts in ([0, 2, 1, 6], [1, 2, 3, 6], [0, 2, 3, 5], [0, 9, 3, 6], [0, -1, 3, 6]):
        x = shared.full_rows(shared.make([(64, [3, 4]), (96, [5]), (32, [1, 70, 2])], hq, hkv, 128,
                                         16, BF16, seed=7))
        x["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        decode(x, build, bound)
        shared.verify(x, err=pa.DEVERR_CU_SEQLENS)
    for bad in (-1, -2 ** 31, 2 ** 31 - 1):
        x = shared.full_rows(shared.make([(64, [3, 4]), (96, [5, 6]), (32, [1, 70])], hq, hkv, 128,
                                         16, BF16, seed=8))
        x["prefix"][1] = bad
        decode(x, build, bound)
        shared.verify(x, err=pa.DEVERR_CONTEXT)


@SHARED
def test_bad_blocks_and_lengths(build, hq, hkv, bound):
    require_gpu()
    # a bad id in one group's prefix: reported, that part adds nothing, the
    # other group is whole
    x = shared.make([(500, [3, 4, 2]), (200, [5, 6, 1])], hq, hkv, 128, 16, BF16, seed=9)
    x["table"][0, 7] = x["k_pool"].shape[0]
    decode(x, build, bound)
    shared.verify(x, seqs={3, 4, 5}, err=pa.DEVERR_BLOCK_ID)
    assert bool(torch.isfinite(x["out"].float()).all())
    # a bad id among a sequence's own blocks
    x = shared.make([(160, [30, 40, 2]), (208, [5, 6, 1])], hq, hkv, 128, 16, BF16, seed=10)
    x["table"][1, 160 // 16] = -7
    decode(x, build, bound)
    shared.verify(x, seqs={0, 2, 3, 4, 5}, err=pa.DEVERR_BLOCK_ID)
    # lengths no table can hold, or beyond the host's bound: an empty sequence
    for n in (-1, 10 ** 6, 2 ** 31 - 1):
        x = shared.make([(160, [30, 40, 2]), (208, [5, 6])], hq, hkv, 128, 16, BF16, seed=11)
        x["ctx"][1] = n
        decode(x, build, bound)
        shared.verify(x, seqs={0, 2, 3, 4}, err=pa.DEVERR_CONTEXT)
        assert bool((x["out"][1] == 0).all())


@SHARED
def test_shared_captured_and_two_at_once(build, hq, hkv, bound):
    require_gpu()
    x = shared.make([(700, [3, 40, 9, 100, 1])], hq, hkv, 128, 16, BF16, seed=12)
    y = shared.make([(130, [3] * 20), (64, [7, 8])], hq, hkv, 128, 16, BF16, seed=13)
    calls = []
    for z in (x, y):
        b = z["max_prefix"] if bound is None else bound
        n = pa.pa_decode_shared_plan(len(z["ctx_list"]), len(z["prefix_list"]), hq, hkv, 128,
                                     z["max_ctx"], b)
        w = torch.full((n,), 0xff, dtype=torch.uint8, device="cuda")
        decode(z, build, bound)
        calls.append(lambda s, z=z, w=w, b=b: shared.run(z, workspace=w, max_prefix=b, stream=s))
    replayed(calls, [x["out"], y["out"]])
    shared.verify(x)
    shared.verify(y)


@SHARED
def test_shared_wait_that_runs_out(build, hq, hkv, bound):
    require_gpu()
    x = shared.make([(900, [30, 40, 1, 2, 3, 4, 5])], hq, hkv, 128, 16, BF16, seed=15)
    pa.pa_debug_set_wait_limit_ns(1)
    try:
        decode(x, build, bound)
        torch.cuda.synchronize()
    finally:
        pa.pa_debug_set_wait_limit_ns(0)
    assert int(x["err"]) == pa.DEVERR_TIMEOUT
    x["err"].zero_()
    decode(x, build, bound)
    shared.verify(x)


@pytest.mark.parametrize("first,tiles", [(2, 76), (6, 85), (8, 97), (1, 129), (4, 141), (7, 151),
                                         (1, 229), (6, 361)])
def test_a_last_block_of_one_tile_behind_another_group(first, tiles):
    # four query tiles: a line of K/V tiles cut into blocks of half a run, the
    # last of one tile, so that a run can hold two rows of one pair; their
    # states stay apart.  (A group before it moves the line against the runs.)
    require_gpu()
    cost, runs = shared_runs(16, 2, tiles * 128, 32, 1)
    run = -(-(first + 4 * tiles) // runs)
    assert tiles % ((run + 1) // 2) == 1
    assert runs_with_two_rows_of_a_pair(first, 4, tiles, run) > 0
    x = shared.make([(first * 128, [2, 0, 1]), (tiles * 128 - 5, [1] * 13)], 32, 1, 64, 64, BF16,
                    seed=tiles)
    shared.run(x, max_prefix=tiles * 128)
    shared.verify(x, seqs=[0, 2, 3, 6, 7, 10, 11, 14, 15])

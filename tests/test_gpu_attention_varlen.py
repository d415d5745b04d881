"""pa_attention_varlen on the GPU against attention in 64 bits (attn_util: the
bound on each element is derived there)."""
import random

import pytest
import torch

from attn_util import attend, check
from gpu_util import gpu, new_err, pa, require_gpu

pytestmark = gpu

F16, BF16 = torch.float16, torch.bfloat16
CANARY = -3.0


def make(lens, hq, hkv, d, dtype, seed=0, pad=0, packed_kv=True):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t = sum(lens) + pad
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)  # noqa: E731
    if packed_kv:  # one interleaved buffer, as a QKV projection leaves it
        qkv = rand(t, hq + 2 * hkv, d)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        q, k, v = rand(t, hq, d), rand(t, hkv, d), rand(t, hkv, d)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    wide = torch.full((t, hq + 1, d), CANARY, device="cuda", dtype=dtype)
    return dict(lens=lens, cu_list=cu, q=q, k=k, v=v, wide=wide, out=wide[:, :hq],
                cu=torch.tensor(cu, dtype=torch.int32, device="cuda"), err=new_err(),
                scale=d ** -0.5)


def run(x, causal=True, **kw):
    pa.pa_attention_varlen(x["out"], x["q"], x["k"], x["v"], x["cu"], scale=x["scale"],
                           max_seqlen=kw.pop("max_seqlen", max(x["lens"] + [0])), causal=causal,
                           d_error=x["err"], **kw)


def verify(x, causal=True, seqs=None, err=0, what=""):
    torch.cuda.synchronize()
    assert int(x["err"]) == err
    g = x["q"].shape[1] // x["k"].shape[1]
    for b, n in enumerate(x["lens"]):
        if n == 0 or (seqs is not None and b not in seqs):
            continue
        a = x["cu_list"][b]
        i = torch.arange(n, device="cuda")
        vis = (i[None] <= i[:, None]).repeat(g, 1) if causal else None
        for h in range(x["k"].shape[1]):
            q = x["q"][a:a + n, h * g:(h + 1) * g].transpose(0, 1).reshape(g * n, -1)
            want, bound = attend(q, x["k"][a:a + n, h], x["v"][a:a + n, h], x["scale"], vis)
            got = x["out"][a:a + n, h * g:(h + 1) * g].transpose(0, 1).reshape(g * n, -1)
            check(got, want, bound, f"{what} sequence {b} of {n}, KV head {h}")
    # the row behind the heads, and the padding rows
    assert bool((x["wide"][:, -1] == CANARY).all())
    assert bool((x["wide"][x["cu_list"][-1]:] == CANARY).all())


# A long bound takes the build for long prompts, the lengths' own the one for
# short ones.
BUILDS = pytest.mark.parametrize("bound", [None, 1 << 20])


def built(bound):
    return {} if bound is None else {"max_seqlen": bound}


HEADS = [(1, 1), (2, 2), (8, 2), (5, 1), (12, 4), (26, 2), (96, 1), (32, 4)]


@pytest.mark.parametrize("n", [1, 2, 31, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300])
@pytest.mark.parametrize("hq,hkv,d,dtype", [(1, 1, 128, BF16), (8, 2, 64, F16)])
@BUILDS
def test_one_prompt(n, hq, hkv, d, dtype, bound):
    require_gpu()
    x = make([n], hq, hkv, d, dtype, seed=n)
    run(x, **built(bound))
    verify(x)


@pytest.mark.parametrize("hq,hkv", HEADS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("causal", [True, False])
@BUILDS
def test_heads(hq, hkv, d, dtype, causal, bound):
    require_gpu()
    x = make([130, 0, 1, 77, 256, 3, 391], hq, hkv, d, dtype, seed=hq + d)
    run(x, causal, **built(bound))
    verify(x, causal)


@pytest.mark.parametrize("lens", [[900, 1], [1, 900], [640, 640, 640], [1153], [0, 0, 5, 0],
                                  [2000, 40, 1024]])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 128), (40, 40, 128), (80, 40, 64)])
@BUILDS
def test_longer_prompts(lens, causal, hq, hkv, d, bound):
    # query tiles alone (few of them) and in pairs, odd tile counts, a last tile
    # on both streams
    require_gpu()
    x = make(lens, hq, hkv, d, BF16, seed=len(lens))
    run(x, causal, **built(bound))
    for n, heads in (("q", 4), ("out", 4), ("k", 4 * hkv // hq), ("v", 4 * hkv // hq)):
        x[n] = x[n][:, :heads]  # the first heads' worth of checking
    verify(x, causal)


@pytest.mark.parametrize("d", [64, 128])
def test_query_tiles_alone_and_in_pairs(d):
    # a prompt's heads alone in a batch, and among so many that tiles go in pairs
    require_gpu()
    x = make([1400, 33], 64, 64, d, BF16, seed=d, packed_kv=False)
    run(x)
    few = dict(x, wide=torch.full((1433, 5, d), CANARY, device="cuda", dtype=BF16),
               **{n: x[n][:, :4].contiguous() for n in ("q", "k", "v")})
    few["out"] = few["wide"][:, :4]
    run(few)
    verify(few)
    verify(dict(x, out=x["out"][:, :4], **{n: few[n] for n in ("q", "k", "v")}))


def test_long_prompt():
    require_gpu()
    x = make([5003], 8, 1, 128, F16, seed=4)
    run(x)
    verify(x)


@pytest.mark.parametrize("s,hi", [(64, 200), (65, 200), (300, 40), (1500, 3)])
def test_many_prompts(s, hi):
    # up to 64 sequences are dealt out by cost, more of them in order
    require_gpu()
    rng = random.Random(s)
    x = make([rng.randint(0, hi) for _ in range(s)], 4, 2, 64, BF16, seed=s)
    run(x)
    verify(x)


@BUILDS
def test_more_items_than_ctas(bound):
    # each CTA walks a long list of short and long items
    require_gpu()
    rng = random.Random(9)
    x = make([rng.choice([1, 100, 128, 200, 333, 700]) for _ in range(40)], 32, 8, 128, BF16,
             seed=9)
    run(x, **built(bound))
    verify(x, seqs=[0, 1, 7, 20, 38, 39])


@pytest.mark.parametrize("scale", [0.0, -0.11, 1.0, 3.0])
@pytest.mark.parametrize("dtype", [F16, BF16])
@BUILDS
def test_scales(scale, dtype, bound):
    # no preference, reversed preference, nearly one-hot weights
    require_gpu()
    x = make([200, 129], 6, 2, 64, dtype, seed=3)
    x["scale"] = scale
    run(x, **built(bound))
    verify(x)


@BUILDS
def test_rising_scores_rescale_the_running_sum(bound):
    # keys that grow along the sequence: the running maximum jumps by far
    # more than the threshold from tile to tile, in some rows only
    require_gpu()
    x = make([700], 4, 1, 128, BF16, seed=5, packed_kv=False)
    ramp = torch.linspace(0.1, 12.0, 700, device="cuda")[:, None, None]
    x["k"] = (x["k"].float() * ramp).to(BF16)
    x["q"][::3] *= 0.01
    run(x, **built(bound))
    verify(x)


def test_padding_and_neighbours_may_hold_anything():
    # rows past the last sequence hold NaN and are left alone; one sequence's
    # infinities and NaN reach no other sequence
    require_gpu()
    for bad in (float("nan"), float("inf"), torch.finfo(BF16).min):
        x = make([150, 70, 200], 8, 2, 128, BF16, seed=6, pad=90, packed_kv=False)
        end = x["cu_list"][-1]
        for n in ("q", "k", "v"):
            x[n][end:] = bad
            x[n][150:220] = bad
        run(x)
        verify(x, seqs=[0, 2])


@pytest.mark.parametrize("at,row", [(8, 32), (0, 8), (16, 24)])
def test_output_rows_on_16_bytes(at, row):
    # output rows that start on 16 bytes but not on 32 (by the first row, by
    # the row stride, by both)
    require_gpu()
    x = make([200, 1, 150], 8, 2, 64, F16, seed=9)
    t, n = 351, 8 * 64
    flat = torch.full((t * (n + row) + at,), CANARY, dtype=F16, device="cuda")
    x["out"] = flat[at:].view(t, n + row)[:, :n].view(t, 8, 64)
    run(x)
    verify(x)
    assert bool((flat[:at] == CANARY).all())
    assert bool((flat[at:].view(t, n + row)[:, n:] == CANARY).all())


def test_rows_beyond_32_bits_of_elements():
    # rows of one wide buffer, the last prompts' more than 2^32 bytes and 2^31
    # elements behind the first's
    require_gpu()
    lens, hq, hkv, d, width = [100] * 660, 4, 2, 128, 1 << 15
    t = sum(lens)
    assert t * width > 1 << 31
    buf = torch.empty((t, width // d, d), dtype=F16, device="cuda")
    q, k, v, out = buf[:, :hq], buf[:, 9:9 + hkv], buf[:, 20:20 + hkv], buf[:, 200:200 + hq]
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    for x in (q, k, v):
        x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
    buf[:, 200 + hq] = CANARY
    cu = list(range(0, t + 1, 100))
    x = dict(lens=lens, cu_list=cu, q=q, k=k, v=v, out=out, wide=buf[:, 200:201 + hq],
             cu=torch.tensor(cu, dtype=torch.int32, device="cuda"), err=new_err(),
             scale=d ** -0.5)
    run(x)
    verify(x, seqs=[0, 1, 327, 328, 655, 656, 658, 659])


def test_equals_the_paged_prefill_in_value():
    # the same prompts through the cache: both are within half of the paged
    # call's stated bound of the exact values, so within it of each other
    require_gpu()
    lens, hq, hkv, d, bs = [300, 77], 8, 2, 128, 16
    x = make(lens, hq, hkv, d, BF16, seed=8)
    run(x)
    t = sum(lens)
    nb = sum(-(-n // bs) for n in lens)
    kp = torch.zeros((nb, bs, hkv, d), dtype=BF16, device="cuda")
    vp = torch.zeros_like(kp)
    table = torch.full((2, 19), -1, dtype=torch.int32, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    ctx, cu, left = i32([0, 0]), i32([0, 0, 0]), i32([0])
    slots = torch.empty(t, dtype=torch.int64, device="cuda")
    pa.pa_build_tables(table, i32([0, 0]), i32(lens), torch.arange(nb, dtype=torch.int32,
                                                                   device="cuda"),
                       i32([nb]), ctx, cu, slots, left, block_size=bs, num_blocks=nb)
    pa.pa_reshape_and_cache(x["k"], x["v"], kp, vp, slots)
    q = x["q"].contiguous()
    paged = torch.empty_like(q)
    pa.pa_prefill_varlen(paged, q, kp, vp, table, cu, ctx, scale=x["scale"], max_seqlen_q=300,
                         max_context_len=300)
    torch.cuda.synchronize()
    verify(x)
    assert float((paged.double() - x["out"].double()).abs().max()) <= 2e-2


def test_bad_cu_seqlens_are_reported_and_skipped():
    require_gpu()
    x = make([100, 50, 60], 4, 2, 64, BF16, seed=1, pad=10)
    x["cu"][2] = 300                      # beyond the rows: sequences 1 and 2 are none
    run(x)
    verify(x, seqs=[0], err=pa.DEVERR_CU_SEQLENS)
    assert bool((x["out"][100:] == CANARY).all())
    x = make([100, 50, 60], 4, 2, 64, BF16, seed=1, pad=10)
    run(x, max_seqlen=60)                 # sequence 0 is longer than the host said
    verify(x, seqs=[1, 2], err=pa.DEVERR_CU_SEQLENS)
    assert bool((x["out"][:100] == CANARY).all())


def test_captured_repeated_and_on_two_streams():
    require_gpu()
    x = make([400, 33, 257], 8, 2, 128, BF16, seed=2)
    y = make([129, 640], 8, 2, 128, BF16, seed=3)
    run(x)
    run(y)
    torch.cuda.synchronize()
    first = x["out"].clone(), y["out"].clone()
    # two calls at once
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        run(x, stream=s1)
        run(y, stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(x["out"], first[0]) and torch.equal(y["out"], first[1])
    graphs = []
    for z in (x, y):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(z)
        graphs.append(g)
    x["out"].fill_(0)
    y["out"].fill_(0)
    for g, s in zip(graphs * 3, (s1, s2) * 3):
        with torch.cuda.stream(s):
            s.wait_stream(torch.cuda.current_stream())
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(x["out"], first[0]) and torch.equal(y["out"], first[1])
    assert int(x["err"]) == 0


@pytest.mark.parametrize("hq,hkv", [(8, 2), (64, 64)])  # tiles alone, in pairs
def test_a_wait_that_runs_out_is_reported(hq, hkv):
    # a 1 ns bound: the launch gives up somewhere, says so and leaves the
    # device usable; the next launches give the same values as before
    require_gpu()
    x = make([300, 200], hq, hkv, 128, BF16, seed=7)
    run(x)
    torch.cuda.synchronize()
    want = x["out"].clone()
    pa.pa_debug_set_wait_limit_ns(1)
    try:
        run(x)
        torch.cuda.synchronize()
    finally:
        pa.pa_debug_set_wait_limit_ns(0)
    assert int(x["err"]) == pa.DEVERR_TIMEOUT
    x["err"].zero_()
    run(x)
    verify(x)
    assert torch.equal(x["out"], want)

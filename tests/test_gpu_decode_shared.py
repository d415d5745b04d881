"""pa_decode_shared on the GPU against attention in 64 bits over the tokens the
definition names (attn_util: the bound on each element is derived there)."""
import random

import pytest
import torch

from attn_util import attend, check
from gpu_util import gpu, new_err, pa, require_gpu

pytestmark = gpu

F16, BF16 = torch.float16, torch.bfloat16
NAN = float("nan")


def make(groups, hq, hkv, d, bs, dtype, seed=0, short=()):
    """groups: (prefix length, [own token counts]).  `short`: (sequence,
    length) pairs cut below their prefix.  Pool rows that the definition does
    not name hold NaN: other blocks, rows past a context, and a sequence's own
    block before the prefix's end."""
    rng = random.Random(seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    starts, prefix, ctx = [0], [], []
    for p, owns in groups:
        prefix.append(p)
        ctx += [p + n for n in owns]
        starts.append(len(ctx))
    for b, n in short:
        ctx[b] = n
    s = len(ctx)
    width = max([1] + [-(-max(c, p) // bs) for c, p in
                       [(c, 0) for c in ctx] + [(0, p) for p in prefix]])
    need = sum(-(-p // bs) for p in prefix) + sum(-(-c // bs) + 1 for c in ctx)
    ids = list(range(need + 3))
    rng.shuffle(ids)
    it = iter(ids)
    table = [[-1] * width for _ in range(s)]
    rows = []                               # pool row of each token of each sequence
    for k, p in enumerate(prefix):
        pre = [next(it) for _ in range(-(-p // bs))]
        for b in range(starts[k], starts[k + 1]):
            # a sequence of its own tokens has its own copy of the block the
            # prefix ends in; the first sequence's row is the prefix's
            n = -(-ctx[b] // bs)
            own = list(pre)
            if ctx[b] > p:
                if p % bs and b > starts[k]:
                    own[-1] = next(it)
                own += [next(it) for _ in range(n - len(own))]
            elif b > starts[k]:
                own = [-1] * len(pre)       # never read: all of it is the prefix
            table[b][:len(own)] = own
            at = [pre[j // bs] if j < p else own[j // bs] for j in range(ctx[b])]
            rows.append([x * bs + j % bs for j, x in enumerate(at)])
    nb = len(ids)
    rand = lambda *sh: torch.randn(sh, generator=g, device="cuda").to(dtype)  # noqa: E731
    k_pool = torch.full((nb, bs, hkv, d), NAN, dtype=dtype, device="cuda")
    v_pool = k_pool.clone()
    used = sorted({r for row in rows for r in row}
                  | {r for k, p in enumerate(prefix) if starts[k + 1] > starts[k]
                     for j in range(p) for r in [table[starts[k]][j // bs] * bs + j % bs]})
    if used:
        u = torch.tensor(used, device="cuda")
        k_pool.view(nb * bs, hkv, d)[u] = rand(len(used), hkv, d)
        v_pool.view(nb * bs, hkv, d)[u] = rand(len(used), hkv, d)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    wide = torch.full((s, hq + 2, d), -3.0, dtype=dtype, device="cuda")
    qw = rand(s, hq + 1, d)
    return dict(starts_list=starts, prefix_list=prefix, ctx_list=ctx, rows=rows, hq=hq, hkv=hkv,
                d=d, bs=bs, q=qw[:, :hq], k_pool=k_pool, v_pool=v_pool, table=i32(table),
                ctx=i32(ctx), starts=i32(starts), prefix=i32(prefix), wide=wide,
                out=wide[:, :hq], err=new_err(), scale=d ** -0.5,
                max_ctx=max(ctx + [0]), max_prefix=max(prefix + [0]))


def run(x, **kw):
    return pa.pa_decode_shared(x["out"], x["q"], x["k_pool"], x["v_pool"], x["table"], x["ctx"],
                               x["starts"], x["prefix"], scale=x["scale"],
                               max_context_len=kw.pop("max_ctx", x["max_ctx"]),
                               max_prefix_len=kw.pop("max_prefix", x["max_prefix"]),
                               d_error=x["err"], **kw)


def verify(x, seqs=None, err=0):
    torch.cuda.synchronize()
    assert int(x["err"]) == err
    g = x["hq"] // x["hkv"]
    kf, vf = x["k_pool"].flatten(0, 1), x["v_pool"].flatten(0, 1)
    for b, rows in enumerate(x["rows"]):
        if seqs is not None and b not in seqs:
            continue
        if not rows:
            assert bool((x["out"][b] == 0).all())
            continue
        r = torch.tensor(rows, device="cuda")
        for h in range(x["hkv"]):
            want, bound = attend(x["q"][b, h * g:(h + 1) * g], kf[r, h], vf[r, h], x["scale"])
            check(x["out"][b, h * g:(h + 1) * g], want, bound,
                  f"sequence {b} of {len(rows)}, KV head {h}")
    assert bool((x["wide"][:, x["hq"]:] == -3.0).all())


# A long bound gives the prefix pass more runs, and the build for long runs.
BUILDS = pytest.mark.parametrize("bound", [None, 1 << 20])


def built(bound):
    return {} if bound is None else {"max_prefix": bound}


@pytest.mark.parametrize("p", [1, 15, 16, 17, 127, 128, 129, 300, 1000])
@pytest.mark.parametrize("bs", [8, 16, 128])
def test_prefix_lengths(p, bs):
    require_gpu()
    x = make([(p, [1, 0, 5, 40, 130])], 8, 2, 64 if p % 2 else 128, bs,
             BF16 if bs == 16 else F16, seed=p + bs)
    run(x)
    verify(x)


@pytest.mark.parametrize("hq,hkv", [(8, 2), (32, 8), (5, 1), (16, 16), (32, 1), (96, 1), (40, 4),
                                    (26, 2)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [F16, BF16])
@BUILDS
def test_heads(hq, hkv, d, dtype, bound):
    # several groups, one of a single sequence, one without a prefix, an empty
    # one, one of empty sequences
    require_gpu()
    x = make([(200, [1, 7, 33]), (70, [9]), (0, [50, 300]), (50, []), (0, [0, 0]), (129, [0, 2])],
             hq, hkv, d, 16, dtype, seed=hq + d)
    run(x, **built(bound))
    verify(x)


@pytest.mark.parametrize("n,hq,hkv,p", [(3, 4, 4, 900), (31, 8, 2, 400), (32, 8, 2, 400),
                                        (33, 8, 2, 260), (70, 8, 2, 384), (200, 4, 4, 257),
                                        (300, 2, 1, 1000)])
@BUILDS
def test_group_sizes(n, hq, hkv, p, bound):
    # rows of one tile, of two, of a tile pair and a half
    require_gpu()
    rng = random.Random(n)
    x = make([(p, [rng.randint(0, 30) for _ in range(n)])], hq, hkv, 128, 32, BF16, seed=n)
    run(x, **built(bound))
    verify(x, seqs=set(rng.sample(range(n), min(n, 40))) | {0, n - 1})


@pytest.mark.parametrize("hq,hkv,groups", [
    # (prefix, sequences): groups of 1 to 5 query tiles and more side by side, lines
    # of many short head units and of few long ones, rows cut across head units
    (32, 4, [(900, 50), (130, 3), (600, 70), (1, 40), (2000, 17)]),
    (32, 4, [(128, 130), (0, 5), (4000, 33), (129, 49)]),
    (5, 5, [(700, 400), (300, 260), (50, 129)]),
    (16, 1, [(3000, 24), (250, 25), (640, 9)]),
    (2, 2, [(6000, 513)]),
    (1, 1, [(19500, 400)]),
])
@BUILDS
def test_groups_of_many_query_tiles(hq, hkv, groups, bound):
    require_gpu()
    rng = random.Random(hq * len(groups))
    x = make([(p, [rng.randint(0, 20) for _ in range(n)]) for p, n in groups], hq, hkv, 64, 16,
             BF16, seed=hq)
    run(x, **built(bound))
    s = x["starts_list"]
    verify(x, seqs=set(rng.sample(range(s[-1]), min(s[-1], 60))) | set(s[:-1])
           | {e - 1 for e in s[1:]})


@pytest.mark.parametrize("bs", [8, 32])
def test_sequences_shorter_than_their_prefix(bs):
    # as in a padded batch: rows of length 0, 1 and less than the prefix
    require_gpu()
    x = make([(300, [4, 0, 9, 0, 3, 1]), (40, [2, 2])], 8, 2, 128, bs, BF16, seed=5,
             short=[(0, 0), (1, 0), (3, 1), (4, 299), (5, 130), (6, 0)])
    run(x)
    verify(x)


def test_long_prefix_few_rows():
    require_gpu()
    x = make([(20000, [3, 100]), (9001, [1])], 4, 2, 128, 128, BF16, seed=2)
    run(x)
    verify(x)


def test_many_groups():
    require_gpu()
    rng = random.Random(3)
    x = make([(rng.randint(0, 200), [rng.randint(0, 20) for _ in range(rng.randint(0, 4))])
              for _ in range(90)], 4, 2, 64, 16, F16, seed=3)
    run(x)
    verify(x)


@pytest.mark.parametrize("scale", [0.0, -0.2, 2.0])
def test_scales(scale):
    require_gpu()
    x = make([(260, [5, 17, 0])], 8, 2, 64, 16, BF16, seed=4)
    x["scale"] = scale
    run(x)
    verify(x)


def test_no_groups_and_no_prefix_is_the_plain_decode():
    require_gpu()
    x = make([(0, [100, 7, 300])], 8, 2, 128, 16, BF16, seed=6)
    want = torch.empty(x["out"].shape, dtype=BF16, device="cuda")
    pa.pa_decode(want, x["q"], x["k_pool"], x["v_pool"], x["table"], x["ctx"], scale=x["scale"],
                 max_context_len=x["max_ctx"])
    run(x)
    torch.cuda.synchronize()
    assert torch.equal(x["out"], want)
    x["starts"], x["prefix"] = x["starts"][:1], x["prefix"][:0]
    x["wide"].fill_(-3.0)
    run(x)
    verify(x)
    assert torch.equal(x["out"], want)


def full_rows(x):
    """The same batch with every row naming all of its tokens' blocks (a
    prefix of whole blocks), as pa_decode wants them."""
    for k, p in enumerate(x["prefix_list"]):
        assert p % x["bs"] == 0
        a, e = x["starts_list"][k], x["starts_list"][k + 1]
        x["table"][a:e, :p // x["bs"]] = x["table"][a, :p // x["bs"]].clone()
    return x


def test_bad_groups_fall_back_to_each_own_row():
    require_gpu()
    for starts in ([0, 2, 1, 5], [1, 2, 3, 5], [0, 2, 3, 4], [0, 9, 3, 5], [0, -1, 3, 5]):
        x = full_rows(make([(64, [3, 4]), (96, [5]), (32, [1, 70])], 8, 2, 128, 16, BF16, seed=7))
        x["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        run(x)
        verify(x, err=pa.DEVERR_CU_SEQLENS)


def test_bad_prefix_lengths_fall_back_to_each_own_row():
    require_gpu()
    for bad in (-1, -2**31, 10**6, 2**31 - 1):
        x = full_rows(make([(64, [3, 4]), (96, [5, 6]), (32, [1, 70])], 8, 2, 128, 16, BF16,
                           seed=8))
        x["prefix"][1] = bad
        run(x)
        verify(x, err=pa.DEVERR_CONTEXT)


def test_bad_blocks_and_lengths():
    require_gpu()
    # a bad id in one group's prefix: reported, that part adds nothing, the
    # other group is whole
    x = make([(500, [3, 4]), (200, [5, 6])], 8, 2, 128, 16, BF16, seed=9)
    x["table"][0, 7] = x["k_pool"].shape[0]
    run(x)
    verify(x, seqs={2, 3}, err=pa.DEVERR_BLOCK_ID)
    assert torch.isfinite(x["out"].float()).all()
    # a bad id among a sequence's own blocks
    x = make([(160, [30, 40]), (208, [5, 6])], 8, 2, 128, 16, BF16, seed=10)
    x["table"][1, 160 // 16] = -7
    run(x)
    verify(x, seqs={0, 2, 3}, err=pa.DEVERR_BLOCK_ID)
    # lengths no table can hold, or beyond the host's bound: an empty sequence
    for n in (-1, 10**6, 2**31 - 1):
        x = make([(160, [30, 40, 2]), (208, [5, 6])], 8, 2, 128, 16, BF16, seed=11)
        x["ctx"][1] = n
        run(x)
        verify(x, seqs={0, 2, 3, 4}, err=pa.DEVERR_CONTEXT)
        assert bool((x["out"][1] == 0).all())


def test_repeated_captured_and_on_two_streams():
    require_gpu()
    x = make([(700, [3, 40, 9, 100])], 8, 2, 128, 16, BF16, seed=12)
    y = make([(130, [3] * 20), (64, [7, 8])], 8, 2, 128, 16, BF16, seed=13)
    spaces = []
    for z in (x, y):
        n = pa.pa_decode_shared_plan(len(z["ctx_list"]), len(z["prefix_list"]), 8, 2, 128,
                                     z["max_ctx"], z["max_prefix"])
        spaces.append(torch.full((n,), 0xff, dtype=torch.uint8, device="cuda"))
        run(z, workspace=spaces[-1])
        verify(z)
    first = [z["out"].clone() for z in (x, y)]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        run(x, workspace=spaces[0], stream=s1)
        run(y, workspace=spaces[1], stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(x["out"], first[0]) and torch.equal(y["out"], first[1])
    graphs = []
    for z, w in zip((x, y), spaces):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(3):
                run(z, workspace=w)
        z["wide"].fill_(-3.0)
        graphs.append(g)
    for g, s in zip(graphs * 3, (s1, s2) * 3):
        with torch.cuda.stream(s):
            s.wait_stream(torch.cuda.current_stream())
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(x["out"], first[0]) and torch.equal(y["out"], first[1])
    assert int(x["err"]) == 0 and int(y["err"]) == 0


def test_pools_beyond_32_bits_of_elements():
    # the batch's blocks moved to the end of pools of more than 2^31 elements
    require_gpu()
    x = make([(300, [5, 70, 1]), (130, [9, 200])], 16, 8, 128, 128, BF16, seed=16)
    nb, n = 16800, x["k_pool"].shape[0]
    assert nb * 128 * 8 * 128 > 1 << 31
    for name in ("k_pool", "v_pool"):
        pool = torch.empty((nb, 128, 8, 128), dtype=BF16, device="cuda")
        pool[nb - n:] = x[name]
        x[name] = pool
    x["table"] = torch.where(x["table"] >= 0, x["table"] + (nb - n), x["table"])
    x["rows"] = [[r + (nb - n) * 128 for r in rows] for rows in x["rows"]]
    run(x)
    verify(x)


def test_own_workspace_on_another_stream():
    # no workspace given: the call's own belongs to the stream it runs on, so
    # what the current stream allocates and writes meanwhile is not it
    require_gpu()
    x = make([(700, [3, 40, 9, 100])], 8, 2, 128, 16, BF16, seed=15)
    n = pa.pa_decode_shared_plan(4, 1, 8, 2, 128, x["max_ctx"], x["max_prefix"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        run(x, stream=s)
        torch.full((n,), 0xff, dtype=torch.uint8, device="cuda")
    verify(x)


def test_behind_a_write_and_before_a_read():
    # the launches around the call in its stream: the step's cache write
    # before it, a copy of its output and a reuse of its inputs behind it
    require_gpu()
    x = make([(96, [2, 3, 50])], 8, 2, 128, 16, BF16, seed=14)
    want = None
    for i in range(10):
        slots = torch.tensor([r[-1] for r in x["rows"]], dtype=torch.int64, device="cuda")
        g = torch.Generator(device="cuda")
        g.manual_seed(i)
        k = torch.randn((3, 2, 128), generator=g, device="cuda").to(BF16)
        v = torch.randn((3, 2, 128), generator=g, device="cuda").to(BF16)
        pa.pa_reshape_and_cache(k, v, x["k_pool"], x["v_pool"], slots)
        run(x)
        want = x["out"].clone()
        x["wide"].fill_(0.0)
    x["wide"].fill_(-3.0)
    x["out"].copy_(want)
    verify(x)


def test_a_wait_that_runs_out_is_reported():
    require_gpu()
    x = make([(900, [30, 40])], 8, 2, 128, 16, BF16, seed=15)
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

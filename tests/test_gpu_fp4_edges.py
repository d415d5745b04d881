"""The calls over FP4 pools at the edges of what they document: keys far below a dominant
one, rows that nothing wrote, batches of one long and many short sequences, many
sequences."""
import pytest
import torch

import fp4_util as F
import paged_kv_cache_34_gb300 as pa

pytestmark = pytest.mark.gpu
DEV = "cuda"
BOTH = [torch.float16, torch.bfloat16]


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def new_err():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def done(err, want=0):
    torch.cuda.synchronize()
    assert int(err) == want


def cache(lens, hkv, d, bs, seed):
    """(block table, pools, head scales) of contexts `lens`: codes of every kind, group
    scales a few steps apart, and NaN scales behind each context."""
    g = gen(seed)
    count = torch.tensor([-(-n // bs) for n in lens])
    nb, width = int(count.sum()) + 2, int(count.max())
    held = (torch.arange(width) < count[:, None]).to(DEV)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEV)
    table[held] = torch.randperm(nb, generator=g, device=DEV)[:int(held.sum())].to(torch.int32)
    n = torch.tensor(lens, device=DEV)
    last = [(table[b, -(-m // bs) - 1], m % bs) for b, m in enumerate(lens) if m % bs]
    pools = []
    for _ in range(2):
        pool = torch.randint(0, 256, (nb, hkv, bs // 8, 9 * d // 2), generator=g, device=DEV,
                             dtype=torch.uint8)
        pool[..., 4 * d:] = 90 + pool[..., 4 * d:] % 32
        ps = F.parts(pool, d)[1]
        for block, m in last:
            behind = torch.arange(bs, device=DEV).view(-1, 8) >= m
            ps[block.long()] = torch.where(behind[..., None], 0x7f, ps[block.long()])
        pools.append(pool)
    scales = [0.001 + 0.002 * torch.rand(hkv, generator=g, device=DEV) for _ in range(2)]
    assert int(n.max()) > 0
    return table, pools, scales


def slots_of(table, b, n, bs):
    j = torch.arange(n, device=DEV)
    return table[b].long()[j // bs] * bs + j % bs


def rows64(pool, S, slots, d):
    return F.values(*F.get(pool, slots, d)) * S.double()[:, None]


def device_us(call, calls=5):
    """Device time of a call among others, the median of nine replays of a graph."""
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        for _ in range(calls):
            call()
    times = []
    for _ in range(11):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        graph.replay()
        b.record()
        torch.cuda.synchronize()
        times.append(1000 * a.elapsed_time(b) / calls)
    return sorted(times[2:])[4]


# ----------------------------------------------------------------- weights --
@pytest.mark.parametrize("dtype", BOTH)
def test_weights_far_below_a_dominant_key(dtype):
    # One key of each head's context is 2^24 to 2^26.8 times as likely as every other, and
    # its value is 0 where theirs is 1: what is left of theirs is the output.  Batches of
    # long contexts, so that a worker meets some hundred thousand keys behind the
    # dominant one (all sequences share one context's blocks).
    d, bs, n, seqs, heads = 64, 128, 1 << 20, 600, 8
    pools = [F.new_pool(n // bs, 1, bs, d, code=0, scale=0x38) for _ in range(2)]
    F.parts(pools[1], d)[0][:] = 0x22  # value 1
    slot = torch.tensor([7], device=DEV)
    row, one = torch.zeros(1, 1, d, device=DEV, dtype=torch.long), \
        torch.full((1, 1, d // 16), 0x38, device=DEV)
    F.put(pools[1], slot, row, one)
    row[..., 0] = 7  # 6
    F.put(pools[0], slot, row, one)
    S = torch.ones(1, device=DEV)
    q = torch.zeros(seqs, heads, d, device=DEV)
    q[:, :, 0] = (24 + 0.4 * torch.arange(heads, device=DEV)) * 0.6931471805599453 / 6
    q = q.to(dtype)
    table = torch.arange(n // bs, dtype=torch.int32, device=DEV).repeat(seqs, 1)
    out, err = torch.empty_like(q), new_err()
    pa.pa_decode_fp4(out, q, *pools, table, i32([n] * seqs), S, S, scale=1.0, max_context_len=n,
                     d_error=err)
    done(err)
    # weights of 1 beside exp(6 q): out = m / (m + exp(6 q)), m = n - 1 keys, in 64 bits;
    # the score 6 q is exact (one product of 2 and 8 or 11 bits), scaled and turned into a
    # power of two in fp32 (relative 2^-23 of up to 20, twice, and the exponential's 2^-21);
    # weights keep 2^-11 (fp16), fp32 sums of 2^18 equal values a lane: n / 32 steps of
    # 2^-24 at most, the output rounded.  Below 2^-14 fp16's steps are 2^-24 whatever the
    # weight, so one is off by up to 2^-25 where the dominant key's is 2^7 or more: 2^-32 of
    # the sum for each of the at most 2^18 keys that share its worker.
    big = torch.exp(6 * q[0, :, 0].double())
    want = ((n - 1) / (n - 1 + big))[None, :, None].expand(seqs, heads, d)
    u = torch.finfo(dtype).eps / 2
    rel = u + 2.0 ** -11 + 20 * 2.0 ** -22 + 2.0 ** -20 + n / 32 * 2.0 ** -24
    F.check(out, want, 1.01 * (rel * want + 2.0 ** (18 - 32)), "what is left beside the dominant key")


@pytest.mark.parametrize("lens,hq,hkv,d", [([700, 3, 1999, 64], 32, 8, 128), ([9000], 16, 2, 64),
                                           ([150, 20, 90], 8, 2, 64), ([2500] * 40, 32, 2, 128)])
def test_a_decode_repeats_itself(lens, hq, hkv, d):
    # no order of work depends on timing: the same bits again, whatever ran in between
    table, pools, scales = cache(lens, hkv, d, 16, 3)
    q = torch.randn(len(lens), hq, d, generator=gen(4), device=DEV).bfloat16()
    args = (*pools, table, i32(lens), *scales)
    first, again = torch.empty_like(q), torch.empty_like(q)
    pa.pa_decode_fp4(first, q, *args, scale=0.1, max_context_len=max(lens))
    for _ in range(5):
        pa.pa_decode_fp4(again, q.roll(1, 0), *args, scale=0.3, max_context_len=max(lens))
        pa.pa_decode_fp4(again, q, *args, scale=0.1, max_context_len=max(lens))
        assert torch.equal(first, again)


# ------------------------------------------------------------------ gather --
@pytest.mark.parametrize("dtype", BOTH)
def test_an_unusable_head_scale_reads_zeros_whatever_the_pool_holds(dtype):
    d, bs = 128, 16
    pools = [F.new_pool(2, 3, bs, d) for _ in range(2)]  # NaN group scales everywhere
    for bad in (0.0, float("nan"), float("inf"), -1.0, 2.0 ** -65, 2.0 ** 65):
        S = torch.tensor([1.0, bad, 1.0], device=DEV)
        out, err = torch.full((2, 40, 3, d), 7.0, dtype=dtype, device=DEV), new_err()
        pa.pa_gather_cache_fp4(out[0], out[1], *pools, i32([[0, 1]]), i32([30]), i32([4]), S, S,
                               max_context_len=32, d_error=err)
        done(err, pa.DEVERR_SCALE)
        assert bool((out[:, 4:34, 1] == 0).all())
        assert bool(out[:, 4:34, ::2].isnan().all())
        assert bool((out[:, :4] == 7).all()) and bool((out[:, 34:] == 7).all())


@pytest.mark.parametrize("dtype", BOTH)
def test_rows_are_rounded_to_fp32_and_then_to_16_bits(dtype):
    # every code under every group scale, under head scales near enough to ties that the
    # two roundings are not one
    d, bs, hkv = 64, 128, 1000
    code = torch.arange(16, device=DEV).repeat(4).expand(128, hkv, d)
    c = torch.arange(128, device=DEV).clamp(max=126)[:, None, None].expand(128, hkv, 4)
    pool = F.new_pool(1, hkv, bs, d)
    F.put(pool, torch.arange(128, device=DEV), code, c)
    S = 0.001 + 0.002 * torch.rand(hkv, generator=gen(5), device=DEV)
    S[:5] = torch.tensor([float.fromhex(x) for x in (
        "0x1.13e8bap-9", "0x1.9305bp-10", "0x1.8d89d8p-10", "0x1.ce6668p-10", "0x1.a3b13cp-10")])
    out, err = torch.empty(2, 128, hkv, d, dtype=dtype, device=DEV), new_err()
    pa.pa_gather_cache_fp4(out[0], out[1], pool, pool, i32([[0]]), i32([128]), i32([0]), S, S,
                           max_context_len=128, d_error=err)
    done(err)
    exact = F.values(code, c) * S.double()[:, None]
    want = exact.float().to(dtype)
    assert torch.equal(out[0], want) and torch.equal(out[1], want)
    # the test would not tell the two apart without such values
    step = (torch.nextafter(want, torch.full_like(want, float("inf"))).double(),
            torch.nextafter(want, torch.full_like(want, float("-inf"))).double())
    off = (want.double() - exact).abs()
    assert bool(((step[0] - exact).abs() < off).any() | ((step[1] - exact).abs() < off).any())


def gathered(lens, hkv, d, bs, dtype, seed, most=None):
    """The gather of `lens` in another order than the sequences', checked exactly."""
    table, pools, scales = cache(lens, hkv, d, bs, seed)
    starts, r = [0] * len(lens), 1
    for b in reversed(range(len(lens))):
        starts[b] = r
        r += lens[b] + b % 2
    out, err = torch.full((2, r, hkv, d), 7.0, dtype=dtype, device=DEV), new_err()
    args = (*pools, table, i32(lens), i32(starts), *scales)
    most = most or max(lens)
    pa.pa_gather_cache_fp4(out[0], out[1], *args, max_context_len=most, d_error=err)
    done(err)
    n = torch.tensor(lens, device=DEV)
    seq = torch.repeat_interleave(torch.arange(len(lens), device=DEV), n)
    j = torch.arange(seq.numel(), device=DEV) - (n.cumsum(0) - n)[seq]
    slots = table[seq, j // bs].long() * bs + j % bs
    at = torch.tensor(starts, device=DEV)[seq] + j
    for o, pool, S in zip(out, pools, scales):
        want = torch.full_like(o, 7.0)
        for a in range(0, at.numel(), 1 << 15):
            k = slice(a, a + (1 << 15))
            v = F.values(*F.get(pool, slots[k], d)).float() * S[:, None]
            want[at[k]] = v.to(dtype)
        assert torch.equal(o, want)
    return lambda: pa.pa_gather_cache_fp4(out[0], out[1], *args, max_context_len=most)


@pytest.mark.parametrize("lens,hkv,d,bs,dtype", [
    ([20000] + [3, 0, 17] * 40, 8, 128, 32, torch.float16),
    ([5, 0, 30000, 9] * 2 + [1] * 250, 1, 64, 16, torch.bfloat16),
    ([0] * 700 + [9000] + [33] * 1300, 2, 64, 8, torch.float16),
    ([40] * 300 + [12000], 3, 128, 16, torch.bfloat16),
    ([4000] + [1] * 90, 40, 128, 128, torch.bfloat16),
    ([0] * 300, 8, 64, 8, torch.float16), ([2500] * 70, 5, 64, 64, torch.float16),
])
def test_gather_of_one_long_and_many_short(lens, hkv, d, bs, dtype):
    gathered(lens if max(lens) else lens[:-1] + [1], hkv, d, bs, dtype, len(lens), most=40000)


def test_gather_time_of_one_long_among_many():
    # the work of 127 contexts of 100 tokens is an eighth of the long one's
    alone = device_us(gathered([100000], 8, 128, 32, torch.bfloat16, 1))
    among = device_us(gathered([100000] + [100] * 127, 8, 128, 32, torch.bfloat16, 1))
    assert among < 2 * alone, f"{among:.0f} us beside {alone:.0f} us alone"


# ------------------------------------------------------------------ decode --
def decoded(lens, hq, hkv, d, bs, dtype, seed):
    """The decode of `lens`, checked against 64 bits for some of its sequences."""
    table, pools, scales = cache(lens, hkv, d, bs, seed)
    q = torch.randn(len(lens), hq, d, generator=gen(seed + 1), device=DEV).to(dtype)
    out, err = torch.full_like(q, float("nan")), new_err()
    args = (*pools, table, i32(lens), *scales)
    ws = torch.empty(pa.pa_decode_fp4_plan(len(lens), hq, hkv, d, max(lens)), dtype=torch.uint8,
                     device=DEV)

    def call(error=None):
        pa.pa_decode_fp4(out, q, *args, scale=d ** -0.5, max_context_len=max(lens), workspace=ws,
                         d_error=error)

    call(err)
    done(err)
    assert bool(out.isfinite().all())
    longest = sorted(range(len(lens)), key=lambda b: -lens[b])
    grp = hq // hkv
    for b in set(longest[:4] + longest[-4:] + [0, len(lens) - 1]):
        if lens[b] == 0:
            assert bool((out[b] == 0).all())
            continue
        slots = slots_of(table, b, lens[b], bs)
        k, v = (rows64(pool, S, slots, d) for pool, S in zip(pools, scales))
        for h in range(hkv):
            r = slice(h * grp, (h + 1) * grp)
            F.check(out[b, r], *F.attend(q[b, r], k[:, h], v[:, h], d ** -0.5), f"sequence {b}")
    return call


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("lens,hq,hkv,d,bs", [
    ([60000] + [100] * 31, 64, 8, 128, 64), ([3, 30000, 0, 200] * 16, 32, 8, 128, 32),
    ([200] * 255 + [40000], 32, 8, 64, 16), ([300] * 64 + [0] * 3 + [20000, 50], 32, 32, 64, 32),
    ([50000] + [200] * 15, 64, 8, 128, 128), ([30000, 30000] + [257] * 130, 128, 8, 64, 128),
    ([25000] + [40] * 180, 12, 4, 128, 8), ([100000, 700] + [30] * 40, 7, 7, 64, 16),
])
def test_decode_of_one_long_and_many_short(lens, hq, hkv, d, bs, dtype):
    decoded(lens, hq, hkv, d, bs, dtype, len(lens))


@pytest.mark.parametrize("short,n", [(100, 31), (200, 255)])
def test_decode_time_of_one_long_among_many(short, n):
    # the short ones are 2 % and 51 % of the long one's work
    alone = device_us(decoded([100000], 64, 8, 128, 128, torch.bfloat16, 1))
    others = device_us(decoded([short] * n, 64, 8, 128, 128, torch.bfloat16, 1))
    among = device_us(decoded([100000] + [short] * n, 64, 8, 128, 128, torch.bfloat16, 1))
    assert among < 1.15 * (alone + others), \
        f"{among:.0f} us; {alone:.0f} us alone, the others {others:.0f}"


@pytest.mark.parametrize("n,most", [(600, 400), (640, 400), (700, 400), (1200, 200)])
def test_many_sequences_leave_as_many_workers_as_fit(n, most):
    # The plan's size says how many partial states a call may leave: one for each sequence's
    # unit and worker.  Lengths and prefix sums, 8 bytes a sequence, leave room for two CTAs
    # of four workers an SM beside rings of two stages up to thousands of sequences.  (Contexts
    # that are not cut, up to 256 tokens, have no use for more workers than there are units:
    # here one each.)
    d, heads = 128, 8
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rows = pa.pa_decode_fp4_plan(n, heads, 1, d, most) // (heads * (d + 2) * 4)
    assert rows - n >= min(2 * 4 * sms - 1, n if most <= 256 else 1 << 30)
    decoded([most, 0, 1, most // 2] * (n // 4), heads, 1, d, 16, torch.float16, n)


# --------------------------------------------------------- errors in builds --
def test_gather_of_uneven_lengths_skips_what_is_wrong():
    # as for even lengths: bad lengths, rows and blocks cost their own part only, whichever
    # round of sequences they are in, and a bad scale leaves zeros
    n, d, hkv, bs = 600, 64, 2, 8
    lens = [20] * n
    lens[300] = 5000
    table, pools, scales = cache(lens, hkv, d, bs, 21)
    starts = [0] * n
    for b in range(1, n):
        starts[b] = starts[b - 1] + lens[b - 1]
    rows = starts[-1] + lens[-1]
    bad_len, bad_rows, bad_block = {0: -3, 299: 5001, 520: 1 << 30}, {1: -1, 255: rows, 599: rows - 19}, \
        {2: (1, 1 << 30), 300: (400, -1), 512: (0, pools[0].shape[0])}
    out, err = torch.full((2, rows, hkv, d), 7.0, dtype=torch.float16, device=DEV), new_err()
    ctx, at, ids = list(lens), list(starts), table.clone()
    for b, v in bad_len.items():
        ctx[b] = v
    for b, v in bad_rows.items():
        at[b] = v
    for b, (block, v) in bad_block.items():
        ids[b, block] = v
    scales[1][1] = 0.0
    pa.pa_gather_cache_fp4(out[0], out[1], *pools, ids, i32(ctx), i32(at), *scales,
                           max_context_len=5000, d_error=err)
    done(err, pa.DEVERR_CONTEXT | pa.DEVERR_CU_SEQLENS | pa.DEVERR_BLOCK_ID | pa.DEVERR_SCALE)
    want = torch.full_like(out, 7.0)
    for b in range(n):
        if b in bad_len or b in bad_rows:
            continue
        slots, to = slots_of(table, b, lens[b], bs), torch.arange(lens[b], device=DEV)
        if b in bad_block:
            keep = to // bs != bad_block[b][0]
            slots, to = slots[keep], to[keep]
        for o, pool, S in zip(want, pools, scales):
            o[starts[b] + to] = (F.values(*F.get(pool, slots, d)).float() * S[:, None]).half()
    assert torch.equal(out, want)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("lens,hq,hkv,d", [
    ([100] * 40 + [30000] + [100] * 30, 32, 32, 128), ([60] * 20 + [20000] + [200] * 20, 64, 8, 128),
    ([20000] + [100] * 40, 16, 16, 128), ([50] * 30 + [40000, 9], 14, 7, 64),
])
def test_long_rows_keep_errors_and_nan_to_themselves(lens, hq, hkv, d, dtype):
    # the long context's rows are joined by several warps; a NaN query, a bad block and a bad
    # scale stay in their own rows
    bs, long = 16, max(range(len(lens)), key=lambda b: lens[b])
    table, pools, scales = cache(lens, hkv, d, bs, 31)
    q = torch.randn(len(lens), hq, d, generator=gen(32), device=DEV).to(dtype)
    args = dict(scale=d ** -0.5, max_context_len=max(lens))
    clean = torch.empty_like(q)
    pa.pa_decode_fp4(clean, q, *pools, table, i32(lens), *scales, **args)
    slots = slots_of(table, long, lens[long], bs)
    grp = hq // hkv
    for h in (0, hkv - 1):
        k, v = (rows64(pool, S, slots, d)[:, h] for pool, S in zip(pools, scales))
        r = slice(h * grp, (h + 1) * grp)
        F.check(clean[long, r], *F.attend(q[long, r], k, v, d ** -0.5), f"head {h}")
    bits = clean.view(torch.int16)
    # NaN in one query head of the long context
    qn, out, err = q.clone(), torch.empty_like(q), new_err()
    qn[long, hq - 1, 3] = float("nan")
    pa.pa_decode_fp4(out, qn, *pools, table, i32(lens), *scales, d_error=err, **args)
    done(err)
    assert bool(out[long, hq - 1].isnan().all())
    out[long, hq - 1] = clean[long, hq - 1]
    assert torch.equal(out.view(torch.int16), bits)
    # a block of the long context: finite, and the others as they were
    ids = table.clone()
    ids[long, 7] = pools[0].shape[0]
    pa.pa_decode_fp4(out, q, *pools, ids, i32(lens), *scales, d_error=err, **args)
    done(err, pa.DEVERR_BLOCK_ID)
    assert bool(out[long].isfinite().all())
    out[long] = clean[long]
    assert torch.equal(out.view(torch.int16), bits)
    # one head's scale
    err.zero_()
    bad = scales[0].clone()
    bad[hkv - 1] = float("inf")
    pa.pa_decode_fp4(out, q, *pools, table, i32(lens), bad, scales[1], d_error=err, **args)
    done(err, pa.DEVERR_SCALE)
    assert bool((out[:, hq - grp:] == 0).all())
    out[:, hq - grp:] = clean[:, hq - grp:]
    assert torch.equal(out.view(torch.int16), bits)

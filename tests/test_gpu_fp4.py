"""The FP4 pools on the GPU: the write's bytes and the gather's rows exactly, the
decode within its 64-bit bound."""
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


# ------------------------------------------------------------------- write --
@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("shuffled", [False, True])
def test_every_16_bit_pattern(dtype, shuffled):
    # every pattern (NaN, infinities, both zeros, subnormals) as a key and, in another
    # order, as a value, under scales from 2^-64 to 2^64
    scales = [2.0 ** -64, 1.7e-9, 1e-4, 0.0017, 0.33, 1.0, 1.5, 77.7, 2.0 ** 40, 2.0 ** 64]
    bits = torch.arange(65536, device=DEV)
    if shuffled:
        bits = bits[torch.randperm(65536, generator=gen(1), device=DEV)]
    x = bits.to(torch.int32).to(torch.int16).view(dtype).view(512, 1, 128).repeat(1, len(scales), 1)
    y = x.flip(0, 2).contiguous()
    S = torch.tensor(scales, device=DEV)
    kc, vc = (F.new_pool(32, len(scales), 16, 128) for _ in range(2))
    slots = torch.randperm(512, generator=gen(2), device=DEV)
    err = new_err()
    pa.pa_reshape_and_cache_fp4(x, y, kc, vc, slots, S, S, d_error=err)
    done(err)
    for rows, pool in ((x, kc), (y, vc)):
        code, c = F.quantise(rows, S)
        got, got_c = F.get(pool, slots, 128)
        assert torch.equal(got_c.long(), c)
        assert torch.equal(got.long(), code)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("t,hkv,d,bs", [(1, 1, 64, 8), (5, 2, 64, 16), (37, 8, 128, 32),
                                        (300, 32, 128, 128), (129, 3, 64, 64), (2000, 8, 128, 16),
                                        (9, 40, 128, 8)])
def test_write(t, hkv, d, bs, dtype):
    g = gen(t + hkv)
    qkv = torch.randn(t, 3 * hkv, d, generator=g, device=DEV).to(dtype)
    k, v = qkv[:, hkv:2 * hkv], qkv[:, 2 * hkv:]
    ks, vs = (0.001 + 0.002 * torch.rand(hkv, generator=g, device=DEV) for _ in range(2))
    nb = -(-t // bs) + 2
    slots = torch.randperm(nb * bs, generator=g, device=DEV)[:t]
    slots[::4] = -1
    kc, vc = F.new_pool(nb, hkv, bs, d), F.new_pool(nb, hkv, bs, d, code=0x13, scale=0x55)
    want = [kc.clone(), vc.clone()]
    real = slots >= 0
    for pool, x, s in ((want[0], k, ks), (want[1], v, vs)):
        F.put(pool, slots[real], *F.quantise(x[real], s))
    err = new_err()
    pa.pa_reshape_and_cache_fp4(k, v, kc, vc, slots, ks, vs, d_error=err)
    done(err)
    assert torch.equal(kc, want[0]) and torch.equal(vc, want[1])


def test_write_bad_slots_and_scales():
    k, v = torch.randn(2, 6, 3, 64, generator=gen(3), device=DEV).half()
    for bad in (0.0, -1.0, float("nan"), float("inf"), 2.0 ** -65, 2.0 ** 65):
        ks, vs = torch.tensor([[0.01, bad, 0.02], [0.01, 0.01, 0.01]], device=DEV)
        kc, vc = F.new_pool(2, 3, 8, 64), F.new_pool(2, 3, 8, 64)
        want = [kc.clone(), vc.clone()]
        slots = torch.tensor([0, 3, 16, 15, -5, 1 << 40], device=DEV)
        err = new_err()
        pa.pa_reshape_and_cache_fp4(k, v, kc, vc, slots, ks, vs, d_error=err)
        done(err, pa.DEVERR_SLOT | pa.DEVERR_SCALE)
        ok = torch.tensor([0, 1, 3], device=DEV)
        F.put(want[0], slots[ok], *F.quantise(k[ok], ks))
        F.put(want[1], slots[ok], *F.quantise(v[ok], vs))
        assert torch.equal(kc, want[0]) and torch.equal(vc, want[1])


# ------------------------------------------------------------------ gather --
def state(lens, hkv, d, bs, seed, spare=3):
    """Pools of random rows for contexts `lens`; rows of no position hold NaN scales."""
    g = gen(seed)
    count = [-(-max(n, 0) // bs) for n in lens]
    nb = sum(count) + spare
    ids = torch.randperm(nb, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(lens), max(count + [1])), -1, dtype=torch.int32, device=DEV)
    used = 0
    for b, c in enumerate(count):
        table[b, :c] = ids[used:used + c]
        used += c
    pools, scales = [], []
    slots = torch.cat([torch.zeros(0, dtype=torch.int64, device=DEV)] + [
        table[b].long().repeat_interleave(bs)[:n] * bs
        + torch.arange(n, device=DEV) % bs for b, n in enumerate(lens)])
    for _ in range(2):
        pool = F.new_pool(nb, hkv, bs, d)
        S = 0.001 + 0.002 * torch.rand(hkv, generator=g, device=DEV)
        code = torch.randint(0, 16, (slots.numel(), hkv, d), generator=g, device=DEV)
        c = torch.randint(0, 120, (slots.numel(), hkv, d // 16), generator=g, device=DEV)
        F.put(pool, slots, code, c)
        pools.append(pool)
        scales.append(S)
    return table, pools, scales, slots


def rows16(pool, slots, S, d, dtype):
    v = F.values(*F.get(pool, slots, d)).float() * S[:, None]
    return v.to(dtype)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("lens,hkv,d,bs", [([1], 1, 64, 8), ([7, 0, 130, 64], 2, 128, 16),
                                           ([33, 1000, 5], 8, 128, 128), ([200] * 40, 2, 64, 32),
                                           ([0, 0], 2, 64, 16), ([3000], 32, 128, 64)])
def test_gather(lens, hkv, d, bs, dtype):
    table, (kc, vc), (ks, vs), slots = state(lens, hkv, d, bs, seed=len(lens) + hkv)
    # rows of every sequence behind a gap, in another order than the sequences'
    starts, r = [0] * len(lens), 2
    for b in reversed(range(len(lens))):
        starts[b] = r
        r += lens[b] + 3
    buf = torch.full((2, r, 2 * hkv, d), 7.0, dtype=dtype, device=DEV)
    k_out, v_out = buf[0, :, :hkv], buf[1, :, hkv:]  # strided rows
    err = new_err()
    pa.pa_gather_cache_fp4(k_out, v_out, kc, vc, table, i32(lens), i32(starts), ks, vs,
                           max_context_len=max(lens) + 5, d_error=err)
    done(err)
    want = torch.full_like(buf, 7.0)
    at = torch.cat([torch.arange(n, device=DEV) + s for n, s in zip(lens, starts)])
    want[0, at, :hkv] = rows16(kc, slots, ks, d, dtype)
    want[1, at, hkv:] = rows16(vc, slots, vs, d, dtype)
    assert torch.equal(buf, want)


def test_gather_errors_skip_their_part():
    lens, hkv, d, bs = [20, 20, 20, 20, 20, 20], 2, 64, 8
    table, (kc, vc), (ks, vs), slots = state(lens, hkv, d, bs, seed=9)
    good = rows16(kc, slots, ks, d, torch.float16).view(6, 20, hkv, d)
    lens[1], lens[2] = -3, 41
    starts = [0, 20, 40, -1, 101, 60]
    table[5, 1] = kc.shape[0]
    table[0, 2] = -7
    out = torch.full((2, 120, hkv, d), 7.0, dtype=torch.float16, device=DEV)
    err = new_err()
    pa.pa_gather_cache_fp4(out[0], out[1], kc, vc, table, i32(lens), i32(starts), ks, vs,
                           max_context_len=100, d_error=err)
    done(err, pa.DEVERR_CONTEXT | pa.DEVERR_CU_SEQLENS | pa.DEVERR_BLOCK_ID)
    want = torch.full_like(out[0], 7.0)
    want[0:16], want[60:68], want[76:80] = good[0, :16], good[5, :8], good[5, 16:]
    assert torch.equal(out[0], want)
    # a bad scale: zeros for that head
    ks[1] = float("nan")
    pa.pa_gather_cache_fp4(out[0], out[1], kc, vc, table[4:5], i32([20]), i32([0]), ks, vs,
                           max_context_len=100, d_error=err)
    torch.cuda.synchronize()
    assert int(err) & pa.DEVERR_SCALE
    assert bool((out[0, :20, 1] == 0).all()) and torch.equal(out[0, :20, 0], good[4, :, 0])


# ------------------------------------------------------------------ decode --
def reference(q, pools, scales, table, lens, bs, scale):
    kc, vc = pools
    hkv, d = kc.shape[1], q.shape[2]
    grp = q.shape[1] // hkv
    want = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    bound = torch.zeros_like(want)
    for b, n in enumerate(lens):
        if n <= 0:
            continue
        slots = table[b].long().repeat_interleave(bs)[:n] * bs + torch.arange(n, device=DEV) % bs
        k, v = (F.values(*F.get(pool, slots, d)) * S.double()[:, None]
                for pool, S in zip(pools, scales))
        for h in range(hkv):
            r = slice(h * grp, (h + 1) * grp)
            want[b, r], bound[b, r] = F.attend(q[b, r], k[:, h], v[:, h], scale)
    return want, bound


def run(lens, hq, hkv, d, bs, dtype, seed, scale=None, spread=1.0, most=None):
    table, pools, scales, _ = state(lens, hkv, d, bs, seed)
    # real caches hold values of about one standard deviation: a few code scales apart
    for pool in pools:
        ps = F.parts(pool, d)[1]
        ps.copy_(torch.where(ps == 0x7f, ps, 90 + ps % 32))
    q = (torch.randn(len(lens), hq, d, generator=gen(seed + 1), device=DEV) * spread).to(dtype)
    scale = d ** -0.5 if scale is None else scale
    out = torch.full_like(q, float("nan"))
    err = new_err()
    pa.pa_decode_fp4(out, q, *pools, table, i32(lens), *scales, scale=scale,
                     max_context_len=max(lens) if most is None else most, d_error=err)
    done(err)
    want, bound = reference(q, pools, scales, table, lens, bs, scale)
    F.check(out, want, bound, f"{lens[:4]} {hq}/{hkv}")
    assert all(bool((out[b] == 0).all()) for b, n in enumerate(lens) if n == 0)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("bs", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (8, 2, 128), (4, 4, 128), (24, 2, 64)])
def test_block_sizes(bs, hq, hkv, d, dtype):
    run([1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 65, 130, 0, 257], hq, hkv, d, bs, dtype, bs)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("grp", [1, 2, 3, 5, 8, 9, 15, 16, 17, 33, 64])
def test_groups(grp, dtype):
    run([300, 41, 1], 2 * grp, 2, 128, 16, dtype, grp)
    run([77], grp, 1, 64, 32, dtype, grp)


@pytest.mark.parametrize("lens,hq,hkv,d,bs", [
    ([512, 2048, 1333, 701, 1999, 600, 888, 1024], 32, 32, 128, 16),
    ([50, 2000, 130, 0, 777, 1999, 64, 51], 32, 8, 128, 32),
    ([40001, 20000], 64, 8, 128, 128), ([9000], 8, 1, 64, 64), ([20000, 3], 128, 8, 128, 32),
    ([16] * 700, 8, 2, 64, 8), ([1] * 1500 + [0] * 30, 4, 2, 64, 16),
    ([200, 1, 0, 256, 130, 33] * 16, 8, 2, 128, 16), ([256, 128, 0, 129] * 4, 16, 8, 64, 32),
])
def test_long_and_many(lens, hq, hkv, d, bs):
    run(lens, hq, hkv, d, bs, torch.bfloat16 if hkv == 8 else torch.float16, len(lens) + hq)


@pytest.mark.parametrize("lens,hq,hkv,d,bs", [
    ([700, 0, 333, 900] * 33, 32, 8, 128, 32),  # many rows, more sequences than a warp sums up
    ([900, 33, 0, 1500] * 16, 64, 8, 64, 32), ([2700, 1, 500] * 8, 128, 8, 128, 16),
    ([600] * 128, 16, 2, 64, 64), ([600] * 129, 16, 2, 64, 64), ([2000] * 130, 4, 1, 128, 16),
    ([1500, 20, 900], 32, 8, 128, 32), ([3000, 0, 2500], 6, 2, 64, 16),
])
def test_pieces_of_many_and_few_rows(lens, hq, hkv, d, bs):
    for dtype in BOTH:
        run(lens, hq, hkv, d, bs, dtype, len(lens) + d, most=max(lens) + 500)


@pytest.mark.parametrize("dtype", BOTH)
def test_scales_and_sizes_of_queries(dtype):
    for scale in (0.0, -0.1, 1e-30, 3.0):
        run([100, 33], 8, 2, 128, 16, dtype, 5, scale=scale)
    run([100, 33], 8, 2, 128, 16, dtype, 6, spread=30.0)
    if dtype is torch.bfloat16:  # beyond fp16's range, and below it
        run([100, 33], 8, 2, 128, 16, dtype, 7, spread=1e6, scale=1e-7)
        run([100, 33], 32, 2, 64, 16, dtype, 8, spread=1e-9, scale=1e8)


def test_loose_bounds_and_a_padded_table():
    run([100, 33, 260], 8, 2, 128, 16, torch.float16, 9, most=272)
    table, pools, scales, _ = state([50], 2, 64, 16, 3)
    wide = torch.full((1, 5000), 1 << 30, dtype=torch.int32, device=DEV)
    wide[0, :4] = table[0]
    q = torch.randn(1, 4, 64, device=DEV).half()
    a, b = torch.empty_like(q), torch.empty_like(q)
    pa.pa_decode_fp4(a, q, *pools, table, i32([50]), *scales, scale=0.1, max_context_len=50)
    pa.pa_decode_fp4(b, q, *pools, wide, i32([50]), *scales, scale=0.1, max_context_len=80000)
    want, bound = reference(q, pools, scales, table, [50], 16, 0.1)
    F.check(a, want, bound)
    F.check(b, want, bound)


def test_nan_queries_stay_in_their_head():
    for lens in ([40, 40], [9000, 40]):
        table, pools, scales, _ = state(lens, 2, 128, 16, 4)
        for dtype in BOTH:
            q = torch.randn(2, 16, 128, generator=gen(5), device=DEV).to(dtype)
            q[0, 3, 7] = float("nan")
            out = torch.empty_like(q)
            pa.pa_decode_fp4(out, q, *pools, table, i32(lens), *scales, scale=0.1,
                             max_context_len=max(lens))
            assert bool(out[0, 3].isnan().all())
            out[0, 3], q[0, 3] = 0, 0
            want, bound = reference(q, pools, scales, table, lens, 16, 0.1)
            want[0, 3] = 0
            F.check(out, want, bound)


def test_errors():
    lens = [40, 40, 40, 40]
    table, pools, scales, _ = state(lens, 2, 64, 16, 6)
    q = torch.randn(4, 4, 64, generator=gen(5), device=DEV).half()
    want, bound = reference(q, pools, scales, table, lens, 16, 0.1)
    got, err = torch.empty_like(q), new_err()
    bad = i32([-1, 49, 200, 40])
    pa.pa_decode_fp4(got, q, *pools, table, bad, *scales, scale=0.1, max_context_len=200,
                     d_error=err)
    done(err, pa.DEVERR_CONTEXT)
    assert bool((got[:3] == 0).all())
    F.check(got[3], want[3], bound[3])
    # a bad block: its pieces add nothing (they begin at multiples of 16 tokens at most)
    for id in (-1, pools[0].shape[0], 1 << 30):
        t = table.clone()
        t[1, 1] = id
        err.zero_()
        pa.pa_decode_fp4(got, q, *pools, t, i32(lens), *scales, scale=0.1, max_context_len=40,
                         d_error=err)
        done(err, pa.DEVERR_BLOCK_ID)
        assert bool(got.isfinite().all())
        F.check(got[[0, 2, 3]], want[[0, 2, 3]], bound[[0, 2, 3]])
    for s in (0.0, float("nan"), 2.0 ** 65):
        for which in (0, 1):
            sc = [x.clone() for x in scales]
            sc[which][1] = s
            err.zero_()
            pa.pa_decode_fp4(got, q, *pools, table, i32(lens), *sc, scale=0.1, max_context_len=40,
                             d_error=err)
            done(err, pa.DEVERR_SCALE)
            assert bool((got[:, 2:] == 0).all())
            F.check(got[:, :2], want[:, :2], bound[:, :2])
    with pytest.raises(pa.PaError):
        pa.pa_decode_fp4(got, q, *pools, table, i32(lens), *scales, scale=0.1, max_context_len=40,
                         workspace=torch.empty(64, dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("dtype", BOTH)
def test_write_and_decode_in_one_call(dtype):
    lens = [17, 600, 1, 129]
    table, pools, scales, _ = state(lens, 2, 128, 16, 7)
    g = gen(8)
    q, k = (torch.randn(4, n, 128, generator=g, device=DEV).to(dtype) for n in (8, 4))
    k, v = k[:, :2], k[:, 2:]
    last = torch.tensor([n - 1 for n in lens], device=DEV)
    slots = table[torch.arange(4, device=DEV), last // 16].long() * 16 + last % 16
    two = [p.clone() for p in pools]
    a, b, err = torch.empty_like(q), torch.empty_like(q), new_err()
    pa.pa_reshape_and_cache_fp4(k, v, *two, slots, *scales)
    pa.pa_decode_fp4(a, q, *two, table, i32(lens), *scales, scale=0.1, max_context_len=600)
    pa.pa_decode_write_fp4(b, q, k, v, *pools, slots, table, i32(lens), *scales, scale=0.1,
                           max_context_len=600, d_error=err)
    done(err)
    assert torch.equal(a, b) and all(torch.equal(x, y) for x, y in zip(two, pools))
    want, bound = reference(q, pools, scales, table, lens, 16, 0.1)
    F.check(b, want, bound)


def test_graphs_streams_and_two_calls_at_once():
    lens = [3000, 1, 0, 777]
    table, pools, scales, _ = state(lens, 2, 128, 16, 10)
    g = gen(11)
    qs = [torch.randn(4, 8, 128, generator=g, device=DEV).half() for _ in range(2)]
    outs = [torch.empty_like(q) for q in qs]
    need = pa.pa_decode_fp4_plan(4, 8, 2, 128, 3000)
    spaces = [torch.empty(need, dtype=torch.uint8, device=DEV) for _ in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    ctx = i32(lens)

    def call(n, stream=None):
        pa.pa_decode_fp4(outs[n], qs[n], *pools, table, ctx, *scales, scale=0.1,
                         max_context_len=3000, workspace=spaces[n], stream=stream)

    torch.cuda.synchronize()
    for _ in range(20):
        for n in (0, 1):
            call(n, streams[n])
    torch.cuda.synchronize()
    for n in (0, 1):
        want, bound = reference(qs[n], pools, scales, table, lens, 16, 0.1)
        F.check(outs[n], want, bound)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(0)
    first = outs[0].clone()
    qs[0].copy_(qs[1])
    ctx[0] = 1500
    graph.replay()
    torch.cuda.synchronize()
    lens[0] = 1500
    want, bound = reference(qs[0], pools, scales, table, lens, 16, 0.1)
    F.check(outs[0], want, bound)
    assert not torch.equal(first, outs[0])


def test_pools_past_2_32_bytes():
    hkv, d, bs = 8, 128, 128
    nb = (1 << 32) // (hkv * bs // 8 * 576) + 20
    pools = [torch.zeros(nb, hkv, bs // 8, 576, dtype=torch.uint8, device=DEV) for _ in range(2)]
    lens = [300]
    table = i32([[nb - 1, 0, nb - 7]])
    slots = table[0].long().repeat_interleave(bs)[:300] * bs + torch.arange(300, device=DEV) % bs
    k, v = torch.randn(2, 300, hkv, d, generator=gen(12), device=DEV).half()
    S = torch.full((hkv,), 0.0017, device=DEV)
    pa.pa_reshape_and_cache_fp4(k, v, *pools, slots, S, S)
    code, c = F.quantise(k, S)
    got, got_c = F.get(pools[0], slots, d)
    assert torch.equal(got.long(), code) and torch.equal(got_c.long(), c)
    rows = torch.empty(2, 300, hkv, d, dtype=torch.float16, device=DEV)
    pa.pa_gather_cache_fp4(rows[0], rows[1], *pools, table, i32(lens), i32([0]), S, S,
                           max_context_len=300)
    assert torch.equal(rows[1], rows16(pools[1], slots, S, d, torch.float16))
    q = torch.randn(1, 16, d, generator=gen(13), device=DEV).half()
    out = torch.empty_like(q)
    pa.pa_decode_fp4(out, q, *pools, table, i32(lens), S, S, scale=0.1, max_context_len=300)
    F.check(out, *reference(q, pools, (S, S), table, lens, bs, 0.1))


def test_copy_blocks():
    table, pools, scales, _ = state([64, 64], 2, 64, 16, 14)
    before = [p.clone() for p in pools]
    pairs = torch.tensor([[int(table[0, 0]), int(table[1, 3])]], device=DEV)
    pa.pa_copy_blocks(*pools, pairs)
    torch.cuda.synchronize()
    for a, b in zip(pools, before):
        assert torch.equal(a[pairs[0, 1]], b[pairs[0, 0]])


@pytest.mark.parametrize("d", [64, 128])
def test_a_wait_that_runs_out(d):
    # pools larger than L2, so that copies are waited for longer than one try of a wait
    # takes; the launches after it are as before
    lens = [4000] * (48 if d == 128 else 96)
    table, pools, scales, _ = state(lens, 8, d, 128, 15)
    q = torch.randn(len(lens), 8, d, generator=gen(16), device=DEV).half()
    first, again, err = torch.empty_like(q), torch.empty_like(q), new_err()
    args = (q, *pools, table, i32(lens), *scales)
    pa.pa_decode_fp4(first, *args, scale=0.1, max_context_len=4000)
    pa.pa_debug_set_wait_limit_ns(1)
    try:
        pa.pa_decode_fp4(again, *args, scale=0.1, max_context_len=4000, d_error=err)
        torch.cuda.synchronize()
    finally:
        pa.pa_debug_set_wait_limit_ns(0)
    assert int(err) == pa.DEVERR_TIMEOUT
    err.zero_()
    for _ in range(3):
        pa.pa_decode_fp4(again, *args, scale=0.1, max_context_len=4000, d_error=err)
        assert torch.equal(first, again)
    done(err)


def test_empty_calls():
    table, pools, scales, _ = state([40, 5], 2, 64, 16, 17)
    before = [p.clone() for p in pools]
    q = torch.full((2, 8, 64), 3.0, dtype=torch.float16, device=DEV)
    out, err = torch.full_like(q, 7.0), new_err()
    pa.pa_decode_fp4(out, q, *pools, table, i32([0, 0]), *scales, scale=0.1, max_context_len=0,
                     d_error=err)
    done(err)
    assert bool((out == 0).all())
    none = torch.empty(0, 2, 64, dtype=torch.float16, device=DEV)
    slots = torch.empty(0, dtype=torch.int64, device=DEV)
    pa.pa_reshape_and_cache_fp4(none, none, *pools, slots, *scales, d_error=err)
    pa.pa_gather_cache_fp4(none, none, *pools, table, i32([0, 0]), i32([9, -1]), *scales,
                           max_context_len=40, d_error=err)
    pa.pa_decode_fp4(q[:0], q[:0], *pools, table[:0], i32([]), *scales, scale=0.1,
                     max_context_len=40, d_error=err)
    # a step whose batch decodes nothing still writes
    pa.pa_decode_write_fp4(q[:0], q[:0], q[:1, :2], q[1:, 2:4], *pools, table[0, :1].long() * 16,
                           table[:0], i32([]), *scales, scale=0.1, max_context_len=40, d_error=err)
    done(err)
    for pool, was, s in zip(pools, before, scales):
        F.put(was, table[0, :1].long() * 16, *F.quantise(q[:1, :2], s))
        assert torch.equal(pool, was)

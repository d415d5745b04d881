"""pa_rope_and_cache and pa_qk_norm_rope against the formula in 64 bits."""
import pytest
import torch

import paged_kv_cache_34_gb300 as pa

gpu = pytest.mark.gpu
DEV = "cuda"


def table(most, rot):
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(most, dtype=torch.float64)[:, None] * f[None]
    return torch.cat([a.cos(), a.sin()], 1).float().to(DEV)


def formula(x, pos, cos_sin, w, eps, pairs):
    """(value, scale of the fp32 errors) of heads x [T, H, D], in 64 bits."""
    y = x.double()
    if w is not None:
        y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
    out, size = y.clone(), y.abs()
    if cos_sin is not None and cos_sin.shape[1]:
        half = cos_sin.shape[1] // 2
        at = cos_sin[pos.long()].double()[:, None, :]
        c, s = at[..., :half], at[..., half:]
        i = torch.arange(half, device=x.device)
        a, b = (2 * i, 2 * i + 1) if pairs else (i, i + half)
        ya, yb = y[..., a], y[..., b]
        out[..., a], out[..., b] = ya * c - yb * s, yb * c + ya * s
        size[..., a] = (ya * c).abs() + (yb * s).abs()
        size[..., b] = (yb * c).abs() + (ya * s).abs()
    return out, size


def check(got, want, size, dtype, what):
    # half a step of the output's type (fp16: of its subnormals at least), and the fp32
    # steps before it: 128 squares summed along 16 lanes' terms and three shuffles (at
    # most 19 roundings, halved by the root), rsqrt (2 units), three products, the
    # rotation's product and sum: at most 20 units of 2^-24 of the terms' sizes
    u = torch.finfo(dtype).eps / 2
    least = 2.0 ** -25 if dtype is torch.float16 else 0.0
    bound = u * want.abs() + (1 + u) * 20 * 2.0 ** -24 * size + least
    off = (got.double() - want).abs() - bound
    assert bool((off <= 0).all()), f"{what}: off its bound by {float(off.max())}"


def make(t, hq, hkv, d, dtype, seed, spread=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    qkv = (torch.randn(t, hq + 2 * hkv, d, generator=g, device=DEV) * spread).to(dtype)
    w = (1 + 0.3 * torch.randn(2, d, generator=g, device=DEV)).to(dtype)
    pos = torch.randint(0, 4096, (t,), generator=g, device=DEV, dtype=torch.int32)
    return qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], w[0], w[1], pos, g


def run(t, hq, hkv, d, dtype, rot, pairs, norm, bs, rows, seed, spread=1.0, stream=None):
    q, k, v, qw, kw, pos, g = make(t, hq, hkv, d, dtype, seed, spread)
    qw, kw = (qw if "q" in norm else None), (kw if "k" in norm else None)
    cs = table(4096, rot) if rot else None
    nb = -(-t // bs) + 3
    slots = torch.randperm(nb * bs, generator=g, device=DEV)[:t]
    slots[::5] = -1 - torch.arange(slots[::5].numel(), device=DEV)  # padding tokens
    kc = torch.full((nb, bs, hkv, d), 7.0, dtype=dtype, device=DEV)
    vc = torch.full((nb, bs, hkv, d), 9.0, dtype=dtype, device=DEV)
    q_out = torch.empty(t, hq, d, dtype=dtype, device=DEV)
    k_out = torch.empty(t, hkv, d, dtype=dtype, device=DEV) if rows else None
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    before = [x.clone() for x in (q, k, v)]
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    pa.pa_rope_and_cache(q_out, q, k, v, kc, vc, slots, pos, cs, key_out=k_out, interleaved=pairs,
                         q_weight=qw, k_weight=kw, eps=1e-5, d_error=err, stream=stream)
    torch.cuda.synchronize()
    assert int(err) == 0
    assert all(torch.equal(a, b) for a, b in zip(before, (q, k, v)))
    want, size = formula(q, pos, cs, qw, 1e-5, pairs)
    check(q_out, want, size, dtype, "query_out")
    want, size = formula(k, pos, cs, kw, 1e-5, pairs)
    real = slots >= 0
    flat_k, flat_v = kc.view(-1, hkv, d), vc.view(-1, hkv, d)
    check(flat_k[slots[real]], want[real], size[real], dtype, "key_cache")
    assert torch.equal(flat_v[slots[real]], v[real])
    if rows:
        check(k_out, want, size, dtype, "key_out")
        assert torch.equal(k_out[real], flat_k[slots[real]])
    left = torch.ones(nb * bs, dtype=torch.bool, device=DEV)
    left[slots[real]] = False
    assert bool((flat_k[left] == 7).all()) and bool((flat_v[left] == 9).all())


@gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("t,hq,hkv,d,rot,pairs,norm,bs,rows", [
    (1, 8, 2, 64, 64, False, "", 16, False), (4, 8, 2, 64, 16, True, "qk", 8, True),
    (5, 32, 32, 128, 128, False, "", 16, False), (33, 32, 8, 128, 128, False, "qk", 32, True),
    (7, 40, 8, 128, 64, True, "k", 128, False), (64, 12, 4, 64, 48, False, "q", 12, True),
    (3, 128, 8, 128, 128, True, "qk", 64, True), (2, 32, 1, 128, 16, False, "qk", 1, False),
    (9, 1, 1, 64, 0, False, "qk", 16, True), (2, 7, 3, 128, 112, False, "q", 16, False),
    (6, 64, 8, 64, 32, True, "", 16, True), (2500, 16, 16, 128, 128, False, "qk", 16, False),
    (3001, 8, 2, 64, 64, True, "k", 32, True), (1, 256, 64, 128, 128, False, "qk", 16, True),
])
def test_matches_formula(t, hq, hkv, d, rot, pairs, norm, bs, rows, dtype):
    run(t, hq, hkv, d, dtype, rot, pairs, norm, bs, rows, seed=t * 131 + d + rot)


@gpu
@pytest.mark.parametrize("t,hq,hkv,d,rot,pairs,norm", [
    (305, 8, 2, 128, 128, False, "qk"), (701, 3, 1, 64, 48, True, ""),
    (4901, 8, 4, 128, 96, True, "qk"), (5003, 1, 1, 64, 64, False, "q"),
    (6007, 12, 4, 64, 64, False, "qk"), (20011, 5, 3, 64, 32, True, "k"),
])
def test_many_tokens_of_few_heads(t, hq, hkv, d, rot, pairs, norm):
    # several tokens share a CTA, the last CTA's places are not all taken
    run(t, hq, hkv, d, torch.bfloat16, rot, pairs, norm, 16, True, seed=t)


@gpu
def test_a_bad_position_leaves_the_tokens_beside_it():
    q, k, v, qw, kw, pos, g = make(5000, 4, 2, 64, torch.float16, 11)
    bad = torch.randperm(5000, generator=g, device=DEV)[:300]
    cs = table(4096, 64)
    want_q, size_q = formula(q, pos, cs, qw, 1e-6, False)
    want_k, size_k = formula(k, pos, cs, kw, 1e-6, False)
    pos[bad] = 4096
    q_out, k_out = torch.full((5000, 4, 64), 5.0, dtype=q.dtype, device=DEV), \
        torch.full((5000, 2, 64), 6.0, dtype=q.dtype, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.pa_qk_norm_rope(q_out, k_out, q, k, pos, cs, q_weight=qw, k_weight=kw, d_error=err)
    torch.cuda.synchronize()
    assert int(err) == pa.DEVERR_POSITION
    assert bool((q_out[bad] == 5).all()) and bool((k_out[bad] == 6).all())
    good = torch.ones(5000, dtype=torch.bool, device=DEV)
    good[bad] = False
    check(q_out[good], want_q[good], size_q[good], q.dtype, "query_out")
    check(k_out[good], want_k[good], size_k[good], q.dtype, "key_out")


@gpu
@pytest.mark.parametrize("spread", [1e-4, 300.0])
def test_sizes_of_values(spread):
    for norm in ("", "qk"):
        run(17, 8, 2, 128, torch.float16, 128, False, norm, 16, True, seed=3, spread=spread)
        run(17, 8, 2, 128, torch.bfloat16, 64, True, norm, 16, True, seed=4, spread=spread)


@gpu
@pytest.mark.parametrize("pairs", [False, True])
def test_in_place_equals_out_of_place(pairs):
    q, k, v, qw, kw, pos, _ = make(50, 8, 2, 128, torch.bfloat16, 5)
    cs = table(4096, 96)
    more = dict(interleaved=pairs, q_weight=qw, k_weight=kw)
    q_out, k_out = torch.empty(50, 8, 128, dtype=q.dtype, device=DEV), \
        torch.empty(50, 2, 128, dtype=q.dtype, device=DEV)
    pa.pa_qk_norm_rope(q_out, k_out, q, k, pos, cs, **more)
    was = v.clone()
    pa.pa_qk_norm_rope(q, k, q, k, pos, cs, **more)
    torch.cuda.synchronize()
    assert torch.equal(q, q_out) and torch.equal(k, k_out) and torch.equal(v, was)


@gpu
def test_bad_positions_and_slots_are_skipped():
    q, k, v, qw, kw, pos, _ = make(12, 8, 2, 64, torch.float16, 6)
    cs = table(4096, 64)
    pos[2], pos[5] = -1, 4096
    slots = torch.arange(12, device=DEV) + 4
    slots[7] = 64  # one past the pool
    kc = torch.full((4, 16, 2, 64), 7.0, dtype=q.dtype, device=DEV)
    vc = torch.full_like(kc, 9.0)
    q_out, k_out = torch.full((12, 8, 64), 5.0, dtype=q.dtype, device=DEV), \
        torch.full((12, 2, 64), 6.0, dtype=q.dtype, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.pa_rope_and_cache(q_out, q, k, v, kc, vc, slots, pos, cs, key_out=k_out, d_error=err)
    torch.cuda.synchronize()
    assert int(err) == pa.DEVERR_POSITION | pa.DEVERR_SLOT
    bad = torch.tensor([2, 5], device=DEV)
    assert bool((q_out[bad] == 5).all()) and bool((k_out[bad] == 6).all())
    good = [t for t in range(12) if t not in (2, 5)]
    want, size = formula(q, pos.clamp(0, 4095), cs, None, 0, False)
    check(q_out[good], want[good], size[good], q.dtype, "query_out")
    want, size = formula(k, pos.clamp(0, 4095), cs, None, 0, False)
    check(k_out[good], want[good], size[good], q.dtype, "key_out")
    written = [t for t in good if t != 7]
    flat = kc.view(-1, 2, 64)
    check(flat[slots[written]], want[written], size[written], q.dtype, "key_cache")
    left = torch.ones(64, dtype=torch.bool, device=DEV)
    left[slots[written]] = False
    assert bool((flat[left] == 7).all()) and bool((vc.view(-1, 2, 64)[left] == 9).all())


@gpu
def test_nan_and_infinity_stay_in_their_head_row():
    q, k, v, qw, kw, pos, _ = make(6, 8, 2, 128, torch.bfloat16, 7)
    cs = table(4096, 128)
    clean_q, clean_k = torch.empty(6, 8, 128, dtype=q.dtype, device=DEV), \
        torch.empty(6, 2, 128, dtype=q.dtype, device=DEV)
    pa.pa_qk_norm_rope(clean_q, clean_k, q, k, pos, cs, q_weight=qw, k_weight=kw)
    q[1, 3, 5], k[4, 1, 127] = float("nan"), float("inf")
    got_q, got_k = torch.empty_like(clean_q), torch.empty_like(clean_k)
    pa.pa_qk_norm_rope(got_q, got_k, q, k, pos, cs, q_weight=qw, k_weight=kw)
    torch.cuda.synchronize()
    assert bool(got_q[1, 3].isnan().all()) and bool(got_k[4, 1].isnan().any())
    clean_q[1, 3], clean_k[4, 1] = got_q[1, 3], got_k[4, 1]
    assert torch.equal(got_q.view(torch.int16), clean_q.view(torch.int16))
    assert torch.equal(got_k.view(torch.int16), clean_k.view(torch.int16))


@gpu
def test_on_another_stream_and_in_a_graph():
    run(9, 8, 2, 128, torch.float16, 128, False, "qk", 16, True, seed=8,
        stream=torch.cuda.Stream())
    q, k, v, qw, kw, pos, _ = make(9, 8, 2, 128, torch.float16, 9)
    cs = table(4096, 128)
    kc, vc = (torch.zeros(3, 16, 2, 128, dtype=q.dtype, device=DEV) for _ in range(2))
    slots = torch.arange(9, device=DEV)
    q_out = torch.empty(9, 8, 128, dtype=q.dtype, device=DEV)
    args = (q_out, q, k, v, kc, vc, slots, pos, cs)
    pa.pa_rope_and_cache(*args, q_weight=qw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_rope_and_cache(*args, q_weight=qw)
    q.copy_(torch.randn_like(q, dtype=torch.float32))
    pos.add_(1).clamp_(max=4095)
    graph.replay()
    torch.cuda.synchronize()
    want, size = formula(q, pos, cs, qw, 1e-6, False)
    check(q_out, want, size, q.dtype, "query_out")


@gpu
def test_rows_past_2_31_elements():
    # two tokens 2^31 elements apart, and a slot past 2^31 elements of the pool
    d, hkv, bs = 128, 8, 128
    stride = (1 << 31) + 8 * 128
    qkv = torch.zeros(stride + 12 * 128, dtype=torch.float16, device=DEV)
    rows = qkv.as_strided((2, 12, d), (stride, d, 1))
    rows.copy_(torch.randn(2, 12, d, device=DEV))
    nb = (1 << 31) // (bs * hkv * d) + 2
    kc = torch.zeros(nb, bs, hkv, d, dtype=torch.float16, device=DEV)
    vc = torch.zeros_like(kc)
    pos = torch.tensor([3, 4000], dtype=torch.int32, device=DEV)
    slots = torch.tensor([5, nb * bs - 1], device=DEV)
    cs = table(4096, d)
    key = qkv.as_strided((2, hkv, d), (stride, d, 1), 2 * d)
    q, q_out = rows[:, :2], torch.empty(2, 2, d, dtype=torch.float16, device=DEV)
    pa.pa_rope_and_cache(q_out, q, key, key, kc, vc, slots, pos, cs)
    torch.cuda.synchronize()
    want, size = formula(key, pos, cs, None, 0, False)
    check(kc.view(-1, hkv, d)[slots], want, size, torch.float16, "key_cache")
    assert torch.equal(vc.view(-1, hkv, d)[slots], key)
    want, size = formula(q, pos, cs, None, 0, False)
    check(q_out, want, size, torch.float16, "query_out")

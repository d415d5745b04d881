"""Cases for the operators between a projection and a paged KV cache, and for a
cache held in 4 bits.

  rope    pa_rope_and_cache / pa_qk_norm_rope: the norms of a step's query and
          key heads, the rotation by their positions, and the write of keys
          and values into the cache, in one pass;
  append  pa_reshape_and_cache_fp4, then pa_gather_cache_fp4: new rows quantised
          into a 4-bit cache, and the requests' rows read back in 16 bits (a
          chunk of a prompt over what a 4-bit cache holds already);
  decode  pa_decode_fp4: one query per request over a 4-bit cache.

A 4-bit cache is uint8 [num_blocks, num_kv_heads, block_size / 8, 4.5 D]: tiles of
eight tokens, first their 4-bit codes (E2M1, element 2i in the low half of byte
i), D / 2 bytes a token, then their scales (E4M3, one for 16 elements), D / 16
bytes a token.  A value is code * scale * (the head's fp32 scale).

``listed()`` and ``draw(rng)`` give cases, ``prepare`` their inputs, ``run``
one pass (the plain form, or with ``own`` the library's kernels), ``work`` the
bytes and operations a pass cannot do without, ``exact`` the outputs in 64
bits.  Lengths come from the case (``lens``), everything else from the seed.
"""
import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases --
def _rope(name, seqs, ctx, new, hq, hkv, d, bs, dtype, lens, rot, norm="", pairs=False, rows=False,
          cache=True, pad=0):
    return dict(name=name, op="rope", seqs=seqs, ctx_lo=ctx[0], ctx_hi=ctx[1], new_lo=new[0],
                new_hi=new[1], hq=hq, hkv=hkv, d=d, bs=bs, dtype=dtype, lens=lens, rot=rot,
                norm=norm, pairs=pairs, rows=rows, cache=cache, pad=pad)


def _append(name, seqs, ctx, new, hkv, d, bs, dtype, lens):
    return dict(name=name, op="append", seqs=seqs, ctx_lo=ctx[0], ctx_hi=ctx[1], new_lo=new[0],
                new_hi=new[1], hkv=hkv, d=d, bs=bs, dtype=dtype, lens=lens)


def _decode(name, seqs, ctx, hq, hkv, d, bs, dtype, lens, log=False, empty=0):
    return dict(name=name, op="decode", seqs=seqs, ctx_lo=ctx[0], ctx_hi=ctx[1], hq=hq, hkv=hkv,
                d=d, bs=bs, dtype=dtype, lens=lens, log=log, empty=empty)


def listed():
    return [
        # the smallest step: four requests, small heads; latency
        _rope("rope decode 4, 8/2 d 64", 4, (1, 127), (1, 1), 8, 2, 64, 16, "f16", 1, 64),
        # a decode step of eight requests, one KV head per query head
        _rope("rope decode 8, 32/32", 8, (512, 2047), (1, 1), 32, 32, 128, 16, "bf16", 2, 128),
        # a decode step ahead of a 4-bit cache's own write: norms and rotation alone
        _rope("norm rope decode 32, 32/8", 32, (50, 2000), (1, 1), 32, 8, 128, 32, "f16", 3, 128,
              norm="qk", cache=False),
        # decodes and prompt chunks side by side, padded to a fixed token count; neighbouring
        # elements rotated, half of the head, a group that is no power of two
        _rope("norm rope mixed 40/8", 48, (0, 8000), (1, 129), 40, 8, 128, 32, "f16", 4, 64,
              norm="k", pairs=True, pad=333),
        # a packed batch of prompts: rotated key rows for the attention, and the cache
        _rope("norm rope prompts 32/8", 16, (0, 0), (50, 2000), 32, 8, 128, 128, "bf16", 5, 128,
              norm="qk", rows=True),
        # a few requests append one token each and are read back
        _append("append 8 tokens", 8, (20, 200), (1, 1), 8, 128, 16, "bf16", 6),
        # chunks of prompts over what the cache holds
        _append("append chunks", 6, (1500, 8000), (65, 513), 8, 128, 32, "f16", 7),
        # a packed batch of whole prompts, one KV head per query head
        _append("append prompts", 16, (0, 0), (50, 2000), 32, 128, 128, "bf16", 8),
        # four requests, small heads: latency
        _decode("decode 4, 8/2 d 64", 4, (1, 128), 8, 2, 64, 16, "f16", 9),
        # eight requests, one KV head per query head
        _decode("decode 8, 32/32", 8, (512, 2048), 32, 32, 128, 16, "bf16", 10),
        # a continuous batch of mixed lengths, some of its rows empty
        _decode("decode 32, 32/8", 32, (50, 2000), 32, 8, 128, 32, "f16", 11, log=True, empty=3),
        # long documents, grouped heads
        _decode("decode long 4, 64/8", 4, (32768, 131072), 64, 8, 128, 128, "bf16", 12),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = [(8, 2), (32, 32), (32, 8), (64, 8), (40, 8), (16, 16), (12, 4), (32, 1), (128, 8)]


def draw(rng):
    op = rng.choice(["rope", "append", "decode", "decode"])
    lens, dtype, d = rng.randrange(1 << 30), rng.choice(["f16", "bf16"]), rng.choice([64, 128, 128])
    hq, hkv = rng.choice(HEADS)
    bs = rng.choice([8, 16, 32, 64, 128])
    if op == "rope":
        seqs, new, ctx = _log(rng, 1, 256), _log(rng, 1, 2000), _log(rng, 1, 100000)
        while seqs * new * (hq + 2 * hkv) * d > 8.0e7:
            new = new * 2 // 3
        new = max(1, new)
        c = _rope("", seqs, (rng.choice([0, ctx // 2]), ctx), (rng.choice([1, new]), new), hq, hkv,
                  d, bs, dtype, lens, rng.choice([d, d, d // 2, 16]),
                  norm=rng.choice(["", "qk", "qk", "q", "k"]), pairs=rng.random() < 0.4,
                  rows=rng.random() < 0.4, cache=rng.random() < 0.75,
                  pad=rng.choice([0, 0, rng.randrange(1, 300)]))
    elif op == "append":
        seqs, new, ctx = _log(rng, 1, 128), _log(rng, 1, 2000), _log(rng, 1, 16000)
        while seqs * (new + ctx) * hkv * d > 6.0e7:
            new, ctx = new * 2 // 3 + 1, ctx * 2 // 3
        c = _append("", seqs, (rng.choice([0, ctx // 2]), ctx), (rng.choice([1, new]), new), hkv,
                    d, bs, dtype, lens)
    else:
        seqs, hi = _log(rng, 1, 256), _log(rng, 16, 131072)
        while seqs * hi * hkv * d > 2.5e8 or seqs * hi * hq * d > 2.0e9:
            hi = hi * 2 // 3 + 1
        c = _decode("", seqs, (rng.choice([1, hi // 3 + 1, hi]), hi), hq, hkv, d, bs, dtype, lens,
                    log=rng.random() < 0.5, empty=rng.choice([0, 0, rng.randrange(1, 5)]))
    c.pop("name")
    return c


def _lens(c):
    """Each request's cached and new tokens (rope, append)."""
    r = random.Random(c["lens"])
    return ([r.randint(c["ctx_lo"], c["ctx_hi"]) for _ in range(c["seqs"])],
            [r.randint(c["new_lo"], c["new_hi"]) for _ in range(c["seqs"])])


def _contexts(c):
    """Each request's context (decode); the empty rows of the batch come last."""
    r = random.Random(c["lens"])
    lo, hi = c["ctx_lo"], c["ctx_hi"]
    n = [_log(r, lo, hi) if c["log"] else r.randint(lo, hi) for _ in range(c["seqs"])]
    return n + [0] * c["empty"]


# ----------------------------------------------------------------- inputs --
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _tables(g, lens, bs):
    """A block table over a shuffled pool: (table, number of blocks)."""
    count = [-(-n // bs) for n in lens]
    width, nb = max(1, max(count)), sum(count) + 4
    order = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    held = torch.arange(width, device="cuda")[None, :] < torch.tensor(count, device="cuda")[:, None]
    table[held] = order[:sum(count)]
    return table, nb


def _steps(ctx, new, table, bs):
    """Positions and slots of the new tokens, request by request."""
    n = torch.tensor(new, device="cuda")
    seq = torch.repeat_interleave(torch.arange(len(new), device="cuda"), n)
    first = torch.cumsum(n, 0) - n
    pos = torch.arange(seq.numel(), device="cuda") - first[seq] + torch.tensor(ctx, device="cuda")[seq]
    return pos.to(torch.int32), table[seq, pos // bs].long() * bs + pos % bs


def _angles(most, rot):
    """The cos and sin of every position: fp32 [most, rot]."""
    freq = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    a = torch.arange(most, device="cuda", dtype=torch.float64)[:, None] * freq[None, :]
    return torch.cat([a.cos(), a.sin()], 1).float()


def _encode(x, scale):
    """fp32 [..., Hkv, D] and per-head scales -> codes [..., D/2], scales [..., D/16] (bytes)."""
    x = x.unflatten(-1, (-1, 16))
    s = scale[:, None]
    c = (x.abs().amax(-1) / (6.0 * s)).clamp(max=448.0).to(torch.float8_e4m3fn)
    w = (c.float() * s)[..., None]
    q = torch.where(w > 0, x / w, 0.0)
    m = q.abs()
    # the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6: ties to the even code
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5)
            + (m >= 3.5) + (m > 5.0) + 8 * torch.signbit(q))
    code = code.to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), c.view(torch.uint8)


def _split(pool, d):
    """A pool's codes [NB, Hkv, bs/8, 8, D/2] and scales [NB, Hkv, bs/8, 8, D/16] (views)."""
    return (pool[..., :4 * d].unflatten(-1, (8, d // 2)),
            pool[..., 4 * d:].unflatten(-1, (8, d // 16)))


def _pool(g, nb, hkv, bs, d, dtype, scale):
    """A pool whose every row is a quantised row of 16-bit normal values."""
    pool = torch.empty((nb, hkv, bs // 8, 9 * d // 2), dtype=torch.uint8, device="cuda")
    codes, scales = _split(pool, d)
    step = max(1, (1 << 26) // (hkv * bs * d))
    for a in range(0, nb, step):
        n = min(step, nb - a)
        x = _normal(g, (n, bs // 8, 8, hkv, d), dtype).float()
        co, sc = _encode(x, scale)
        codes[a:a + n] = co.permute(0, 3, 1, 2, 4)
        scales[a:a + n] = sc.permute(0, 3, 1, 2, 4)
    return pool


def _head_scales(g, hkv):
    """Largest magnitudes of 4 to 6 standard deviations take the largest scale and code."""
    return (4.0 + 2.0 * torch.rand(hkv, generator=g, device="cuda")) / (6.0 * 448.0)


def prepare(case, seed):
    g = _gen(seed)
    dt, hkv, d, bs = DTYPES[case["dtype"]], case["hkv"], case["d"], case["bs"]
    if case["op"] == "decode":
        ctx = _contexts(case)
        table, nb = _tables(g, ctx, bs)
        ks, vs = _head_scales(g, hkv), _head_scales(g, hkv)
        q = _normal(g, (len(ctx), case["hq"], d), dt)
        return dict(op="decode", q=q, table=table, ctx=_i32(ctx), most=max(ctx), bs=bs, ks=ks,
                    vs=vs, kc=_pool(g, nb, hkv, bs, d, dt, ks), vc=_pool(g, nb, hkv, bs, d, dt, vs),
                    scale=1.0 / math.sqrt(d), out=torch.empty_like(q))
    ctx, new = _lens(case)
    total = [a + b for a, b in zip(ctx, new)]
    table, nb = _tables(g, total, bs)
    pos, slots = _steps(ctx, new, table, bs)
    t = slots.numel()
    if case["op"] == "append":
        ks, vs = _head_scales(g, hkv), _head_scales(g, hkv)
        kv = _normal(g, (t, 2, hkv, d), dt)  # views into one buffer of projections
        first = [sum(total[:b]) for b in range(len(total))]
        rows = torch.empty((2, sum(total), hkv, d), dtype=dt, device="cuda")
        return dict(op="append", k=kv[:, 0], v=kv[:, 1], slots=slots, table=table,
                    lens=_i32(total), first=_i32(first), most=max(total), bs=bs, ks=ks, vs=vs,
                    kc=_pool(g, nb, hkv, bs, d, dt, ks), vc=_pool(g, nb, hkv, bs, d, dt, vs),
                    k_rows=rows[0], v_rows=rows[1])
    hq = case["hq"]
    if case["pad"]:
        pos = torch.cat([pos, torch.zeros(case["pad"], dtype=torch.int32, device="cuda")])
        slots = torch.cat([slots, torch.full((case["pad"],), -1, device="cuda")])
        t += case["pad"]
    qkv = _normal(g, (t, hq + 2 * hkv, d), dt)
    weight = {n: (1.0 + 0.2 * _normal(g, (d,), torch.float32)).to(dt) if n in case["norm"] else None
              for n in "qk"}
    st = dict(op="rope", q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], pos=pos,
              cos_sin=_angles(max(total), case["rot"]), qw=weight["q"], kw=weight["k"], eps=1e-6,
              pairs=case["pairs"], bs=bs, slots=slots,
              q_out=torch.empty((t, hq, d), dtype=dt, device="cuda"))
    if case["rows"] or not case["cache"]:
        st["k_out"] = torch.empty((t, hkv, d), dtype=dt, device="cuda")
    if case["cache"]:
        st["kc"] = torch.zeros((nb, bs, hkv, d), dtype=dt, device="cuda")
        st["vc"] = torch.zeros((nb, bs, hkv, d), dtype=dt, device="cuda")
    return st


# ------------------------------------------------------------ plain forms --
def _turned(x, w, st):
    """Heads [T, H, D], normed and rotated, in fp32."""
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + st["eps"]) * w.float()
    at = st["cos_sin"][st["pos"].long()][:, None, :]
    half = at.shape[-1] // 2
    c, s = at[..., :half], at[..., half:]
    rest = y[..., 2 * half:]
    if st["pairs"]:
        a, b = y[..., 0:2 * half:2], y[..., 1:2 * half:2]
        r = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = y[..., :half], y[..., half:2 * half]
        r = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([r, rest], -1)


def _plain_rope(st):
    dt = st["q"].dtype
    k = _turned(st["k"], st["kw"], st).to(dt)
    r = dict(q_out=_turned(st["q"], st["qw"], st).to(dt))
    if "k_out" in st:
        r["k_out"] = k
    if "kc" in st:
        real = st["slots"] >= 0
        at = st["slots"][real]
        r["kc"], r["vc"] = st["kc"], st["vc"]
        r["kc"].flatten(0, 1)[at] = k[real]
        r["vc"].flatten(0, 1)[at] = st["v"][real]
    return r


def _values(codes, scales, scale):
    """fp32 values of code and scale bytes [..., D/2], [..., D/16] (scale: broadcast)."""
    e2m1 = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=codes.device)
    x = torch.stack([e2m1[(codes & 15).long()], e2m1[(codes >> 4).long()]], -1).flatten(-2)
    s = scales.view(torch.float8_e4m3fn).float()
    return (x.unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2) * scale


def _plain_append(st):
    d, bs, slots = st["k"].shape[2], st["bs"], st["slots"]
    lens, first = st["lens"].long(), st["first"].long()
    blk, tile, row = slots // bs, slots % bs // 8, slots % 8
    n = st["k_rows"].shape[0]
    seq = torch.repeat_interleave(torch.arange(lens.numel(), device=lens.device), lens,
                                  output_size=n)
    pos = torch.arange(n, device=lens.device) - first[seq]
    ids, at, of = st["table"][seq, pos // bs].long(), pos % bs // 8, pos % 8

    def one(x, pool, scale):
        codes, scales = _split(pool, d)
        co, sc = _encode(x.float(), scale)
        codes[blk, :, tile, row] = co
        scales[blk, :, tile, row] = sc
        return _values(codes[ids, :, at, of], scales[ids, :, at, of], scale[:, None]).to(x.dtype)

    return dict(k_rows=one(st["k"], st["kc"], st["ks"]), v_rows=one(st["v"], st["vc"], st["vs"]))


def _plain_decode(st):
    s, hq, d = st["q"].shape
    hkv = st["kc"].shape[1]
    ids = st["table"].long().clamp(min=0)
    hidden = torch.arange(ids.shape[1] * st["bs"], device=ids.device) >= st["ctx"][:, None]

    def rows(pool, scale):  # [S, Hkv, tokens, D], every request padded to the longest
        codes, scales = _split(pool[ids].transpose(1, 2), d)
        x = _values(codes, scales, scale[:, None, None, None, None])
        return x.reshape(s, hkv, -1, d)

    q = st["q"].float().view(s, hkv, hq // hkv, d)
    a = torch.matmul(q, rows(st["kc"], st["ks"]).transpose(2, 3)) * st["scale"]
    a = a.masked_fill_(hidden[:, None, None, :], float("-inf"))
    p = torch.exp(a - a.amax(-1, keepdim=True).clamp(min=-3.0e38))
    p = p / p.sum(-1, keepdim=True).clamp(min=1.0e-30)
    return torch.matmul(p, rows(st["vc"], st["vs"])).view(s, hq, d).to(st["q"].dtype)


# ---------------------------------------------------------------- one pass --
def _own_rope(st):
    import paged_kv_cache_34_gb300 as pa
    more = dict(interleaved=st["pairs"], q_weight=st["qw"], k_weight=st["kw"], eps=st["eps"])
    if "kc" not in st:
        pa.pa_qk_norm_rope(st["q_out"], st["k_out"], st["q"], st["k"], st["pos"], st["cos_sin"],
                           **more)
    else:
        pa.pa_rope_and_cache(st["q_out"], st["q"], st["k"], st["v"], st["kc"], st["vc"],
                             st["slots"], st["pos"], st["cos_sin"], key_out=st.get("k_out"), **more)
    return {n: st[n] for n in ("q_out", "k_out", "kc", "vc") if n in st}


def _own_append(st):
    import paged_kv_cache_34_gb300 as pa
    pa.pa_reshape_and_cache_fp4(st["k"], st["v"], st["kc"], st["vc"], st["slots"], st["ks"],
                                st["vs"])
    pa.pa_gather_cache_fp4(st["k_rows"], st["v_rows"], st["kc"], st["vc"], st["table"], st["lens"],
                           st["first"], st["ks"], st["vs"], max_context_len=st["most"])
    return dict(k_rows=st["k_rows"], v_rows=st["v_rows"])


def _own_decode(st):
    import paged_kv_cache_34_gb300 as pa
    if "workspace" not in st:  # kept from step to step
        s, hq, d = st["q"].shape
        need = pa.pa_decode_fp4_plan(s, hq, st["kc"].shape[1], d, st["most"])
        st["workspace"] = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    return pa.pa_decode_fp4(st["out"], st["q"], st["kc"], st["vc"], st["table"], st["ctx"],
                            st["ks"], st["vs"], scale=st["scale"], max_context_len=st["most"],
                            workspace=st["workspace"])


def run(st):
    if own:
        return {"rope": _own_rope, "append": _own_append, "decode": _own_decode}[st["op"]](st)
    return {"rope": _plain_rope, "append": _plain_append, "decode": _plain_decode}[st["op"]](st)


# --------------------------------------------------------- floor and truth --
def work(case):
    hkv, d, bs = case["hkv"], case["d"], case["bs"]
    row4 = 2 * hkv * 9 * d // 16  # a token's K and V in 4 bits
    if case["op"] == "decode":
        n = sum(_contexts(case))
        return {"bytes": n * row4 + 4 * d * case["hq"] * case["seqs"] + 4 * -(-n // bs),
                "flops": 4 * case["hq"] * d * n}
    ctx, new = _lens(case)
    if case["op"] == "append":
        # new rows in and their codes out; the cached codes in, every row out
        return {"bytes": sum(new) * (4 * hkv * d + row4 + 8) + sum(ctx) * row4
                + (sum(ctx) + sum(new)) * 4 * hkv * d, "flops": 0}
    t, hq = sum(new) + case["pad"], case["hq"]
    heads = 2 * (hq + hkv) + (2 * hkv if case["cache"] else 0)
    if case["cache"] and case["rows"]:
        heads += hkv
    return {"bytes": t * (2 * d * heads + 4) + sum(new) * (8 if case["cache"] else 0)
            + 4 * case["rot"] * len({p for a, b in zip(ctx, new) for p in range(a, a + b)}),
            "flops": t * (hq + hkv) * (3 * case["rot"] + 4 * d * bool(case["norm"]))}


def _e2m1(b):
    """The value of a 4-bit code in 64 bits: sign, two exponent bits of bias 1, one fraction bit."""
    e, m = (b >> 1 & 3).double(), (b & 1).double()
    v = torch.where(e > 0, (1 + m / 2) * torch.exp2(e - 1), m / 2)
    return torch.where(b >= 8, -v, v)


def _e4m3(b):
    """The value of an 8-bit scale in 64 bits: four exponent bits of bias 7, three fraction bits."""
    e, m = (b >> 3 & 15).double(), (b & 7).double()
    return torch.where(e > 0, (1 + m / 8) * torch.exp2(e - 7), m / 512)


def _cached(pool, head, row, scale):
    """Rows of one head from a pool's bytes, in 64 bits: row = block * bs + offset."""
    d, tiles = pool.shape[3] * 2 // 9, pool.shape[2]
    flat = pool[:, head].reshape(-1, pool.shape[3])
    t, r = torch.div(row, 8, rounding_mode="floor"), (row % 8)[:, None]
    assert flat.shape[0] % tiles == 0
    i = torch.arange(d, device=pool.device)
    code = (flat[t[:, None], r * (d // 2) + i // 2].int() >> (4 * (i % 2))) & 15
    sc = flat[t[:, None], 4 * d + r * (d // 16) + i // 16].int()
    return _e2m1(code) * _e4m3(sc) * float(scale)


def _exact_rope(st, case):
    p = st["pos"].long()
    half = case["rot"] // 2
    c, s = (x.double()[:, None, :] for x in (st["cos_sin"][p, :half], st["cos_sin"][p, half:]))
    first = torch.arange(half, device=p.device) * (2 if case["pairs"] else 1)
    second = first + (1 if case["pairs"] else half)

    def heads(x, w):
        y = x.double()
        if w is not None:
            y = y / (y.pow(2).sum(-1, keepdim=True) / y.shape[-1] + st["eps"]).sqrt() * w.double()
        z = y.clone()
        z[..., first] = y[..., first] * c - y[..., second] * s
        z[..., second] = y[..., first] * s + y[..., second] * c
        return z

    k = heads(st["k"], st["kw"])
    r = dict(q_out=heads(st["q"], st["qw"]))
    if "k_out" in st:
        r["k_out"] = k
    if "kc" in st:
        rows = torch.nonzero(st["slots"] >= 0)[:, 0]
        for n, x in (("kc", k), ("vc", st["v"].double())):
            full = torch.zeros(st[n].shape, dtype=torch.float64, device=p.device)
            full.view(-1, *full.shape[2:]).index_copy_(0, st["slots"][rows], x[rows])
            r[n] = full
    return r


def _exact_append(st, case):
    """The nearest representable values by search: quotients as the definition rounds them, to
    fp32, from 64 bits."""
    grid = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    bytes8 = torch.arange(127, device="cuda")
    scales8 = _e4m3(bytes8)
    pos = [(b, j) for b, n in enumerate(st["lens"].tolist()) for j in range(0, n, st["bs"])]
    ids = st["table"].tolist()
    rows = torch.cat([torch.arange(min(st["bs"], int(st["lens"][b]) - j), device="cuda")
                      + ids[b][j // st["bs"]] * st["bs"] for b, j in pos])

    def nearest(q, table):  # ties to the even place
        hi = torch.searchsorted(table, q.clamp(max=float(table[-1])).contiguous())
        hi = hi.clamp(1, table.numel() - 1)
        lo = hi - 1
        a, b = q - table[lo], table[hi] - q
        return torch.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)

    out = {}
    for n, x, pool, scale in (("k_rows", st["k"], st["kc"], st["ks"]),
                              ("v_rows", st["v"], st["vc"], st["vs"])):
        got = torch.empty(st[n].shape, dtype=torch.float64, device="cuda")
        for h in range(case["hkv"]):
            s = scale[h]
            every = torch.empty((pool.shape[0] * st["bs"], case["d"]), dtype=torch.float64,
                                device="cuda")
            every[rows] = _cached(pool, h, rows, s)
            y = x[:, h].double().unflatten(-1, (-1, 16))
            six = (6.0 * s.double()).float().double()
            c = scales8[nearest((y.abs().amax(-1) / six).float().double(), scales8)]
            w = (c * s.double()).float().double()[..., None]
            q = torch.where(w > 0, y / w, 0.0).float().double()
            v = grid[nearest(q.abs(), grid)] * torch.sign(q) * c[..., None] * s.double()
            every[st["slots"]] = v.flatten(-2)
            got[:, h] = every[rows]
        out[n] = got
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(st, case)
    if case["op"] == "append":
        return _exact_append(st, case)
    q = st["q"].double()
    out = torch.zeros_like(q)
    g = case["hq"] // case["hkv"]
    for b, n in enumerate(_contexts(case)):
        if n == 0:
            continue
        j = torch.arange(n, device="cuda")
        row = st["table"][b].long()[j // case["bs"]] * case["bs"] + j % case["bs"]
        for h in range(case["hkv"]):
            k = _cached(st["kc"], h, row, st["ks"][h])
            z = q[b, h * g:(h + 1) * g] @ k.T * st["scale"]
            e = torch.exp(z - z.max(dim=1, keepdim=True).values)
            v = _cached(st["vc"], h, row, st["vs"][h])
            out[b, h * g:(h + 1) * g] = e @ v / e.sum(dim=1, keepdim=True)
    return out

"""Cases for three operators of a serving step over a paged KV cache.

  tables   pa_build_tables: from each request's cached and new token counts,
           the step's cumulative query lengths, token positions, cache slots
           and the block-table entries of newly taken blocks;
  prompt   pa_attention_varlen: causal attention of whole prompts packed one
           behind the other, straight from their K and V rows;
  shared   pa_decode_shared: one query per request over the paged cache, for
           groups of requests that share a prefix, the prefix read once for
           its whole group.

``listed()`` and ``draw(rng)`` give cases, ``prepare`` their inputs, ``run``
one pass (the plain form, or with ``own`` the library's kernels), ``work`` the
bytes and operations a pass cannot do without, ``exact`` the outputs in 64
bits.  Lengths come from the case (``lens``), everything else from the seed.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases --
def _tables(name, seqs, ctx, new, bs, lens, short=False, pad=0):
    return dict(name=name, op="tables", seqs=seqs, ctx_lo=ctx[0], ctx_hi=ctx[1], new_lo=new[0],
                new_hi=new[1], bs=bs, lens=lens, short=short, pad=pad)


def _prompt(name, seqs, length, hq, hkv, d, dtype, lens):
    return dict(name=name, op="prompt", seqs=seqs, lo=length[0], hi=length[1], hq=hq, hkv=hkv,
                d=d, dtype=dtype, lens=lens)


def _shared(name, seqs, groups, prefix, suffix, hq, hkv, d, bs, dtype, lens, pad=0):
    return dict(name=name, op="shared", seqs=seqs, groups=groups, prefix_lo=prefix[0],
                prefix_hi=prefix[1], suffix_lo=suffix[0], suffix_hi=suffix[1], hq=hq, hkv=hkv,
                d=d, bs=bs, dtype=dtype, lens=lens, pad=pad)


def listed():
    return [
        # a decode step of a small batch: every request gets one token
        _tables("tables decode 8", 8, (512, 2048), (1, 1), 16, 1),
        # a continuous-batching step: decodes and prompt chunks side by side,
        # the slot array padded to the step's token budget
        _tables("tables mixed 256", 256, (0, 2000), (1, 64), 32, 2, pad=777),
        # a large admission: a thousand prompts of a long-document workload
        _tables("tables prompts 1024", 1024, (0, 500), (50, 2000), 16, 3),
        # one short prompt, small heads: latency
        _prompt("prompt one short", 1, (37, 37), 8, 2, 64, "f16", 4),
        # the packed-prefill batch: 16 prompts of mixed lengths, one KV head per query head
        _prompt("prompt packed 32/32", 16, (50, 2000), 32, 32, 128, "bf16", 5),
        # grouped heads, a group that is no power of two, odd lengths
        _prompt("prompt packed 40/8", 24, (33, 3001), 40, 8, 128, "f16", 6),
        # long documents, grouped heads
        _prompt("prompt long 32/8", 2, (16001, 16384), 32, 8, 128, "bf16", 7),
        # a few requests behind one short system prompt, small heads
        _shared("shared 4 x 500", 4, 1, (500, 500), (1, 128), 8, 2, 64, 16, "f16", 8),
        # a chat batch behind one system prompt, some rows of the batch empty
        _shared("shared 32 x 4000", 32, 1, (4000, 4000), (1, 1000), 32, 8, 128, 16, "bf16", 9,
                pad=4),
        # several prompts in use at once, each by part of the batch
        _shared("shared 64 in 6 groups", 64, 6, (300, 9000), (1, 600), 64, 8, 128, 32, "f16", 10),
        # samples of one long document, one KV head per query head
        _shared("shared 8 x 16384 32/32", 8, 1, (16384, 16384), (20, 200), 32, 32, 128, 128,
                "bf16", 11),
        # a large batch over one long document
        _shared("shared 256 x 32768", 256, 1, (32768, 32768), (50, 2000), 64, 8, 128, 128,
                "bf16", 12),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _drawn(case):
    case.pop("name")
    return case


def draw(rng):
    op = rng.choice(["tables", "prompt", "shared"])
    lens = rng.randrange(1 << 30)
    if op == "tables":
        seqs, new_hi = _log(rng, 1, 2048), _log(rng, 1, 2000)
        while seqs * new_hi > 1000000:
            new_hi = max(1, new_hi // 2)
        return _drawn(_tables("", seqs, (0, _log(rng, 1, 8000)), (rng.choice([0, 1]), new_hi),
                              rng.choice([8, 16, 32, 64, 128]), lens,
                              short=rng.random() < 0.25,
                              pad=rng.choice([0, 0, _log(rng, 1, 3000)])))
    hq, hkv = rng.choice([(8, 2), (32, 32), (32, 8), (64, 8), (40, 8), (16, 16), (12, 4), (32, 1)])
    d, dtype = rng.choice([64, 128, 128]), rng.choice(["f16", "bf16"])
    if op == "prompt":
        seqs, hi = _log(rng, 1, 64), _log(rng, 1, 16000)
        while seqs * hi * hi * hq * d > 1.5e12 or seqs * hi * (hq + hkv) * d > 2.0e8:
            hi = hi * 2 // 3 + 1
        return _drawn(_prompt("", seqs, (rng.choice([1, hi // 3 + 1, hi]), hi), hq, hkv, d, dtype,
                              lens))
    seqs = _log(rng, 1, 256)
    groups = min(seqs, rng.choice([1, 1, 2, _log(rng, 1, 16)]))
    plo, phi = sorted((_log(rng, 1, 30000), _log(rng, 16, 30000)))
    slo, shi = rng.choice([0, 1]), _log(rng, 1, 2000)
    while ((groups * phi + seqs * shi) * hkv * d > 1.5e8
           or seqs * (phi + shi) * hq * d > 6.0e10):
        phi, shi = phi * 2 // 3 + 1, shi * 2 // 3 + 1
    return _drawn(_shared("", seqs, groups, (min(plo, phi), phi), (slo, shi), hq, hkv, d,
                          rng.choice([8, 16, 32, 64, 128]), dtype, lens,
                          pad=rng.choice([0, 0, rng.randrange(1, 9)])))


def _uniform(rng, lo, hi):
    return rng.randint(lo, hi)


def _tables_lens(c):
    r = random.Random(c["lens"])
    ctx = [_uniform(r, c["ctx_lo"], c["ctx_hi"]) for _ in range(c["seqs"])]
    new = [_uniform(r, c["new_lo"], c["new_hi"]) for _ in range(c["seqs"])]
    if sum(new) == 0:
        new[-1] = 1
    return ctx, new


def _tables_free(c, ctx, new):
    """Blocks the step takes, and how many the free list holds."""
    bs = c["bs"]
    need = sum(-(-(a + n) // bs) - -(-a // bs) for a, n in zip(ctx, new))
    return need, max(0, need // 2) if c["short"] else need + 64


def _prompt_lens(c):
    r = random.Random(c["lens"])
    return [_uniform(r, c["lo"], c["hi"]) for _ in range(c["seqs"])]


def _shared_lens(c):
    """(group starts, prefix lengths, context lengths); the padded rows of the
    batch are a last group of empty sequences with no prefix."""
    r = random.Random(c["lens"])
    s, g = c["seqs"], c["groups"]
    cuts = sorted(r.sample(range(1, s), g - 1)) if g > 1 else []
    starts = [0] + cuts + [s]
    prefix = [_uniform(r, c["prefix_lo"], c["prefix_hi"]) for _ in range(g)]
    ctx = []
    for k in range(g):
        for _ in range(starts[k], starts[k + 1]):
            lo, hi = c["suffix_lo"], c["suffix_hi"]
            own_part = lo if hi <= lo else min(hi, max(lo, int(math.exp(
                r.uniform(math.log(max(lo, 1)), math.log(hi + 1)))) - (lo == 0)))
            ctx.append(prefix[k] + own_part)
    if c["pad"]:
        starts.append(s + c["pad"])
        prefix.append(0)
        ctx += [0] * c["pad"]
    return starts, prefix, ctx


# ----------------------------------------------------------------- inputs --
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "tables":
        ctx, new = _tables_lens(case)
        bs, s = case["bs"], len(ctx)
        _, nfree = _tables_free(case, ctx, new)
        have = [-(-a // bs) for a in ctx]
        width = max(1, max(-(-(a + n) // bs) for a, n in zip(ctx, new)))
        nb = sum(have) + nfree + 16
        order = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
        table = torch.full((s, width), -1, dtype=torch.int32, device="cuda")
        col = torch.arange(width, device="cuda")
        h = torch.tensor(have, device="cuda")
        table[col[None, :] < h[:, None]] = order[:sum(have)]
        free = order[sum(have):].clone()  # the list's first nfree entries are free
        tokens = sum(new) + case["pad"]
        return dict(op="tables", bs=bs, num_blocks=nb, block_table=table, context_lens=_i32(ctx),
                    query_lens=_i32(new), free_blocks=free, num_free=_i32([nfree]),
                    context_lens_out=torch.empty(s, dtype=torch.int32, device="cuda"),
                    cu_seqlens_q=torch.empty(s + 1, dtype=torch.int32, device="cuda"),
                    slot_mapping=torch.empty(tokens, dtype=torch.int64, device="cuda"),
                    positions=torch.empty(tokens, dtype=torch.int32, device="cuda"),
                    num_free_out=torch.empty(1, dtype=torch.int32, device="cuda"))
    dt, hq, hkv, d = DTYPES[case["dtype"]], case["hq"], case["hkv"], case["d"]
    if case["op"] == "prompt":
        lens = _prompt_lens(case)
        t = sum(lens)
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        # K and V are views into one buffer of interleaved projections
        kv = _normal(g, (t, 2, hkv, d), dt)
        return dict(op="prompt", lens=lens, q=_normal(g, (t, hq, d), dt), k=kv[:, 0], v=kv[:, 1],
                    cu=_i32(cu), scale=1.0 / math.sqrt(d), max_seqlen=max(lens),
                    out=torch.empty((t, hq, d), dtype=dt, device="cuda"))
    starts, prefix, ctx = _shared_lens(case)
    bs, s = case["bs"], len(ctx)
    # block tables: a group's first ceil(prefix / bs) entries name the same
    # blocks; a request's own tokens follow in blocks of its own, so a prefix
    # that ends inside a block has that block's leading part in both
    width = max(1, -(-max(ctx) // bs))
    rows = []
    used = 0
    for k in range(len(prefix)):
        whole = prefix[k] // bs
        shared_ids = list(range(used, used + -(-prefix[k] // bs)))
        used += len(shared_ids)
        for m, b in enumerate(range(starts[k], starts[k + 1])):
            n = -(-ctx[b] // bs)
            keep = len(shared_ids) if m == 0 else min(whole, n)
            row = shared_ids[:keep]
            row = row + list(range(used, used + n - len(row)))
            used += n - min(keep, n)
            rows.append(row + [-1] * (width - len(row)))
    nb = used + 8
    order = torch.cat([torch.randperm(nb, generator=g, device="cuda"),
                       torch.full((1,), -1, device="cuda")])
    table = order[torch.tensor(rows, device="cuda")].to(torch.int32)  # entry -1 stays -1
    k_pool = _normal(g, (nb, bs, hkv, d), dt)
    v_pool = _normal(g, (nb, bs, hkv, d), dt)
    # a prefix that ends inside a block: every member's copy of it is the same
    flat_k, flat_v = k_pool.view(nb * bs, hkv, d), v_pool.view(nb * bs, hkv, d)
    for k in range(len(prefix)):
        tail = prefix[k] % bs
        if tail:
            at = table[starts[k]:starts[k + 1], prefix[k] // bs].long()
            src = torch.arange(tail, device="cuda") + at[0] * bs
            dst = (torch.arange(tail, device="cuda")[None, :] + at[:, None] * bs).reshape(-1)
            flat_k[dst] = flat_k[src].repeat(at.numel(), 1, 1)
            flat_v[dst] = flat_v[src].repeat(at.numel(), 1, 1)
    return dict(op="shared", bs=bs, starts=starts, prefix=prefix, ctx=ctx,
                q=_normal(g, (s, hq, d), dt), k_pool=k_pool, v_pool=v_pool, block_table=table,
                context_lens=_i32(ctx), group_starts=_i32(starts), prefix_lens=_i32(prefix),
                scale=1.0 / math.sqrt(d), max_context_len=max(ctx), max_prefix_len=max(prefix),
                out=torch.empty((s, hq, d), dtype=dt, device="cuda"))


# ------------------------------------------------------------ plain forms --
def _plain_tables(st):
    bs = st["bs"]
    ctx, new = st["context_lens"].long(), st["query_lens"].long()
    table, free, nfree = st["block_table"], st["free_blocks"].long(), st["num_free"].long()
    have, need = (ctx + bs - 1) // bs, (ctx + new + bs - 1) // bs
    take = need - have
    upto = torch.cumsum(take, 0)
    first = upto - take
    ok = (take == 0) | (upto <= nfree)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device=ctx.device), torch.cumsum(new, 0)])
    # block table: request b's blocks have .. need - 1 come off the end of the list
    col = torch.arange(table.shape[1], device=ctx.device)[None, :]
    fresh = (col >= have[:, None]) & (col < need[:, None]) & ok[:, None]
    at = (nfree - 1 - (first[:, None] + col - have[:, None])).clamp(0, free.numel() - 1)
    table = torch.where(fresh, free[at].to(torch.int32), table)
    # tokens
    t = torch.arange(st["slot_mapping"].numel(), device=ctx.device)
    real = t < cu[-1]
    seq = torch.searchsorted(cu[1:], t, right=True).clamp(max=ctx.numel() - 1)
    pos = torch.where(real, ctx[seq] + t - cu[seq], 0)
    ids = table[seq, pos // bs].long()
    slot = torch.where(real & ok[seq], ids * bs + pos % bs, -1)
    left = nfree - torch.where(upto <= nfree, upto, 0).amax()
    return dict(block_table=table, context_lens_out=torch.where(ok, ctx + new, 0).to(torch.int32),
                cu_seqlens_q=cu.to(torch.int32), slot_mapping=slot,
                positions=pos.to(torch.int32), num_free_out=left.to(torch.int32))


def _softmax(s):
    s = torch.exp(s - s.amax(-1, keepdim=True))
    return s / s.sum(-1, keepdim=True)


def _prompt_attention(st, dtype):
    q, k, v = st["q"], st["k"], st["v"]
    hq, hkv, g = q.shape[1], k.shape[1], q.shape[1] // k.shape[1]
    out = torch.empty_like(q, dtype=dtype)
    row = 0
    for n in st["lens"]:
        own_q = q[row:row + n].to(dtype).view(n, hkv, g, -1).permute(1, 2, 0, 3)
        own_k = k[row:row + n].to(dtype).permute(1, 2, 0)[:, None]
        own_v = v[row:row + n].to(dtype).permute(1, 0, 2)[:, None]
        hidden = torch.ones((n, n), dtype=torch.bool, device=q.device).triu_(1)
        step = max(1, (1 << 30) // (g * n * n))  # KV heads at a time
        for h in range(0, hkv, step):
            s = torch.matmul(own_q[h:h + step], own_k[h:h + step]) * st["scale"]
            p = _softmax(s.masked_fill_(hidden, float("-inf")))
            o = torch.matmul(p, own_v[h:h + step])  # [heads, g, n, d]
            out[row:row + n, h * g:(h + step) * g] = o.permute(2, 0, 1, 3).reshape(n, -1, q.shape[2])
        row += n
    return out


def _shared_attention(st, dtype):
    q, bs = st["q"], st["bs"]
    nb, _, hkv, d = st["k_pool"].shape
    hq = q.shape[1]
    g = hq // hkv
    k_rows, v_rows = st["k_pool"].view(nb * bs, hkv, d), st["v_pool"].view(nb * bs, hkv, d)
    out = torch.zeros_like(q, dtype=dtype)
    for j, n_pre in enumerate(st["prefix"]):
        a, b = st["starts"][j], st["starts"][j + 1]
        lens = st["ctx"][a:b]
        if max(lens) == 0:
            continue
        pos = torch.arange(n_pre, device=q.device)
        pre = st["block_table"][a, pos // bs].long() * bs + pos % bs
        pos = torch.arange(n_pre, max(max(lens), n_pre + 1), device=q.device)
        ids = st["block_table"][a:b, (pos // bs).clamp(max=st["block_table"].shape[1] - 1)].long()
        hidden = pos[None, :] >= st["context_lens"][a:b, None]  # [m, own]
        rest = torch.where(hidden, 0, ids * bs + (pos % bs)[None, :])
        hidden = hidden[:, None, :]
        for h in range(hkv):
            qh = q[a:b, h * g:(h + 1) * g].to(dtype)
            s0 = torch.matmul(qh, k_rows[pre, h].to(dtype).t())
            s1 = torch.matmul(qh, k_rows[rest, h].to(dtype).transpose(1, 2))
            s = torch.cat([s0, s1.masked_fill_(hidden, float("-inf"))], -1) * st["scale"]
            p = _softmax(s)
            out[a:b, h * g:(h + 1) * g] = (
                torch.matmul(p[..., :n_pre], v_rows[pre, h].to(dtype))
                + torch.matmul(p[..., n_pre:], v_rows[rest, h].to(dtype)))
    return out


# ---------------------------------------------------------------- one pass --
def _own_tables(st):
    import paged_kv_cache_34_gb300 as pa
    pa.pa_build_tables(st["block_table"], st["context_lens"], st["query_lens"], st["free_blocks"],
                       st["num_free"], st["context_lens_out"], st["cu_seqlens_q"],
                       st["slot_mapping"], st["num_free_out"], positions=st["positions"],
                       block_size=st["bs"], num_blocks=st["num_blocks"])
    return {n: st[n] for n in ("block_table", "context_lens_out", "cu_seqlens_q", "slot_mapping",
                               "positions")} | {"num_free_out": st["num_free_out"]}


def _own_prompt(st):
    import paged_kv_cache_34_gb300 as pa
    return pa.pa_attention_varlen(st["out"], st["q"], st["k"], st["v"], st["cu"],
                                  scale=st["scale"], max_seqlen=st["max_seqlen"])


def _own_shared(st):
    import paged_kv_cache_34_gb300 as pa
    if "workspace" not in st:  # kept from step to step
        s, hq, d = st["q"].shape
        need = pa.pa_decode_shared_plan(s, len(st["prefix"]), hq, st["k_pool"].shape[2], d,
                                        st["max_context_len"], st["max_prefix_len"])
        st["workspace"] = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    return pa.pa_decode_shared(st["out"], st["q"], st["k_pool"], st["v_pool"], st["block_table"],
                               st["context_lens"], st["group_starts"], st["prefix_lens"],
                               scale=st["scale"], max_context_len=st["max_context_len"],
                               max_prefix_len=st["max_prefix_len"], workspace=st["workspace"])


def run(st):
    op = st["op"]
    if own:
        return {"tables": _own_tables, "prompt": _own_prompt, "shared": _own_shared}[op](st)
    if op == "tables":
        r = _plain_tables(st)
        r["num_free_out"] = r["num_free_out"].reshape(1)
        return r
    f = _prompt_attention if op == "prompt" else _shared_attention
    return f(st, torch.float32).to(st["q"].dtype)


# --------------------------------------------------------- floor and truth --
def work(case):
    if case["op"] == "tables":
        ctx, new = _tables_lens(case)
        need, nfree = _tables_free(case, ctx, new)
        s, t = len(ctx), sum(new) + case["pad"]
        # two counts in and two out per request, the taken blocks' ids in and
        # out, the block in use, slot and position of every token
        return {"bytes": 16 * s + 8 * min(need, nfree) + 4 * s + 12 * t, "flops": 0}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "prompt":
        lens = _prompt_lens(case)
        return {"bytes": 2 * d * (2 * hq + 2 * hkv) * sum(lens),
                "flops": 4 * hq * d * sum(n * (n + 1) // 2 for n in lens)}
    starts, prefix, ctx = _shared_lens(case)
    tokens = sum(prefix) + sum(ctx[b] - prefix[k] for k in range(len(prefix))
                               for b in range(starts[k], starts[k + 1]))
    return {"bytes": 4 * d * hkv * tokens + 4 * d * hq * len(ctx) + 4 * -(-tokens // case["bs"]),
            "flops": 4 * hq * d * sum(ctx)}


def _exact_tables(st):
    bs = st["bs"]
    ctx, new = st["context_lens"].tolist(), st["query_lens"].tolist()
    free, left = st["free_blocks"].tolist(), int(st["num_free"])
    table = st["block_table"].cpu().numpy().copy()
    slots = np.full(st["slot_mapping"].numel(), -1, np.int64)
    places = np.zeros(slots.size, np.int32)
    lens_out, cu, closed = [], [0], False
    for b, (c, n) in enumerate(zip(ctx, new)):
        have, need = (c + bs - 1) // bs, (c + n + bs - 1) // bs
        pos = np.arange(c, c + n)
        places[cu[-1]:cu[-1] + n] = pos
        if need > have and (closed or need - have > left):
            closed = True  # nobody behind it takes blocks either
            lens_out.append(0)
        else:
            for j in range(have, need):
                left -= 1
                table[b, j] = free[left]
            slots[cu[-1]:cu[-1] + n] = table[b, pos // bs].astype(np.int64) * bs + pos % bs
            lens_out.append(c + n)
        cu.append(cu[-1] + n)
    return dict(block_table=table, context_lens_out=np.array(lens_out, np.int32),
                cu_seqlens_q=np.array(cu, np.int32), slot_mapping=slots, positions=places,
                num_free_out=np.array([left], np.int32))


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "tables":
        return _exact_tables(st)
    q = st["q"].double()
    out = torch.zeros_like(q)
    hq, hkv = case["hq"], case["hkv"]
    g = hq // hkv

    def weights(s):  # natural exponentials of the scores, normalised, in 64 bits
        e = torch.exp(s - s.max(dim=-1, keepdim=True).values)
        return e / e.sum(dim=-1, keepdim=True)

    if case["op"] == "prompt":
        k, v = st["k"].double(), st["v"].double()
        a = 0
        for n in st["lens"]:
            for h in range(hq):
                for i in range(0, n, 4096):  # query rows i .. e - 1 see keys 0 .. e - 1
                    e = min(n, i + 4096)
                    s = q[a + i:a + e, h] @ k[a:a + e, h // g].T * st["scale"]
                    rows = torch.arange(i, e, device=q.device)[:, None]
                    s[torch.arange(e, device=q.device)[None, :] > rows] = float("-inf")
                    out[a + i:a + e, h] = weights(s) @ v[a:a + e, h // g]
            a += n
        return out
    bs = st["bs"]
    for b, n in enumerate(st["ctx"]):
        if n == 0:
            continue
        j = torch.arange(n, device=q.device)
        blk = st["block_table"][b].long()[j // bs]
        # the definition: the request's own row of the table, prefix and all,
        # but for the group's first row where the prefix ends inside a block
        k, v = st["k_pool"][blk, j % bs].double(), st["v_pool"][blk, j % bs].double()
        s = torch.einsum("hgd,nhd->hgn", q[b].view(hkv, g, -1), k) * st["scale"]
        out[b] = torch.einsum("hgn,nhd->hgd", weights(s), v).reshape(hq, -1)
    return out

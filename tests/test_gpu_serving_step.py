"""The step operators together, as a serving loop uses them: tables from
lengths, a prompt's attention from its own rows, the cache write, and decode
steps of requests admitted behind that prompt; every attention output against
64 bits over the tokens fed so far."""
import pytest
import torch

from attn_util import attend, check
from gpu_util import gpu, new_err, pa, require_gpu

pytestmark = gpu


@pytest.mark.parametrize("n_prompt,bs", [(333, 16), (256, 32)])
def test_prompt_then_shared_decode_steps(n_prompt, bs):
    require_gpu()
    hq, hkv, d, s, nb, width = 8, 2, 128, 6, 96, 40
    dt = torch.bfloat16
    g = torch.Generator(device="cuda")
    g.manual_seed(n_prompt)
    rand = lambda *sh: torch.randn(sh, generator=g, device="cuda").to(dt)  # noqa: E731
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    k_pool = torch.full((nb, bs, hkv, d), float("nan"), dtype=dt, device="cuda")
    v_pool = k_pool.clone()
    free, nfree, err = torch.randperm(nb, dtype=torch.int32, device="cuda"), i32([nb]), new_err()
    scale = d ** -0.5

    def tables(table, lens, new, tokens):
        out, cu = torch.empty_like(lens), torch.empty(len(new) + 1, dtype=torch.int32,
                                                      device="cuda")
        slots = torch.empty(tokens, dtype=torch.int64, device="cuda")
        left = torch.empty_like(nfree)
        pa.pa_build_tables(table, lens, i32(new), free, nfree, out, cu, slots, left,
                           block_size=bs, num_blocks=nb, d_error=err)
        return out, cu, slots, left

    def expect(q, k, v, got, what, causal=False):
        n, m = q.shape[0], k.shape[0]
        vis = None
        if causal:
            i = torch.arange(n, device="cuda")
            vis = (i[None] <= i[:, None]).repeat(hq // hkv, 1)
        for h in range(hkv):
            hs = slice(h * hq // hkv, (h + 1) * hq // hkv)
            want, bound = attend(q[:, hs].transpose(0, 1).reshape(-1, d), k[:, h], v[:, h], scale,
                                 vis)
            check(got[:, hs].transpose(0, 1).reshape(-1, d), want, bound, f"{what}, {m} keys")

    # the prompt: tables, attention from its rows, the write
    row = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
    plen, cu, slots, nfree = tables(row, i32([0]), [n_prompt], n_prompt)
    qkv = rand(n_prompt, hq + 2 * hkv, d)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    out = torch.empty((n_prompt, hq, d), dtype=dt, device="cuda")
    pa.pa_attention_varlen(out, q, k, v, cu, scale=scale, max_seqlen=n_prompt, d_error=err)
    pa.pa_reshape_and_cache(k, v, k_pool, v_pool, slots, d_error=err)
    torch.cuda.synchronize()
    expect(q, k, v, out, "prompt", causal=True)

    # s requests fork from it; the prefix they share is its whole blocks (the
    # rest of its last block is copied into a block of each one's own)
    whole = n_prompt // bs * bs
    table = row.repeat(s, 1)
    if n_prompt % bs:
        src = int(row[0, whole // bs])
        take = free[int(nfree) - s:int(nfree)].clone()
        nfree = nfree - s
        pairs = torch.stack([torch.full((s,), src, device="cuda"), take.long()], 1).contiguous()
        pa.pa_copy_blocks(k_pool, v_pool, pairs, d_error=err)
        table[:, whole // bs] = take
    lens, starts, prefix = i32([n_prompt] * s), i32([0, s]), i32([whole])
    keys, values = [[k] for _ in range(s)], [[v] for _ in range(s)]
    for step in range(bs + 3):
        # request s - 1 pauses in every other step
        new = [1] * (s - 1) + [step % 2]
        lens, cu, slots, nfree = tables(table, lens, new, s)
        n = sum(new)
        qn, kn, vn = rand(s, hq, d), rand(s, hkv, d), rand(s, hkv, d)
        pa.pa_reshape_and_cache(kn, vn, k_pool, v_pool, slots, d_error=err)
        out = torch.empty((s, hq, d), dtype=dt, device="cuda")
        pa.pa_decode_shared(out, qn, k_pool, v_pool, table, lens, starts, prefix, scale=scale,
                            max_context_len=n_prompt + bs + 3, max_prefix_len=whole, d_error=err)
        torch.cuda.synchronize()
        for b in range(n):
            keys[b].append(kn[b:b + 1])
            values[b].append(vn[b:b + 1])
        if step in (0, 1, bs - 1, bs, bs + 2):
            for b in range(s):
                expect(qn[b:b + 1], torch.cat(keys[b]), torch.cat(values[b]), out[b:b + 1],
                       f"step {step}, request {b}")
    assert int(err) == 0
    used = s * (-(-(n_prompt + bs + 3) // bs) - whole // bs) + whole // bs
    assert nb - int(nfree) <= used + s + 1

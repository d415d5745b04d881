"""The operators between a projection and the cache, and those over a 4-bit cache, in the
order in which a server calls them: prompts, a chunk over what the cache holds, a decode
step; each stage against 64 bits on what the stage before left."""
import pytest
import torch

import attn_util as A
import fp4_util as F
import paged_kv_cache_34_gb300 as pa
import test_gpu_rope as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
HQ, HKV, D, BS, NB = 8, 2, 128, 16, 200


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class Server:
    def __init__(self, dtype, four):
        self.g = torch.Generator(device=DEV)
        self.g.manual_seed(11)
        self.dtype, self.four = dtype, four
        self.table = torch.full((3, 40), -1, dtype=torch.int32, device=DEV)
        self.free = torch.randperm(NB, generator=self.g, device=DEV).to(torch.int32)
        self.left = i32([NB])
        self.lens = i32([0, 0, 0])
        self.cs = R.table(1024, D)
        self.w = (1 + 0.2 * torch.randn(2, D, generator=self.g, device=DEV)).to(dtype)
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)
        if four:
            self.pools = [F.new_pool(NB, HKV, BS, D) for _ in range(2)]
            self.scales = [torch.tensor([0.0019, 0.0024], device=DEV) for _ in range(2)]
        else:
            self.pools = [torch.full((NB, BS, HKV, D), float("nan"), dtype=dtype, device=DEV)
                          for _ in range(2)]
        # what the cache should hold, in 64 bits, request by request
        self.kept = [[torch.zeros(0, HKV, D, dtype=torch.float64, device=DEV) for _ in range(2)]
                     for _ in range(3)]

    def project(self, new):
        """A step's tables and its rotated, normed rows; the cache is written."""
        t = sum(new)
        qkv = torch.randn(t, HQ + 2 * HKV, D, generator=self.g, device=DEV).to(self.dtype)
        q, k, v = qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:]
        raw_q, raw_k = q.clone(), k.clone()
        lens, cu, left = i32([0, 0, 0]), i32([0] * 4), i32([0])
        slots = torch.empty(t, dtype=torch.int64, device=DEV)
        pos = torch.empty(t, dtype=torch.int32, device=DEV)
        pa.pa_build_tables(self.table, self.lens, i32(new), self.free, self.left, lens, cu, slots,
                           left, positions=pos, block_size=BS, num_blocks=NB, d_error=self.err)
        norms = dict(q_weight=self.w[0], k_weight=self.w[1])
        if self.four:
            pa.pa_qk_norm_rope(q, k, q, k, pos, self.cs, d_error=self.err, **norms)
            pa.pa_reshape_and_cache_fp4(k, v, *self.pools, slots, *self.scales, d_error=self.err)
        else:
            pa.pa_rope_and_cache(q, q, k, v, *self.pools, slots, pos, self.cs, key_out=k,
                                 d_error=self.err, **norms)
        torch.cuda.synchronize()
        for got, raw, w, what in ((q, raw_q, self.w[0], "q"), (k, raw_k, self.w[1], "k")):
            want, size = R.formula(raw, pos, self.cs, w, 1e-6, False)
            R.check(got, want, size, self.dtype, what)
        ends = cu.tolist()
        for b in range(3):
            for n, x in enumerate((k, v)):
                row = x[ends[b]:ends[b + 1]].double()
                if self.four:
                    row = F.values(*F.quantise(x[ends[b]:ends[b + 1]], self.scales[n])) \
                        * self.scales[n].double()[:, None]
                self.kept[b][n] = torch.cat([self.kept[b][n], row])
        self.lens, self.left = lens, left
        return q, k, v, cu, ends

    def want(self, b, q, scale):
        """(64 bits, bound) of request b's newest queries q [n, HQ, D] over its cache."""
        k, v = self.kept[b]
        n, m, g = q.shape[0], k.shape[0], HQ // HKV
        out, bound = (torch.zeros(q.shape, dtype=torch.float64, device=DEV) for _ in range(2))
        for i in range(n):  # row i sees all but the n - 1 - i newest
            e = m - (n - 1 - i)
            for h in range(HKV):
                r = slice(h * g, (h + 1) * g)
                out[i, r], bound[i, r] = F.attend(q[i, r], k[:e, h], v[:e, h], scale)
        return out, bound


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("four", [False, True])
def test_prompts_chunk_and_decode(four, dtype):
    s, scale = Server(dtype, four), D ** -0.5
    # prompts: attention from their own rows
    q, k, v, cu, ends = s.project([70, 1, 33])
    out = torch.empty(q.shape, dtype=dtype, device=DEV)
    pa.pa_attention_varlen(out, q, k, v, cu, scale=scale, max_seqlen=70, d_error=s.err)
    torch.cuda.synchronize()
    for b in range(3):
        rows = slice(ends[b], ends[b + 1])
        n = ends[b + 1] - ends[b]
        see = torch.ones(n, n, dtype=torch.bool, device=DEV).tril()
        for h in range(HQ):
            A.check(out[rows, h], *A.attend(q[rows, h], k[rows, h // 4], v[rows, h // 4], scale, see))
    # a chunk of new tokens over what the cache holds
    q, k, v, cu, ends = s.project([20, 45, 3])
    out = torch.empty(q.shape, dtype=dtype, device=DEV)
    lens = s.lens.tolist()
    if four:  # read back into blocks of a 16-bit pool, request by request
        blocks = [-(-n // BS) for n in lens]
        first = [sum(blocks[:b]) for b in range(3)]
        rows = torch.zeros(2, sum(blocks) * BS, HKV, D, dtype=dtype, device=DEV)
        pa.pa_gather_cache_fp4(rows[0], rows[1], *s.pools, s.table, s.lens,
                               i32([f * BS for f in first]), *s.scales, max_context_len=200,
                               d_error=s.err)
        pools = rows.view(2, -1, BS, HKV, D)
        table = torch.arange(10, device=DEV, dtype=torch.int32)[None, :] + i32(first)[:, None]
        s_kept = s.kept
        s.kept = [[rows[n, first[b] * BS:first[b] * BS + lens[b]].double() for n in range(2)]
                  for b in range(3)]
        for b in range(3):  # the rows are the cache's values, rounded once
            for n in range(2):
                off = (s.kept[b][n] - s_kept[b][n]).abs()
                u = torch.finfo(dtype).eps / 2 + 2.0 ** -24
                assert bool((off <= u * s_kept[b][n].abs()).all())
    else:
        pools, table = s.pools, s.table
    pa.pa_prefill_varlen(out, q, *pools, table.contiguous(), cu, s.lens, scale=scale,
                         max_seqlen_q=45, max_context_len=200, d_error=s.err)
    torch.cuda.synchronize()
    for b in range(3):
        rows = slice(ends[b], ends[b + 1])
        n, m = ends[b + 1] - ends[b], lens[b]
        see = torch.ones(n, m, dtype=torch.bool, device=DEV).tril(m - n)
        for h in range(HQ):
            kk, vv = (x[:, h // 4].to(dtype) for x in s.kept[b])
            A.check(out[rows, h], *A.attend(q[rows, h], kk, vv, scale, see))
    if four:
        s.kept = s_kept
    # a decode step of all three
    q, k, v, cu, ends = s.project([1, 1, 1])
    out = torch.empty(q.shape, dtype=dtype, device=DEV)
    if four:
        pa.pa_decode_fp4(out, q, *s.pools, s.table, s.lens, *s.scales, scale=scale,
                         max_context_len=200, d_error=s.err)
    else:
        pa.pa_decode(out, q, *s.pools, s.table, s.lens, scale=scale, max_context_len=200,
                     d_error=s.err)
    torch.cuda.synchronize()
    for b in range(3):
        if four:
            F.check(out[b:b + 1], *s.want(b, q[b:b + 1], scale))
        else:
            for h in range(HQ):
                kk, vv = (x[:, h // 4].to(dtype) for x in s.kept[b])
                A.check(out[b:b + 1, h], *A.attend(q[b:b + 1, h], kk, vv, scale))
    assert int(s.err) == 0

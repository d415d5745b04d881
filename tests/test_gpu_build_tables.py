"""pa_build_tables on the GPU against the definition, request by request in
Python integers: every output value must be equal."""
import random

import pytest
import torch

import oracle
from gpu_util import gpu, new_err, pa, require_gpu

pytestmark = gpu

CANARY = -7


def plain(table, ctx, new, free, nfree, tokens, bs, nb):
    """The definition (table: list of rows, changed in place)."""
    err = 0
    cap = len(table[0]) * bs if table else 0
    f = min(max(nfree, 0), len(free))
    if f != nfree:
        err |= pa.DEVERR_NO_BLOCKS
    slots, pos, lens, cu, used, left = [-1] * tokens, [0] * tokens, [], [0], 0, f
    for b, (c, n) in enumerate(zip(ctx, new)):
        if c < 0 or n < 0 or c + n > cap:
            err |= pa.DEVERR_CONTEXT
            lens.append(0)
            cu.append(cu[-1])
            continue
        have, need = -(-c // bs), -(-(c + n) // bs)
        first, used = used, used + need - have
        fits = n == 0 or cu[-1] + n <= tokens
        blocks = need == have or used <= f
        if not fits:
            err |= pa.DEVERR_CU_SEQLENS
        if not blocks:
            err |= pa.DEVERR_NO_BLOCKS
        ok = fits and blocks
        if ok:
            for j in range(have, need):
                i = free[f - 1 - (first + j - have)]
                table[b][j] = i if 0 <= i < nb else -1
                left = min(left, f - 1 - (first + j - have))
        for i in range(n):
            t = cu[-1] + i
            if t >= tokens:
                break
            pos[t] = c + i
            if ok:
                blk = table[b][(c + i) // bs]
                if 0 <= blk < nb:
                    slots[t] = blk * bs + (c + i) % bs
                else:
                    err |= pa.DEVERR_BLOCK_ID
        lens.append(c + n if ok else 0)
        cu.append(cu[-1] + n)
    return dict(table=table, lens=lens, cu=[min(x, 2**31 - 1) for x in cu], slots=slots, pos=pos,
                left=left), err


class Step:
    """One call's tensors; the table has columns of a wider buffer around it."""

    def __init__(self, table, ctx, new, free, nfree, tokens, bs, nb, shift=0):
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        s, w = len(ctx), len(table[0]) if table else 1
        self.wide = torch.full((s, w + 5), CANARY, dtype=torch.int32, device="cuda")
        self.table = self.wide[:, 2:2 + w]
        if s:
            self.table.copy_(i32(table))
        self.ctx, self.new, self.free, self.nfree = i32(ctx), i32(new), i32(free), i32([nfree])
        self.lens, self.cu = i32([CANARY] * s), i32([CANARY] * (s + 1))
        # `shift` elements off the allocation's start: unaligned vectors
        self.slot_buf = torch.full((tokens + shift + 4,), CANARY, dtype=torch.int64, device="cuda")
        self.pos_buf = torch.full((tokens + shift + 4,), CANARY, dtype=torch.int32, device="cuda")
        self.slots, self.pos = (x[shift:shift + tokens] for x in (self.slot_buf, self.pos_buf))
        self.left, self.err = i32([CANARY]), new_err()
        self.bs, self.nb, self.shift, self.tokens = bs, nb, shift, tokens

    def run(self, positions=True):
        pa.pa_build_tables(self.table, self.ctx, self.new, self.free, self.nfree, self.lens,
                           self.cu, self.slots, self.left, block_size=self.bs, num_blocks=self.nb,
                           positions=self.pos if positions else None, d_error=self.err)

    def check(self, want, err, positions=True):
        torch.cuda.synchronize()
        assert self.table.tolist() == want["table"]
        assert self.lens.tolist() == want["lens"] and self.cu.tolist() == want["cu"]
        assert self.slots.tolist() == want["slots"]
        assert self.pos.tolist() == (want["pos"] if positions else [CANARY] * self.tokens)
        assert self.left.tolist() == [want["left"]]
        assert int(self.err) == err
        # nothing around the outputs was touched
        edge = torch.cat([self.wide[:, :2], self.wide[:, -3:]], 1)
        assert bool((edge == CANARY).all())
        for buf in (self.slot_buf, self.pos_buf):
            out = torch.cat([buf[:self.shift], buf[self.shift + self.tokens:]])
            assert bool((out == CANARY).all())


def make(rng, s, ctx_hi, new_hi, bs, extra=3, pad=0, width=None, shift=0):
    ctx = [rng.randint(0, ctx_hi) for _ in range(s)]
    new = [rng.choice([0, 1, rng.randint(0, new_hi)]) for _ in range(s)]
    width = width or max([1] + [-(-(c + n) // bs) for c, n in zip(ctx, new)])
    held = sum(-(-c // bs) for c in ctx)
    need = sum(-(-(c + n) // bs) - -(-c // bs) for c, n in zip(ctx, new))
    nb = held + need + extra
    ids = list(range(nb))
    rng.shuffle(ids)
    it = iter(ids)
    table = [[next(it) if j < -(-c // bs) else -1 for j in range(width)] for c in ctx]
    free = list(it)
    return dict(table=table, ctx=ctx, new=new, free=free, nfree=need + min(extra, 2),
                tokens=sum(new) + pad, bs=bs, nb=nb, shift=shift)


def run_both(d, positions=True):
    require_gpu()
    step = Step(**d)
    step.run(positions)
    want, err = plain([list(r) for r in d["table"]], d["ctx"], d["new"], d["free"], d["nfree"],
                      d["tokens"], d["bs"], d["nb"])
    step.check(want, err, positions)
    return step, want, err


@pytest.mark.parametrize("bs", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("s,ctx_hi,new_hi", [(1, 0, 1), (1, 300, 500), (2, 40, 3), (7, 0, 130),
                                             (33, 500, 1), (511, 90, 9), (513, 20, 40)])
def test_steps(bs, s, ctx_hi, new_hi):
    rng = random.Random(s * 1000 + bs)
    run_both(make(rng, s, ctx_hi, new_hi, bs, pad=rng.choice([0, 1, 50])))


@pytest.mark.parametrize("shift", [0, 1, 2, 3])
def test_unaligned_outputs_and_no_positions(shift):
    d = make(random.Random(shift), 9, 100, 77, 16, pad=5, shift=shift)
    run_both(d)
    run_both(d, positions=False)


@pytest.mark.parametrize("s", [2049, 4096, 4097, 8193, 20000])
def test_many_requests(s):
    # beyond 4096 requests one shared sum stands for several of them
    run_both(make(random.Random(s), s, 33, 3, 16, pad=3))


def test_many_tokens():
    # more tokens than one wave of threads takes in a step
    run_both(make(random.Random(3), 40, 1000, 60000, 128, pad=11))


@pytest.mark.parametrize("seed", range(6))
def test_short_lists_bad_lengths_and_bad_blocks(seed):
    rng = random.Random(seed)
    d = make(rng, 60, 200, 90, 16, pad=20)
    d["nfree"] = rng.randint(0, d["nfree"])                     # requests behind go without
    for _ in range(3):                                          # lengths that do not fit a row
        b = rng.randrange(60)
        which = rng.choice(["ctx", "new"])
        d[which][b] = rng.choice([-1, -2**31, 2**31 - 1, 5000])
    if seed % 2:
        d["tokens"] = rng.randint(0, d["tokens"] // 2)          # tokens past the array
    if seed >= 2:                                               # ids outside the pool
        d["free"][rng.randrange(len(d["free"]))] = rng.choice([-1, d["nb"], 2**31 - 1])
        held = [(b, j) for b, r in enumerate(d["table"]) for j, x in enumerate(r) if x >= 0]
        b, j = rng.choice(held)
        d["table"][b][j] = rng.choice([-5, d["nb"]])
    _, _, err = run_both(d)
    assert err != 0


@pytest.mark.parametrize("nfree", [-1, -2**31, 10**6])
def test_list_length_outside_its_array(nfree):
    d = make(random.Random(8), 12, 60, 40, 16)
    d["nfree"] = nfree
    _, _, err = run_both(d)
    assert err & pa.DEVERR_NO_BLOCKS


def test_sums_beyond_32_bits():
    # every length is legal, their sum is not an int32: no slot is wrong, cu
    # stays at its largest value
    require_gpu()
    s, width = 40, 1 << 21                             # 2^28 tokens a row
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    new = [3] + [1 << 28] * (s - 1)                    # sum far above 2^31
    out, cu = i32([CANARY] * s), i32([CANARY] * (s + 1))
    slots = torch.full((8,), CANARY, dtype=torch.int64, device="cuda")
    left, err = i32([0]), new_err()
    table = torch.full((s, width), -1, dtype=torch.int32, device="cuda")
    pa.pa_build_tables(table, i32([0] * s), i32(new), i32([5]), i32([1]), out, cu, slots, left,
                       block_size=128, num_blocks=9, d_error=err)
    torch.cuda.synchronize()
    assert slots.tolist() == [5 * 128, 5 * 128 + 1, 5 * 128 + 2] + [-1] * 5
    assert out.tolist() == [3] + [0] * (s - 1) and left.tolist() == [0]
    run, want = 0, [0]
    for n in new:
        run += n
        want.append(min(run, 2**31 - 1))
    assert cu.tolist() == want
    assert int(err) == pa.DEVERR_CU_SEQLENS | pa.DEVERR_NO_BLOCKS


def test_no_requests_and_no_tokens():
    require_gpu()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    e = torch.zeros((0,), dtype=torch.int32, device="cuda")
    cu, left = i32([9]), i32([9])
    slots = torch.full((6,), CANARY, dtype=torch.int64, device="cuda")
    pa.pa_build_tables(e.view(0, 1), e, e, i32([3, 4]), i32([2]), e, cu, slots, left,
                       block_size=16, num_blocks=8)
    torch.cuda.synchronize()
    assert cu.tolist() == [0] and left.tolist() == [2] and slots.tolist() == [-1] * 6
    d = make(random.Random(1), 5, 50, 0, 16)
    d["new"], d["tokens"] = [0] * 5, 0
    run_both(d)


def test_repeated_captured_and_on_another_stream():
    # the same inputs give the same outputs again, eagerly, from a graph and
    # on a side stream
    d = make(random.Random(5), 100, 300, 50, 32, pad=7)
    step, want, err = run_both(d)
    step.run()
    step.check(want, err)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step.run()
    for buf in (step.lens, step.cu, step.slots, step.pos, step.left):
        buf.fill_(CANARY)
    g.replay()
    step.check(want, err)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step.run()
    torch.cuda.current_stream().wait_stream(side)
    step.check(want, err)


def test_steps_follow_one_another():
    # three steps of one batch: a prompt, then decode steps; each step's
    # outputs are the next one's inputs, and the tables address every token
    # of every request exactly once
    require_gpu()
    s, bs, nb = 6, 16, 64
    new = [[40, 3, 17, 100, 1, 16], [1] * s, [1, 0, 1, 5, 1, 1]]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.full((s, 12), -1, dtype=torch.int32, device="cuda")
    free, nfree = torch.randperm(nb, dtype=torch.int32, device="cuda"), i32([nb])
    lens, written = i32([0] * s), []
    for n in new:
        out, cu = torch.empty_like(lens), torch.empty(s + 1, dtype=torch.int32, device="cuda")
        slots = torch.empty(sum(n), dtype=torch.int64, device="cuda")
        left, err = torch.empty_like(nfree), new_err()
        pa.pa_build_tables(table, lens, i32(n), free, nfree, out, cu, slots, left,
                           block_size=bs, num_blocks=nb, d_error=err)
        torch.cuda.synchronize()
        assert int(err) == 0
        written += slots.tolist()
        lens, nfree = out, left
    assert lens.tolist() == [sum(x) for x in zip(*new)]
    want = []
    for b, n in enumerate(lens.tolist()):
        row = table[b].tolist()
        want += [row[j // bs] * bs + j % bs for j in range(n)]
    assert sorted(written) == sorted(want) and len(set(written)) == len(written)


def test_matches_the_host_formulas():
    # slots and cumulative lengths equal the Runner-side formulas of the pages
    d = make(random.Random(21), 17, 200, 60, 16)
    _, want, _ = run_both(d)
    assert want["cu"] == [int(x) for x in oracle.cu_seqlens(d["new"])]
    for b, (c, n) in enumerate(zip(d["ctx"], d["new"])):
        for i in range(n):
            assert want["slots"][want["cu"][b] + i] == oracle.slot_of([want["table"][b]], 0,
                                                                      c + i, 16)

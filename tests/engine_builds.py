"""Which build of the attention tile engine a call takes, restated from the
launchers' rules, and batches that reach each of them.  The tests assert the
build they mean to run, so that a changed rule cannot silently leave one out.

pa_attention_varlen has three: one query tile per item ("single"), pairs of
them with the compact softmax ("compact"), and pairs with the unrolled one
("pairs"); pa_decode_shared's prefix pass the same three.
"""
import torch


def packed_heads(group):
    for d in range(min(group, 128), 1, -1):
        if group % d == 0 and (128 // d) * d >= 112:
            return d
    return 1


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def varlen_build(num_seqs, total, max_seqlen, hq, hkv):
    pg = packed_heads(hq // hkv)
    rows = 128 // pg
    items = min(total // rows + num_seqs,
                num_seqs * -(-min(max_seqlen, total) // rows)) * (hq // pg)
    if items <= (4 if max_seqlen >= 640 else 1) * sms():
        return "single"
    return "compact" if max_seqlen <= 2048 else "pairs"


def shared_build(num_seqs, num_groups, max_prefix, hq, hkv):
    pg = packed_heads(hq // hkv)
    if num_seqs <= 128 // pg:
        return "single"
    cost, runs = shared_runs(num_seqs, num_groups, max_prefix, hq, hkv)
    return "compact" if cost <= 64 * runs else "pairs"


def shared_runs(num_seqs, num_groups, max_prefix, hq, hkv):
    """(the most the prefix pass can cost, its runs) of a batch of tile pairs."""
    pg = packed_heads(hq // hkv)
    cost = (num_seqs // (128 // pg) + num_groups) * (hq // pg) * -(-max_prefix // 128)
    most = sms() // 2 if cost <= 6 * sms() else sms()
    return cost, max(1, min((cost + 1) // 2, most))


def runs_with_two_rows_of_a_pair(start, tiles, line, run):
    """How many of the prefix pass's runs (of `run` cost) hold tiles of one pair of
    query tiles from two blocks of a line of `line` K/V tiles, in a group of
    `tiles` query tiles that starts at cost position `start`."""
    ks = min(line, run if tiles == 3 else (run + 1) // 2)
    held = {}
    for blk in range(-(-line // ks)):
        n = min(ks, line - blk * ks)
        at = start + blk * ks * tiles
        for q in range((tiles + 1) // 2):
            w = 2 if 2 * q + 1 < tiles else 1
            for i in range(n):
                held.setdefault(((at + w * i) // run, q), set()).add(blk)
            at += w * n
    return sum(len(b) > 1 for b in held.values())


def reach(x, build):
    """A batch of test_gpu_attention_varlen.make() and its host bound for a
    call that takes `build`: its heads are repeated until the call has that
    many items.  Returns (batch, bound); ``copies`` is in the batch."""
    lens, hq, hkv = x["lens"], x["q"].shape[1], x["k"].shape[1]
    longest = max(lens + [1])
    bound = max(longest, 4096) if build == "pairs" else longest
    copies = 1
    while varlen_build(len(lens), x["q"].shape[0], bound, hq * copies, hkv * copies) != build:
        copies *= 2
        assert copies <= 1024, (lens, hq, hkv, build)
    y = dict(x, copies=copies, heads=(hq, hkv))
    for n in ("q", "k", "v"):
        y[n] = x[n].repeat(1, copies, 1)
    y["wide"] = torch.full((x["q"].shape[0], hq * copies + 1, x["q"].shape[2]), -3.0,
                           dtype=x["q"].dtype, device="cuda")
    y["out"] = y["wide"][:, :hq * copies]
    return y, bound


def first_copy(y):
    """The batch of `reach`, cut to its first copy's heads; the other copies'
    outputs must be the first's, bit for bit."""
    hq, hkv = y["heads"]
    outs = y["out"].unflatten(1, (y["copies"], hq))
    same = torch.equal(outs.view(torch.int16), outs[:, :1].expand_as(outs).view(torch.int16))
    assert same, "copies of the same heads differ"
    return dict(y, q=y["q"][:, :hq], k=y["k"][:, :hkv], v=y["v"][:, :hkv], out=y["out"][:, :hq])

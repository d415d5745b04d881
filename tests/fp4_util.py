"""The 4-bit pools' format in 64 bits, and attention over it with a bound on a
correct kernel's error; written from the definitions alone."""
import torch

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def e4m3_values():
    """The 127 finite values without a sign, in code order: exponent bias 7, three
    fraction bits, exponent 0 subnormal."""
    v = []
    for b in range(127):
        e, m = b >> 3, b & 7
        v.append((1 + m / 8) * 2.0 ** (e - 7) if e else m / 8 * 2.0 ** -6)
    return v


def nearest(q, values):
    """Index of the nearest of `values` (increasing) to q >= 0, ties to the even index."""
    t = torch.tensor(values, dtype=torch.float64, device=q.device)
    q = q.clamp(max=values[-1]).contiguous()
    hi = torch.searchsorted(t, q).clamp(1, len(values) - 1)
    lo = hi - 1
    down, up = q - t[lo], t[hi] - q
    return torch.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)


def fp32(x):
    return x.float().double()


def quantise(x, scale):
    """Rows [..., Hkv, D] of 16-bit values -> (codes [..., Hkv, D], group scale bytes
    [..., Hkv, D/16]) of the heads' fp32 scales; every step rounded to fp32."""
    y = x.double().unflatten(-1, (-1, 16))
    y = torch.where(y.isnan(), 0.0, y)
    S = scale.double()[:, None]
    good = (S >= 2.0 ** -64) & (S <= 2.0 ** 64)
    S = torch.where(good, S, 1.0)
    c = nearest(fp32(y.abs().amax(-1) / fp32(6 * S)), e4m3_values())
    c = torch.where(good, c, 0)
    w = fp32(torch.tensor(e4m3_values(), dtype=torch.float64, device=x.device)[c] * S)[..., None]
    some = w > 0
    q = fp32(y / torch.where(some, w, 1.0))
    code = nearest(q.abs(), E2M1) + 8 * (torch.signbit(q)).long()
    code = torch.where(some, code, 0)
    return code.flatten(-2), c


def values(code, c):
    """code * group scale in 64 bits (without the head's scale)."""
    t = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device=code.device)
    # 0x7f: NaN
    s = torch.tensor(e4m3_values() + [float("nan")], dtype=torch.float64, device=code.device)
    return (t[code.long()].unflatten(-1, (-1, 16)) * s[c.long()][..., None]).flatten(-2)


def parts(pool, d):
    """(codes, scales) of a pool: views [NB, Hkv, bs/8, 8, D/2] and [.., 8, D/16]."""
    assert pool.shape[3] == 9 * d // 2
    return (pool[..., :4 * d].unflatten(-1, (8, d // 2)),
            pool[..., 4 * d:].unflatten(-1, (8, d // 16)))


def new_pool(nb, hkv, bs, d, device="cuda", code=0xff, scale=0x7f):
    """A pool of rows that no call may take for anything: NaN scales."""
    pool = torch.empty(nb, hkv, bs // 8, 9 * d // 2, dtype=torch.uint8, device=device)
    pool[..., :4 * d] = code
    pool[..., 4 * d:] = scale
    return pool


def put(pool, slots, codes, c):
    """Rows' codes [T, Hkv, D] and scales [T, Hkv, D/16] into the pool's slots [T]."""
    bs, d = pool.shape[2] * 8, codes.shape[-1]
    pc, ps = parts(pool, d)
    b, o = slots // bs, slots % bs
    both = (codes[..., 0::2] | codes[..., 1::2] << 4).to(torch.uint8)
    pc[b, :, o // 8, o % 8] = both
    ps[b, :, o // 8, o % 8] = c.to(torch.uint8)


def get(pool, slots, d):
    """Codes [T, Hkv, D] and scale bytes [T, Hkv, D/16] of the pool's slots."""
    bs = pool.shape[2] * 8
    pc, ps = parts(pool, d)
    b, o = slots // bs, slots % bs
    x = pc[b, :, o // 8, o % 8]
    return torch.stack([x & 15, x >> 4], -1).flatten(-2), ps[b, :, o // 8, o % 8]


def attend(q, k, v, scale):
    """Queries q [n, d] of one KV head over keys and values k, v [m, d] in 64 bits:
    (out, bound on a correct kernel's error).

    As in attn_util, for weights w_j that are rounded to fp16 (u = 2^-11) before they
    are summed and multiplied: out - o = sum_j w_j (x_j + d_j) (v_j - o) + rounding, with
    |d_j| <= u, or 2^-25 next to a sum of at least 1 for weights below 2^-14; x_j from the
    score's fp32 sum of d terms, its scaling and the exponential; fp32 sums over m keys;
    the output rounded to its type."""
    u, d, m = torch.finfo(q.dtype).eps / 2, q.shape[1], k.shape[0]
    fp16 = q.dtype is torch.float16
    q = q.double()
    s = q @ k.T * scale
    mag = (q.abs() @ k.abs().T * abs(scale)).amax(-1, keepdim=True)
    e = torch.exp(s - s.amax(-1, keepdim=True))
    total = e.sum(-1, keepdim=True)
    w = e / total
    o = w @ v
    x = torch.expm1(2 * ((d + 8) * 2.0 ** -24 * mag + 2.0 ** -21))
    spread, flat = torch.empty_like(o), torch.empty_like(o)
    for i in range(q.shape[0]):
        dist = (v - o[i]).abs()
        spread[i] = w[i] @ dist
        flat[i] = dist.sum(0)
    bound = ((x + 2.0 ** -11) * spread + 2.0 ** -25 / total * flat + u * o.abs()
             + m * 2.0 ** -23 * (w @ v.abs()))
    if fp16:
        bound = bound + 2.0 ** -25
    return o, 1.01 * bound + 1e-30


def check(got, want, bound, what=""):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: non-finite output"
    over = (got - want).abs() - bound
    if over.numel() and float(over.max()) > 0:
        i = int(over.flatten().argmax())
        raise AssertionError(f"{what}: {got.flatten()[i]:.6g} at {i}, want "
                             f"{want.flatten()[i]:.6g} within {bound.flatten()[i]:.3g}")
